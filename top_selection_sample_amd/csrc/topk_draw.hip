// The next token of each row of logits.
//
//   w_i = exp((z_i - m) / temperature), m the largest logit; of the tokens in
//   the order (z falling, i rising) the first top_k stay, of those the shortest
//   beginning with top_p of their sum, of those the ones with w_i >= min_p;
//   the token is the first, by index, at which the sum of the w that stayed
//   exceeds u times their sum
//
// Which token it is hangs on sums over the whole row next to a border, so the
// weights are whole multiples of 2^-F, F = 62 - ceil(log2 n), in 64 bits: sums
// are exact, in whatever order and whatever pieces they are taken (atomics
// included), and the comparisons with top_p and u are exact as well.  The
// exponential is a polynomial in 64-bit floats: of 2^t, t = (z - m) log2(e) /
// temperature, it is off by less than (1 + |t|) 2^-51 of its value (three roundings
// of t, each up to 2^-53 of it, and those of the polynomial), so by less than 2^-50
// of the largest weight.
//
// top_k and top_p keep a beginning of the one order, so together they are one
// cut: a logit and an index.  A row is cut into chunks, a workgroup each:
//
//   k_sample_first    the chunks' maxima; where top_k is small, those of every
//                     GROUP entries too: if k groups reach a bin, the k largest
//                     entries lie in the bins up to it, and in such groups
//   k_sample_bins     other rows with a cut: counts and sums of weights by bins
//                     of m - z (its float's leading bits: 128 bins to an octave)
//   k_sample_plan     from those the bins that the cut can lie in
//   k_sample_collect  their entries, and each chunk's sum over the bins before
//   k_sample_finish   the entries sorted, the cut, the chunk that the token
//                     lies in, the token
//
// Calls without a cut do without the second and third, those whose top_k is small
// in all rows without the middle three.  (A row's last workgroup doing the next step
// saves a launch, but the fence that this takes in every workgroup writes its
// cache back: 790 us for 256 rows of 65536, against 30.)
//
// One row of 131072 f32 with top_k 50 and top_p takes 3 + 9 us, each a chain of
// dependent steps; 64 rows of 100003 bf16 with settings of their own 27 (6 the
// first pass, 15 the last, 2 to 3 each of the three that find nothing to do); 256
// rows of 65536 f32 (67 MB) with min_p 33: 11.8 for the maxima, 5.7 TB/s, 15 for
// the sums, which reads the logits once more, and 6.7.  153 rows of 78201 bf16
// with top_p alone 92: 6, 30 for the bins, bound by their atomics in LDS, 5, 32
// and 23.
#include <algorithm>

#include "topk_model.hpp"
#include "topk_ops_device.hpp"

namespace tk {

namespace {

constexpr uint32_t FIRST_THREADS = 256;
constexpr uint32_t ROW_THREADS = 512;
constexpr uint32_t ROW_WAVES = ROW_THREADS / 64;
constexpr uint32_t TILE = 4096;             // entries that a workgroup takes at a time; a chunk is one or more
constexpr uint32_t MAX_CHUNKS = 1024;       // of a row
constexpr uint32_t BINS = 2048;             // 16 octaves of m - z from 2^-7 on, 128 to an octave
constexpr uint32_t FIRST_BIN = (127 - 7) << 7;
constexpr uint32_t CAP = 4096;              // entries of a row around its cut that are sorted
constexpr uint32_t GROUP = TILE / FIRST_THREADS;   // entries of a thread of k_sample_first
constexpr uint32_t SMALL_K = 384;           // a small top_k
constexpr uint32_t PAIRS = 512;             // entries that are compared each with each rather than sorted

// What is known of a row between the launches.
struct SampleRow {
  uint64_t before;        // weight of the bins below `lo`
  uint64_t before_k;      // weight of the bins below `bk`
  uint32_t lo, hi, bk;    // entries of bins lo to hi, and of bin bk, are collected; bk: where the k-th is (BINS: top_k is off)
  uint32_t count, count_k;// entries of the bins below lo and bk
  uint32_t k;             // top_k, where bk says so
  uint32_t cut;           // whether there is a cut
  uint32_t inside;        // all that can stay is collected
};

// The settings of a row, worked out once for all its workgroups.
struct Settings {
  double rate;       // log2(e) / temperature; 0 if greedy
  float far;         // logits further than this below the maximum have no weight that counts
  uint32_t greedy;
};

struct SampleArgs {
  const void* logits;
  const float* u;
  int64_t* tokens;
  float* logprobs;
  const float* temperatures;
  const int64_t* top_ks;
  const float* top_ps;
  const float* min_ps;
  float* maxima;          // [rows][chunks]
  Settings* settings;     // [rows]
  uint32_t* collected;    // [rows]: entries in `cand`, or more than CAP
  float* groups;          // [rows][chunks * FIRST_THREADS]: the groups' maxima, where top_k is small; null: it never is
  uint64_t* sums;         // [rows][chunks]: weight that surely stays
  uint32_t* bin_count;    // [rows][BINS]
  uint64_t* bin_sum;
  uint64_t* cand;         // [rows][CAP]
  SampleRow* row;
  uint64_t ld, work;
  int64_t top_k;
  float temperature, top_p, min_p;
  uint32_t n, chunk, chunks, bits;   // bits: F
};

__device__ __forceinline__ float temperature_of(const SampleArgs& a, uint64_t r) { return a.temperatures ? a.temperatures[r] : a.temperature; }
__device__ __forceinline__ float top_p_of(const SampleArgs& a, uint64_t r) { return a.top_ps ? a.top_ps[r] : a.top_p; }
__device__ __forceinline__ double min_p_of(const SampleArgs& a, uint64_t r) {
  const float p = a.min_ps ? a.min_ps[r] : a.min_p;
  return p > 1.f ? 1.0 : (double)p;
}

// `far`: well below min_p, or below half of 2^-62.
__device__ __forceinline__ Settings make_settings(const SampleArgs& a, uint64_t r) {
  const float t = temperature_of(a, r);
  const double p = min_p_of(a, r);
  Settings s;
  s.greedy = !(t > 0.f);
  s.rate = s.greedy ? 0.0 : 1.4426950408889634 / (double)t;
  const double least = p > 0.0 ? fmax(log2(p) - 1e-3, -64.0) : -64.0;
  const double far = s.rate > 0.0 ? -least / s.rate * (1.0 + 1e-6) : INFINITY;
  s.far = s.greedy ? 0.f : far < 3e38 ? __uint_as_float(__float_as_uint((float)far) + 1) : INFINITY;   // rounded up
  return s;
}

template <class T>
__device__ __forceinline__ float logit_of(const T* row, uint32_t i) {
  const float z = to_f32(row[i]);
  return z != z ? -INFINITY : z;
}

// The weight of a logit: 2^t, t = (z - m) log2(e) / temperature, as 2^i times a
// polynomial in f = t - i, |f| <= 1/2, with the coefficients ln(2)^j / j!; the
// first one left out is below 2^-57.
__device__ __forceinline__ double weight_of(float z, float m, const Settings& s) {
  if (z == m) return 1.0;
  if (s.greedy) return 0.0;
  const double t = ((double)z - (double)m) * s.rate;
  if (!(t > -64.0)) return 0.0;   // below half of 2^-62
  const double i = rint(t), f = t - i;
  double p = 1.3691488853904128e-12;
  p = fma(f, p, 2.5678435993488206e-11);
  p = fma(f, p, 4.4455382718708116e-10);
  p = fma(f, p, 7.054911620801123e-09);
  p = fma(f, p, 1.01780860092397e-07);
  p = fma(f, p, 1.321548679014431e-06);
  p = fma(f, p, 1.5252733804059841e-05);
  p = fma(f, p, 0.0001540353039338161);
  p = fma(f, p, 0.0013333558146428443);
  p = fma(f, p, 0.009618129107628477);
  p = fma(f, p, 0.05550410866482158);
  p = fma(f, p, 0.24022650695910072);
  p = fma(f, p, 0.6931471805599453);
  p = fma(f, p, 1.0);
  return ldexp(p, (int)i);
}
__device__ __forceinline__ uint64_t fixed_of(double w, uint32_t bits) { return (uint64_t)rint(ldexp(w, (int)bits)); }

// Order of the tokens: larger logits, then lower indices, have larger codes.
__device__ __forceinline__ uint64_t code_of(float z, uint32_t i) {
  const uint32_t u = __float_as_uint(z + 0.f);
  const uint32_t key = u & 0x80000000u ? ~u : u | 0x80000000u;
  return (uint64_t)key << 32 | (uint32_t)~i;
}
__device__ __forceinline__ float logit_of_code(uint64_t c) {
  const uint32_t key = (uint32_t)(c >> 32);
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// Whether a logit can be taken at all: of an infinite maximum only its equals.
__device__ __forceinline__ bool live(float z, float m) { return z > -INFINITY && (z == m || m < INFINITY); }

// Bins rise with m - z, whose rounding keeps the order.
__device__ __forceinline__ uint32_t bin_of(float z, float m) {
  if (z == m) return 0;
  const uint32_t b = __float_as_uint(m - z) >> 16;
  return b <= FIRST_BIN ? 0u : min(b - FIRST_BIN, BINS - 1);
}

// m - z of all logits in bins up to b, but the equals of an infinite m, is below
// this; that of a logit of -inf is not, nor is one that overflows (last bin).
__device__ __forceinline__ float bin_end(uint32_t b) { return b >= BINS - 1 ? INFINITY : __uint_as_float((FIRST_BIN + b + 1) << 16); }

// ceil(p * w) and floor(p * w), exact; p a float in (0, 1).
__device__ __forceinline__ void scaled(float p, uint64_t w, uint64_t* floor_, uint64_t* ceil_) {
  const uint32_t u = __float_as_uint(p);
  const uint32_t e = u >> 23;
  const uint64_t mant = e ? (u & 0x7FFFFFu) | 0x800000u : u & 0x7FFFFFu;
  const uint32_t shift = 150 - (e ? e : 1);   // p = mant * 2^-shift, shift from 24 to 149
  const uint64_t hi = __umul64hi(mant, w), lo = mant * w;   // below 2^86
  uint64_t q, rest;
  if (shift < 64) {
    q = hi << (64 - shift) | lo >> shift;
    rest = lo << (64 - shift);
  } else if (shift == 64) {
    q = hi;
    rest = lo;
  } else {
    const uint32_t s = shift - 64;
    q = s < 64 ? hi >> s : 0;
    rest = lo | (s < 64 ? hi << (64 - s) : hi);
  }
  *floor_ = q;
  *ceil_ = q + (rest != 0);
}

// The weight that the beginning has to stay below: an entry stays if the sum
// before it is less than this (1: the first entry only).
__device__ __forceinline__ uint64_t limit_of(float p, uint64_t w) {
  if (p >= 1.f) return ~uint64_t(0);
  if (!(p > 0.f)) return 1;
  uint64_t f, c;
  scaled(p, w, &f, &c);
  return c ? c : 1;
}

// *to, shared and no less than 0, becomes the most of all threads' x.  One lane of
// a wave takes part for all: as atomics of whole waves, one for each of a thread's
// bins, this took two thirds of k_sample_plan (16.5 us, now 5.2).
__device__ __forceinline__ void raise_to(uint32_t* to, uint32_t x) {
#pragma unroll
  for (uint32_t d = 32; d; d /= 2) x = max(x, (uint32_t)__shfl_xor((int)x, d));
  if (threadIdx.x % 64 == 0 && x) atomicMax(to, x);
}

__device__ __forceinline__ float row_max(const SampleArgs& a, uint64_t r) {
  float m = -INFINITY;
  for (uint32_t i = threadIdx.x % 64; i < a.chunks; i += 64) m = fmaxf(m, a.maxima[r * a.chunks + i]);
  return wave_top(m);
}

// A row whose k is at most this gets its first k by way of its groups.  Where k
// of G groups reach a bin, about n (1 - (1 - k / G)^(1 / GROUP)) entries do: 1.15
// k for a quarter of the groups, a twelfth of the row for three quarters.  So
// many are compared each with each, if they are at most PAIRS.
__host__ __device__ __forceinline__ int64_t small_limit(int64_t n) {
  if (n <= (int64_t)PAIRS) return n;
  const int64_t k = n < 12 * (int64_t)PAIRS ? 3 * n / (4 * GROUP) : n / (4 * GROUP);
  return k < (int64_t)SMALL_K ? k : (int64_t)SMALL_K;
}

// How many of a row's first entries are looked at, where that is a small number
// (of a short row with top_p all of them); 0: it is not, or there is no cut.
__device__ __forceinline__ uint32_t small_k(const SampleArgs& a, uint64_t r) {
  if (!a.groups) return 0;
  if (!(temperature_of(a, r) > 0.f)) return 1;
  const int64_t k = a.top_ks ? a.top_ks[r] : a.top_k;
  if (k > 0 && k <= small_limit(a.n)) return (uint32_t)k;
  return a.n <= PAIRS && !(top_p_of(a, r) >= 1.f) ? a.n : 0u;
}

// TILE logits from i0 on, whole vectors to a thread; -inf behind `end`.  (NaN is
// not live, and no maximum.)
template <class T, uint32_t THREADS>
struct Tile {
  static constexpr uint32_t VEC = Vec<T>::N, PER = TILE / THREADS, VECS = PER / VEC;
  static_assert(VECS * VEC == PER, "whole vectors");
  float z[PER];
  __device__ __forceinline__ static uint32_t index(uint32_t i0, uint32_t j) {
    return i0 + (j / VEC * THREADS + threadIdx.x) * VEC + j % VEC;
  }
  __device__ __forceinline__ void load(const T* row, uint32_t i0, uint32_t end) {
    if (i0 + TILE <= end) {
#pragma unroll
      for (uint32_t v = 0; v < VECS; ++v) Vec<T>::load(row + index(i0, v * VEC), z + v * VEC);
    } else {
#pragma unroll
      for (uint32_t j = 0; j < PER; ++j) {
        const uint32_t i = index(i0, j);
        z[j] = i < end ? to_f32(row[i]) : -INFINITY;
      }
    }
  }
};

// The first bin at which the counts reach k, or the last one; all threads get it.
template <uint32_t THREADS>
__device__ __forceinline__ uint32_t bin_reaching(const uint32_t* count, uint32_t k, uint32_t* part, uint32_t* found) {
  constexpr uint32_t PER = BINS / THREADS;
  if (threadIdx.x == 0) *found = BINS - 1;
  uint32_t c[PER], sum = 0, all;
#pragma unroll
  for (uint32_t i = 0; i < PER; ++i) sum += c[i] = count[threadIdx.x * PER + i];
  uint32_t at = thread_scan<THREADS>(sum, part, &all);
  if (at < k && k <= at + sum) {
#pragma unroll
    for (uint32_t i = 0; i < PER; ++i) {
      if (at < k && k <= at + c[i]) *found = threadIdx.x * PER + i;
      at += c[i];
    }
  }
  __syncthreads();
  return *found;
}

template <class T>
__global__ __launch_bounds__(FIRST_THREADS) void k_sample_first(SampleArgs a) {
  __shared__ float part[FIRST_THREADS / 64];
  const uint64_t id = block_id();
  if (id >= a.work) return;
  const uint64_t r = id / a.chunks;
  const uint32_t c = (uint32_t)(id - r * a.chunks);
  const T* row = static_cast<const T*>(a.logits) + r * a.ld;
  const uint32_t i0 = c * a.chunk, i1 = min(i0 + a.chunk, a.n);
  Tile<T, FIRST_THREADS> tile;
  tile.load(row, i0, i1);
  const bool bins = a.bin_count && !small_k(a, r);
  float m = -INFINITY;
  for (uint32_t at = i0;;) {
#pragma unroll
    for (uint32_t j = 0; j < GROUP; ++j) m = fmaxf(m, tile.z[j]);
    at += TILE;
    if (at >= i1) break;
    tile.load(row, at, i1);
  }
  if (a.groups) a.groups[id * FIRST_THREADS + threadIdx.x] = m;   // one tile is the whole chunk here
  m = wave_top(m);
  if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = m;
  if (bins)   // the chunks of a row share the clearing of its bins
    for (uint32_t i = c * FIRST_THREADS + threadIdx.x; i < BINS; i += a.chunks * FIRST_THREADS) {
      a.bin_count[r * BINS + i] = 0;
      a.bin_sum[r * BINS + i] = 0;
    }
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (uint32_t w = 1; w < FIRST_THREADS / 64; ++w) m = fmaxf(m, part[w]);
    a.maxima[id] = m;
    if (c == 0) {
      a.settings[r] = make_settings(a, r);
      if (a.collected) a.collected[r] = 0;
    }
  }
}

// A workgroup for each row.  (Found by every chunk's workgroup for itself, it
// took most of k_sample_collect: 153 rows of 78201 109 us.)
__global__ __launch_bounds__(ROW_THREADS) void k_sample_plan(SampleArgs a) {
  __shared__ uint64_t w_before[BINS + 1];
  __shared__ uint32_t c_before[BINS + 1];
  __shared__ uint32_t part32[ROW_WAVES], mark[3];
  __shared__ uint64_t part64[ROW_WAVES];
  const uint64_t r = block_id();
  if (r >= a.work || small_k(a, r)) return;
  constexpr uint32_t PER = BINS / ROW_THREADS;
  const uint32_t t = threadIdx.x;
  uint32_t c[PER], call;
  uint64_t w[PER], wall;
  uint32_t cs = 0;
  uint64_t ws = 0;
  int64_t k = a.top_ks ? a.top_ks[r] : a.top_k;
  if (!(temperature_of(a, r) > 0.f)) k = 1;
#pragma unroll
  for (uint32_t i = 0; i < PER; ++i) {
    ws += w[i] = a.bin_sum[r * BINS + t * PER + i];
    cs += c[i] = k > 0 ? a.bin_count[r * BINS + t * PER + i] : w[i] != 0;   // without top_k only whether there are any counts
  }
  uint32_t cb = thread_scan<ROW_THREADS>(cs, part32, &call);
  uint64_t wb = thread_scan<ROW_THREADS>(ws, part64, &wall);
#pragma unroll
  for (uint32_t i = 0; i < PER; ++i) {
    c_before[t * PER + i] = cb;
    w_before[t * PER + i] = wb;
    cb += c[i];
    wb += w[i];
  }
  uint32_t &bk = mark[0], &lo = mark[1], &hi = mark[2];
  if (t == 0) {
    c_before[BINS] = call;
    w_before[BINS] = wall;
    bk = BINS;
    lo = hi = 0;
  }
  __syncthreads();
  const bool cut_k = k > 0 && k < (int64_t)call;
  if (cut_k) {
#pragma unroll
    for (uint32_t i = 0; i < PER; ++i)
      if (c_before[t * PER + i] < (uint64_t)k && (uint64_t)k <= c_before[t * PER + i + 1]) bk = t * PER + i;
  }
  __syncthreads();
  const float p = top_p_of(a, r);
  const bool cut_p = !(p >= 1.f);
  if (cut_p) {
    // the last bin with an entry whose preceding weight is below the limit, for
    // the least and the most weight that top_k can leave
    const uint64_t l0 = limit_of(p, bk < BINS ? w_before[bk] : wall), l1 = limit_of(p, bk < BINS ? w_before[bk + 1] : wall);
    uint32_t x = 0, y = 0;
#pragma unroll
    for (uint32_t i = 0; i < PER; ++i) {
      if (c[i] && w_before[t * PER + i] < l0) x = t * PER + i;
      if (c[i] && w_before[t * PER + i] < l1) y = t * PER + i;
    }
    raise_to(&lo, x);
    raise_to(&hi, y);
  } else if (t == 0) {
    lo = hi = bk;
  }
  __syncthreads();
  SampleRow v;
  v.cut = cut_k || cut_p;
  const uint32_t last = bk < BINS ? max(hi, bk) : hi;
  const bool few = v.cut && k > 0 && c_before[min(last, BINS - 1) + 1] <= PAIRS;   // few entries: all that can stay
  v.inside = few;
  v.lo = few ? 0 : lo;
  v.hi = few ? last : hi;
  v.bk = bk;
  v.before = w_before[v.lo];
  v.count = c_before[v.lo];
  v.before_k = bk < BINS ? w_before[bk] : wall;
  v.count_k = bk < BINS ? c_before[bk] : call;
  v.k = cut_k ? (uint32_t)k : 0u;
  if (t == 0) a.row[r] = v;
}

template <class T>
__global__ __launch_bounds__(ROW_THREADS) void k_sample_bins(SampleArgs a) {
  __shared__ uint64_t sum[BINS];
  __shared__ uint32_t count[BINS];
  const uint64_t id = block_id();
  if (id >= a.work) return;
  const uint64_t r = id / a.chunks;
  const uint32_t c = (uint32_t)(id - r * a.chunks);
  if (small_k(a, r)) return;
  const Settings s = a.settings[r];
  const T* row = static_cast<const T*>(a.logits) + r * a.ld;
  const uint32_t i0 = c * a.chunk, i1 = min(i0 + a.chunk, a.n);
  Tile<T, ROW_THREADS> tile;
  tile.load(row, i0, i1);
  for (uint32_t i = threadIdx.x; i < BINS; i += ROW_THREADS) sum[i] = count[i] = 0;
  const float m = row_max(a, r);
  const bool counted = (a.top_ks ? a.top_ks[r] : a.top_k) > 0 || s.greedy;
  __syncthreads();
  for (uint32_t at = i0;;) {
#pragma unroll
    for (uint32_t j = 0; j < tile.PER; ++j) {
      const float z = tile.z[j];
      if (!live(z, m)) continue;
      const uint32_t b = bin_of(z, m);
      if (counted) atomicAdd(&count[b], 1u);
      const uint64_t w = fixed_of(weight_of(z, m, s), a.bits);
      if (w) atomicAdd(reinterpret_cast<unsigned long long*>(&sum[b]), (unsigned long long)w);
    }
    at += TILE;
    if (at >= i1) break;
    tile.load(row, at, i1);
  }
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < BINS; i += ROW_THREADS) {
    if (count[i]) atomicAdd(&a.bin_count[r * BINS + i], count[i]);
    if (sum[i]) atomicAdd(reinterpret_cast<unsigned long long*>(&a.bin_sum[r * BINS + i]), (unsigned long long)sum[i]);
  }
}

// Of a row without a cut, every bin is before it.  CUT: some row has one.
//
// The logits that surely stay and whose weight counts are listed first and then
// looked at by consecutive threads: few do, and a weight takes a wave the same
// time for one of them as for 64.
template <class T, bool CUT>
__global__ __launch_bounds__(ROW_THREADS) void k_sample_collect(SampleArgs a) {
  __shared__ uint64_t code[CUT ? TILE : 1];   // entries to be handed on
  __shared__ float listed[TILE];
  __shared__ uint32_t part32[ROW_WAVES], base;
  __shared__ uint64_t part64[ROW_WAVES];
  const uint64_t id = block_id();
  if (id >= a.work) return;
  const uint64_t r = id / a.chunks;
  const uint32_t c = (uint32_t)(id - r * a.chunks);
  if (small_k(a, r)) return;
  const Settings s = a.settings[r];
  const T* row = static_cast<const T*>(a.logits) + r * a.ld;
  const uint32_t i0 = c * a.chunk, i1 = min(i0 + a.chunk, a.n);
  Tile<T, ROW_THREADS> tile;
  tile.load(row, i0, i1);
  const float m = row_max(a, r);
  SampleRow v;
  v.cut = 0;
  v.lo = v.hi = v.bk = BINS;
  if constexpr (CUT) v = a.row[r];
  const float near = v.lo ? bin_end(v.lo - 1) : 0.f;   // logits nearer to the maximum than this lie in bins before lo
  const double min_p = min_p_of(a, r);
  uint64_t sum = 0;
  for (uint32_t at = i0;;) {
    uint32_t sure = 0, cand = 0, all;   // a bit for each of this thread's logits
#pragma unroll
    for (uint32_t j = 0; j < tile.PER; ++j) {
      const float z = tile.z[j];
      bool in = !(m - z > s.far) && z > -INFINITY;
      if constexpr (CUT) in = in && (!v.cut || (z == m ? v.lo > 0 : m - z < near));
      sure |= in ? 1u << j : 0u;
      if constexpr (CUT) {
        const uint32_t b = bin_of(z, m);
        cand |= v.cut && live(z, m) && b >= v.lo && (b <= v.hi || b == v.bk) ? 1u << j : 0u;
      }
    }
    // places of both, in the halves of one sum (a tile has 4096)
    const uint32_t place = thread_scan<ROW_THREADS>((uint32_t)__popc(sure) | (uint32_t)__popc(cand) << 16, part32, &all);
    uint32_t to = place & 0xFFFF, hand = place >> 16;
#pragma unroll
    for (uint32_t j = 0; j < tile.PER; ++j) {
      if (sure >> j & 1) listed[to++] = tile.z[j];
      if constexpr (CUT)
        if (cand >> j & 1) code[hand++] = code_of(tile.z[j], tile.index(at, j));
    }
    const uint32_t sures = all & 0xFFFF, cands = all >> 16;
    if (CUT && cands && threadIdx.x == 0) base = atomicAdd(&a.collected[r], cands);
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < sures; i += ROW_THREADS) {
      const double w = weight_of(listed[i], m, s);
      if (w >= min_p) sum += fixed_of(w, a.bits);
    }
    if constexpr (CUT)
      for (uint32_t i = threadIdx.x; i < cands; i += ROW_THREADS)
        if (base + i < CAP) a.cand[r * CAP + base + i] = code[i];
    at += TILE;
    if (at >= i1) break;
    tile.load(row, at, i1);
    __syncthreads();
  }
  sum = wave_total(sum);
  if (threadIdx.x % 64 == 0) part64[threadIdx.x / 64] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (uint32_t w = 1; w < ROW_WAVES; ++w) sum += part64[w];
    a.sums[id] = sum;
  }
}

// The cut of a row whose entries around it are more than CAP (many equal
// logits): radix selection over the whole row, by one workgroup.  `allowed`:
// only codes from there on count.  by_count: the entry of rank `want` - 1;
// otherwise the last entry with less than `want` weight before it.
template <class T>
__device__ uint64_t select_code(const SampleArgs& a, const T* row, float m, const Settings& s,
                                uint64_t allowed, bool by_count, uint64_t want, uint64_t* hist, uint64_t* found) {
  uint64_t prefix = 0, base = 0;
  const uint32_t t = threadIdx.x;
  for (int shift = 56; shift >= 0; shift -= 8) {
    if (shift == 24 || (shift == 16 && a.n <= 1u << 16)) {   // a digit that all indices have: n is at most 2^24
      prefix |= uint64_t(255) << shift;
      continue;
    }
    if (t < 256) hist[t] = 0;
    __syncthreads();
    for (uint32_t i = t; i < a.n; i += ROW_THREADS) {
      const float z = logit_of(row, i);
      if (!live(z, m)) continue;
      const uint64_t c = code_of(z, i);
      if (c < allowed || (shift < 56 && (c ^ prefix) >> (shift + 8))) continue;
      const uint64_t w = by_count ? 1 : fixed_of(weight_of(z, m, s), a.bits);
      if (w) atomicAdd(reinterpret_cast<unsigned long long*>(&hist[c >> shift & 255]), (unsigned long long)w);
    }
    __syncthreads();
    if (t == 0) {   // from the largest digit down: the last bin that begins below `want`
      uint64_t at = base;
      uint32_t best = 0;
      uint64_t best_at = base;
      for (int i = 255; i >= 0; --i) {
        if (!hist[i]) continue;
        if (at < want) {
          best = (uint32_t)i;
          best_at = at;
        }
        at += hist[i];
      }
      found[0] = prefix | (uint64_t)best << shift;
      found[1] = best_at;
    }
    __syncthreads();
    prefix = found[0];
    base = found[1];
    __syncthreads();
  }
  return prefix;
}

// Sum of the weights that stay in entries [i0, i1), by a wave.
template <class T>
__device__ __forceinline__ uint64_t staying(const SampleArgs& a, const T* row, uint32_t i0, uint32_t i1, float m, const Settings& s,
                                            double min_p, uint64_t cut) {
  uint64_t sum = 0;
  for (uint32_t i = i0 + threadIdx.x % 64; i < i1; i += 64) {
    const float z = logit_of(row, i);
    if (!live(z, m) || code_of(z, i) < cut) continue;
    const double w = weight_of(z, m, s);
    if (w >= min_p) sum += fixed_of(w, a.bits);
  }
  return wave_total(sum);
}

// What a workgroup that ends a row keeps in LDS.
struct alignas(16) RowShared {
  uint64_t code[CAP];
  uint64_t sorted[PAIRS], pair[PAIRS];
  uint64_t sums[MAX_CHUNKS];   // weight that stays, by chunk
  uint64_t part64[ROW_WAVES], found[2], rest;
  uint32_t count[BINS];
  uint32_t part32[ROW_WAVES], pick;
};

// A token of weight w, the whole in fixed point; -1: none.  The weight counts as it
// is, not as the multiple that it is drawn by: of a rare token's that has few bits.
__device__ __forceinline__ void write_token(const SampleArgs& a, uint64_t r, int64_t token, double w, uint64_t all) {
  a.tokens[r] = token;
  a.logprobs[r] = token < 0 ? -INFINITY : (float)log(ldexp(w, (int)a.bits) / (double)all);
}

// Each of the n <= PAIRS threads' value: the sum over all j < n of what `take`
// says of l.code[j], l.sorted[j].  All threads share the pairs; one holds two
// rows of them, which halves what is read from LDS.
template <class F>
__device__ __forceinline__ uint64_t over_pairs(RowShared& l, uint32_t n, F take) {
  constexpr uint32_t AHEAD = 8;
  const uint32_t t = threadIdx.x;
  uint32_t shift = 0;      // half the entries, rounded up to a power of two, 1 << shift
  while ((2u << shift) < n) ++shift;
  const uint32_t half = 1u << shift, i = t & (half - 1), parts = ROW_THREADS >> shift, part = t >> shift;
  const uint32_t end = (n + AHEAD - 1) / AHEAD * AHEAD;     // zeros from n on
  const uint32_t per = (end / AHEAD + parts - 1) / parts * AHEAD, j0 = part * per, j1 = min(j0 + per, end);
  if (t < PAIRS) l.pair[t] = 0;
  if (n + t < end) l.code[n + t] = l.sorted[n + t] = 0;
  __syncthreads();
  const bool low = i < n, high = i + half < n;
  if (low) {
    const uint64_t own0 = l.code[i], own1 = l.code[high ? i + half : i];
    uint64_t sum0 = 0, sum1 = 0;
    for (uint32_t j = j0; j < j1; j += AHEAD) {
      uint64_t c[AHEAD], w[AHEAD];
#pragma unroll
      for (uint32_t x = 0; x < AHEAD; ++x) {
        c[x] = l.code[j + x];
        w[x] = l.sorted[j + x];
      }
#pragma unroll
      for (uint32_t x = 0; x < AHEAD; ++x) {
        sum0 += take(own0, c[x], w[x]);
        sum1 += take(own1, c[x], w[x]);
      }
    }
    if (sum0) atomicAdd(reinterpret_cast<unsigned long long*>(&l.pair[i]), (unsigned long long)sum0);
    if (high && sum1) atomicAdd(reinterpret_cast<unsigned long long*>(&l.pair[i + half]), (unsigned long long)sum1);
  }
  __syncthreads();
  return t < n ? l.pair[t] : 0;
}

// The n entries of l.code in order, the first ones first.
__device__ __forceinline__ void sort_codes(RowShared& l, uint32_t n) {
  const uint32_t t = threadIdx.x;
  if (n <= PAIRS) {   // an entry's place is the number of larger ones
    const uint64_t place = over_pairs(l, n, [](uint64_t own, uint64_t c, uint64_t) { return (uint64_t)(c > own); });
    if (t < n) l.sorted[place] = l.code[t];
    __syncthreads();
    if (t < n) l.code[t] = l.sorted[t];
    __syncthreads();
    return;
  }
  uint32_t size = 2 * PAIRS;
  while (size < n) size *= 2;
  for (uint32_t i = n + t; i < size; i += ROW_THREADS) l.code[i] = 0;
  __syncthreads();
  for (uint32_t len = 2; len <= size; len *= 2)
    for (uint32_t step = len / 2; step; step /= 2) {
      for (uint32_t i = t; i < size / 2; i += ROW_THREADS) {
        const uint32_t x = (i & ~(step - 1)) * 2 + (i & (step - 1)), y = x + step;
        const uint64_t cx = l.code[x], cy = l.code[y];
        if ((cx < cy) == ((x & len) == 0)) {   // falling
          l.code[x] = cy;
          l.code[y] = cx;
        }
      }
      __syncthreads();
    }
}

// floor(u * all), of a u outside [0, 1) its end.
__device__ __forceinline__ uint64_t target_of(float u, uint64_t all) {
  if (!(u < 1.f)) return all - 1;
  if (!(u > 0.f)) return 0;
  uint64_t target, up;
  scaled(u, all, &target, &up);
  return target;
}

// The end of a row all of whose entries that can stay are in l.code, at most
// PAIRS, one to a thread: sorted, cut, and the token found from each entry's sum
// over those of lower index.
__device__ void finish_few(const SampleArgs& a, uint64_t r, float m, const Settings& s, const SampleRow& v, uint32_t n, float p,
                           double min_p, float u, RowShared& l) {
  const uint32_t t = threadIdx.x;
  sort_codes(l, n);
  const uint64_t code = t < n ? l.code[t] : 0;
  const double f = t < n ? weight_of(logit_of_code(code), m, s) : 0.0;
  const uint64_t w = fixed_of(f, a.bits);
  uint64_t all;
  const uint64_t before = thread_scan<ROW_THREADS>(w, l.part64, &all);
  if (t == 0) l.found[0] = all;
  __syncthreads();
  if (v.k && t == v.k) l.found[0] = before;   // the sum of the first k
  __syncthreads();
  const bool in = t < n && !(v.k && t >= v.k) && before < limit_of(p, v.k ? l.found[0] : v.before_k);
  const uint64_t mine = in && f >= min_p ? w : 0;
  if (t < PAIRS) l.sorted[t] = mine;
  thread_scan<ROW_THREADS>(mine, l.part64, &all);   // waits for l.sorted as well
  if (all == 0) {      // a min_p of NaN: nothing stays
    if (t == 0) write_token(a, r, -1, 0.0, 1);
    return;
  }
  const uint64_t target = target_of(u, all);
  const uint64_t lower = over_pairs(l, n, [](uint64_t own, uint64_t c, uint64_t x) { return ~(uint32_t)c < ~(uint32_t)own ? x : 0; });
  if (mine && lower <= target && target < lower + mine) write_token(a, r, ~(uint32_t)code, f, all);
}

// The end of a row.  n_cand entries around the cut are in l.code (more than
// CAP: they are not, and the whole row is gone through again); `inside`: all
// that can stay is among them, and the chunks' sums are 0.
template <class T>
__device__ void finish_row(const SampleArgs& a, uint64_t r, const T* row, float m, const Settings& s, const SampleRow& v,
                           uint32_t n_cand, bool inside, RowShared& l) {
  const uint32_t t = threadIdx.x;
  const double min_p = min_p_of(a, r);
  const float u = a.u[r];
  uint64_t cut = 0;
  bool whole = false;       // the chunks' sums have to be taken anew
  uint32_t staying_cands = 0;
  if (v.cut) {
    const float p = top_p_of(a, r);
    if (inside && n_cand <= PAIRS) {
      finish_few(a, r, m, s, v, n_cand, p, min_p, u, l);
      return;
    }
    if (n_cand <= CAP) {
      sort_codes(l, n_cand);
      // consecutive entries to a thread: their weights' sums, and where the k-th is
      const uint32_t per = (n_cand + ROW_THREADS - 1) / ROW_THREADS;
      const uint32_t x0 = min(t * per, n_cand), x1 = min(x0 + per, n_cand);
      uint64_t own = 0, all;
      uint32_t low = 0;     // entries of bins up to hi: before those of a bin bk beyond
      for (uint32_t x = x0; x < x1; ++x) {
        const float z = logit_of_code(l.code[x]);
        own += fixed_of(weight_of(z, m, s), a.bits);
        low += bin_of(z, m) <= v.hi;
      }
      const uint64_t at = thread_scan<ROW_THREADS>(own, l.part64, &all);
      uint32_t lows;
      thread_scan<ROW_THREADS>(low, l.part32, &lows);
      const bool apart = v.bk < BINS && v.bk > v.hi;   // bin bk does not follow on the others
      // where bk's entries begin in the list, and where the k-th ends
      const uint32_t bk_at = v.bk >= BINS ? 0u : apart ? lows : v.count_k - v.count;
      const uint32_t k_at = v.bk >= BINS ? 0u : bk_at + (v.k - v.count_k);
      if (t == 0) {
        l.found[0] = l.found[1] = all;
        l.pick = 0;
      }
      __syncthreads();
      uint64_t run = at;
      if (v.bk < BINS)
        for (uint32_t x = x0; x < x1; ++x) {
          if (x == bk_at) l.found[0] = run;
          if (x == k_at) l.found[1] = run;
          run += fixed_of(weight_of(logit_of_code(l.code[x]), m, s), a.bits);
        }
      __syncthreads();
      const uint64_t bk_start = l.found[0];
      const uint64_t sum_k = v.bk < BINS ? v.before_k + (l.found[1] - bk_start) : v.before_k;
      const uint64_t limit = limit_of(p, sum_k);
      run = at;
      uint32_t last = 0;
      for (uint32_t x = x0; x < x1; ++x) {
        const uint64_t before = apart && x >= lows ? v.before_k + (run - bk_start) : v.before + run;
        const bool in_k = v.bk >= BINS || x < k_at;
        if (in_k && before < limit) last = x;
        run += fixed_of(weight_of(logit_of_code(l.code[x]), m, s), a.bits);
      }
      raise_to(&l.pick, last);
      __syncthreads();
      staying_cands = l.pick + 1;
      cut = l.code[l.pick];
      __syncthreads();
    } else {
      if (v.bk < BINS) cut = select_code(a, row, m, s, 0, true, v.k, l.sums, l.found);
      if (!(p >= 1.f)) {
        uint64_t mine = 0, all;
        for (uint32_t c = t / 64; c < a.chunks; c += ROW_WAVES) {
          const uint32_t i0 = c * a.chunk;
          mine += staying(a, row, i0, min(i0 + a.chunk, a.n), m, s, -1.0, cut);
        }
        thread_scan<ROW_THREADS>(t % 64 ? uint64_t(0) : mine, l.part64, &all);
        cut = select_code(a, row, m, s, cut, false, limit_of(p, all), l.sums, l.found);
      }
      whole = true;
    }
  }
  // the chunks' sums, and the entries around the cut that stay
  if (whole) {
    for (uint32_t c = t / 64; c < a.chunks; c += ROW_WAVES) {
      const uint32_t i0 = c * a.chunk;
      const uint64_t sum = staying(a, row, i0, min(i0 + a.chunk, a.n), m, s, min_p, cut);
      if (t % 64 == 0) l.sums[c] = sum;
    }
  } else {
    for (uint32_t c = t; c < a.chunks; c += ROW_THREADS) l.sums[c] = inside ? 0 : a.sums[r * a.chunks + c];
    __syncthreads();
    for (uint32_t i = t; i < staying_cands; i += ROW_THREADS) {
      const uint64_t x = l.code[i];
      const double w = weight_of(logit_of_code(x), m, s);
      if (w >= min_p) atomicAdd(reinterpret_cast<unsigned long long*>(&l.sums[~(uint32_t)x / a.chunk]), (unsigned long long)fixed_of(w, a.bits));
    }
  }
  __syncthreads();
  constexpr uint32_t SUMS = MAX_CHUNKS / ROW_THREADS;
  uint64_t own[SUMS], mine = 0, all;
#pragma unroll
  for (uint32_t i = 0; i < SUMS; ++i) mine += own[i] = t * SUMS + i < a.chunks ? l.sums[t * SUMS + i] : 0;
  uint64_t before = thread_scan<ROW_THREADS>(mine, l.part64, &all);
  if (all == 0) {   // a min_p of NaN: nothing stays
    if (t == 0) write_token(a, r, -1, 0.0, 1);
    return;
  }
  const uint64_t target = target_of(u, all);
#pragma unroll
  for (uint32_t i = 0; i < SUMS; ++i) {
    if (before <= target && target < before + own[i]) {
      l.pick = t * SUMS + i;
      l.rest = target - before;
    }
    before += own[i];
  }
  __syncthreads();
  // that chunk, a tile at a time, consecutive entries to a thread
  const uint32_t i1 = min((l.pick + 1) * a.chunk, a.n);
  uint64_t rest = l.rest;
  constexpr uint32_t PER = TILE / ROW_THREADS;
  for (uint32_t i0 = l.pick * a.chunk; i0 < i1; i0 += TILE) {
    const uint32_t j0 = i0 + t * PER;
    float z[PER];
    if (j0 + PER <= i1) {
#pragma unroll
      for (uint32_t j = 0; j < PER; j += Vec<T>::N) Vec<T>::load(row + j0 + j, z + j);
    } else {
#pragma unroll
      for (uint32_t j = 0; j < PER; ++j) z[j] = j0 + j < i1 ? to_f32(row[j0 + j]) : -INFINITY;
    }
    uint64_t w[PER], sum = 0, tile_all;
#pragma unroll
    for (uint32_t j = 0; j < PER; ++j) {
      w[j] = 0;
      if (!(m - z[j] > s.far) && live(z[j], m) && code_of(z[j], j0 + j) >= cut) {
        const double f = weight_of(z[j], m, s);
        if (f >= min_p) w[j] = fixed_of(f, a.bits);
      }
      sum += w[j];
    }
    uint64_t run = thread_scan<ROW_THREADS>(sum, l.part64, &tile_all);
    if (rest < tile_all) {
      if (run <= rest && rest < run + sum) {
#pragma unroll
        for (uint32_t j = 0; j < PER; ++j) {
          if (run <= rest && rest < run + w[j]) write_token(a, r, j0 + j, weight_of(z[j], m, s), all);
          run += w[j];
        }
      }
      return;
    }
    rest -= tile_all;
  }
}

// A row with a small top_k: the bin that k groups reach, those groups, and
// their entries in the bins up to it.
template <class T>
__device__ void finish_small(const SampleArgs& a, uint64_t r, const T* row, float m, const Settings& s, uint32_t k, RowShared& l) {
  constexpr uint32_t VEC = Vec<T>::N, VECS = GROUP / VEC, AHEAD = 4;
  const uint32_t t = threadIdx.x;
  const uint32_t groups = a.chunks * FIRST_THREADS;      // a multiple of 256
  const float* tops = a.groups + r * groups;
  constexpr uint32_t BATCH = ROW_THREADS * 4 * AHEAD;
  f32x4 v[AHEAD];
  auto load = [&](uint32_t g0) {
#pragma unroll
    for (uint32_t i = 0; i < AHEAD; ++i) {
      v[i] = f32x4{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (g0 + i * ROW_THREADS * 4 < groups) v[i] = *reinterpret_cast<const f32x4*>(tops + g0 + i * ROW_THREADS * 4);
    }
  };
  load(t * 4);
  for (uint32_t i = t; i < BINS; i += ROW_THREADS) l.count[i] = 0;
  __syncthreads();
  for (uint32_t g0 = t * 4;;) {
#pragma unroll
    for (uint32_t i = 0; i < AHEAD; ++i)
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j)
        if (live(v[i][j], m)) atomicAdd(&l.count[bin_of(v[i][j], m)], 1u);
    g0 += BATCH;
    if (g0 >= groups) break;
    load(g0);
  }
  __syncthreads();
  const uint32_t last = bin_reaching<ROW_THREADS>(l.count, k, l.part32, &l.pick);
  // By half the distance: of finite logits it does not overflow, and it rounds as the whole does.
  const float half_below = 0.5f * bin_end(last), half_m = 0.5f * m;
  auto near = [&](float z) { return fmaf(-0.5f, z, half_m) < half_below || z == m; };   // m > -inf
  uint32_t* hits = reinterpret_cast<uint32_t*>(l.sums);           // 2 * MAX_CHUNKS of them
  uint32_t found = 0;
  for (uint32_t b0 = 0; b0 < groups; b0 += BATCH) {
    const uint32_t g0 = b0 + t * 4;
    if (groups > BATCH) load(g0);
    uint32_t mask = 0, all;
#pragma unroll
    for (uint32_t i = 0; i < AHEAD; ++i)
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j) mask |= near(v[i][j]) ? 1u << (i * 4 + j) : 0u;
    uint32_t at = found + thread_scan<ROW_THREADS>((uint32_t)__popc(mask), l.part32, &all);
    for (; mask; mask &= mask - 1, ++at) {
      const uint32_t x = __builtin_ctz(mask);
      if (at < 2 * MAX_CHUNKS) hits[at] = g0 + x / 4 * ROW_THREADS * 4 + x % 4;
    }
    found += all;
  }
  __syncthreads();
  uint32_t taken = 0;
  if (found <= 2 * MAX_CHUNKS) {
    for (uint32_t x0 = 0; x0 < found * VECS; x0 += ROW_THREADS) {
      const uint32_t x = x0 + t;
      const bool there = x < found * VECS;
      const uint32_t g = hits[there ? x / VECS : 0];
      const uint32_t i0 = g / FIRST_THREADS * TILE + (x % VECS * FIRST_THREADS + g % FIRST_THREADS) * VEC;
      float z[VEC];
      if (i0 + VEC <= a.n) {
        Vec<T>::load(row + i0, z);
      } else {
#pragma unroll
        for (uint32_t j = 0; j < VEC; ++j) z[j] = i0 + j < a.n ? to_f32(row[i0 + j]) : -INFINITY;
      }
      uint32_t mine = 0, all;
#pragma unroll
      for (uint32_t j = 0; j < VEC; ++j) mine += there && near(z[j]);
      uint32_t at = taken + thread_scan<ROW_THREADS>(mine, l.part32, &all);
#pragma unroll
      for (uint32_t j = 0; j < VEC; ++j)
        if (there && near(z[j])) {
          if (at < CAP) l.code[at] = code_of(z[j], i0 + j);
          ++at;
        }
      taken += all;
    }
  }
  __syncthreads();
  SampleRow w;
  w.cut = w.inside = 1;
  w.lo = w.count = w.count_k = 0;
  w.hi = w.bk = BINS - 1;      // the list is a beginning of the row's order
  w.before = w.before_k = 0;
  w.k = k;
  const uint32_t n = found <= 2 * MAX_CHUNKS ? taken : CAP + 1;
  __syncthreads();
  finish_row(a, r, row, m, s, w, n, true, l);
}

template <class T>
__global__ __launch_bounds__(ROW_THREADS) void k_sample_finish(SampleArgs a) {
  __shared__ RowShared l;
  const uint64_t r = block_id();
  if (r >= a.work) return;
  const T* row = static_cast<const T*>(a.logits) + r * a.ld;
  const Settings s = a.settings[r];
  const uint32_t k = small_k(a, r);
  const float m = row_max(a, r);
  if (m == -INFINITY) {
    if (threadIdx.x == 0) write_token(a, r, -1, 0.0, 1);
    return;
  }
  if (k) {
    finish_small(a, r, row, m, s, k, l);
    return;
  }
  SampleRow v;
  v.cut = 0;
  v.lo = BINS;
  uint32_t n = 0;
  if (a.row) v = a.row[r];
  if (v.cut) {
    n = a.collected[r];
    for (uint32_t i = threadIdx.x; i < min(n, CAP); i += ROW_THREADS) l.code[i] = a.cand[r * CAP + i];
    __syncthreads();
  }
  finish_row(a, r, row, m, s, v, n, v.cut && v.inside, l);
}

struct SamplePlan {
  uint32_t chunk = TILE, chunks = 0, bits = 62;
  bool cut = true;       // some row may have a cut that is not among a small number of its first entries
  bool small = false;    // some row may have one that is,
  bool all_small = false;// all rows have
  size_t off_max = 0, off_settings = 0, off_collected = 0, off_sums = 0, off_groups = 0, off_count = 0, off_bins = 0, off_cand = 0, off_row = 0,
         total = 0;
};

SamplePlan sample_plan(const topk_sample_args& a) {
  SamplePlan p;
  while (ceil_div(a.n, p.chunk) > MAX_CHUNKS) p.chunk *= 2;
  p.chunks = (uint32_t)ceil_div(a.n, p.chunk);
  while ((int64_t(1) << (62 - p.bits)) < a.n) --p.bits;
  // what the numbers among the settings say of all rows
  const bool tile = p.chunk == TILE, brief = a.n <= (int64_t)PAIRS;
  const bool greedy = !a.temperatures && !(a.temperature > 0.f);
  const bool nucleus = !a.top_ps && !(a.top_p >= 1.f);
  p.all_small = tile && (greedy || (!a.top_ks && a.top_k > 0 && a.top_k <= small_limit(a.n)) || (brief && nucleus));
  const bool cuts = a.top_ks || (a.top_k > 0 && a.top_k < a.n) || a.top_ps || nucleus;
  p.small = p.all_small || (tile && (a.top_ks || a.temperatures || (brief && cuts)));
  p.cut = !p.all_small && !brief && (cuts || (!tile && (greedy || a.temperatures)));
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  const size_t rows = (size_t)a.rows;
  p.off_max = take(rows * p.chunks * 4);
  p.off_settings = take(rows * sizeof(Settings));
  p.off_sums = take(rows * p.chunks * 8);
  if (p.small) p.off_groups = take(rows * p.chunks * FIRST_THREADS * 4);
  if (p.cut) {
    p.off_count = take(rows * BINS * 4);
    p.off_bins = take(rows * BINS * 8);
    p.off_cand = take(rows * CAP * 8);
    p.off_collected = take(rows * 4);
    p.off_row = take(rows * sizeof(SampleRow));
  }
  p.total = at;
  return p;
}

template <class T>
hipError_t sample_call(SampleArgs a, const SamplePlan& p, uint64_t rows, hipStream_t s) {
  a.work = rows * p.chunks;
  const dim3 chunks = wide_grid(a.work);
  k_sample_first<T><<<chunks, FIRST_THREADS, 0, s>>>(a);
  SampleArgs by_row = a;
  by_row.work = rows;
  if (p.cut) {
    k_sample_bins<T><<<chunks, ROW_THREADS, 0, s>>>(a);
    k_sample_plan<<<wide_grid(rows), ROW_THREADS, 0, s>>>(by_row);
    k_sample_collect<T, true><<<chunks, ROW_THREADS, 0, s>>>(a);
  } else if (!p.all_small) {
    k_sample_collect<T, false><<<chunks, ROW_THREADS, 0, s>>>(a);
  }
  k_sample_finish<T><<<wide_grid(rows), ROW_THREADS, 0, s>>>(by_row);
  return hipGetLastError();
}

}  // namespace

size_t sample_workspace(const topk_sample_args& a) { return a.rows ? sample_plan(a).total : 0; }

hipError_t launch_sample(const topk_sample_args& in, void* ws, hipStream_t s) {
  if (!in.rows) return hipSuccess;
  const SamplePlan p = sample_plan(in);
  char* w = static_cast<char*>(ws);
  SampleArgs a;
  a.logits = in.logits, a.u = in.u, a.tokens = in.tokens, a.logprobs = in.logprobs;
  a.temperatures = in.temperatures, a.top_ks = in.top_ks, a.top_ps = in.top_ps, a.min_ps = in.min_ps;
  a.maxima = reinterpret_cast<float*>(w + p.off_max);
  a.settings = reinterpret_cast<Settings*>(w + p.off_settings);
  a.collected = p.cut ? reinterpret_cast<uint32_t*>(w + p.off_collected) : nullptr;
  a.sums = reinterpret_cast<uint64_t*>(w + p.off_sums);
  a.groups = p.small ? reinterpret_cast<float*>(w + p.off_groups) : nullptr;
  a.bin_count = p.cut ? reinterpret_cast<uint32_t*>(w + p.off_count) : nullptr;
  a.bin_sum = p.cut ? reinterpret_cast<uint64_t*>(w + p.off_bins) : nullptr;
  a.cand = p.cut ? reinterpret_cast<uint64_t*>(w + p.off_cand) : nullptr;
  a.row = p.cut ? reinterpret_cast<SampleRow*>(w + p.off_row) : nullptr;
  a.ld = (uint64_t)in.ld;
  a.top_k = in.top_k;
  a.temperature = in.temperature, a.top_p = in.top_p, a.min_p = in.min_p;
  a.n = (uint32_t)in.n;
  a.chunk = p.chunk, a.chunks = p.chunks, a.bits = p.bits;
  return in.dtype == TOPK_BF16 ? sample_call<bf16_t>(a, p, (uint64_t)in.rows, s) : sample_call<float>(a, p, (uint64_t)in.rows, s);
}

}  // namespace tk
