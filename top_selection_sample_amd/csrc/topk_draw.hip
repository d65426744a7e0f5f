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
// exponential is a table of 64 powers and a polynomial in 64-bit floats, off
// by less than 2^-50 of its value.
//
// top_k and top_p keep a beginning of the one order, so together they are one
// cut: a logit and an index.  A row is cut into chunks, a workgroup each:
//
//   k_sample_max      the chunks' maxima
//   k_sample_hist     counts and sums of weights by bins of m - z (its float's
//                     leading bits: 128 bins to an octave)
//   k_sample_plan     from those the bins that the cut can lie in
//   k_sample_collect  their entries, and each chunk's sum over the bins before
//   k_sample_finish   sorts the entries, finds the cut, then the chunk that the
//                     token lies in, then the token
//
// Without top_k and top_p there is no cut: k_sample_sum stands in the place of
// the middle three.
#include <algorithm>

#include "topk_model.hpp"
#include "topk_ops_device.hpp"

namespace tk {

namespace {

constexpr uint32_t CHUNK_THREADS = 256;
constexpr uint32_t ROW_THREADS = 1024;
constexpr uint32_t ROW_WAVES = ROW_THREADS / 64;
constexpr uint32_t MAX_CHUNKS = 1024;       // of a row
constexpr uint32_t BINS = 2048;             // 16 octaves of m - z from 2^-7 on, 128 to an octave
constexpr uint32_t FIRST_BIN = (127 - 7) << 7;
constexpr uint32_t CAP = 4096;              // entries of a row around its cut that are sorted

// What is known of a row between the launches.
struct SampleRow {
  uint64_t before;        // weight of the bins below `lo`
  uint64_t before_k;      // weight of the bins below `bk`
  uint32_t lo, hi, bk;    // entries of bins lo to hi, and of bin bk, are collected; bk: where the k-th is (BINS: top_k is off)
  uint32_t count, count_k;// entries of the bins below lo and bk
  uint32_t k;             // top_k, where bk says so
  uint32_t cut;           // whether there is a cut
  uint32_t collected;
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

// The settings of a row.
struct Settings {
  double rate;       // log2(e) / temperature
  bool greedy;
};

__device__ __forceinline__ Settings settings_of(const SampleArgs& a, uint64_t r) {
  const float t = a.temperatures ? a.temperatures[r] : a.temperature;
  Settings s;
  s.greedy = !(t > 0.f);
  s.rate = s.greedy ? 0.0 : 1.4426950408889634 / (double)t;
  return s;
}

__device__ __forceinline__ float top_p_of(const SampleArgs& a, uint64_t r) { return a.top_ps ? a.top_ps[r] : a.top_p; }
__device__ __forceinline__ double min_p_of(const SampleArgs& a, uint64_t r) {
  const float p = a.min_ps ? a.min_ps[r] : a.min_p;
  return p > 1.f ? 1.0 : (double)p;
}

template <class T>
__device__ __forceinline__ float logit_of(const T* row, uint32_t i) {
  const float z = to_f32(row[i]);
  return z != z ? -INFINITY : z;
}

// 2^(j / 64).
__device__ const double POWERS[64] = {
    0x1.0000000000000p+0, 0x1.02c9a3e778061p+0, 0x1.059b0d3158574p+0, 0x1.0874518759bc8p+0,
    0x1.0b5586cf9890fp+0, 0x1.0e3ec32d3d1a2p+0, 0x1.11301d0125b51p+0, 0x1.1429aaea92de0p+0,
    0x1.172b83c7d517bp+0, 0x1.1a35beb6fcb75p+0, 0x1.1d4873168b9aap+0, 0x1.2063b88628cd6p+0,
    0x1.2387a6e756238p+0, 0x1.26b4565e27cddp+0, 0x1.29e9df51fdee1p+0, 0x1.2d285a6e4030bp+0,
    0x1.306fe0a31b715p+0, 0x1.33c08b26416ffp+0, 0x1.371a7373aa9cbp+0, 0x1.3a7db34e59ff7p+0,
    0x1.3dea64c123422p+0, 0x1.4160a21f72e2ap+0, 0x1.44e086061892dp+0, 0x1.486a2b5c13cd0p+0,
    0x1.4bfdad5362a27p+0, 0x1.4f9b2769d2ca7p+0, 0x1.5342b569d4f82p+0, 0x1.56f4736b527dap+0,
    0x1.5ab07dd485429p+0, 0x1.5e76f15ad2148p+0, 0x1.6247eb03a5585p+0, 0x1.6623882552225p+0,
    0x1.6a09e667f3bcdp+0, 0x1.6dfb23c651a2fp+0, 0x1.71f75e8ec5f74p+0, 0x1.75feb564267c9p+0,
    0x1.7a11473eb0187p+0, 0x1.7e2f336cf4e62p+0, 0x1.82589994cce13p+0, 0x1.868d99b4492edp+0,
    0x1.8ace5422aa0dbp+0, 0x1.8f1ae99157736p+0, 0x1.93737b0cdc5e5p+0, 0x1.97d829fde4e50p+0,
    0x1.9c49182a3f090p+0, 0x1.a0c667b5de565p+0, 0x1.a5503b23e255dp+0, 0x1.a9e6b5579fdbfp+0,
    0x1.ae89f995ad3adp+0, 0x1.b33a2b84f15fbp+0, 0x1.b7f76f2fb5e47p+0, 0x1.bcc1e904bc1d2p+0,
    0x1.c199bdd85529cp+0, 0x1.c67f12e57d14bp+0, 0x1.cb720dcef9069p+0, 0x1.d072d4a07897cp+0,
    0x1.d5818dcfba487p+0, 0x1.da9e603db3285p+0, 0x1.dfc97337b9b5fp+0, 0x1.e502ee78b3ff6p+0,
    0x1.ea4afa2a490dap+0, 0x1.efa1bee615a27p+0, 0x1.f50765b6e4540p+0, 0x1.fa7c1819e90d8p+0};

__device__ __forceinline__ void load_powers(double* table) {
  if (threadIdx.x < 64) table[threadIdx.x] = POWERS[threadIdx.x];
  __syncthreads();
}

// The weight of a logit as a float, and in multiples of 2^-bits.  t = log2 of
// the weight is split into j / 64 and |f| <= 1/128; the polynomial of 2^f has
// the coefficients ln(2)^i / i!, and (f ln 2)^6 / 720 < 2^-54 is left out.
__device__ __forceinline__ double weight_of(float z, float m, const Settings& s, const double* table) {
  if (z == m) return 1.0;
  if (s.greedy) return 0.0;
  const double t = ((double)z - (double)m) * s.rate;
  if (!(t > -64.0)) return 0.0;   // below half of 2^-62
  const double q = rint(t * 64.0);
  const double f = fma(q, -0.015625, t);
  const int i = (int)q;
  double p = fma(f, 0.0013333558146428443, 0.0096181291076284772);
  p = fma(f, p, 0.055504108664821580);
  p = fma(f, p, 0.24022650695910071);
  p = fma(f, p, 0.69314718055994531);
  p = fma(f, p, 1.0);
  return ldexp(table[i & 63] * p, i >> 6);
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

__device__ __forceinline__ float row_max(const SampleArgs& a, uint64_t r) {
  float m = -INFINITY;
  for (uint32_t i = threadIdx.x % 64; i < a.chunks; i += 64) m = fmaxf(m, a.maxima[r * a.chunks + i]);
#pragma unroll
  for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  return m;
}

// Exclusive sums over the threads of a workgroup; *total: of all.
template <uint32_t THREADS, class V>
__device__ __forceinline__ V thread_scan(V v, V* part, V* total) {
  V up = v;
#pragma unroll
  for (uint32_t o = 1; o < 64; o <<= 1) {
    const V t = __shfl_up(up, o);
    if (threadIdx.x % 64 >= o) up += t;
  }
  if (threadIdx.x % 64 == 63) part[threadIdx.x / 64] = up;
  __syncthreads();
  V before = 0, all = 0;
  for (uint32_t w = 0; w < THREADS / 64; ++w) {
    if (w < threadIdx.x / 64) before += part[w];
    all += part[w];
  }
  __syncthreads();
  *total = all;
  return before + up - v;
}

template <class T>
__global__ __launch_bounds__(CHUNK_THREADS) void k_sample_max(SampleArgs a) {
  __shared__ float part[CHUNK_THREADS / 64];
  const uint64_t id = block_id();
  if (id >= a.work) return;
  const uint64_t r = id / a.chunks;
  const uint32_t c = (uint32_t)(id % a.chunks);
  const T* row = static_cast<const T*>(a.logits) + r * a.ld;
  const uint32_t i0 = c * a.chunk, i1 = min(i0 + a.chunk, a.n);
  float m = -INFINITY;
  for (uint32_t i = i0 + threadIdx.x; i < i1; i += CHUNK_THREADS) m = fmaxf(m, logit_of(row, i));
#pragma unroll
  for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (uint32_t w = 1; w < CHUNK_THREADS / 64; ++w) m = fmaxf(m, part[w]);
    a.maxima[id] = m;
  }
  if (a.bin_count) {   // the chunks of a row share the clearing of its bins
    for (uint32_t i = c * CHUNK_THREADS + threadIdx.x; i < BINS; i += a.chunks * CHUNK_THREADS) {
      a.bin_count[r * BINS + i] = 0;
      a.bin_sum[r * BINS + i] = 0;
    }
  }
}

template <class T>
__global__ __launch_bounds__(CHUNK_THREADS) void k_sample_hist(SampleArgs a) {
  __shared__ uint64_t sum[BINS];
  __shared__ uint32_t count[BINS];
  __shared__ double table[64];
  const uint64_t id = block_id();
  if (id >= a.work) return;
  const uint64_t r = id / a.chunks;
  const uint32_t c = (uint32_t)(id % a.chunks);
  const T* row = static_cast<const T*>(a.logits) + r * a.ld;
  for (uint32_t i = threadIdx.x; i < BINS; i += CHUNK_THREADS) sum[i] = count[i] = 0;
  load_powers(table);
  const float m = row_max(a, r);
  const Settings s = settings_of(a, r);
  const uint32_t i0 = c * a.chunk, i1 = min(i0 + a.chunk, a.n);
  for (uint32_t i = i0 + threadIdx.x; i < i1; i += CHUNK_THREADS) {
    const float z = logit_of(row, i);
    if (!live(z, m)) continue;
    const uint32_t b = bin_of(z, m);
    atomicAdd(&count[b], 1u);
    const uint64_t w = fixed_of(weight_of(z, m, s, table), a.bits);
    if (w) atomicAdd(reinterpret_cast<unsigned long long*>(&sum[b]), (unsigned long long)w);
  }
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < BINS; i += CHUNK_THREADS) {
    if (!count[i]) continue;
    atomicAdd(&a.bin_count[r * BINS + i], count[i]);
    if (sum[i]) atomicAdd(reinterpret_cast<unsigned long long*>(&a.bin_sum[r * BINS + i]), (unsigned long long)sum[i]);
  }
}

// Two bins to a thread.
__global__ __launch_bounds__(ROW_THREADS) void k_sample_plan(SampleArgs a) {
  __shared__ uint32_t part32[ROW_WAVES];
  __shared__ uint64_t part64[ROW_WAVES];
  __shared__ uint32_t c_before[BINS + 1];
  __shared__ uint64_t w_before[BINS + 1];
  __shared__ uint32_t bk, lo, hi;
  const uint64_t r = block_id();
  if (r >= a.work) return;
  const uint32_t t = threadIdx.x;
  const uint32_t* bc = a.bin_count + r * BINS;
  const uint64_t* bs = a.bin_sum + r * BINS;
  const uint32_t c0 = bc[2 * t], c1 = bc[2 * t + 1];
  const uint64_t s0 = bs[2 * t], s1 = bs[2 * t + 1];
  uint32_t call;
  uint64_t wall;
  const uint32_t cb = thread_scan<ROW_THREADS>(c0 + c1, part32, &call);
  const uint64_t wb = thread_scan<ROW_THREADS>(s0 + s1, part64, &wall);
  c_before[2 * t] = cb;
  c_before[2 * t + 1] = cb + c0;
  w_before[2 * t] = wb;
  w_before[2 * t + 1] = wb + s0;
  if (t == 0) {
    c_before[BINS] = call;
    w_before[BINS] = wall;
    bk = BINS;
    lo = hi = 0;
  }
  __syncthreads();
  const Settings s = settings_of(a, r);
  int64_t k = a.top_ks ? a.top_ks[r] : a.top_k;
  if (s.greedy) k = 1;
  const bool cut_k = k > 0 && k < (int64_t)call;
  if (cut_k) {
#pragma unroll
    for (uint32_t i = 0; i < 2; ++i)
      if (c_before[2 * t + i] < (uint64_t)k && (uint64_t)k <= c_before[2 * t + i + 1]) bk = 2 * t + i;
  }
  __syncthreads();
  const float p = top_p_of(a, r);
  const bool cut_p = !(p >= 1.f);
  const uint64_t least = bk < BINS ? w_before[bk] : wall, most = bk < BINS ? w_before[bk + 1] : wall;
  if (cut_p) {
    // the last bin with an entry whose preceding weight is below the limit
    const uint64_t l0 = limit_of(p, least), l1 = limit_of(p, most);
#pragma unroll
    for (uint32_t i = 0; i < 2; ++i) {
      if (!(i ? c1 : c0)) continue;
      if (w_before[2 * t + i] < l0) atomicMax(&lo, 2 * t + i);
      if (w_before[2 * t + i] < l1) atomicMax(&hi, 2 * t + i);
    }
  } else if (t == 0) {
    lo = hi = bk;
  }
  __syncthreads();
  if (t == 0) {
    SampleRow v;
    v.cut = cut_k || cut_p;
    const uint32_t last = bk < BINS ? max(hi, bk) : hi;
    uint32_t from = lo;
    if (v.cut && c_before[min(last, BINS - 1) + 1] <= CAP) from = 0, hi = last;   // few entries: all that can stay
    v.lo = from;
    v.hi = hi;
    v.bk = bk;
    v.before = w_before[from];
    v.count = c_before[from];
    v.before_k = bk < BINS ? w_before[bk] : wall;
    v.count_k = bk < BINS ? c_before[bk] : call;
    v.k = cut_k ? (uint32_t)k : 0u;
    v.collected = 0;
    a.row[r] = v;
  }
}

template <class T>
__global__ __launch_bounds__(CHUNK_THREADS) void k_sample_collect(SampleArgs a) {
  __shared__ double table[64];
  __shared__ uint64_t part[CHUNK_THREADS / 64];
  const uint64_t id = block_id();
  if (id >= a.work) return;
  const uint64_t r = id / a.chunks;
  const uint32_t c = (uint32_t)(id % a.chunks);
  const T* row = static_cast<const T*>(a.logits) + r * a.ld;
  load_powers(table);
  const float m = row_max(a, r);
  const Settings s = settings_of(a, r);
  const double min_p = min_p_of(a, r);
  const SampleRow v = a.row[r];
  const uint32_t i0 = c * a.chunk, i1 = min(i0 + a.chunk, a.n);
  uint64_t sum = 0;
  for (uint32_t i = i0 + threadIdx.x; i < i1; i += CHUNK_THREADS) {
    const float z = logit_of(row, i);
    if (!live(z, m)) continue;
    const uint32_t b = bin_of(z, m);
    if (!v.cut || b < v.lo) {
      const double w = weight_of(z, m, s, table);
      if (w >= min_p) sum += fixed_of(w, a.bits);
    } else if (b <= v.hi || b == v.bk) {
      const uint32_t at = atomicAdd(&a.row[r].collected, 1u);
      if (at < CAP) a.cand[r * CAP + at] = code_of(z, i);
    }
  }
  sum = wave_sum(sum);
  if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (uint32_t w = 1; w < CHUNK_THREADS / 64; ++w) sum += part[w];
    a.sums[id] = sum;
  }
}

// The middle of a call without a cut.
template <class T>
__global__ __launch_bounds__(CHUNK_THREADS) void k_sample_sum(SampleArgs a) {
  __shared__ double table[64];
  __shared__ uint64_t part[CHUNK_THREADS / 64];
  const uint64_t id = block_id();
  if (id >= a.work) return;
  const uint64_t r = id / a.chunks;
  const uint32_t c = (uint32_t)(id % a.chunks);
  const T* row = static_cast<const T*>(a.logits) + r * a.ld;
  load_powers(table);
  const float m = row_max(a, r);
  const Settings s = settings_of(a, r);
  const double min_p = min_p_of(a, r);
  const uint32_t i0 = c * a.chunk, i1 = min(i0 + a.chunk, a.n);
  uint64_t sum = 0;
  for (uint32_t i = i0 + threadIdx.x; i < i1; i += CHUNK_THREADS) {
    const float z = logit_of(row, i);
    if (!live(z, m)) continue;
    const double w = weight_of(z, m, s, table);
    if (w >= min_p) sum += fixed_of(w, a.bits);
  }
  sum = wave_sum(sum);
  if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (uint32_t w = 1; w < CHUNK_THREADS / 64; ++w) sum += part[w];
    a.sums[id] = sum;
  }
}

// The cut of a row whose entries around it are more than CAP (many equal
// logits): radix selection over the whole row, by one workgroup.  `allowed`:
// only codes from there on count.  by_count: the entry of rank `want` - 1;
// otherwise the last entry with less than `want` weight before it.
template <class T>
__device__ uint64_t select_code(const SampleArgs& a, const T* row, float m, const Settings& s, const double* table,
                                uint64_t allowed, bool by_count, uint64_t want, uint64_t* hist, uint64_t* found) {
  uint64_t prefix = 0, base = 0;
  const uint32_t t = threadIdx.x;
  for (int shift = 56; shift >= 0; shift -= 8) {
    if (t < 256) hist[t] = 0;
    __syncthreads();
    for (uint32_t i = t; i < a.n; i += ROW_THREADS) {
      const float z = logit_of(row, i);
      if (!live(z, m)) continue;
      const uint64_t c = code_of(z, i);
      if (c < allowed || (shift < 56 && (c ^ prefix) >> (shift + 8))) continue;
      const uint64_t w = by_count ? 1 : fixed_of(weight_of(z, m, s, table), a.bits);
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
                                            double min_p, uint64_t cut, const double* table) {
  uint64_t sum = 0;
  for (uint32_t i = i0 + threadIdx.x % 64; i < i1; i += 64) {
    const float z = logit_of(row, i);
    if (!live(z, m) || code_of(z, i) < cut) continue;
    const double w = weight_of(z, m, s, table);
    if (w >= min_p) sum += fixed_of(w, a.bits);
  }
  return wave_sum(sum);
}

template <class T>
__global__ __launch_bounds__(ROW_THREADS) void k_sample_finish(SampleArgs a) {
  __shared__ uint64_t code[CAP];
  __shared__ uint64_t sums[MAX_CHUNKS];
  __shared__ uint64_t part[ROW_WAVES], found[2];
  __shared__ double table[64];
  __shared__ uint32_t pick;
  __shared__ uint64_t rest;
  const uint64_t r = block_id();
  if (r >= a.work) return;
  const uint32_t t = threadIdx.x;
  const T* row = static_cast<const T*>(a.logits) + r * a.ld;
  load_powers(table);
  const float m = row_max(a, r);
  if (m == -INFINITY) {
    if (t == 0) {
      a.tokens[r] = -1;
      a.logprobs[r] = -INFINITY;
    }
    return;
  }
  const Settings s = settings_of(a, r);
  const double min_p = min_p_of(a, r);
  uint64_t cut = 0;
  bool whole = false;       // the chunks' sums have to be taken anew
  uint32_t n_cand = 0;
  SampleRow v;
  v.cut = 0;
  if (a.row) v = a.row[r];
  if (v.cut) {
    const float p = top_p_of(a, r);
    if (v.collected <= CAP) {
      n_cand = v.collected;
      uint32_t size = 64;
      while (size < n_cand) size *= 2;
      for (uint32_t i = t; i < size; i += ROW_THREADS) code[i] = i < n_cand ? a.cand[r * CAP + i] : 0;
      __syncthreads();
      for (uint32_t len = 2; len <= size; len *= 2)
        for (uint32_t step = len / 2; step; step /= 2) {
          for (uint32_t i = t; i < size / 2; i += ROW_THREADS) {
            const uint32_t x = (i & ~(step - 1)) * 2 + (i & (step - 1)), y = x + step;
            const uint64_t cx = code[x], cy = code[y];
            if ((cx < cy) == ((x & len) == 0)) {   // falling
              code[x] = cy;
              code[y] = cx;
            }
          }
          __syncthreads();
        }
      // CAP / ROW_THREADS entries to a thread: their weights' sums, and where the k-th is
      constexpr uint32_t PER = CAP / ROW_THREADS;
      uint64_t w[PER], own = 0, all;
      uint32_t low = 0;     // entries of bins up to hi: before those of a bin bk beyond
#pragma unroll
      for (uint32_t i = 0; i < PER; ++i) {
        const uint32_t x = t * PER + i;
        w[i] = 0;
        if (x < n_cand) {
          const float z = logit_of_code(code[x]);
          w[i] = fixed_of(weight_of(z, m, s, table), a.bits);
          low += bin_of(z, m) <= v.hi;
        }
        own += w[i];
      }
      const uint64_t at = thread_scan<ROW_THREADS>(own, part, &all);
      uint64_t lows;
      thread_scan<ROW_THREADS>((uint64_t)low, part, &lows);
      const bool apart = v.bk < BINS && v.bk > v.hi;   // bin bk does not follow on the others
      // sums of the list before an entry: of the first `lows` of bk's own, and up to the k-th
      const uint32_t bk_at = v.bk >= BINS ? 0u : apart ? (uint32_t)lows : v.count_k - v.count;
      const uint32_t k_at = v.bk >= BINS ? 0u : bk_at + (v.k - v.count_k);
      if (t == 0) found[0] = found[1] = all;
      __syncthreads();
      uint64_t run = at;
#pragma unroll
      for (uint32_t i = 0; i < PER; ++i) {
        const uint32_t x = t * PER + i;
        if (v.bk < BINS && x < n_cand) {
          if (x == bk_at) found[0] = run;
          if (x == k_at) found[1] = run;
        }
        run += w[i];
      }
      __syncthreads();
      const uint64_t sum_k = v.bk < BINS ? v.before_k + (found[1] - found[0]) : v.before_k;
      const uint64_t limit = limit_of(p, sum_k);
      const uint64_t bk_start = found[0];
      if (t == 0) pick = 0;
      __syncthreads();
      run = at;
#pragma unroll
      for (uint32_t i = 0; i < PER; ++i) {
        const uint32_t x = t * PER + i;
        if (x < n_cand) {
          const bool second = apart && x >= lows;
          const uint64_t before = second ? v.before_k + (run - bk_start) : v.before + run;
          const bool in_k = v.bk >= BINS || x < k_at;
          if (in_k && before < limit) atomicMax(&pick, x);
        }
        run += w[i];
      }
      __syncthreads();
      cut = code[pick];
      __syncthreads();
    } else {
      if (v.bk < BINS) {
        cut = select_code(a, row, m, s, table, 0, true, v.k, sums, found);
      }
      if (!(p >= 1.f)) {
        uint64_t mine = 0, all;
        for (uint32_t c = t / 64; c < a.chunks; c += ROW_WAVES) {
          const uint32_t i0 = c * a.chunk;
          mine += staying(a, row, i0, min(i0 + a.chunk, a.n), m, s, -1.0, cut, table);
        }
        thread_scan<ROW_THREADS>(t % 64 ? uint64_t(0) : mine, part, &all);
        cut = select_code(a, row, m, s, table, cut, false, limit_of(p, all), sums, found);
      }
      whole = true;
    }
  }
  // the chunks' sums, and the entries around the cut that stay
  if (whole) {
    for (uint32_t c = t / 64; c < a.chunks; c += ROW_WAVES) {
      const uint32_t i0 = c * a.chunk;
      const uint64_t sum = staying(a, row, i0, min(i0 + a.chunk, a.n), m, s, min_p, cut, table);
      if (t % 64 == 0) sums[c] = sum;
    }
  } else {
    for (uint32_t c = t; c < a.chunks; c += ROW_THREADS) sums[c] = a.sums[r * a.chunks + c];
    __syncthreads();
    for (uint32_t i = t; i < n_cand; i += ROW_THREADS) {
      const uint64_t x = code[i];
      if (x < cut) continue;
      const double w = weight_of(logit_of_code(x), m, s, table);
      if (w >= min_p) atomicAdd(reinterpret_cast<unsigned long long*>(&sums[(uint32_t)~(uint32_t)x / a.chunk]), (unsigned long long)fixed_of(w, a.bits));
    }
  }
  __syncthreads();
  const uint64_t mine = t < a.chunks ? sums[t] : 0;   // MAX_CHUNKS = ROW_THREADS
  uint64_t all;
  const uint64_t before = thread_scan<ROW_THREADS>(mine, part, &all);
  if (all == 0) {   // a min_p of NaN: nothing stays
    if (t == 0) {
      a.tokens[r] = -1;
      a.logprobs[r] = -INFINITY;
    }
    return;
  }
  const float u = a.u[r];
  uint64_t target, up;
  if (!(u < 1.f)) target = all - 1;      // the last one
  else if (!(u > 0.f)) target = 0;
  else scaled(u, all, &target, &up);
  if (t == 0) {
    pick = 0;
    rest = 0;
  }
  __syncthreads();
  if (before <= target && target < before + mine) {
    pick = t;
    rest = target - before;
  }
  __syncthreads();
  // that chunk, consecutive entries to a thread
  const uint32_t i0 = pick * a.chunk, i1 = min(i0 + a.chunk, a.n);
  const uint32_t per = (a.chunk + ROW_THREADS - 1) / ROW_THREADS;
  const uint32_t j0 = min(i0 + t * per, i1), j1 = min(j0 + per, i1);
  uint64_t own = 0, chunk_all;
  for (uint32_t i = j0; i < j1; ++i) {
    const float z = logit_of(row, i);
    if (!live(z, m) || code_of(z, i) < cut) continue;
    const double w = weight_of(z, m, s, table);
    if (w >= min_p) own += fixed_of(w, a.bits);
  }
  uint64_t run = thread_scan<ROW_THREADS>(own, part, &chunk_all);
  if (run <= rest && rest < run + own) {
    for (uint32_t i = j0; i < j1; ++i) {
      const float z = logit_of(row, i);
      if (!live(z, m) || code_of(z, i) < cut) continue;
      const double w = weight_of(z, m, s, table);
      if (!(w >= min_p)) continue;
      const uint64_t f = fixed_of(w, a.bits);
      if (rest < run + f) {
        a.tokens[r] = i;
        a.logprobs[r] = (float)log((double)f / (double)all);
        break;
      }
      run += f;
    }
  }
}

struct SamplePlan {
  uint32_t chunk = 0, chunks = 0, bits = 0;
  bool cut = true;
  size_t off_max = 0, off_sums = 0, off_count = 0, off_bins = 0, off_cand = 0, off_row = 0, total = 0;
};

SamplePlan sample_plan(const topk_sample_args& a) {
  SamplePlan p;
  p.cut = a.top_ks || a.top_ps || a.temperatures || (a.top_k > 0 && a.top_k < a.n) || !(a.top_p >= 1.f) || !(a.temperature > 0.f);
  p.chunk = 1024;
  while (ceil_div(a.n, p.chunk) > MAX_CHUNKS || (p.chunk < 8192 && a.rows * ceil_div(a.n, p.chunk) > 1024)) p.chunk *= 2;
  p.chunks = (uint32_t)ceil_div(a.n, p.chunk);
  p.bits = 62;
  while ((int64_t(1) << (62 - p.bits)) < a.n) --p.bits;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  const size_t rows = (size_t)a.rows;
  p.off_max = take(rows * p.chunks * 4);
  p.off_sums = take(rows * p.chunks * 8);
  if (p.cut) {
    p.off_count = take(rows * BINS * 4);
    p.off_bins = take(rows * BINS * 8);
    p.off_cand = take(rows * CAP * 8);
    p.off_row = take(rows * sizeof(SampleRow));
  }
  p.total = at;
  return p;
}

template <class T>
hipError_t sample_call(SampleArgs a, const SamplePlan& p, uint64_t rows, hipStream_t s) {
  a.work = rows * p.chunks;
  const dim3 chunks = wide_grid(a.work), whole = wide_grid(rows);
  SampleArgs by_row = a;
  by_row.work = rows;
  k_sample_max<T><<<chunks, CHUNK_THREADS, 0, s>>>(a);
  if (p.cut) {
    k_sample_hist<T><<<chunks, CHUNK_THREADS, 0, s>>>(a);
    k_sample_plan<<<whole, ROW_THREADS, 0, s>>>(by_row);
    k_sample_collect<T><<<chunks, CHUNK_THREADS, 0, s>>>(a);
  } else {
    k_sample_sum<T><<<chunks, CHUNK_THREADS, 0, s>>>(a);
  }
  k_sample_finish<T><<<whole, ROW_THREADS, 0, s>>>(by_row);
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
  a.sums = reinterpret_cast<uint64_t*>(w + p.off_sums);
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
