// The operators on a selection's entries: each entry e has a row r_e, a
// latent j_e and a coefficient.
//
//   by row      out[r] = bias + sum of coef_e src[j_e] over the entries of row r
//   by latent   out[j] = sum of coef_e src[r_e] over the entries of latent j
//   dots        dv_e = <g[r_e], w[j_e]>
//
// A selection comes in rank order, so its entries are first grouped by key
// (the row or the latent): a stable counting sort, in which equal keys keep
// rank order, so that every sum has one order whatever the timing.  Sorted
// entries are then summed in chunks of equal size, whatever their keys: a
// latent that is active in every row costs its wave no more than a rare one.
// A run of one key inside a chunk is written at once; runs that cross a chunk's
// edge leave partial sums, which a last pass adds in order, and which also
// writes the keys that have no entry.
//
// Row-wise selections are grouped by row as they come, and a short flattened
// one is cheaper to search by every row than to sort.
#include <algorithm>

#include "topk_ops_device.hpp"

namespace tk {

namespace {

// What the kernels know of a selection.
struct KSel {
  const int64_t* idx;
  uint64_t n, rows;
  uint32_t k, total;
  int flat;
};

KSel ksel(const Selection& s) {
  return KSel{s.indices, (uint64_t)s.n, (uint64_t)s.rows, (uint32_t)s.k, (uint32_t)s.total, s.flat};
}

// Row and latent of entry e; false for a padded slot or an index out of range.
__device__ __forceinline__ bool entry_of(const KSel& s, uint32_t e, int64_t i, uint32_t* row, uint32_t* latent) {
  if (s.flat) {
    if (i < 0 || s.n == 0) return false;
    uint64_t r;
    if (((uint64_t)i >> 32) == 0) r = (uint32_t)i / (uint32_t)s.n;   // n < 2^31
    else r = (uint64_t)i / s.n;
    if (r >= s.rows) return false;
    *row = (uint32_t)r;
    *latent = (uint32_t)((uint64_t)i - r * s.n);
    return true;
  }
  if ((uint64_t)i >= s.n) return false;
  *row = e / s.k;
  *latent = (uint32_t)i;
  return true;
}

// The coefficient of entry e: 0 where its gate is not above 0.
template <class T>
__device__ __forceinline__ float coef_of(const T* coef, const T* gate, uint32_t e) {
  if (gate && !(to_f32(gate[e]) > 0.f)) return 0.f;
  return to_f32(coef[e]);
}

// ---------------------------------------------------------------- grouping
// Stable counting sort of the entries by key, one or two digits of at most 14
// bits, the lower first; up to 16383 keys need one pass (keys are below 2^28).
// Each of `blocks` workgroups counts the digits of its consecutive entries
// (k_count); k_scan turns the counts into the place of each block's first
// entry of each digit; k_place writes the entries there.  Within a block the
// order is kept by taking 1024 entries at a time and, among those, wave by
// wave; within a wave a lane's place is the number of lower lanes with the
// same digit, from one ballot per digit bit.  Entries out of range have the
// key `keys`, behind all others.
//
// The launches are short and bound by latency, not by their bytes: 131072
// entries of 4096 rows take 5.0 + 6.9 + 6.3 us; by 12288 latents, whose counts
// are 6 MB, 8.4 + 9.3 + 6.7; by 65536 latents in two passes, with the rows'
// single pass in the same launches, 19 + 16.
constexpr uint32_t SORT_THREADS = 1024;
constexpr uint32_t MAX_BINS = 16384;
constexpr uint32_t GROUP = 64;          // bins of one k_scan workgroup
constexpr uint32_t SMALL = 4096;        // entries that one workgroup sorts

struct SortPlan {
  uint32_t keys = 0, total = 0;
  bool small = false;                   // one workgroup sorts them all (k_sort_small)
  uint32_t passes = 1, width = 0;       // digit bits of a pass (0: the whole key)
  uint32_t max_bins = 0;
  uint32_t blocks = 0, per_block = 0;
  size_t off_cnt = 0, off_coarse = 0, off_pair = 0, off_rec = 0, off_run = 0, total_bytes = 0;
};

uint32_t bins_of(const SortPlan& p, uint32_t pass) {
  if (!p.width) return p.keys + 1;
  const uint32_t shift = p.width * pass;
  const uint64_t top = (uint64_t)p.keys >> shift;
  return (uint32_t)std::min<uint64_t>(uint64_t(1) << p.width, top + 1);
}

SortPlan sort_plan(int64_t keys, int64_t total) {
  SortPlan p;
  p.keys = (uint32_t)keys;
  p.total = (uint32_t)total;
  p.small = total <= SMALL;
  if (keys + 1 > (int64_t)MAX_BINS) {
    uint32_t bits = 0;
    while ((uint64_t(1) << bits) <= (uint64_t)keys) ++bits;   // the key `keys` itself is one
    p.passes = bits > 14 ? 2 : 1;
    p.width = (bits + p.passes - 1) / p.passes;
  }
  p.max_bins = p.width ? 1u << p.width : p.keys + 1;
  const int64_t blocks = std::min<int64_t>(256, std::max<int64_t>(1, ceil_div(total, SORT_THREADS)));
  p.per_block = (uint32_t)(ceil_div(std::max<int64_t>(total, 1), blocks * SORT_THREADS) * SORT_THREADS);
  p.blocks = (uint32_t)std::max<int64_t>(1, ceil_div(total, p.per_block));
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  if (!p.small) {
    p.off_cnt = take((size_t)p.blocks * p.max_bins * 4);
    p.off_coarse = take((size_t)p.blocks * (p.max_bins / GROUP + 1) * 4);
  }
  if (!p.small && p.passes > 1) p.off_pair = take((size_t)total * 8);
  p.off_rec = take((size_t)total * 16);
  p.off_run = take((size_t)keys * 8);
  p.total_bytes = at;
  return p;
}

// One pass over (key, entry) pairs; the first makes them from the selection,
// the last writes what the sums read: (key, the other index, coefficient,
// entry), one 16-byte store to a place of its own instead of four.
struct KPass {
  const u32x2* in;            // (key, entry); null: from the selection
  u32x2* out;                 // null in the last pass, which writes records
  u32x4* rec;
  uint32_t* cnt;              // [blocks][bins]
  uint32_t* coarse;           // [groups][blocks]
  uint32_t* run;              // [keys][2]: first entry and end of a key's run, cleared by the first pass
  uint32_t keys, total, per_block, bins, groups, shift, mask, digit_bits, blocks;
  int by_row;
};

// A launch sorts by row and by latent side by side (grid dimension y).
struct KPasses {
  KPass p[2];
};

__device__ __forceinline__ uint32_t key_of(const KSel& s, const KPass& p, uint32_t e) {
  if (p.in) return p.in[e][0];
  uint32_t row, latent;
  if (!entry_of(s, e, s.idx[e], &row, &latent)) return p.keys;
  return p.by_row ? row : latent;
}

constexpr uint32_t NO_ENTRY = 0xFFFFFFFFu;

__global__ __launch_bounds__(SORT_THREADS) void k_count(KSel s, KPasses ps) {
  extern __shared__ uint32_t hist[];
  const KPass& p = ps.p[blockIdx.y];
  for (uint32_t i = threadIdx.x; i < p.bins; i += SORT_THREADS) hist[i] = 0;
  __syncthreads();
  const uint32_t e0 = blockIdx.x * p.per_block;
  const uint32_t e1 = p.total - e0 < p.per_block ? p.total : e0 + p.per_block;
  for (uint32_t e = e0 + threadIdx.x; e < e1; e += SORT_THREADS)
    atomicAdd(&hist[(key_of(s, p, e) >> p.shift) & p.mask], 1u);
  if (!p.in) {
    for (uint64_t i = (uint64_t)blockIdx.x * SORT_THREADS + threadIdx.x; i < p.keys; i += (uint64_t)gridDim.x * SORT_THREADS)
      p.run[2 * i] = NO_ENTRY;
  }
  __syncthreads();
  const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  for (uint32_t g = wave; g < p.groups; g += SORT_THREADS / 64) {
    const uint32_t b = g * GROUP + lane;
    const uint32_t v = b < p.bins ? hist[b] : 0u;
    if (b < p.bins) p.cnt[(size_t)blockIdx.x * p.bins + b] = v;
    const uint32_t sum = wave_sum(v);
    if (lane == 0) p.coarse[(size_t)g * p.blocks + blockIdx.x] = sum;
  }
}

// Workgroup g: places of the GROUP bins from g * GROUP on.  Sixteen waves
// share the blocks; a lane is a bin.  The sum of all lower bins comes from the
// groups' totals that k_count left beside the counts, so no launch is needed
// for a scan of scans.
__global__ __launch_bounds__(SORT_THREADS) void k_scan(KPasses ps) {
  __shared__ uint32_t part[16][GROUP];
  __shared__ uint32_t before[16];
  const KPass& p = ps.p[blockIdx.y];
  const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64, g = blockIdx.x;
  if (g >= p.groups) return;
  const uint32_t bin = g * GROUP + lane;
  const uint32_t per = (p.blocks + 15) / 16;
  const uint32_t b0 = wave * per < p.blocks ? wave * per : p.blocks;
  const uint32_t b1 = b0 + per < p.blocks ? b0 + per : p.blocks;
  uint32_t v[16];         // at most 256 blocks
#pragma unroll
  for (uint32_t i = 0; i < 16; ++i)
    v[i] = (b0 + i < b1 && bin < p.bins) ? p.cnt[(size_t)(b0 + i) * p.bins + bin] : 0u;
  uint32_t lower = 0;     // entries of the bins below this group
  const uint32_t n = g * p.blocks;
#pragma unroll 8
  for (uint32_t i = threadIdx.x; i < n; i += SORT_THREADS) lower += p.coarse[i];
  uint32_t sum = 0;
#pragma unroll
  for (uint32_t i = 0; i < 16; ++i) sum += v[i];
  part[wave][lane] = sum;
  lower = wave_sum(lower);
  if (lane == 0) before[wave] = lower;
  __syncthreads();
  uint32_t base = 0, own = 0, all = 0;
#pragma unroll
  for (uint32_t w = 0; w < 16; ++w) {
    base += before[w];
    if (w < wave) own += part[w][lane];
    all += part[w][lane];
  }
  uint32_t up = all;      // inclusive sum over the group's bins
#pragma unroll
  for (uint32_t o = 1; o < 64; o <<= 1) {
    const uint32_t t = __shfl_up(up, o);
    if (lane >= o) up += t;
  }
  uint32_t at = base + up - all + own;
#pragma unroll
  for (uint32_t i = 0; i < 16; ++i) {
    if (b0 + i < b1 && bin < p.bins) p.cnt[(size_t)(b0 + i) * p.bins + bin] = at;
    at += v[i];
  }
}

template <class T>
__global__ __launch_bounds__(SORT_THREADS) void k_place(KSel s, KPasses ps, const T* __restrict__ coef,
                                                        const T* __restrict__ gate) {
  extern __shared__ uint32_t taken[];     // entries of each bin that the block has placed
  const KPass& p = ps.p[blockIdx.y];
  for (uint32_t i = threadIdx.x; i < p.bins; i += SORT_THREADS) taken[i] = 0;
  __syncthreads();
  const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  const uint32_t e0 = blockIdx.x * p.per_block;
  const uint32_t e1 = p.total - e0 < p.per_block ? p.total : e0 + p.per_block;
  for (uint32_t c = e0; c < e1; c += SORT_THREADS) {
    const uint32_t e = c + threadIdx.x;
    const bool in = e < e1;
    uint32_t key = 0, pos = e, other = 0;
    float w = 0.f;
    if (in) {
      if (p.in) {
        const u32x2 q = p.in[e];
        key = q[0];
        pos = q[1];
      }
      if (!p.in || !p.out) {
        uint32_t row = 0, latent = 0;
        const int64_t i = s.idx[pos];
        if (!p.out) w = coef_of(coef, gate, pos);
        const bool good = entry_of(s, pos, i, &row, &latent);
        if (!p.in) key = good ? (p.by_row ? row : latent) : p.keys;
        other = good ? (p.by_row ? latent : row) : 0u;
        w = good ? w : 0.f;
      }
    }
    const uint32_t d = (key >> p.shift) & p.mask;
    uint32_t at = in ? p.cnt[(size_t)blockIdx.x * p.bins + d] : 0u;
    uint64_t same = __ballot(in);
    for (uint32_t b = 0; b < p.digit_bits; ++b) {
      const bool bit = d >> b & 1u;
      const uint64_t m = __ballot(bit);
      same &= bit ? m : ~m;
    }
    const uint32_t rank = __popcll(same & ((uint64_t(1) << lane) - 1));
    at += rank;
    for (uint32_t w2 = 0; w2 < SORT_THREADS / 64; ++w2) {
      if (w2 == wave && in) {
        const uint32_t t = taken[d];
        at += t;
        if (rank == 0) taken[d] = t + (uint32_t)__popcll(same);
      }
      __syncthreads();
    }
    if (in) {
      if (p.out) p.out[at] = u32x2{key, pos};
      else p.rec[at] = u32x4{key, other, __float_as_uint(w), pos};
    }
  }
}

// Few entries: one workgroup sorts them in LDS, eight bits of the key at a
// time, in one launch instead of three or six (4000 entries of 12288 latents
// 14 us).  Each of its 16 waves holds
// consecutive entries, at most four to a lane, and counts their digits on its
// own (lanes with equal digits are found by ballots, so the order is kept);
// the counts' prefix over digits, then waves, gives the places.  Workgroups
// beyond the first only clear their share of the runs' bounds.
template <class T>
__global__ __launch_bounds__(SORT_THREADS) void k_sort_small(KSel s, KPasses ps, const T* __restrict__ coef,
                                                             const T* __restrict__ gate) {
  constexpr uint32_t ROUNDS = SMALL / SORT_THREADS, WAVES = SORT_THREADS / 64;
  __shared__ uint32_t keys[SMALL], ents[SMALL], other[SMALL];
  __shared__ uint32_t cnt[WAVES][256];
  __shared__ uint32_t below[4];
  const KPass& p = ps.p[blockIdx.y];
  for (uint64_t i = (uint64_t)blockIdx.x * SORT_THREADS + threadIdx.x; i < p.keys; i += (uint64_t)gridDim.x * SORT_THREADS)
    p.run[2 * i] = NO_ENTRY;
  if (blockIdx.x) return;
  const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  const uint32_t rounds = (p.total + SORT_THREADS - 1) / SORT_THREADS;   // at most ROUNDS
  const uint32_t first = wave * rounds * 64 + lane;
  uint32_t key[ROUNDS], ent[ROUNDS];
#pragma unroll
  for (uint32_t r = 0; r < ROUNDS; ++r) {
    const uint32_t e = first + r * 64;
    key[r] = p.keys;
    ent[r] = e;
    if (r < rounds && e < p.total) {
      uint32_t row = 0, latent = 0;
      const bool good = entry_of(s, e, s.idx[e], &row, &latent);
      key[r] = good ? (p.by_row ? row : latent) : p.keys;
      other[e] = good ? (p.by_row ? latent : row) : 0u;
    }
  }
  for (uint32_t shift = 0; shift < p.digit_bits; shift += 8) {
    for (uint32_t i = lane; i < 256; i += 64) cnt[wave][i] = 0;
    uint32_t rank[ROUNDS];
#pragma unroll
    for (uint32_t r = 0; r < ROUNDS; ++r) {
      if (r >= rounds) break;
      const bool in = first + r * 64 < p.total;
      const uint32_t d = key[r] >> shift & 255u;
      uint64_t same = __ballot(in);
#pragma unroll
      for (uint32_t b = 0; b < 8; ++b) {
        const bool bit = d >> b & 1u;
        const uint64_t m = __ballot(bit);
        same &= bit ? m : ~m;
      }
      const uint32_t before = __popcll(same & ((uint64_t(1) << lane) - 1));
      if (in) {
        const uint32_t c = cnt[wave][d];
        rank[r] = c + before;
        if (before == 0) cnt[wave][d] = c + (uint32_t)__popcll(same);
      }
    }
    __syncthreads();
    if (threadIdx.x < 256) {     // a thread is a digit
      uint32_t c[WAVES], sum = 0;
#pragma unroll
      for (uint32_t w = 0; w < WAVES; ++w) {
        c[w] = cnt[w][threadIdx.x];
        sum += c[w];
      }
      uint32_t up = sum;
#pragma unroll
      for (uint32_t o = 1; o < 64; o <<= 1) {
        const uint32_t t = __shfl_up(up, o);
        if (lane >= o) up += t;
      }
      if (lane == 63) below[wave] = up;
      uint32_t at = up - sum;
#pragma unroll
      for (uint32_t w = 0; w < WAVES; ++w) {
        cnt[w][threadIdx.x] = at;
        at += c[w];
      }
    }
    __syncthreads();
#pragma unroll
    for (uint32_t r = 0; r < ROUNDS; ++r) {
      if (r >= rounds || first + r * 64 >= p.total) break;
      const uint32_t d = key[r] >> shift & 255u;
      uint32_t at = cnt[wave][d] + rank[r];
      for (uint32_t q = 0; q < d / 64; ++q) at += below[q];
      keys[at] = key[r];
      ents[at] = ent[r];
    }
    __syncthreads();
#pragma unroll
    for (uint32_t r = 0; r < ROUNDS; ++r) {
      if (r >= rounds || first + r * 64 >= p.total) break;
      key[r] = keys[first + r * 64];
      ent[r] = ents[first + r * 64];
    }
  }
  __syncthreads();
#pragma unroll
  for (uint32_t r = 0; r < ROUNDS; ++r) {
    const uint32_t i = first + r * 64;
    if (r >= rounds || i >= p.total) break;
    const float w = key[r] < p.keys ? coef_of(coef, gate, ent[r]) : 0.f;
    p.rec[i] = u32x4{key[r], other[ent[r]], __float_as_uint(w), ent[r]};
  }
}

// ---------------------------------------------------------------- sums
struct KSeg {
  const u32x4* rec;     // sorted (key, the other index, coefficient, entry)
  uint32_t* run;        // [keys][2]
  const void* src;
  const void* bias;
  void* out;            // null: not wanted
  void* coef_sum;
  const void* wsrc;     // dots: a row per key
  void* dots;
  float* part;          // [chunks][2][d]: a run that came in, a run that goes on
  float* part_c;        // [chunks][2]
  int64_t lds, ldo, ldw;
  uint32_t keys, total, chunk, d;
  int stream;           // store out past the caches
  uint32_t join;        // keys of one workgroup of k_join_runs
};

// A launch sums by row and by latent side by side (grid dimension z).
struct KSegs {
  KSeg s[2];
};

// A lane's share of the d columns: NV vectors of VEC of them, 64 VEC apart.
template <int VEC, int NV>
struct Share {
  uint32_t at[NV];     // first column of each vector
  uint32_t twice[NV];  // its first columns that another lane holds too
  bool in[NV];
  __device__ __forceinline__ Share(uint32_t c, uint32_t d) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const uint32_t b = c + v * 64 * VEC;
      in[v] = b < d;
      at[v] = in[v] ? column_of<VEC>(b, d) : 0u;
      twice[v] = in[v] ? b - at[v] : 0u;
    }
  }
};

// One lane's share of a row, kept as it was read until it is used.
template <class T, int VEC, int NV>
struct Row {
  u32x4 q[NV];
  __device__ __forceinline__ void load(const T* p, const Share<VEC, NV>& c, bool there) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      q[v] = u32x4{0u, 0u, 0u, 0u};
      if (there && c.in[v]) {
        if constexpr (VEC == 1) q[v][0] = __float_as_uint(to_f32(p[c.at[v]]));
        else q[v] = read16(p + c.at[v]);
      }
    }
  }
  __device__ __forceinline__ void unpack(int v, float* f) const {
    if constexpr (VEC == 1) f[0] = __uint_as_float(q[v][0]);
    else Vec<T>::unpack(q[v], f);
  }
};

// VEC elements of an output row.
template <class T, int VEC>
__device__ __forceinline__ void store_out(T* o, const float* v, int stream) {
  if (VEC > 1 && stream) {
    // (the empty statements keep the compiler from merging the two stores into a plain one)
    asm volatile("");
    stream_vec<T>(o, v);
    asm volatile("");
  } else {
    store_vec<T, VEC>(o, v);
  }
}

template <int VEC>
__device__ __forceinline__ void store_part(float* o, const float* v) {
  if constexpr (VEC == 1) {
    o[0] = v[0];
  } else {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) Vec<float>::store(o + i, v + i);
  }
}

// Eight sums over 64 lanes: each of the first three exchanges halves the
// number of sums a lane carries, so lane l ends with the sum of entry l % 8.
__device__ __forceinline__ float eight_sums(float* sum, uint32_t lane) {
#pragma unroll
  for (uint32_t h = 4; h; h >>= 1) {
    const bool up = lane & h;
#pragma unroll
    for (uint32_t u = 0; u < h; ++u) {
      const float keep = up ? sum[u + h] : sum[u], give = up ? sum[u] : sum[u + h];
      sum[u] = keep + __shfl_xor(give, h);
    }
  }
  float v = sum[0];
#pragma unroll
  for (uint32_t o = 8; o < 64; o <<= 1) v += __shfl_xor(v, o);
  return v;
}

// A wave sums the chunk's entries for 64 VEC NV columns, AHEAD rows of src in
// flight: the pass is bound by the gathered rows, of which L2 and the memory
// cache deliver 6 to 7 TB/s (131072 entries of 512: by row out of 64 MB of
// bf16 weights 21 us, 6.4 TB/s; by latent with dots, f32, 44 us, 6.1 TB/s of
// gathered gradients alone).  The entries' keys, source rows and coefficients are wave-uniform
// (read from one lane), so a row's address is scalar and a run's end a scalar
// branch.  With DOTS the wave also takes each entry's dot product of its
// source row and its key's row of wsrc, which neighbouring entries of a run
// find in the first-level cache.
// RAGGED: the last vector of a row begins in the one before it.
template <class T, int VEC, int NV, int AHEAD, bool DOTS, bool RAGGED>
__global__ __launch_bounds__(256) void k_seg(KSegs ss) {
  const KSeg& p = ss.s[blockIdx.z];
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
  const uint32_t chunk = blockIdx.x * 4 + wave;
  const uint64_t first = (uint64_t)chunk * p.chunk;
  if (first >= p.total) return;
  const uint32_t e0 = (uint32_t)first;
  const uint32_t e1 = p.total - e0 < p.chunk ? p.total : e0 + p.chunk;
  const Share<VEC, NV> cols((blockIdx.y * 64 * NV + lane) * VEC, p.d);
  const bool one = blockIdx.y == 0 && lane == 0;
  const T* src = static_cast<const T*>(p.src);
  const T* wsrc = static_cast<const T*>(p.wsrc);
  const uint32_t before = e0 ? p.rec[e0 - 1][0] : NO_ENTRY;
  const uint32_t behind = e1 < p.total ? p.rec[e1][0] : NO_ENTRY;
  float acc[NV][VEC] = {}, csum = 0.f;
  uint32_t cur = p.rec[e0][0];
  bool came = cur == before;
  if (one && !came && cur < p.keys) p.run[2 * (size_t)cur] = e0;

  auto flush = [&](uint32_t end, bool goes) {   // `end`: the entry behind the run
    if (cur < p.keys) {
      if (one && !goes) p.run[2 * (size_t)cur + 1] = end;
      if (came || goes) {
        const size_t slot = (size_t)chunk * 2 + (came ? 0 : 1);
        if (p.out) {
#pragma unroll
          for (int v = 0; v < NV; ++v)
            if (cols.in[v]) store_part<VEC>(p.part + slot * p.d + cols.at[v], acc[v]);
        }
        if (p.coef_sum && one) p.part_c[slot] = csum;
      } else {
        if (p.out) {
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            if (!cols.in[v]) continue;
            const uint32_t at = cols.at[v];
            if (p.bias) {
              float b[VEC];
              load_vec<T, VEC>(static_cast<const T*>(p.bias) + at, b);
#pragma unroll
              for (int i = 0; i < VEC; ++i) acc[v][i] += b[i];
            }
            store_out<T, VEC>(static_cast<T*>(p.out) + (int64_t)cur * p.ldo + at, acc[v], p.stream);
          }
        }
        if (p.coef_sum && one) static_cast<T*>(p.coef_sum)[cur] = from_f32<T>(csum);
      }
    }
    came = false;
    csum = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[v][i] = 0.f;
  };

  for (uint32_t b = e0; b < e1; b += 64) {
    const uint32_t have = e1 - b < 64 ? e1 - b : 64;
    const bool mine = lane < have;
    u32x4 r = {p.keys, 0u, 0u, 0u};
    if (mine) r = p.rec[b + lane];
    const uint32_t lk = r[0], lo = r[1], lc = r[2], le = r[3];
    for (uint32_t i0 = 0; i0 < have; i0 += AHEAD) {
      Row<T, VEC, NV> row[AHEAD], wrow[DOTS ? AHEAD : 1];
#pragma unroll
      for (uint32_t u = 0; u < AHEAD; ++u) {   // i0 + u < 64; lanes beyond `have` hold no key
        const uint32_t o = __builtin_amdgcn_readlane(lo, i0 + u);
        const uint32_t k = __builtin_amdgcn_readlane(lk, i0 + u);
        row[u].load(src + (int64_t)o * p.lds, cols, k < p.keys);
        if constexpr (DOTS) wrow[u].load(wsrc + (int64_t)k * p.ldw, cols, k < p.keys);
      }
      float dot[AHEAD];
#pragma unroll
      for (uint32_t u = 0; u < AHEAD; ++u) {
        const uint32_t k = __builtin_amdgcn_readlane(lk, i0 + u);
        const float w = __uint_as_float(__builtin_amdgcn_readlane(lc, i0 + u));
        if (k != cur && i0 + u < have) {
          flush(b + i0 + u, false);
          cur = k;
          if (one && cur < p.keys) p.run[2 * (size_t)cur] = b + i0 + u;
        }
        csum += w;
        dot[u] = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          float f[VEC];
          row[u].unpack(v, f);
          if constexpr (DOTS) {
            float g[VEC];
            wrow[u].unpack(v, g);
            if constexpr (RAGGED) {   // columns that another lane takes
#pragma unroll
              for (int i = 0; i < VEC; ++i) g[i] = (uint32_t)i < cols.twice[v] ? 0.f : g[i];
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) dot[u] = fmaf(f[i], g[i], dot[u]);
          }
          // (an entry behind the end has weight and row 0)
#pragma unroll
          for (int i = 0; i < VEC; ++i) acc[v][i] = fmaf(w, f[i], acc[v][i]);
        }
      }
      if constexpr (DOTS) {
        static_assert(AHEAD == 8, "eight_sums");
        const float v = eight_sums(dot, lane);
        const uint32_t e = __shfl(le, i0 + lane % AHEAD);   // (sums of lane l: entry l % 8)
        if (lane < AHEAD && i0 + lane < have) static_cast<T*>(p.dots)[e] = from_f32<T>(v);
      }
    }
  }
  flush(e1, behind == cur);
}

// Adds the partial sums of chunks [q, end) of a run (its first chunk keeps
// them in the second slot) for the VEC columns from c on.
template <int VEC>
__device__ __forceinline__ void add_parts(float* acc, const KSeg& p, uint32_t first, uint32_t q, uint32_t end, uint32_t c) {
#pragma unroll 8
  for (; q < end; ++q) {
    const float* b = p.part + ((size_t)q * 2 + (q == first)) * p.d + c;
    if constexpr (VEC == 1) {
      acc[0] += b[0];
    } else {
#pragma unroll
      for (int j = 0; j < VEC; j += 4) {
        float v[4];
        Vec<float>::load(b + j, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j + i] += v[i];
      }
    }
  }
}

template <class T, int VEC>
__device__ __forceinline__ void write_key(const KSeg& p, uint64_t key, uint32_t c, float* acc) {
  if (p.bias) {
    float b[VEC];
    load_vec<T, VEC>(static_cast<const T*>(p.bias) + c, b);
#pragma unroll
    for (int j = 0; j < VEC; ++j) acc[j] += b[j];
  }
  store_out<T, VEC>(static_cast<T*>(p.out) + (int64_t)key * p.ldo + c, acc, p.stream);
}

// Writes the keys without an entry, and joins the runs of several chunks.  A
// workgroup takes `join` keys, a lane of every wave each to look at; the waves
// share first the empty ones, whose stores wait for nothing, then the runs
// that cross a chunk's edge.  There is at most one of those per chunk, so the
// keys of a workgroup are as many as to hold two at most (131072 entries of
// 65536 latents and, beside them, of 4096 rows: 10.3 us; 14.8 with 16 keys to a
// workgroup whatever their number).  Runs of more than LONG chunks are shared
// by the four waves.
constexpr uint32_t LONG = 12;

uint32_t join_keys(uint32_t keys, uint32_t chunks) {
  return (uint32_t)std::min<uint64_t>(64, std::max<uint64_t>(1, 2ull * keys / std::max(1u, chunks)));
}

template <class T, int VEC>
__global__ __launch_bounds__(256) void k_join_runs(KSegs ss) {
  __shared__ float join[4][64 * VEC];
  const KSeg& p = ss.s[blockIdx.z];
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
  const uint64_t k0 = (uint64_t)block_id() * p.join;
  if (k0 >= p.keys) return;
  const bool mine = lane < p.join && k0 + lane < p.keys;
  uint32_t first = NO_ENTRY, end = 0;     // of the lane's key
  if (p.total && mine) {
    first = p.run[2 * (k0 + lane)];
    end = p.run[2 * (k0 + lane) + 1];
  }
  // chunks [q0, q1) of the run; none: q1 = 0
  const uint32_t lq0 = first == NO_ENTRY ? 0u : first / p.chunk, lq1 = first == NO_ENTRY ? 0u : (end - 1) / p.chunk + 1;
  const bool none = mine && lq1 == 0;
  if (p.coef_sum && none && wave == 0) static_cast<T*>(p.coef_sum)[k0 + lane] = from_f32<T>(0.f);
  const uint64_t empty = __ballot(none);
  if (p.out && empty) {
    for (uint32_t b = lane * VEC; b < p.d; b += 64 * VEC) {
      const uint32_t c = column_of<VEC>(b, p.d);
      float v[VEC] = {};
      if (p.bias) load_vec<T, VEC>(static_cast<const T*>(p.bias) + c, v);
      uint32_t turn = 0;
      for (uint64_t m = empty; m; m &= m - 1) {
        if (turn++ % 4 != wave) continue;
        const uint64_t key = k0 + (uint32_t)__ffsll((unsigned long long)m) - 1;
        store_out<T, VEC>(static_cast<T*>(p.out) + (int64_t)key * p.ldo + c, v, p.stream);
      }
    }
  }
  uint32_t turn = 0;
  for (uint64_t m = __ballot(mine && lq1 > lq0 + 1); m; m &= m - 1) {   // (one chunk: written there)
    if (turn++ % 4 != wave) continue;
    const uint32_t i = (uint32_t)__ffsll((unsigned long long)m) - 1;
    const uint32_t q0 = __builtin_amdgcn_readlane(lq0, i), q1 = __builtin_amdgcn_readlane(lq1, i);
    if (p.coef_sum) {
      float s = 0.f;
      for (uint32_t q = q0 + lane; q < q1; q += 64) s += p.part_c[(size_t)q * 2 + (q == q0)];
      s = wave_sum(s);
      if (lane == 0) static_cast<T*>(p.coef_sum)[k0 + i] = from_f32<T>(s);
    }
    if (!p.out || q1 - q0 > LONG) continue;
    for (uint32_t b = lane * VEC; b < p.d; b += 64 * VEC) {
      const uint32_t c = column_of<VEC>(b, p.d);
      float acc[VEC] = {};
      add_parts<VEC>(acc, p, q0, q0, q1, c);
      write_key<T, VEC>(p, k0 + i, c, acc);
    }
  }
  if (!p.out) return;
  for (uint64_t m = __ballot(mine && lq1 - lq0 > LONG); m; m &= m - 1) {
    const uint32_t i = (uint32_t)__ffsll((unsigned long long)m) - 1;
    const uint32_t q0 = __builtin_amdgcn_readlane(lq0, i), q1 = __builtin_amdgcn_readlane(lq1, i);
    const uint32_t per = (q1 - q0 + 3) / 4, a0 = q0 + wave * per, a1 = a0 + per < q1 ? a0 + per : q1;
    for (uint32_t b = 0; b < p.d; b += 64 * VEC) {
      const bool in = b + lane * VEC < p.d;
      const uint32_t c = in ? column_of<VEC>(b + lane * VEC, p.d) : 0u;
      float acc[VEC] = {};
      if (in) add_parts<VEC>(acc, p, q0, a0, a1, c);
#pragma unroll
      for (int j = 0; j < VEC; ++j) join[wave][lane * VEC + j] = acc[j];
      __syncthreads();
      if (wave == 0 && in) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const uint32_t a = lane * VEC + j;
          acc[j] = (join[0][a] + join[1][a]) + (join[2][a] + join[3][a]);
        }
        write_key<T, VEC>(p, k0 + i, c, acc);
      }
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------- rows without a sort
// One workgroup per row and column block.  Row-wise selections: the four
// waves share the row's entries.  Flattened ones: the workgroup reads every
// index, 256 at a time, and keeps those of its row, in order, in LDS.  The
// waves' sums are joined in wave order.
//
// A wave has ROWS_AHEAD rows on their way at a time, so a workgroup takes about
// 10 us for 256 entries, wherever it runs: few rows of many entries are split
// over several workgroups, each with `chunk` of them, whose sums go to the
// workspace and are added in order by a second launch (one row of 1024, 4096
// and 65536 entries of 512 bf16: 38, 164 and 2697 us unsplit; 15, 16 and 24
// split; 18, 34 and 173 through the sort).  1024 rows of 256 entries of 512
// bf16, out of 64 MB of weights: 39 us, 6.9 TB/s of source rows.
constexpr uint32_t KEEP = 1024;        // entries held in LDS
constexpr uint32_t ROWS_AHEAD = 8;     // rows of src in flight per wave

template <class T, int VEC>
__global__ __launch_bounds__(256) void k_rows(KSel s, KSeg p, uint32_t splits, const T* __restrict__ coef,
                                              const T* __restrict__ gate) {
  __shared__ uint32_t ent[KEEP];
  __shared__ float cf[KEEP];
  __shared__ uint32_t found[4];
  __shared__ float join[4][64 * VEC];
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
  const uint32_t row = block_id();
  if (row >= s.rows) return;
  const uint32_t split = blockIdx.z % splits;
  const Share<VEC, 1> cols((blockIdx.z / splits * 64 + lane) * VEC, p.d);
  const uint32_t c = cols.at[0];
  const bool in = cols.in[0];
  const T* src = static_cast<const T*>(p.src);
  float acc[VEC] = {};
  const uint32_t first = s.flat ? 0u : row * s.k, end = s.flat ? s.total : first + s.k;
  const uint32_t e0 = first + split * p.chunk, e1 = end - e0 < p.chunk ? end : e0 + p.chunk;
  uint32_t held = 0;     // entries in LDS; the same in every thread
  for (uint32_t b = e0; b < e1 || held; b += 256) {
    if (b < e1) {
      const uint32_t e = b + threadIdx.x;
      uint32_t r = 0, latent = 0;
      const bool mine = e < e1 && entry_of(s, e, s.idx[e], &r, &latent) && r == row;
      const uint64_t m = __ballot(mine);
      if (lane == 0) found[wave] = (uint32_t)__popcll(m);
      __syncthreads();
      uint32_t at = held + __popcll(m & ((uint64_t(1) << lane) - 1));
      for (uint32_t w = 0; w < 4; ++w) {
        if (w < wave) at += found[w];
        held += found[w];
      }
      if (mine) {
        ent[at] = latent;
        cf[at] = coef_of(coef, gate, e);
      }
      __syncthreads();
      if (held + 256 <= KEEP && b + 256 < e1) continue;
    }
    // sum what is held
    for (uint32_t i0 = wave * ROWS_AHEAD; i0 < held; i0 += 4 * ROWS_AHEAD) {
      Row<T, VEC, 1> v[ROWS_AHEAD];
      float w[ROWS_AHEAD];
#pragma unroll
      for (uint32_t u = 0; u < ROWS_AHEAD; ++u) {
        const bool there = i0 + u < held;
        const uint32_t o = __builtin_amdgcn_readfirstlane(there ? ent[i0 + u] : 0u);
        w[u] = there ? cf[i0 + u] : 0.f;
        v[u].load(src + (int64_t)o * p.lds, cols, there);
      }
#pragma unroll
      for (uint32_t u = 0; u < ROWS_AHEAD; ++u) {
        float f[VEC];
        v[u].unpack(0, f);
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[i] = fmaf(w[u], f[i], acc[i]);
      }
    }
    held = 0;
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) join[wave][lane * VEC + i] = acc[i];
  __syncthreads();
  if (wave == 0 && in) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const uint32_t a = lane * VEC + i;
      acc[i] = (join[0][a] + join[1][a]) + (join[2][a] + join[3][a]);
    }
    if (splits > 1) store_part<VEC>(p.part + ((size_t)split * s.rows + row) * ((p.d + 3) / 4 * 4) + c, acc);
    else write_key<T, VEC>(p, row, c, acc);
  }
}

// ---------------------------------------------------------------- dots
// A wave takes eight entries; its lanes hold 16-byte pieces of both rows, all
// sixteen on their way before the first product.  131072 entries of 512, in
// rank order: bf16 29.5 us, f32 63 us, 8.5 TB/s of rows out of the caches.
constexpr uint32_t DOTS = 8;

template <class T, int VEC>
__global__ __launch_bounds__(256) void k_dots(KSel s, const T* __restrict__ g, int64_t ldg,
                                              const T* __restrict__ w, int64_t ldw, uint32_t d,
                                              T* __restrict__ dv) {
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
  const uint64_t first = ((uint64_t)block_id() * 4 + wave) * DOTS;
  if (first >= s.total) return;
  const uint32_t e0 = (uint32_t)first;
  uint32_t row = 0, latent = 0;
  const bool good = lane < DOTS && e0 + lane < s.total && entry_of(s, e0 + lane, s.idx[e0 + lane], &row, &latent);
  const uint64_t ok = __ballot(good);
  float sum[DOTS] = {};
  for (uint32_t b = 0; b < d; b += 64 * VEC) {
    const Share<VEC, 1> cols(b + lane * VEC, d);
    Row<T, VEC, 1> x[DOTS], y[DOTS];
#pragma unroll
    for (uint32_t u = 0; u < DOTS; ++u) {
      const uint32_t r = __builtin_amdgcn_readlane(row, u), j = __builtin_amdgcn_readlane(latent, u);
      const bool there = ok >> u & 1;
      x[u].load(g + (int64_t)r * ldg, cols, there);
      y[u].load(w + (int64_t)j * ldw, cols, there);
    }
#pragma unroll
    for (uint32_t u = 0; u < DOTS; ++u) {
      float f[VEC], h[VEC];
      x[u].unpack(0, f);
      y[u].unpack(0, h);
#pragma unroll
      for (int i = 0; i < VEC; ++i) sum[u] = fmaf(f[i], (uint32_t)i < cols.twice[0] ? 0.f : h[i], sum[u]);
    }
  }
  const float v = eight_sums(sum, lane);
  if (lane < DOTS && e0 + lane < s.total) dv[e0 + lane] = from_f32<T>(v);
}

// ---------------------------------------------------------------- host side
// Rows straight from the selection: row-wise, or few enough reads that every
// row may look at every index.  512 bf16, against the way through the sort:
// 64 rows and 65536 entries 30.5 us to 31.6, 128 rows 39 to 31; 1024 rows and
// 4096 entries 20 to 25, 8192 entries 29 to 25; 16 rows and 65536 entries 22 to
// 38; 8 rows and 2^20 entries 199 to 330.
bool rows_direct(const Selection& s) {
  if (!s.flat) return true;
  return s.rows <= 8 ? s.total <= (int64_t(1) << 20) : s.total <= 65536 && s.rows * s.total <= (int64_t(1) << 22);
}

// How the entries that a row's workgroup goes through are split: into pieces of
// 256 or more while the rows alone do not give eight workgroups for each of
// 256 compute units, at most 256 (16 threads of the join share their sums).
struct RowsPlan {
  uint32_t columns = 1, splits = 1, chunk = 1, ldpart = 0;
  size_t bytes = 0;
};

RowsPlan rows_plan(const Selection& s, int64_t d) {
  RowsPlan p;
  const int64_t v = s.dtype == DT_BF16 ? 8 : 4, span = s.flat ? s.total : s.k;
  p.columns = (uint32_t)std::max<int64_t>(1, ceil_div(d, 64 * (d >= v ? v : 1)));
  const int64_t room = 2048 / std::max<int64_t>(1, s.rows * (int64_t)p.columns);
  const int64_t splits = std::max<int64_t>(1, std::min<int64_t>({room, 256, ceil_div(span, 256)}));
  p.chunk = (uint32_t)(ceil_div(std::max<int64_t>(1, span), splits * 256) * 256);
  p.splits = (uint32_t)std::max<int64_t>(1, ceil_div(span, p.chunk));
  p.ldpart = (uint32_t)(ceil_div(d, 4) * 4);
  if (p.splits > 1) p.bytes = align256((size_t)p.splits * (size_t)s.rows * p.ldpart * 4);
  return p;
}

struct SegPlan {
  SortPlan sort;
  uint32_t chunk = 64, chunks = 0;
  size_t off_part = 0, off_part_c = 0, total = 0;
};

// Chunks of 64 entries (the width of a wave), fewer while there are not
// enough chunks for eight waves on each of 256 compute units, more where the
// partial sums would otherwise grow with the selection.
SegPlan seg_plan(const Selection& s, int64_t d, bool by_row) {
  SegPlan p;
  p.sort = sort_plan(by_row ? s.rows : s.n, s.total);
  int64_t chunk = 64;
  while (chunk > 16 && ceil_div(s.total, chunk) < 2048) chunk /= 2;
  chunk *= std::max<int64_t>(1, ceil_div(s.total, chunk * 16384));
  p.chunk = (uint32_t)chunk;
  p.chunks = (uint32_t)ceil_div(s.total, chunk);
  p.off_part = p.sort.total_bytes;
  p.off_part_c = p.off_part + align256((size_t)p.chunks * 2 * (size_t)d * 4);
  p.total = p.off_part_c + align256((size_t)p.chunks * 2 * 4);
  return p;
}

// The sorts of one or two parts: their first passes share launches.
template <class T>
hipError_t run_sorts(const SegCall& a, const SegArgs* const* parts, const SegPlan* plans, char* const* ws, int n,
                     hipStream_t s) {
  const KSel sel = ksel(a.sel);
  const T* coef = static_cast<const T*>(a.coef);
  const T* gate = static_cast<const T*>(a.gate);
  if (plans[0].sort.small) {   // (the same for both: it follows from the entries)
    KPasses ks{};
    uint32_t keys = 0;
    for (int i = 0; i < n; ++i) {
      const SortPlan& p = plans[i].sort;
      KPass& k = ks.p[i];
      k.rec = reinterpret_cast<u32x4*>(ws[i] + p.off_rec);
      k.run = reinterpret_cast<uint32_t*>(ws[i] + p.off_run);
      k.keys = p.keys;
      k.total = p.total;
      k.by_row = parts[i]->by_row;
      while (k.digit_bits < 32 && (uint64_t(1) << k.digit_bits) <= p.keys) ++k.digit_bits;   // of the key `keys`
      keys = std::max(keys, p.keys);
    }
    const uint32_t x = 1 + std::min<uint32_t>(keys / (4 * SORT_THREADS), 255);
    hipLaunchKernelGGL((k_sort_small<T>), dim3(x, n), dim3(SORT_THREADS), 0, s, sel, ks, coef, gate);
    return hipGetLastError();
  }
  uint32_t most = 0;
  for (int i = 0; i < n; ++i) most = std::max(most, plans[i].sort.passes);
  for (uint32_t pass = 0; pass < most; ++pass) {
    KPasses ks;
    uint32_t y = 0, groups = 0, bins = 0, blocks = 0;
    for (int i = 0; i < n; ++i) {
      const SortPlan& p = plans[i].sort;
      if (pass >= p.passes) continue;
      KPass& k = ks.p[y++];
      u32x2* pair = reinterpret_cast<u32x2*>(ws[i] + p.off_pair);
      const bool last = pass + 1 == p.passes;
      k.in = pass ? pair : nullptr;    // at most two passes
      k.out = last ? nullptr : pair;
      k.rec = reinterpret_cast<u32x4*>(ws[i] + p.off_rec);
      k.cnt = reinterpret_cast<uint32_t*>(ws[i] + p.off_cnt);
      k.coarse = reinterpret_cast<uint32_t*>(ws[i] + p.off_coarse);
      k.run = reinterpret_cast<uint32_t*>(ws[i] + p.off_run);
      k.keys = p.keys;
      k.total = p.total;
      k.per_block = p.per_block;
      k.bins = bins_of(p, pass);
      k.groups = (uint32_t)ceil_div(k.bins, GROUP);
      k.shift = p.width * pass;
      k.mask = p.width ? (1u << p.width) - 1 : 0xFFFFFFFFu;
      k.digit_bits = 0;
      while ((1u << k.digit_bits) < k.bins) ++k.digit_bits;
      k.blocks = blocks = p.blocks;     // the same for both: it follows from the entries
      k.by_row = parts[i]->by_row;
      groups = std::max(groups, k.groups);
      bins = std::max(bins, k.bins);
    }
    if (y == 1) ks.p[1] = ks.p[0];
    const size_t lds = (size_t)bins * 4;
    hipLaunchKernelGGL(k_count, dim3(blocks, y), dim3(SORT_THREADS), lds, s, sel, ks);
    hipLaunchKernelGGL(k_scan, dim3(groups, y), dim3(SORT_THREADS), 0, s, ks);
    hipLaunchKernelGGL((k_place<T>), dim3(blocks, y), dim3(SORT_THREADS), lds, s, sel, ks, coef, gate);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <class T>
hipError_t launch_sums(const KSegs& ks, int n, bool wide, uint32_t chunks, int64_t d, bool dots, hipStream_t s) {
  constexpr int V = Vec<T>::N;
  const int64_t span = 64 * (wide ? V : 1), vecs = std::max<int64_t>(1, ceil_div(d, span));
  if (chunks) {
    const uint32_t x = (uint32_t)ceil_div(chunks, 4);
    const dim3 one(x, 1, n), all(x, (uint32_t)vecs, n);
    const bool ragged = d % V;
    if (dots && vecs == 1 && ragged) hipLaunchKernelGGL((k_seg<T, V, 1, 8, true, true>), one, dim3(256), 0, s, ks);
    else if (dots && vecs == 1) hipLaunchKernelGGL((k_seg<T, V, 1, 8, true, false>), one, dim3(256), 0, s, ks);
    else if (dots && ragged) hipLaunchKernelGGL((k_seg<T, V, 2, 8, true, true>), one, dim3(256), 0, s, ks);
    else if (dots) hipLaunchKernelGGL((k_seg<T, V, 2, 8, true, false>), one, dim3(256), 0, s, ks);
    else if (wide) hipLaunchKernelGGL((k_seg<T, V, 1, 16, false, false>), all, dim3(256), 0, s, ks);
    else hipLaunchKernelGGL((k_seg<T, 1, 1, 16, false, false>), all, dim3(256), 0, s, ks);
  }
  int64_t joins = 0;
  for (int i = 0; i < n; ++i) joins = std::max(joins, ceil_div(ks.s[i].keys, ks.s[i].join));
  const dim3 grid = wide_grid((uint64_t)joins, n);
  if (wide) hipLaunchKernelGGL((k_join_runs<T, V>), grid, dim3(256), 0, s, ks);
  else hipLaunchKernelGGL((k_join_runs<T, 1>), grid, dim3(256), 0, s, ks);
  return hipGetLastError();
}

template <class T>
hipError_t run_seg(const SegCall& a, char* ws, hipStream_t s) {
  constexpr int64_t V = Vec<T>::N;
  const SegArgs* sorted[2];
  SegPlan plans[2];
  char* at[2];
  KSegs ks;
  int n = 0;
  const bool wide = a.d >= V;   // rows of at least one vector
  bool dots = false;
  for (int i = 0; i < a.parts; ++i) {
    const SegArgs& p = a.part[i];
    const int64_t keys = p.by_row ? a.sel.rows : a.sel.n;
    KSeg k{};
    k.src = p.src;
    k.bias = p.bias;
    k.out = p.out;
    k.coef_sum = p.coef_sum;
    k.lds = p.lds;
    k.ldo = p.ldo;
    k.keys = (uint32_t)keys;
    k.total = (uint32_t)a.sel.total;
    k.d = p.out || p.dots ? (uint32_t)a.d : 0u;   // without an output src is not read, and may be null
    k.stream = keys * a.d * (int64_t)sizeof(T) >= STREAM_BYTES;
    if (p.dots) {
      // fused where a lane holds its whole share of both rows (and there is a
      // sum to fuse with: without latents every entry gets its 0 from k_dots)
      if (wide && a.d <= 128 * V && a.sel.total && keys) {
        dots = true;
        k.wsrc = p.other;
        k.ldw = p.ldother;
        k.dots = p.dots;
      } else {
        DotArgs q;
        q.sel = a.sel;
        q.g = p.src;
        q.ldg = p.lds;
        q.w = p.other;
        q.ldw = p.ldother;
        q.d = a.d;
        q.dv = p.dots;
        const hipError_t e = launch_dots(q, s);
        if (e != hipSuccess) return e;
      }
    }
    if (keys == 0 || ((a.d == 0 || !p.out) && !p.coef_sum && !k.dots)) continue;
    if (p.by_row && rows_direct(a.sel)) {
      const RowsPlan q = rows_plan(a.sel, a.d);
      const dim3 grid = wide_grid(k.keys, q.columns * q.splits);
      k.chunk = q.chunk;
      k.part = reinterpret_cast<float*>(ws);
      ws += q.bytes;
      const T* coef = static_cast<const T*>(a.coef);
      const T* gate = static_cast<const T*>(a.gate);
      if (wide) hipLaunchKernelGGL((k_rows<T, (int)V>), grid, dim3(256), 0, s, ksel(a.sel), k, q.splits, coef, gate);
      else hipLaunchKernelGGL((k_rows<T, 1>), grid, dim3(256), 0, s, ksel(a.sel), k, q.splits, coef, gate);
      hipError_t e = hipGetLastError();
      if (e == hipSuccess && q.splits > 1) {
        JoinArgs j;
        j.part = k.part;
        j.split = q.splits;
        j.ldpart = q.ldpart;
        j.m = keys;
        j.n = a.d;
        j.dtype = a.sel.dtype;
        j.bias = p.bias;
        j.out = p.out;
        j.ldo = p.ldo;
        e = launch_join(j, s);
      }
      if (e != hipSuccess) return e;
      continue;
    }
    plans[n] = seg_plan(a.sel, a.d, p.by_row);
    const SortPlan& q = plans[n].sort;
    k.rec = reinterpret_cast<const u32x4*>(ws + q.off_rec);
    k.run = reinterpret_cast<uint32_t*>(ws + q.off_run);
    k.part = reinterpret_cast<float*>(ws + plans[n].off_part);
    k.part_c = reinterpret_cast<float*>(ws + plans[n].off_part_c);
    k.chunk = plans[n].chunk;
    k.join = join_keys(k.keys, plans[n].chunks);
    sorted[n] = &p;
    at[n] = ws;
    ks.s[n++] = k;
    ws += plans[n - 1].total;
  }
  if (!n) return hipSuccess;
  if (n == 1) ks.s[1] = ks.s[0];
  if (a.sel.total) {
    const hipError_t e = run_sorts<T>(a, sorted, plans, at, n, s);
    if (e != hipSuccess) return e;
  }
  return launch_sums<T>(ks, n, wide, plans[0].chunks, std::max(ks.s[0].d, ks.s[1].d), dots, s);
}

template <class T>
hipError_t run_dots(const DotArgs& a, hipStream_t s) {
  constexpr int64_t V = Vec<T>::N;
  const bool wide = a.d >= V;
  const dim3 grid = wide_grid((uint64_t)ceil_div(a.sel.total, 4 * DOTS));
  const T* g = static_cast<const T*>(a.g);
  const T* w = static_cast<const T*>(a.w);
  T* dv = static_cast<T*>(a.dv);
  if (wide) hipLaunchKernelGGL((k_dots<T, (int)V>), grid, dim3(256), 0, s, ksel(a.sel), g, a.ldg, w, a.ldw, (uint32_t)a.d, dv);
  else hipLaunchKernelGGL((k_dots<T, 1>), grid, dim3(256), 0, s, ksel(a.sel), g, a.ldg, w, a.ldw, (uint32_t)a.d, dv);
  return hipGetLastError();
}

}  // namespace

size_t seg_workspace(const Selection& sel, int64_t d, bool by_row, bool by_latent) {
  size_t bytes = 0;
  if (by_row) bytes += rows_direct(sel) ? rows_plan(sel, d).bytes : seg_plan(sel, d, true).total;
  if (by_latent) bytes += seg_plan(sel, d, false).total;
  return bytes;
}

hipError_t launch_seg(const SegCall& a, void* ws, hipStream_t s) {
  return a.sel.dtype == DT_BF16 ? run_seg<bf16_t>(a, static_cast<char*>(ws), s)
                                : run_seg<float>(a, static_cast<char*>(ws), s);
}

hipError_t launch_dots(const DotArgs& a, hipStream_t s) {
  if (a.sel.total == 0) return hipSuccess;
  return a.sel.dtype == DT_BF16 ? run_dots<bf16_t>(a, s) : run_dots<float>(a, s);
}

}  // namespace tk
