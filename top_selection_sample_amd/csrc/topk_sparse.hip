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
// Stable counting sort of the entries by key, digits of at most 14 bits, the
// lowest first; up to 16383 keys need one pass.  Each of `blocks` workgroups
// counts the digits of its consecutive entries (k_count); k_scan turns the
// counts into the place of each block's first entry of each digit; k_place
// writes the entries there.  Within a block the order is kept by taking 1024
// entries at a time and, among those, wave by wave; within a wave a lane's
// place is the number of lower lanes with the same digit, from one ballot per
// digit bit.  Entries out of range have the key `keys`, behind all others.
constexpr uint32_t SORT_THREADS = 1024;
constexpr uint32_t MAX_BINS = 16384;
constexpr uint32_t GROUP = 64;          // bins of one k_scan workgroup

struct SortPlan {
  uint32_t keys = 0, total = 0;
  uint32_t passes = 1, width = 0;       // digit bits of a pass (0: the whole key)
  uint32_t max_bins = 0;
  uint32_t blocks = 0, per_block = 0;
  size_t off_cnt = 0, off_coarse = 0, off_key = 0, off_pos = 0, off_skey = 0, off_other = 0, off_coef = 0, total_bytes = 0;
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
  if (keys + 1 > (int64_t)MAX_BINS) {
    uint32_t bits = 0;
    while ((uint64_t(1) << bits) <= (uint64_t)keys) ++bits;   // the key `keys` itself is one
    p.passes = (bits + 13) / 14;
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
  p.off_cnt = take((size_t)p.blocks * p.max_bins * 4);
  p.off_coarse = take((size_t)p.blocks * (p.max_bins / GROUP + 1) * 4);
  if (p.passes > 1) {   // the even passes write here, the odd ones behind it
    p.off_key = take((size_t)total * 8);
    p.off_pos = take((size_t)total * 8);
  }
  p.off_skey = take((size_t)total * 4);
  p.off_other = take((size_t)total * 4);
  p.off_coef = take((size_t)total * 4);
  p.total_bytes = at;
  return p;
}

// One pass over (key, entry) pairs; the first makes them from the selection.
struct KPass {
  const uint32_t* key_in;     // null: from the selection
  const uint32_t* pos_in;
  uint32_t* key_out;
  uint32_t* pos_out;          // null: the last pass, which writes what the sums read
  uint32_t* other;
  float* coef;
  uint32_t* cnt;              // [blocks][bins]
  uint32_t* coarse;           // [blocks][bins / GROUP rounded up]
  uint32_t keys, total, per_block, bins, groups, shift, mask, digit_bits, blocks;
  int by_row;
};

__device__ __forceinline__ uint32_t key_of(const KSel& s, const KPass& p, uint32_t e) {
  if (p.key_in) return p.key_in[e];
  uint32_t row, latent;
  if (!entry_of(s, e, s.idx[e], &row, &latent)) return p.keys;
  return p.by_row ? row : latent;
}

__global__ __launch_bounds__(SORT_THREADS) void k_count(KSel s, KPass p) {
  extern __shared__ uint32_t hist[];
  for (uint32_t i = threadIdx.x; i < p.bins; i += SORT_THREADS) hist[i] = 0;
  __syncthreads();
  const uint32_t e0 = blockIdx.x * p.per_block;
  const uint32_t e1 = p.total - e0 < p.per_block ? p.total : e0 + p.per_block;
  for (uint32_t e = e0 + threadIdx.x; e < e1; e += SORT_THREADS)
    atomicAdd(&hist[(key_of(s, p, e) >> p.shift) & p.mask], 1u);
  __syncthreads();
  const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  for (uint32_t g = wave; g < p.groups; g += SORT_THREADS / 64) {
    const uint32_t b = g * GROUP + lane;
    const uint32_t v = b < p.bins ? hist[b] : 0u;
    if (b < p.bins) p.cnt[(size_t)blockIdx.x * p.bins + b] = v;
    const uint32_t sum = wave_sum(v);
    if (lane == 0) p.coarse[(size_t)blockIdx.x * p.groups + g] = sum;
  }
}

// Workgroup g: places of the GROUP bins from g * GROUP on.  Sixteen waves
// share the blocks; a lane is a bin.
__global__ __launch_bounds__(SORT_THREADS) void k_scan(KPass p) {
  __shared__ uint32_t part[16][GROUP];
  __shared__ uint32_t before[16];
  const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64, g = blockIdx.x;
  uint32_t lower = 0;     // entries of the bins below this group
  for (uint32_t b = wave; b < p.blocks; b += 16)
    for (uint32_t c = lane; c < g; c += 64) lower += p.coarse[(size_t)b * p.groups + c];
  lower = wave_sum(lower);
  if (lane == 0) before[wave] = lower;
  const uint32_t bin = g * GROUP + lane;
  const uint32_t per = (p.blocks + 15) / 16;
  const uint32_t b0 = wave * per < p.blocks ? wave * per : p.blocks;
  const uint32_t b1 = b0 + per < p.blocks ? b0 + per : p.blocks;
  uint32_t v[16];         // at most 256 blocks
  uint32_t sum = 0;
#pragma unroll
  for (uint32_t i = 0; i < 16; ++i) {
    v[i] = (b0 + i < b1 && bin < p.bins) ? p.cnt[(size_t)(b0 + i) * p.bins + bin] : 0u;
    sum += v[i];
  }
  part[wave][lane] = sum;
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
__global__ __launch_bounds__(SORT_THREADS) void k_place(KSel s, KPass p, const T* __restrict__ coef,
                                                        const T* __restrict__ gate) {
  extern __shared__ uint32_t taken[];     // entries of each bin that the block has placed
  for (uint32_t i = threadIdx.x; i < p.bins; i += SORT_THREADS) taken[i] = 0;
  __syncthreads();
  const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  const uint32_t e0 = blockIdx.x * p.per_block;
  const uint32_t e1 = p.total - e0 < p.per_block ? p.total : e0 + p.per_block;
  for (uint32_t c = e0; c < e1; c += SORT_THREADS) {
    const uint32_t e = c + threadIdx.x;
    const bool in = e < e1;
    const uint32_t key = in ? key_of(s, p, e) : 0u;
    const uint32_t d = (key >> p.shift) & p.mask;
    uint64_t same = __ballot(in);
    for (uint32_t b = 0; b < p.digit_bits; ++b) {
      const bool bit = d >> b & 1u;
      const uint64_t m = __ballot(bit);
      same &= bit ? m : ~m;
    }
    const uint32_t rank = __popcll(same & ((uint64_t(1) << lane) - 1));
    uint32_t at = in ? p.cnt[(size_t)blockIdx.x * p.bins + d] + rank : 0u;
    for (uint32_t w = 0; w < SORT_THREADS / 64; ++w) {
      if (w == wave && in) {
        const uint32_t t = taken[d];
        at += t;
        if (rank == 0) taken[d] = t + (uint32_t)__popcll(same);
      }
      __syncthreads();
    }
    if (in) {
      const uint32_t pos = p.key_in ? p.pos_in[e] : e;
      p.key_out[at] = key;
      if (p.pos_out) {
        p.pos_out[at] = pos;
      } else {
        uint32_t row = 0, latent = 0;
        const bool good = entry_of(s, pos, s.idx[pos], &row, &latent);
        p.other[at] = good ? (p.by_row ? latent : row) : 0u;
        p.coef[at] = good ? coef_of(coef, gate, pos) : 0.f;
      }
    }
  }
}

// ---------------------------------------------------------------- sums
constexpr uint32_t ROWS_AHEAD = 8;      // rows of src in flight per wave

struct KSeg {
  const uint32_t* skey;
  const uint32_t* other;
  const float* coef;
  const void* src;
  const void* bias;
  void* out;
  void* coef_sum;
  float* part;          // [chunks][2][d]: a run that came in, a run that goes on
  float* part_c;        // [chunks][2]
  int64_t lds, ldo;
  uint32_t keys, total, chunk, d;
};

// A wave sums the chunk's entries for 64 VEC columns.  The entries' keys,
// source rows and coefficients are wave-uniform (read from one lane), so a
// row's address is scalar and a run's end a scalar branch.
template <class T, int VEC>
__global__ __launch_bounds__(256) void k_seg(KSeg p) {
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
  const uint32_t chunk = blockIdx.x * 4 + wave;
  const uint64_t first = (uint64_t)chunk * p.chunk;
  if (first >= p.total) return;
  const uint32_t e0 = (uint32_t)first;
  const uint32_t e1 = p.total - e0 < p.chunk ? p.total : e0 + p.chunk;
  const uint32_t c = (blockIdx.y * 64 + lane) * VEC;
  const bool in = c < p.d;
  const T* src = static_cast<const T*>(p.src);
  const uint32_t before = e0 ? p.skey[e0 - 1] : 0xFFFFFFFFu;
  const uint32_t behind = e1 < p.total ? p.skey[e1] : 0xFFFFFFFFu;
  float acc[VEC] = {}, csum = 0.f;
  uint32_t cur = p.skey[e0];
  bool came = cur == before;

  auto flush = [&](bool goes) {
    if (cur < p.keys) {
      if (came || goes) {
        const size_t slot = (size_t)chunk * 2 + (came ? 0 : 1);
        if (in) {
          float* o = p.part + slot * p.d + c;
          if constexpr (VEC == 1) {
            o[0] = acc[0];
          } else {
#pragma unroll
            for (int i = 0; i < VEC; i += 4) Vec<float>::store(o + i, acc + i);
          }
        }
        if (p.coef_sum && lane == 0 && blockIdx.y == 0) p.part_c[slot] = csum;
      } else {
        if (in) {
          if (p.bias) {
            float b[VEC];
            load_vec<T, VEC>(static_cast<const T*>(p.bias) + c, b);
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[i] += b[i];
          }
          store_vec<T, VEC>(static_cast<T*>(p.out) + (int64_t)cur * p.ldo + c, acc);
        }
        if (p.coef_sum && lane == 0 && blockIdx.y == 0) static_cast<T*>(p.coef_sum)[cur] = from_f32<T>(csum);
      }
    }
    came = false;
    csum = 0.f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
  };

  for (uint32_t b = e0; b < e1; b += 64) {
    const uint32_t have = e1 - b < 64 ? e1 - b : 64;
    const bool mine = lane < have;
    const uint32_t lk = mine ? p.skey[b + lane] : p.keys;
    const uint32_t lo = mine ? p.other[b + lane] : 0u;
    const float lc = mine ? p.coef[b + lane] : 0.f;
    for (uint32_t i0 = 0; i0 < have; i0 += ROWS_AHEAD) {
      float row[ROWS_AHEAD][VEC];
#pragma unroll
      for (uint32_t u = 0; u < ROWS_AHEAD; ++u) {
        const uint32_t o = __builtin_amdgcn_readlane(lo, i0 + u);   // i0 + u < 64; lanes beyond `have` hold row 0
        const uint32_t k = __builtin_amdgcn_readlane(lk, i0 + u);
#pragma unroll
        for (int i = 0; i < VEC; ++i) row[u][i] = 0.f;
        if (in && k < p.keys) load_vec<T, VEC>(src + (int64_t)o * p.lds + c, row[u]);
      }
#pragma unroll
      for (uint32_t u = 0; u < ROWS_AHEAD; ++u) {
        if (i0 + u >= have) break;
        const uint32_t k = __builtin_amdgcn_readlane(lk, i0 + u);
        const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(lc), i0 + u));
        if (k != cur) {
          flush(false);
          cur = k;
        }
        csum += w;
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[i] = fmaf(w, row[u][i], acc[i]);
      }
    }
  }
  flush(behind == cur);
}

// First entry whose key is at least `key`.
__device__ __forceinline__ uint32_t lower_bound(const uint32_t* __restrict__ skey, uint32_t total, uint32_t key) {
  uint32_t lo = 0, hi = total;
  while (lo < hi) {
    const uint32_t mid = (lo + hi) / 2;
    if (skey[mid] < key) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// Writes the keys without an entry, and joins the runs of several chunks: 64
// keys per workgroup, a wave per key.
constexpr uint32_t JOIN_KEYS = 64;

template <class T, int VEC>
__global__ __launch_bounds__(256) void k_join_runs(KSeg p) {
  __shared__ uint32_t start[JOIN_KEYS + 1];
  const uint32_t k0 = blockIdx.x * JOIN_KEYS;
  if (threadIdx.x <= JOIN_KEYS) {
    const uint32_t k = k0 + threadIdx.x;
    start[threadIdx.x] = lower_bound(p.skey, p.total, k < p.keys ? k : p.keys);
  }
  __syncthreads();
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
  for (uint32_t i = wave; i < JOIN_KEYS && k0 + i < p.keys; i += 4) {
    const uint32_t key = k0 + i;
    const uint32_t lo = __builtin_amdgcn_readfirstlane(start[i]), hi = __builtin_amdgcn_readfirstlane(start[i + 1]);
    const uint32_t q0 = lo / p.chunk, q1 = hi > lo ? (hi - 1) / p.chunk : q0;
    if (hi > lo && q0 == q1) continue;     // written by its chunk
    for (uint32_t c = lane * VEC; c < p.d; c += 64 * VEC) {
      float acc[VEC] = {};
      if (hi > lo) {
        const float* a = p.part + ((size_t)q0 * 2 + 1) * p.d + c;
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc[j] = a[j];
#pragma unroll 4
        for (uint32_t q = q0 + 1; q <= q1; ++q) {
          const float* b = p.part + (size_t)q * 2 * p.d + c;
#pragma unroll
          for (int j = 0; j < VEC; ++j) acc[j] += b[j];
        }
      }
      if (p.bias) {
        float b[VEC];
        load_vec<T, VEC>(static_cast<const T*>(p.bias) + c, b);
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc[j] += b[j];
      }
      store_vec<T, VEC>(static_cast<T*>(p.out) + (int64_t)key * p.ldo + c, acc);
    }
    if (p.coef_sum && lane == 0) {
      float s = 0.f;
      if (hi > lo) {
        s = p.part_c[(size_t)q0 * 2 + 1];
        for (uint32_t q = q0 + 1; q <= q1; ++q) s += p.part_c[(size_t)q * 2];
      }
      static_cast<T*>(p.coef_sum)[key] = from_f32<T>(s);
    }
  }
}

// ---------------------------------------------------------------- rows without a sort
// One workgroup per row and column block.  Row-wise selections: the four
// waves share the row's entries.  Flattened ones: the workgroup reads every
// index, 256 at a time, and keeps those of its row, in order, in LDS.  The
// waves' sums are joined in wave order.
constexpr uint32_t KEEP = 1024;        // entries held in LDS

template <class T, int VEC>
__global__ __launch_bounds__(256) void k_rows(KSel s, KSeg p, const T* __restrict__ coef,
                                              const T* __restrict__ gate) {
  __shared__ uint32_t ent[KEEP];
  __shared__ float cf[KEEP];
  __shared__ uint32_t found[4];
  __shared__ float join[4][64 * VEC];
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
  const uint32_t row = blockIdx.x;
  const uint32_t c = (blockIdx.y * 64 + lane) * VEC;
  const bool in = c < p.d;
  const T* src = static_cast<const T*>(p.src);
  float acc[VEC] = {};
  const uint32_t e0 = s.flat ? 0u : row * s.k, e1 = s.flat ? s.total : e0 + s.k;
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
      float v[ROWS_AHEAD][VEC], w[ROWS_AHEAD];
#pragma unroll
      for (uint32_t u = 0; u < ROWS_AHEAD; ++u) {
        const bool there = i0 + u < held;
        const uint32_t o = __builtin_amdgcn_readfirstlane(there ? ent[i0 + u] : 0u);
        w[u] = there ? cf[i0 + u] : 0.f;
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[u][i] = 0.f;
        if (in && there) load_vec<T, VEC>(src + (int64_t)o * p.lds + c, v[u]);
      }
#pragma unroll
      for (uint32_t u = 0; u < ROWS_AHEAD; ++u)
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[i] = fmaf(w[u], v[u][i], acc[i]);
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
    if (p.bias) {
      float b[VEC];
      load_vec<T, VEC>(static_cast<const T*>(p.bias) + c, b);
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[i] += b[i];
    }
    store_vec<T, VEC>(static_cast<T*>(p.out) + (int64_t)row * p.ldo + c, acc);
  }
}

// ---------------------------------------------------------------- dots
// A wave takes eight entries; its lanes hold 16-byte pieces of both rows.
constexpr uint32_t DOTS = 8;

template <class T, int VEC>
__global__ __launch_bounds__(256) void k_dots(KSel s, const T* __restrict__ g, int64_t ldg,
                                              const T* __restrict__ w, int64_t ldw, uint32_t d,
                                              T* __restrict__ dv) {
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
  const uint64_t first = ((uint64_t)blockIdx.x * 4 + wave) * DOTS;
  if (first >= s.total) return;
  const uint32_t e0 = (uint32_t)first;
  uint32_t row = 0, latent = 0;
  const bool good = lane < DOTS && e0 + lane < s.total && entry_of(s, e0 + lane, s.idx[e0 + lane], &row, &latent);
  const uint64_t ok = __ballot(good);
  float sum[DOTS] = {};
  for (uint32_t c = lane * VEC; c < (d + 64 * VEC - 1) / (64 * VEC) * (64 * VEC); c += 64 * VEC) {
    float a[DOTS][VEC], b[DOTS][VEC];
#pragma unroll
    for (uint32_t u = 0; u < DOTS; ++u) {
      const uint32_t r = __builtin_amdgcn_readlane(row, u), j = __builtin_amdgcn_readlane(latent, u);
#pragma unroll
      for (int i = 0; i < VEC; ++i) a[u][i] = b[u][i] = 0.f;
      if (c < d && (ok >> u & 1)) {
        load_vec<T, VEC>(g + (int64_t)r * ldg + c, a[u]);
        load_vec<T, VEC>(w + (int64_t)j * ldw + c, b[u]);
      }
    }
#pragma unroll
    for (uint32_t u = 0; u < DOTS; ++u)
#pragma unroll
      for (int i = 0; i < VEC; ++i) sum[u] = fmaf(a[u][i], b[u][i], sum[u]);
  }
  // eight sums over 64 lanes: each of the first three exchanges halves the
  // number of sums a lane carries, so lane l ends with the sum of entry l % 8
#pragma unroll
  for (uint32_t h = 4, o = 4; h; h >>= 1, o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (uint32_t u = 0; u < h; ++u) {
      const float keep = up ? sum[u + h] : sum[u], give = up ? sum[u] : sum[u + h];
      sum[u] = keep + __shfl_xor(give, o);
    }
  }
  float v = sum[0];
#pragma unroll
  for (uint32_t o = 8; o < 64; o <<= 1) v += __shfl_xor(v, o);
  if (lane < DOTS && e0 + lane < s.total) dv[e0 + lane] = from_f32<T>(v);
}

// ---------------------------------------------------------------- host side
bool aligned16(const void* p, int64_t ld, int64_t es) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * es) % 16 == 0;
}

// Rows straight from the selection: row-wise, or few enough reads that every
// row may look at every index (4096 rows and entries: 128 MB out of the
// caches, where the sort's three launches alone take longer).
bool rows_direct(const Selection& s) {
  return !s.flat || (s.total <= 8192 && s.rows * s.total <= (int64_t(1) << 24));
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
  const int64_t columns = std::max<int64_t>(1, ceil_div(d, 512));
  int64_t chunk = 64;
  while (chunk > 8 && ceil_div(s.total, chunk) * columns < 2048) chunk /= 2;
  chunk *= std::max<int64_t>(1, ceil_div(s.total, chunk * 16384));
  p.chunk = (uint32_t)chunk;
  p.chunks = (uint32_t)ceil_div(s.total, chunk);
  p.off_part = p.sort.total_bytes;
  p.off_part_c = p.off_part + align256((size_t)p.chunks * 2 * (size_t)d * 4);
  p.total = p.off_part_c + align256((size_t)p.chunks * 2 * 4);
  return p;
}

template <class T>
hipError_t run_sort(const SegArgs& a, const SortPlan& p, char* ws, hipStream_t s) {
  const KSel sel = ksel(a.sel);
  const T* coef = static_cast<const T*>(a.coef);
  const T* gate = static_cast<const T*>(a.gate);
  for (uint32_t pass = 0; pass < p.passes; ++pass) {
    KPass k;
    const bool last = pass + 1 == p.passes;
    uint32_t* keys = reinterpret_cast<uint32_t*>(ws + p.off_key);
    uint32_t* pos = reinterpret_cast<uint32_t*>(ws + p.off_pos);
    k.key_in = pass ? keys + (size_t)((pass - 1) & 1) * p.total : nullptr;
    k.pos_in = pass ? pos + (size_t)((pass - 1) & 1) * p.total : nullptr;
    k.key_out = last ? reinterpret_cast<uint32_t*>(ws + p.off_skey) : keys + (size_t)(pass & 1) * p.total;
    k.pos_out = last ? nullptr : pos + (size_t)(pass & 1) * p.total;
    k.other = reinterpret_cast<uint32_t*>(ws + p.off_other);
    k.coef = reinterpret_cast<float*>(ws + p.off_coef);
    k.cnt = reinterpret_cast<uint32_t*>(ws + p.off_cnt);
    k.coarse = reinterpret_cast<uint32_t*>(ws + p.off_coarse);
    k.keys = p.keys;
    k.total = p.total;
    k.per_block = p.per_block;
    k.bins = bins_of(p, pass);
    k.groups = (uint32_t)ceil_div(k.bins, GROUP);
    k.shift = p.width * pass;
    k.mask = p.width ? (1u << p.width) - 1 : 0xFFFFFFFFu;
    k.digit_bits = 0;
    while ((1u << k.digit_bits) < k.bins) ++k.digit_bits;
    k.blocks = p.blocks;
    k.by_row = a.by_row;
    const size_t lds = (size_t)k.bins * 4;
    hipLaunchKernelGGL(k_count, dim3(p.blocks), dim3(SORT_THREADS), lds, s, sel, k);
    hipLaunchKernelGGL(k_scan, dim3(k.groups), dim3(SORT_THREADS), 0, s, k);
    hipLaunchKernelGGL((k_place<T>), dim3(p.blocks), dim3(SORT_THREADS), lds, s, sel, k, coef, gate);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <class T>
hipError_t run_seg(const SegArgs& a, char* ws, hipStream_t s) {
  constexpr int64_t ES = sizeof(T), V = Vec<T>::N;
  const bool wide = a.d % V == 0 && aligned16(a.src, a.lds, ES) && aligned16(a.out, a.ldo, ES) && aligned16(a.bias, 0, ES);
  const int64_t span = 64 * (wide ? V : 1);
  const uint32_t columns = (uint32_t)std::max<int64_t>(1, ceil_div(a.d, span));
  KSeg k;
  k.src = a.src;
  k.bias = a.bias;
  k.out = a.out;
  k.coef_sum = a.coef_sum;
  k.lds = a.lds;
  k.ldo = a.ldo;
  k.keys = (uint32_t)(a.by_row ? a.sel.rows : a.sel.n);
  k.total = (uint32_t)a.sel.total;
  k.d = (uint32_t)a.d;
  if (a.by_row && rows_direct(a.sel)) {
    const dim3 grid(k.keys, columns);
    const T* coef = static_cast<const T*>(a.coef);
    const T* gate = static_cast<const T*>(a.gate);
    if (wide) hipLaunchKernelGGL((k_rows<T, (int)V>), grid, dim3(256), 0, s, ksel(a.sel), k, coef, gate);
    else hipLaunchKernelGGL((k_rows<T, 1>), grid, dim3(256), 0, s, ksel(a.sel), k, coef, gate);
    return hipGetLastError();
  }
  const SegPlan p = seg_plan(a.sel, a.d, a.by_row);
  const SortPlan& q = p.sort;
  if (a.sel.total) {
    const hipError_t e = run_sort<T>(a, q, ws, s);
    if (e != hipSuccess) return e;
  }
  k.skey = reinterpret_cast<const uint32_t*>(ws + q.off_skey);
  k.other = reinterpret_cast<const uint32_t*>(ws + q.off_other);
  k.coef = reinterpret_cast<const float*>(ws + q.off_coef);
  k.part = reinterpret_cast<float*>(ws + p.off_part);
  k.part_c = reinterpret_cast<float*>(ws + p.off_part_c);
  k.chunk = p.chunk;
  if (p.chunks) {
    const dim3 grid((uint32_t)ceil_div(p.chunks, 4), columns);
    if (wide) hipLaunchKernelGGL((k_seg<T, (int)V>), grid, dim3(256), 0, s, k);
    else hipLaunchKernelGGL((k_seg<T, 1>), grid, dim3(256), 0, s, k);
  }
  const dim3 grid((uint32_t)ceil_div(k.keys, JOIN_KEYS));
  if (wide) hipLaunchKernelGGL((k_join_runs<T, (int)V>), grid, dim3(256), 0, s, k);
  else hipLaunchKernelGGL((k_join_runs<T, 1>), grid, dim3(256), 0, s, k);
  return hipGetLastError();
}

template <class T>
hipError_t run_dots(const DotArgs& a, hipStream_t s) {
  constexpr int64_t ES = sizeof(T), V = Vec<T>::N;
  const bool wide = a.d % V == 0 && aligned16(a.g, a.ldg, ES) && aligned16(a.w, a.ldw, ES);
  const dim3 grid((uint32_t)ceil_div(a.sel.total, 4 * DOTS));
  const T* g = static_cast<const T*>(a.g);
  const T* w = static_cast<const T*>(a.w);
  T* dv = static_cast<T*>(a.dv);
  if (wide) hipLaunchKernelGGL((k_dots<T, (int)V>), grid, dim3(256), 0, s, ksel(a.sel), g, a.ldg, w, a.ldw, (uint32_t)a.d, dv);
  else hipLaunchKernelGGL((k_dots<T, 1>), grid, dim3(256), 0, s, ksel(a.sel), g, a.ldg, w, a.ldw, (uint32_t)a.d, dv);
  return hipGetLastError();
}

}  // namespace

size_t seg_workspace(const Selection& sel, int64_t d, bool by_row) {
  if (by_row && rows_direct(sel)) return 0;
  return seg_plan(sel, d, by_row).total;
}

hipError_t launch_seg(const SegArgs& a, void* ws, hipStream_t s) {
  const int64_t keys = a.by_row ? a.sel.rows : a.sel.n;
  if (keys == 0 || (a.d == 0 && !a.coef_sum)) return hipSuccess;
  return a.sel.dtype == DT_BF16 ? run_seg<bf16_t>(a, static_cast<char*>(ws), s)
                                : run_seg<float>(a, static_cast<char*>(ws), s);
}

hipError_t launch_dots(const DotArgs& a, hipStream_t s) {
  if (a.sel.total == 0) return hipSuccess;
  return a.sel.dtype == DT_BF16 ? run_dots<bf16_t>(a, s) : run_dots<float>(a, s);
}

}  // namespace tk
