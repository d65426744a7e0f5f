// Tokens sorted by expert, and back.
//
//   dispatch      rows[p] = x[e / k] for the entry e (token e / k, choice e % k)
//                 at place p: entries sorted by expert, equal experts in the
//                 order of the entries; those without an expert lie behind
//                 all others, as rows of zeros
//   combine       out[t] = sum over j of w[t, j] y[places[t, j]]
//   combine_grad  dy[p] = sum over the entries e at place p of w_e g[t_e],
//                 dw_e = <g[t_e], y[places_e]>
//
// All are bound by the rows that they move: 16384 tokens x 8 of 1024 bf16 (302
// MB) take 62 us, 50 of them the rows, at 6 TB/s, and 10 the sort; back with
// weights 4099 x 4 of 515 f32 (42 MB) 9.1; the gradient of 8192 x 8 of 1024 bf16
// (285 MB) 61, of which 54 the rows at 5.3 TB/s.  Few rows are bound by the
// launch (8 tokens x 2: 4.2 us in one, 3 for the way back).
//
// The sort is a stable counting sort on one digit, so that a place does not
// hang on timing.
#include <algorithm>

#include "topk_model.hpp"
#include "topk_ops_device.hpp"

namespace tk {

namespace {

constexpr uint32_t NONE = 0xFFFFFFFFu;
constexpr uint32_t DROPPED = 0x80000000u;   // an entry's position, of an entry without an expert
constexpr uint32_t SMALL_TOTAL = 4096;      // entries that every workgroup counts by itself
constexpr uint32_t SMALL_EXPERTS = 1024;
constexpr uint32_t SMALL_PER = 16;          // entries that one of those workgroups moves
constexpr uint32_t SORT_THREADS = 1024;
constexpr uint32_t SELF_SCAN = 32768;       // counts that every block of the sort adds up for itself
constexpr uint32_t MOVE_THREADS = 256;
constexpr uint32_t PIECE = 2;               // vectors of a row that a lane moves at a time

struct RoutePlan {
  bool small = false;
  uint32_t total = 0, bins = 0, blocks = 0, per_block = 0, digit_bits = 0;
  size_t off_cnt = 0, off_all = 0, off_pos = 0, total_bytes = 0;
};

RoutePlan route_plan(int64_t tokens, int64_t k, int64_t experts) {
  RoutePlan p;
  p.total = (uint32_t)(tokens * k);
  p.bins = (uint32_t)experts + 1;      // the last: entries without an expert
  while ((uint64_t(1) << p.digit_bits) < p.bins) ++p.digit_bits;
  p.small = p.total <= SMALL_TOTAL && experts <= SMALL_EXPERTS;
  if (p.small) return p;
  const int64_t total = std::max<int64_t>(p.total, 1);
  const int64_t blocks = std::min<int64_t>(256, ceil_div(total, SORT_THREADS));
  p.per_block = (uint32_t)(ceil_div(total, blocks * SORT_THREADS) * SORT_THREADS);
  p.blocks = (uint32_t)ceil_div(total, p.per_block);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  p.off_cnt = take((size_t)p.blocks * p.bins * 4);
  p.off_all = take((size_t)p.bins * 4);
  p.off_pos = take((size_t)p.total * 4);
  p.total_bytes = at;
  return p;
}

__device__ __forceinline__ uint32_t expert_of(const int64_t* experts, uint32_t e, uint32_t bins) {
  const int64_t i = experts[e];
  return (uint64_t)i < bins - 1 ? (uint32_t)i : bins - 1;
}

// Lanes of the wave with the same digit as this one, among those in `in`.
__device__ __forceinline__ uint64_t same_lanes(uint32_t digit, bool in, uint32_t digit_bits) {
  uint64_t same = __ballot(in);
  for (uint32_t b = 0; b < digit_bits; ++b) {
    const bool bit = digit >> b & 1u;
    const uint64_t m = __ballot(bit);
    same &= bit ? m : ~m;
  }
  return same;
}

// Exclusive prefix sums of v[0, n) in place, by the whole workgroup.
template <uint32_t THREADS>
__device__ __forceinline__ void block_scan(uint32_t* v, uint32_t n) {
  __shared__ uint32_t part[THREADS / 64];
  const uint32_t per = (n + THREADS - 1) / THREADS;
  const uint32_t i0 = min(threadIdx.x * per, n), i1 = min(i0 + per, n);
  uint32_t sum = 0;
  for (uint32_t i = i0; i < i1; ++i) sum += v[i];
  uint32_t up = sum;
#pragma unroll
  for (uint32_t o = 1; o < 64; o <<= 1) {
    const uint32_t t = __shfl_up(up, o);
    if (threadIdx.x % 64 >= o) up += t;
  }
  if (threadIdx.x % 64 == 63) part[threadIdx.x / 64] = up;
  __syncthreads();
  uint32_t at = up - sum;
  for (uint32_t w = 0; w < threadIdx.x / 64; ++w) at += part[w];
  for (uint32_t i = i0; i < i1; ++i) {
    const uint32_t x = v[i];
    v[i] = at;
    at += x;
  }
  __syncthreads();
}

// One row, or zeros, by a wave: PIECE vectors a lane in flight.
template <class U, int VEC>
__device__ __forceinline__ void copy_row(const U* src, U* dst, uint32_t d, bool zero) {
  typedef Bits<U, VEC> B;
  const uint32_t lane = threadIdx.x % 64;
  for (uint32_t c0 = 0; c0 < d; c0 += 64 * VEC * PIECE) {
    typename B::type v[PIECE];
#pragma unroll
    for (uint32_t i = 0; i < PIECE; ++i) {
      const uint32_t c = c0 + (i * 64 + lane) * VEC;
      v[i] = c < d && !zero ? B::load(src + column_of<VEC>(c, d)) : B::zero();
    }
#pragma unroll
    for (uint32_t i = 0; i < PIECE; ++i) {
      const uint32_t c = c0 + (i * 64 + lane) * VEC;
      if (c < d) B::store(dst + column_of<VEC>(c, d), v[i]);
    }
  }
}

// Few entries: every workgroup counts them all by itself and moves its own
// SMALL_PER of them, in one launch.
template <class U, int VEC>
__global__ __launch_bounds__(MOVE_THREADS) void k_dispatch_small(
    const U* __restrict__ x, const int64_t* __restrict__ experts, U* __restrict__ rows, int64_t* __restrict__ places,
    int64_t* __restrict__ offsets, uint64_t ldx, uint64_t ldr, uint32_t total, uint32_t k, uint32_t bins,
    uint32_t digit_bits, uint32_t d) {
  __shared__ uint32_t all[SMALL_EXPERTS + 1], before[SMALL_EXPERTS + 1];
  __shared__ uint32_t pos[SMALL_PER];
  for (uint32_t i = threadIdx.x; i < bins; i += MOVE_THREADS) all[i] = before[i] = 0;
  __syncthreads();
  const uint32_t e0 = blockIdx.x * SMALL_PER;
  for (uint32_t e = threadIdx.x; e < total; e += MOVE_THREADS) {
    const uint32_t key = expert_of(experts, e, bins);
    atomicAdd(&all[key], 1u);
    if (e < e0) atomicAdd(&before[key], 1u);
  }
  __syncthreads();
  block_scan<MOVE_THREADS>(all, bins);
  if (blockIdx.x == 0)
    for (uint32_t i = threadIdx.x; i < bins; i += MOVE_THREADS) offsets[i] = all[i];
  if (threadIdx.x < 64) {
    const uint32_t e = e0 + threadIdx.x;
    const bool in = threadIdx.x < SMALL_PER && e < total;
    const uint32_t key = in ? expert_of(experts, e, bins) : 0u;
    const uint64_t same = same_lanes(key, in, digit_bits);
    if (in) {
      const uint32_t at = all[key] + before[key] + __popcll(same & ((uint64_t(1) << threadIdx.x) - 1));
      const bool good = key < bins - 1;
      places[e] = good ? (int64_t)at : -1;
      pos[threadIdx.x] = at | (good ? 0u : DROPPED);
    }
  }
  __syncthreads();
  for (uint32_t i = threadIdx.x / 64; i < SMALL_PER && e0 + i < total; i += MOVE_THREADS / 64) {
    const uint32_t p = pos[i];
    copy_row<U, VEC>(x + (uint64_t)((e0 + i) / k) * ldx, rows + (uint64_t)(p & ~DROPPED) * ldr, d, p & DROPPED);
  }
}

// cnt[block][expert]: entries of each expert in the block's part.
__global__ __launch_bounds__(SORT_THREADS) void k_route_count(const int64_t* __restrict__ experts, uint32_t* __restrict__ cnt,
                                                              uint32_t total, uint32_t per_block, uint32_t bins) {
  extern __shared__ uint32_t hist[];
  for (uint32_t i = threadIdx.x; i < bins; i += SORT_THREADS) hist[i] = 0;
  __syncthreads();
  const uint32_t e0 = blockIdx.x * per_block;
  const uint32_t e1 = total - e0 < per_block ? total : e0 + per_block;
  for (uint32_t e = e0 + threadIdx.x; e < e1; e += SORT_THREADS) atomicAdd(&hist[expert_of(experts, e, bins)], 1u);
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < bins; i += SORT_THREADS) cnt[(size_t)blockIdx.x * bins + i] = hist[i];
}

// Per expert, the exclusive sums over the blocks in place of the counts, and
// their total.  A lane is an expert, sixteen waves share the blocks.
__global__ __launch_bounds__(SORT_THREADS) void k_route_scan(uint32_t* __restrict__ cnt, uint32_t* __restrict__ all,
                                                             uint32_t blocks, uint32_t bins) {
  __shared__ uint32_t part[16][64];
  const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  const uint32_t bin = blockIdx.x * 64 + lane;
  const uint32_t per = (blocks + 15) / 16;   // at most 16
  const uint32_t b0 = min(wave * per, blocks), b1 = min(b0 + per, blocks);
  uint32_t v[16], sum = 0;
#pragma unroll
  for (uint32_t i = 0; i < 16; ++i) {
    v[i] = (b0 + i < b1 && bin < bins) ? cnt[(size_t)(b0 + i) * bins + bin] : 0u;
    sum += v[i];
  }
  part[wave][lane] = sum;
  __syncthreads();
  uint32_t at = 0, whole = 0;
#pragma unroll
  for (uint32_t w = 0; w < 16; ++w) {
    if (w < wave) at += part[w][lane];
    whole += part[w][lane];
  }
#pragma unroll
  for (uint32_t i = 0; i < 16; ++i) {
    if (b0 + i < b1 && bin < bins) cnt[(size_t)(b0 + i) * bins + bin] = at;
    at += v[i];
  }
  if (wave == 0 && bin < bins) all[bin] = whole;
}

// SCANNED: cnt holds the sums over the blocks and `all` their totals
// (k_route_scan); otherwise every block adds the counts up for itself, which
// for up to SELF_SCAN of them takes less than a launch (16384 x 8 entries, 128
// experts: 15 us in three launches, 11 in two).
template <bool SCANNED>
__global__ __launch_bounds__(SORT_THREADS) void k_route_place(const int64_t* __restrict__ experts, const uint32_t* __restrict__ cnt,
                                                              const uint32_t* __restrict__ all, int64_t* __restrict__ places,
                                                              int64_t* __restrict__ offsets, uint32_t* __restrict__ pos,
                                                              uint32_t total, uint32_t per_block, uint32_t bins, uint32_t digit_bits) {
  extern __shared__ uint32_t next[];   // the place of the next entry of each expert; without SCANNED also the blocks' before
  const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  if constexpr (SCANNED) {
    for (uint32_t i = threadIdx.x; i < bins; i += SORT_THREADS) next[i] = all[i];
  } else {
    for (uint32_t i = threadIdx.x; i < 2 * bins; i += SORT_THREADS) next[i] = 0;
    __syncthreads();
    for (uint32_t b = lane; b < bins; b += 64) {
      uint32_t sum = 0, before = 0;
#pragma unroll 8
      for (uint32_t i = wave; i < gridDim.x; i += SORT_THREADS / 64) {
        const uint32_t v = cnt[(size_t)i * bins + b];
        sum += v;
        before += i < blockIdx.x ? v : 0u;
      }
      atomicAdd(&next[b], sum);
      atomicAdd(&next[bins + b], before);
    }
  }
  __syncthreads();
  block_scan<SORT_THREADS>(next, bins);
  if (blockIdx.x == 0)
    for (uint32_t i = threadIdx.x; i < bins; i += SORT_THREADS) offsets[i] = next[i];
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < bins; i += SORT_THREADS) next[i] += SCANNED ? cnt[(size_t)blockIdx.x * bins + i] : next[bins + i];
  __syncthreads();
  const uint32_t e0 = blockIdx.x * per_block;
  const uint32_t e1 = total - e0 < per_block ? total : e0 + per_block;
  for (uint32_t c = e0; c < e1; c += SORT_THREADS) {
    const uint32_t e = c + threadIdx.x;
    const bool in = e < e1;
    const uint32_t key = in ? expert_of(experts, e, bins) : 0u;
    const uint64_t same = same_lanes(key, in, digit_bits);
    const uint32_t rank = __popcll(same & ((uint64_t(1) << lane) - 1));
    uint32_t at = 0;
    for (uint32_t w = 0; w < SORT_THREADS / 64; ++w) {
      if (w == wave && in) {
        at = next[key] + rank;
        if (rank == 0) next[key] = at + (uint32_t)__popcll(same);
      }
      __syncthreads();
    }
    if (in) {
      const bool good = key < bins - 1;
      places[e] = good ? (int64_t)at : -1;
      pos[e] = at | (good ? 0u : DROPPED);
    }
  }
}

// Each row of x is read once and written to the places of its token's entries.
// An item: PIECE * 64 vectors of one token's row, by a wave.
template <class U, int VEC, bool STREAM>
__global__ __launch_bounds__(MOVE_THREADS) void k_dispatch_move(const U* __restrict__ x, const uint32_t* __restrict__ pos,
                                                                U* __restrict__ rows, uint64_t ldx, uint64_t ldr, uint32_t k,
                                                                uint32_t d, uint32_t pieces, uint64_t items) {
  typedef Bits<U, VEC> B;
  const uint32_t lane = threadIdx.x % 64;
  const uint64_t item = (uint64_t)block_id() * (MOVE_THREADS / 64) + threadIdx.x / 64;
  if (item >= items) return;
  const uint64_t t = item / pieces;
  const uint32_t c0 = (uint32_t)(item % pieces) * (64 * VEC * PIECE);
  const U* src = x + t * ldx;
  typename B::type v[PIECE];
#pragma unroll
  for (uint32_t i = 0; i < PIECE; ++i) {
    const uint32_t c = c0 + (i * 64 + lane) * VEC;
    if (c < d) v[i] = B::load(src + column_of<VEC>(c, d));
  }
  for (uint32_t j = 0; j < k; ++j) {
    const uint32_t p = pos[t * k + j];
    U* dst = rows + (uint64_t)(p & ~DROPPED) * ldr;
#pragma unroll
    for (uint32_t i = 0; i < PIECE; ++i) {
      const uint32_t c = c0 + (i * 64 + lane) * VEC;
      if (c >= d) continue;
      const typename B::type w = p & DROPPED ? B::zero() : v[i];
      if constexpr (STREAM) B::stream(dst + column_of<VEC>(c, d), w);
      else B::store(dst + column_of<VEC>(c, d), w);
    }
  }
}

template <class U, int VEC>
hipError_t dispatch_typed(const topk_dispatch_args& a, const RoutePlan& p, char* ws, hipStream_t s) {
  const U* x = static_cast<const U*>(a.x);
  U* rows = static_cast<U*>(a.rows);
  const uint32_t k = (uint32_t)a.k, d = (uint32_t)a.d;
  if (p.small) {
    const uint32_t blocks = std::max<uint32_t>(1, (p.total + SMALL_PER - 1) / SMALL_PER);
    k_dispatch_small<U, VEC><<<blocks, MOVE_THREADS, 0, s>>>(x, a.experts, rows, a.places, a.offsets, (uint64_t)a.ldx, (uint64_t)a.ldr,
                                                             p.total, std::max(k, 1u), p.bins, p.digit_bits, d);
    return hipGetLastError();
  }
  uint32_t* cnt = reinterpret_cast<uint32_t*>(ws + p.off_cnt);
  uint32_t* all = reinterpret_cast<uint32_t*>(ws + p.off_all);
  uint32_t* pos = reinterpret_cast<uint32_t*>(ws + p.off_pos);
  k_route_count<<<p.blocks, SORT_THREADS, p.bins * 4, s>>>(a.experts, cnt, p.total, p.per_block, p.bins);
  if (p.blocks * p.bins <= SELF_SCAN) {
    k_route_place<false><<<p.blocks, SORT_THREADS, p.bins * 8, s>>>(a.experts, cnt, all, a.places, a.offsets, pos, p.total, p.per_block,
                                                                    p.bins, p.digit_bits);
  } else {
    k_route_scan<<<(p.bins + 63) / 64, SORT_THREADS, 0, s>>>(cnt, all, p.blocks, p.bins);
    k_route_place<true><<<p.blocks, SORT_THREADS, p.bins * 4, s>>>(a.experts, cnt, all, a.places, a.offsets, pos, p.total, p.per_block,
                                                                   p.bins, p.digit_bits);
  }
  if (d && p.total) {
    const uint32_t pieces = (d + 64 * VEC * PIECE - 1) / (64 * VEC * PIECE);
    const uint64_t items = (uint64_t)a.tokens * pieces;
    auto* move = (int64_t)p.total * a.d * (int64_t)sizeof(U) >= STREAM_BYTES ? k_dispatch_move<U, VEC, true> : k_dispatch_move<U, VEC, false>;
    move<<<wide_grid((items + 3) / 4), MOVE_THREADS, 0, s>>>(x, pos, rows, (uint64_t)a.ldx, (uint64_t)a.ldr, k, d, pieces, items);
  }
  return hipGetLastError();
}

// ---------------------------------------------------------------- combine
template <class W>
__device__ __forceinline__ float weight_of(const W* w, uint64_t e) {
  return w ? to_f32(w[e]) : 1.f;
}

// An item: 64 vectors of one token's output row, by a wave; the rows of up to
// AHEAD entries are in flight at a time.
template <class T, class W, int VEC>
__global__ __launch_bounds__(MOVE_THREADS) void k_combine(const T* __restrict__ y, const int64_t* __restrict__ places,
                                                          const W* __restrict__ weights, T* __restrict__ out, uint64_t ldy,
                                                          uint64_t ldo, uint64_t n, uint32_t k, uint32_t d, uint32_t pieces,
                                                          uint64_t items) {
  constexpr uint32_t AHEAD = 8;
  const uint32_t lane = threadIdx.x % 64;
  const uint64_t item = (uint64_t)block_id() * (MOVE_THREADS / 64) + threadIdx.x / 64;
  if (item >= items) return;
  const uint64_t t = item / pieces;
  const uint32_t c = ((uint32_t)(item % pieces) * 64 + lane) * VEC;
  if (c >= d) return;
  const uint32_t at = column_of<VEC>(c, d);
  float sum[VEC];
#pragma unroll
  for (int q = 0; q < VEC; ++q) sum[q] = 0.f;
  for (uint32_t j0 = 0; j0 < k; j0 += AHEAD) {
    float v[AHEAD][VEC], w[AHEAD];
#pragma unroll
    for (uint32_t j = 0; j < AHEAD; ++j) {
      const bool in = j0 + j < k;
      const uint64_t e = t * k + (in ? j0 + j : 0);
      const int64_t p = in ? places[e] : -1;
      const bool good = (uint64_t)p < n;
      w[j] = good ? weight_of(weights, e) : 0.f;
#pragma unroll
      for (int q = 0; q < VEC; ++q) v[j][q] = 0.f;
      if (good) load_vec<T, VEC>(y + (uint64_t)p * ldy + at, v[j]);
    }
#pragma unroll
    for (uint32_t j = 0; j < AHEAD; ++j)
#pragma unroll
      for (int q = 0; q < VEC; ++q) sum[q] = fmaf(w[j], v[j][q], sum[q]);
  }
  store_vec<T, VEC>(out + t * ldo + at, sum);
}

template <class T, class W, int VEC>
hipError_t combine_typed(const topk_combine_args& a, hipStream_t s) {
  const uint32_t d = (uint32_t)a.d;
  const uint32_t pieces = (d + 64 * VEC - 1) / (64 * VEC);
  const uint64_t items = (uint64_t)a.tokens * pieces;
  k_combine<T, W, VEC><<<wide_grid((items + 3) / 4), MOVE_THREADS, 0, s>>>(
      static_cast<const T*>(a.y), a.places, static_cast<const W*>(a.weights), static_cast<T*>(a.out), (uint64_t)a.ldy, (uint64_t)a.ldo,
      (uint64_t)a.n, (uint32_t)a.k, d, pieces, items);
  return hipGetLastError();
}

// ---------------------------------------------------------------- combine's gradient
// owner[p]: one entry at place p, or NONE; next[e]: another entry at the same
// place, or NONE.  A place that several entries name is a chain, linked in
// whatever order they came.
__global__ __launch_bounds__(MOVE_THREADS) void k_owner_clear(uint32_t* __restrict__ owner, uint64_t n) {
  const uint64_t i = (uint64_t)block_id() * MOVE_THREADS + threadIdx.x;
  if (i < n) owner[i] = NONE;
}

__global__ __launch_bounds__(MOVE_THREADS) void k_owner_link(const int64_t* __restrict__ places, uint32_t* __restrict__ owner,
                                                             uint32_t* __restrict__ next, uint64_t n, uint32_t total) {
  const uint64_t e = (uint64_t)block_id() * MOVE_THREADS + threadIdx.x;
  if (e >= total) return;
  const int64_t p = places[e];
  next[e] = (uint64_t)p < n ? atomicExch(&owner[p], (uint32_t)e) : NONE;
}

// Up to MAP_TOTAL entries: every workgroup goes through all of them for
// MAP_PLACES places of its own, in one launch instead of two (8 and 8192
// entries, as many places, 1.6 and 3.8 us against 3.0 and 4.7; 65536 would take 13
// against 6 to 10).
constexpr uint32_t MAP_TOTAL = 8192, MAP_PLACES = 1024;
__global__ __launch_bounds__(MAP_PLACES) void k_owner_map(const int64_t* __restrict__ places, uint32_t* __restrict__ owner,
                                                          uint32_t* __restrict__ next, uint64_t n, uint32_t total) {
  __shared__ uint32_t own[MAP_PLACES];
  constexpr uint32_t AHEAD = 8;
  own[threadIdx.x] = NONE;
  __syncthreads();
  const uint64_t p0 = (uint64_t)block_id() * MAP_PLACES;
  for (uint32_t e0 = threadIdx.x; e0 < total; e0 += MAP_PLACES * AHEAD) {
    uint64_t p[AHEAD];
#pragma unroll
    for (uint32_t i = 0; i < AHEAD; ++i) p[i] = (uint64_t)places[min(e0 + i * MAP_PLACES, total - 1)] - p0;
#pragma unroll
    for (uint32_t i = 0; i < AHEAD; ++i) {
      const uint32_t e = e0 + i * MAP_PLACES;
      if (e < total && p[i] < MAP_PLACES && p0 + p[i] < n) next[e] = atomicExch(&own[p[i]], e);
    }
  }
  __syncthreads();
  if (p0 + threadIdx.x < n) owner[p0 + threadIdx.x] = own[threadIdx.x];
}

// VEC columns of the sum over a chain.  Its order is not the same from call to
// call, so the terms are added as whole multiples of a power of two that 62 bits
// hold (a column's largest term tells which): such a sum has no order.  Where a
// term is not finite, neither is the sum, in any order.  A chain is two walks, each
// bound by the latency of its links: 8192 x 8 entries of 1024 bf16 at random places
// among 65536 take 96 us (distinct ones 61), among 512 420, among 64 2300, all at
// one 77000 (1.2 us an entry).
template <class T, class W, int VEC>
__device__ __forceinline__ void chain_sum(const T* column, const W* weights, const uint32_t* next, uint64_t ldg, uint32_t k, uint32_t e,
                                          float* out) {
  float top[VEC], bad[VEC], v[VEC];
  uint32_t count = 0;
#pragma unroll
  for (int q = 0; q < VEC; ++q) top[q] = bad[q] = 0.f;
#pragma unroll 1
  for (uint32_t j = e; j != NONE; j = next[j], ++count) {
    const float w = weight_of(weights, j);
    load_vec<T, VEC>(column + (uint64_t)(j / k) * ldg, v);
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
      const float t = w * v[q];
      top[q] = fmaxf(top[q], fabsf(t));
      if (!(fabsf(t) < INFINITY)) bad[q] += t;
    }
  }
  const int bits = 62 - (32 - __builtin_clz(count));
  int64_t sum[VEC];
#pragma unroll
  for (int q = 0; q < VEC; ++q) {
    int exponent = 0;
    frexpf(top[q], &exponent);   // top < 2^exponent
    top[q] = (float)(bits - exponent);
    sum[q] = 0;
  }
#pragma unroll 1
  for (uint32_t j = e; j != NONE; j = next[j]) {
    const float w = weight_of(weights, j);
    load_vec<T, VEC>(column + (uint64_t)(j / k) * ldg, v);
#pragma unroll
    for (int q = 0; q < VEC; ++q) sum[q] += (int64_t)rint(ldexp((double)(w * v[q]), (int)top[q]));
  }
#pragma unroll
  for (int q = 0; q < VEC; ++q) out[q] = bad[q] != 0.f ? bad[q] : (float)ldexp((double)sum[q], -(int)top[q]);
}

// Items below `total`: the entries, a wave each: dw_e, and dy's row if the entry
// owns it, PIECE vectors of both rows a lane in flight.  Items from `total` on:
// 64 rows of y each, of which the ones that no entry names are set to zero.
// STREAM: y is read, and dy stored, past the caches.  (Two, four and eight
// entries to a wave, their places looked up side by side, are slower: 8192 x 8
// entries of 1024 bf16 take 65, 71 and 82 us against 62.  The chains' sums would
// take 70 registers, and 62.0 us instead of 61.3: eight waves to a SIMD are asked
// for, which 51 without a spill allow.)
template <class T, class W, int VEC, bool STREAM>
__global__ __launch_bounds__(MOVE_THREADS) __attribute__((amdgpu_waves_per_eu(8))) void k_combine_grad(
    const T* __restrict__ g, const T* __restrict__ y, const int64_t* __restrict__ places, const W* __restrict__ weights,
    const uint32_t* __restrict__ owner, const uint32_t* __restrict__ next, T* __restrict__ dy, W* __restrict__ dw, uint64_t ldg,
    uint64_t ldy, uint64_t lddy, uint64_t n, uint32_t total, uint32_t k, uint32_t d, uint64_t items) {
  const uint32_t lane = threadIdx.x % 64;
  const uint64_t item = (uint64_t)block_id() * (MOVE_THREADS / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  if (item >= items) return;
  auto put = [&](T* p, const float* v) {
    if constexpr (STREAM && VEC > 1) stream_vec<T>(p, v);
    else store_vec<T, VEC>(p, v);
  };
  if (item >= total) {
    const uint64_t r0 = (item - total) * 64;
    const bool bare = r0 + lane < n && owner[r0 + lane] == NONE;
    float z[VEC];
#pragma unroll
    for (int q = 0; q < VEC; ++q) z[q] = 0.f;
    for (uint64_t m = __ballot(bare); m; m &= m - 1) {
      T* row = dy + (r0 + __builtin_ctzll(m)) * lddy;
      for (uint32_t c = lane * VEC; c < d; c += 64 * VEC) put(row + column_of<VEC>(c, d), z);
    }
    return;
  }
  const uint32_t e = (uint32_t)item;
  const int64_t p = places[e];
  if ((uint64_t)p >= n) {
    if (dw && lane == 0) dw[e] = from_f32<W>(0.f);
    return;
  }
  const T* grow = g + (uint64_t)(e / k) * ldg;
  const T* yrow = y + (uint64_t)p * ldy;
  T* dyrow = dy + (uint64_t)p * lddy;
  const bool mine = dy && owner[p] == e;
  const bool chain = mine && next[e] != NONE;
  const float w = weight_of(weights, e);
  float dot = 0.f;
  for (uint32_t c0 = 0; c0 < d; c0 += 64 * VEC * PIECE) {
    float a[PIECE][VEC], b[PIECE][VEC];
#pragma unroll
    for (uint32_t x = 0; x < PIECE; ++x) {
      const uint32_t at = column_of<VEC>(min(c0 + (x * 64 + lane) * VEC, d - 1), d);
      load_vec<T, VEC>(grow + at, a[x]);
      if (dw) {
        if constexpr (STREAM && VEC > 1) Vec<T>::unpack(read16_once(yrow + at), b[x]);
        else load_vec<T, VEC>(yrow + at, b[x]);
      }
    }
#pragma unroll
    for (uint32_t x = 0; x < PIECE; ++x) {
      const uint32_t c = c0 + (x * 64 + lane) * VEC;
      if (c >= d) continue;
      const uint32_t at = column_of<VEC>(c, d);
      if (dw) {
#pragma unroll
        for (int q = 0; q < VEC; ++q)
          if (at + q >= c) dot = fmaf(a[x][q], b[x][q], dot);   // a row's last vector counts its new columns only
      }
      if (!mine) continue;
      if (chain) continue;
#pragma unroll
      for (int q = 0; q < VEC; ++q) a[x][q] *= w;
      put(dyrow + at, a[x]);
    }
  }
  if (dw) {
    dot = wave_sum(dot);
    if (lane == 0) dw[e] = from_f32<W>(dot);
  }
  if (!chain) return;
#pragma unroll 1
  for (uint32_t c = lane * VEC; c < d; c += 64 * VEC) {
    const uint32_t at = column_of<VEC>(c, d);
    float sum[VEC];
    chain_sum<T, W, VEC>(g + at, weights, next, ldg, k, e, sum);
    put(dyrow + at, sum);
  }
}

template <class T, class W, int VEC>
hipError_t combine_grad_typed(const topk_combine_grad_args& a, char* ws, hipStream_t s) {
  const uint32_t total = (uint32_t)(a.tokens * a.k), d = (uint32_t)a.d;
  const bool rows = a.dy && a.n > 0 && d > 0;
  uint32_t* owner = reinterpret_cast<uint32_t*>(ws);
  uint32_t* next = reinterpret_cast<uint32_t*>(ws + align256((size_t)a.n * 4));
  if (rows && total <= MAP_TOTAL) {
    k_owner_map<<<wide_grid((uint64_t)ceil_div(a.n, MAP_PLACES)), MAP_PLACES, 0, s>>>(a.places, owner, next, (uint64_t)a.n, total);
  } else if (rows) {
    k_owner_clear<<<wide_grid((uint64_t)ceil_div(a.n, MOVE_THREADS)), MOVE_THREADS, 0, s>>>(owner, (uint64_t)a.n);
    k_owner_link<<<wide_grid((uint64_t)ceil_div(total, MOVE_THREADS)), MOVE_THREADS, 0, s>>>(a.places, owner, next, (uint64_t)a.n, total);
  }
  const uint64_t items = (uint64_t)total + (rows ? (uint64_t)ceil_div(a.n, 64) : 0);
  if (!items) return hipGetLastError();
  auto* grad = a.n * a.d * (int64_t)sizeof(T) >= STREAM_BYTES ? k_combine_grad<T, W, VEC, true> : k_combine_grad<T, W, VEC, false>;
  grad<<<wide_grid((items + 3) / 4), MOVE_THREADS, 0, s>>>(
      static_cast<const T*>(a.grad), static_cast<const T*>(a.y), a.places, static_cast<const W*>(a.weights), owner, next,
      static_cast<T*>(rows ? a.dy : nullptr), static_cast<W*>(a.dweights), (uint64_t)a.ldg, (uint64_t)a.ldy, (uint64_t)a.lddy,
      (uint64_t)a.n, total, std::max((uint32_t)a.k, 1u), d, items);
  return hipGetLastError();
}

template <class T, class F>
hipError_t by_width(int64_t d, F f) {
  if (d >= Vec<T>::N) return f(std::integral_constant<int, Vec<T>::N>());
  return f(std::integral_constant<int, 1>());
}

}  // namespace

size_t dispatch_workspace(int64_t tokens, int64_t k, int64_t experts) { return route_plan(tokens, k, experts).total_bytes; }

hipError_t launch_dispatch(const topk_dispatch_args& a, void* ws, hipStream_t s) {
  const RoutePlan p = route_plan(a.tokens, a.k, a.n_experts);
  char* w = static_cast<char*>(ws);
  if (a.dtype == TOPK_BF16)
    return by_width<bf16_t>(a.d, [&](auto v) { return dispatch_typed<uint16_t, v()>(a, p, w, s); });
  return by_width<float>(a.d, [&](auto v) { return dispatch_typed<uint32_t, v()>(a, p, w, s); });
}

hipError_t launch_combine(const topk_combine_args& a, hipStream_t s) {
  if (a.tokens == 0 || a.d == 0) return hipSuccess;
  if (a.dtype == TOPK_BF16) {
    if (a.wdtype == TOPK_BF16)
      return by_width<bf16_t>(a.d, [&](auto v) { return combine_typed<bf16_t, bf16_t, v()>(a, s); });
    return by_width<bf16_t>(a.d, [&](auto v) { return combine_typed<bf16_t, float, v()>(a, s); });
  }
  return by_width<float>(a.d, [&](auto v) { return combine_typed<float, float, v()>(a, s); });
}

size_t combine_grad_workspace(const topk_combine_grad_args& a) {
  if (!a.dy || a.n == 0 || a.d == 0) return 0;
  return align256((size_t)a.n * 4) + align256((size_t)(a.tokens * a.k) * 4);
}

hipError_t launch_combine_grad(const topk_combine_grad_args& a, void* ws, hipStream_t s) {
  char* w = static_cast<char*>(ws);
  if (a.dtype == TOPK_BF16) {
    if (a.wdtype == TOPK_BF16)
      return by_width<bf16_t>(a.d, [&](auto v) { return combine_grad_typed<bf16_t, bf16_t, v()>(a, w, s); });
    return by_width<bf16_t>(a.d, [&](auto v) { return combine_grad_typed<bf16_t, float, v()>(a, w, s); });
  }
  return by_width<float>(a.d, [&](auto v) { return combine_grad_typed<float, float, v()>(a, w, s); });
}

}  // namespace tk
