// The global 2-norm of many tensors, and their scaling to a largest norm.
//
//   norm = sqrt(sum over all tensors of g^2);  g *= min(1, max_norm / (norm + eps))
//
// Two launches per 256 tensors: squares, then scaling, in which every
// workgroup adds the partial sums of all workgroups itself, in order, rather
// than wait for a launch that does.  Both passes are bound by memory: the
// gradients of an autoencoder of 65536 latents (two of 65536 x 512 f32, 269
// MB) take 40 us to square, 6.7 TB/s, and 121 us in all when they are scaled;
// within the bound the second launch ends after the norm, 4.7 us.  48 tensors
// of a few thousand elements take 4.7 + 2.4 us, less than the host takes to
// list them.
//
// The squares are summed in 64 bits: an element of 1e30 or 1e-30 then
// neither overflows nor vanishes, the order of the sum does not show in the
// 32-bit result, and the pass stays bound by its reads (a conversion and a
// 64-bit multiply-add per element, of which a compute unit does 64 a clock).
#include <algorithm>

#include "topk_ops_device.hpp"

namespace tk {

namespace {

// A tensor is taken in pieces of CHUNK bytes counted from its address rounded
// down to 16, so that every load is a whole aligned vector; the first and last
// vector of a tensor are masked element by element (a load then sees bytes of
// the same 16 that are not the tensor's, and drops them; a store never
// touches them).
constexpr uint32_t THREADS = 256;
constexpr uint32_t AHEAD = 8;                            // vectors in flight per lane
constexpr uint32_t CHUNK = THREADS * AHEAD * 16;         // 32 KB

// The tensors of one launch ride in its argument block (4 KB at most).
constexpr int TABLE = 256;

struct Table {
  uint64_t p[TABLE];        // address; bit 63: bf16
  uint32_t first[TABLE];    // first piece of each tensor
  uint16_t last[TABLE];     // bytes of its last piece, minus 1
  uint32_t tensors, chunks;
};
static_assert(sizeof(Table) + 64 <= 4096, "the argument block");

// Piece `chunk` of a launch: its vectors' address, and the tensor's bytes
// within it.
struct Piece {
  uintptr_t at;
  uint32_t from, to;
  bool half;
};

__device__ __forceinline__ Piece piece_of(const Table& t, uint32_t chunk) {
  uint32_t lo = 0, hi = t.tensors;     // first[lo] <= chunk < first[hi]
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) / 2;
    if (t.first[mid] <= chunk) lo = mid;
    else hi = mid;
  }
  const uint64_t p = t.p[lo] & ~(uint64_t(1) << 63);
  const uint32_t end = lo + 1 < t.tensors ? t.first[lo + 1] : t.chunks;
  const uint32_t k = chunk - t.first[lo];
  Piece r;
  r.at = (p & ~(uint64_t)15) + (uint64_t)k * CHUNK;
  r.from = k ? 0u : (uint32_t)(p & 15);
  r.to = chunk + 1 == end ? (uint32_t)t.last[lo] + 1u : CHUNK;
  r.half = t.p[lo] >> 63;
  return r;
}

__device__ __forceinline__ double block_sum(double v) {
  __shared__ double part[THREADS / 64];
  v = wave_sum(v);
  if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = v;
  __syncthreads();
  const double r = (part[0] + part[1]) + (part[2] + part[3]);
  __syncthreads();
  return r;
}

template <class T>
__device__ __forceinline__ double squares(u32x4 q, uint32_t at, uint32_t from, uint32_t to) {
  constexpr int V = Vec<T>::N;
  float v[V];
  Vec<T>::unpack(q, v);
  if (at < from || at + 16 > to) {   // a tensor's first or last vector
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t b = at + i * sizeof(T);
      if (b < from || b >= to) v[i] = 0.f;
    }
  }
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < V; ++i) s = fma((double)v[i], (double)v[i], s);
  return s;
}

__global__ __launch_bounds__(THREADS) void k_squares(Table t, double* __restrict__ part) {
  double s = 0.0;
  for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const Piece p = piece_of(t, c);
    u32x4 q[AHEAD];
#pragma unroll
    for (uint32_t u = 0; u < AHEAD; ++u) {
      const uint32_t at = (u * THREADS + threadIdx.x) * 16;
      q[u] = u32x4{0u, 0u, 0u, 0u};
      if (at < p.to) q[u] = *reinterpret_cast<const u32x4*>(p.at + at);
    }
#pragma unroll
    for (uint32_t u = 0; u < AHEAD; ++u) {
      const uint32_t at = (u * THREADS + threadIdx.x) * 16;
      s += p.half ? squares<bf16_t>(q[u], at, p.from, p.to) : squares<float>(q[u], at, p.from, p.to);
    }
  }
  s = block_sum(s);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// The norm out of all workgroups' sums, the same in every workgroup.
__device__ __forceinline__ float norm_of(const double* __restrict__ part, uint32_t parts) {
  double s = 0.0;
#pragma unroll 8
  for (uint32_t i = threadIdx.x; i < parts; i += THREADS) s += part[i];
  return (float)sqrt(block_sum(s));
}

__global__ __launch_bounds__(THREADS) void k_norm(const double* __restrict__ part, uint32_t parts,
                                                  float* __restrict__ norm) {
  const float r = norm_of(part, parts);
  if (threadIdx.x == 0) norm[0] = r;
}

// The factor of every element: 1 where the norm is within bounds (and where
// norm + eps is 0), NaN when the norm is.
__device__ __forceinline__ float clip_factor(float norm, float max_norm, float eps) {
  const float den = norm + eps;
  const float f = max_norm / den;
  return den == 0.f ? 1.f : (f >= 1.f ? 1.f : f);
}

template <class T>
__device__ __forceinline__ void scale(u32x4 q, uintptr_t base, uint32_t at, uint32_t from, uint32_t to, float f) {
  constexpr int V = Vec<T>::N;
  float v[V];
  Vec<T>::unpack(q, v);
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] *= f;
  T* o = reinterpret_cast<T*>(base + at);
  if (at >= from && at + 16 <= to) {
    Vec<T>::store(o, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint32_t b = at + i * sizeof(T);
    if (b >= from && b < to) o[i] = from_f32<T>(v[i]);
  }
}

// Pieces last to first: the end of what the first pass read is still in the
// caches.
__global__ __launch_bounds__(THREADS) void k_scale(Table t, const double* __restrict__ part, uint32_t parts,
                                                   float* __restrict__ norm, float max_norm, float eps, int say) {
  const float n = norm_of(part, parts);
  if (say && blockIdx.x == 0 && threadIdx.x == 0) norm[0] = n;
  const float f = clip_factor(n, max_norm, eps);
  if (f == 1.f) return;
  for (uint32_t i = blockIdx.x; i < t.chunks; i += gridDim.x) {
    const Piece p = piece_of(t, t.chunks - 1 - i);
    u32x4 q[AHEAD];
#pragma unroll
    for (uint32_t u = 0; u < AHEAD; ++u) {
      const uint32_t at = (u * THREADS + threadIdx.x) * 16;
      q[u] = u32x4{0u, 0u, 0u, 0u};
      if (at < p.to) q[u] = *reinterpret_cast<const u32x4*>(p.at + at);
    }
#pragma unroll
    for (uint32_t u = 0; u < AHEAD; ++u) {
      const uint32_t at = (u * THREADS + threadIdx.x) * 16;
      if (at >= p.to) break;
      if (p.half) scale<bf16_t>(q[u], p.at, at, p.from, p.to, f);
      else scale<float>(q[u], p.at, at, p.from, p.to, f);
    }
  }
}

uint64_t chunks_of(const void* p, int64_t count, int64_t es) {
  if (!count) return 0;
  return ((reinterpret_cast<uintptr_t>(p) & 15) + (uint64_t)(count * es) + CHUNK - 1) / CHUNK;
}

// Calls fn(table) for each launch's worth of tensors.
template <class F>
hipError_t for_tables(const NormArgs& a, F fn) {
  int64_t i = 0;
  while (i < a.tensors) {
    Table t;
    t.tensors = 0;
    uint64_t chunks = 0;
    for (; i < a.tensors && t.tensors < TABLE; ++i) {
      const int64_t es = a.dtypes[i] == DT_BF16 ? 2 : 4;
      const uint64_t c = chunks_of(a.ptrs[i], a.counts[i], es);
      if (!c) continue;
      if (chunks + c > 0x7FFFFFFFull) break;
      const uint64_t p = reinterpret_cast<uintptr_t>(a.ptrs[i]);
      const uint32_t j = t.tensors++;
      t.p[j] = p | (a.dtypes[i] == DT_BF16 ? uint64_t(1) << 63 : 0);
      t.first[j] = (uint32_t)chunks;
      t.last[j] = (uint16_t)(((p & 15) + (uint64_t)(a.counts[i] * es) - 1) % CHUNK);
      chunks += c;
    }
    t.chunks = (uint32_t)chunks;
    if (!chunks) continue;
    const hipError_t e = fn(t);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Eight workgroups per compute unit, each with its share of the pieces.
uint32_t grid_of(const Table& t, int cus) { return std::min<uint32_t>(t.chunks, (uint32_t)cus * 8); }

}  // namespace

// One partial sum per workgroup: at most one per piece (a tensor of n bytes
// has at most n / CHUNK + 2), at most eight per compute unit of 512 and launch.
size_t norm_workspace(int64_t tensors, const int64_t* counts) {
  uint64_t pieces = 0;
  for (int64_t i = 0; i < tensors; ++i) pieces += counts[i] ? (uint64_t)counts[i] * 4 / CHUNK + 2 : 0;
  // a launch ends at TABLE tensors, or earlier at 2^31 pieces
  const uint64_t launches = (uint64_t)ceil_div(tensors, TABLE) + pieces / 0x40000000ull + 1;
  return align256((size_t)std::min<uint64_t>(pieces, launches * 4096) * 8);
}

hipError_t launch_norm(const NormArgs& a, void* ws, hipStream_t s) {
  double* part = static_cast<double*>(ws);
  const int cus = std::min(a.cus, 512);
  uint64_t parts = 0;
  hipError_t e = for_tables(a, [&](const Table& t) {
    const uint32_t grid = grid_of(t, cus);
    hipLaunchKernelGGL(k_squares, dim3(grid), dim3(THREADS), 0, s, t, part + parts);
    parts += grid;
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  if (!a.scale || !parts) {
    hipLaunchKernelGGL(k_norm, dim3(1), dim3(THREADS), 0, s, part, (uint32_t)parts, a.norm);
    return hipGetLastError();
  }
  int say = 1;
  return for_tables(a, [&](const Table& t) {
    hipLaunchKernelGGL(k_scale, dim3(grid_of(t, cus)), dim3(THREADS), 0, s, t, part, (uint32_t)parts, a.norm,
                       a.max_norm, a.eps, say);
    say = 0;
    return hipGetLastError();
  });
}

}  // namespace tk
