// The global 2-norm of many tensors, and their scaling to a largest norm.
//
//   norm = sqrt(sum over all tensors of g^2);  g *= min(1, max_norm / (norm + eps))
//
// The squares are summed in 64 bits: an element of 1e30 or 1e-30 then
// neither overflows nor vanishes, the order of the sum does not show in the
// 32-bit result, and the pass stays bound by its reads (one 64-bit multiply
// and add per element, of which a compute unit does 64 a clock).
#include "topk_ops_device.hpp"

namespace tk {

namespace {

// The tensors of one launch ride in its argument block.
constexpr int TABLE = 128;
constexpr uint32_t CHUNK = 16384;      // elements per workgroup

struct Table {
  void* p[TABLE];
  uint64_t count[TABLE];
  uint32_t first[TABLE + 1];           // first chunk of each tensor
  uint32_t tensors;
  uint32_t bf16[TABLE / 32];           // one bit per tensor
};

__device__ __forceinline__ uint32_t find(const Table& t, uint32_t chunk) {
  uint32_t lo = 0, hi = t.tensors;     // first[lo] <= chunk < first[hi]
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) / 2;
    if (t.first[mid] <= chunk) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ double block_sum(double v) {
  __shared__ double part[4];
  v = wave_sum(v);
  if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = v;
  __syncthreads();
  const double r = (part[0] + part[1]) + (part[2] + part[3]);
  __syncthreads();
  return r;
}

__global__ __launch_bounds__(256) void k_squares(Table t, double* __restrict__ part) {
  const uint32_t i = find(t, blockIdx.x);
  const uint64_t e0 = (uint64_t)(blockIdx.x - t.first[i]) * CHUNK;
  const uint64_t e1 = e0 + CHUNK < t.count[i] ? e0 + CHUNK : t.count[i];
  double s = 0.0;
  if (t.bf16[i / 32] >> (i % 32) & 1u) {
    const bf16_t* p = static_cast<const bf16_t*>(t.p[i]);
    for (uint64_t e = e0 + threadIdx.x; e < e1; e += 256) {
      const double v = to_f32(p[e]);
      s = fma(v, v, s);
    }
  } else {
    const float* p = static_cast<const float*>(t.p[i]);
    for (uint64_t e = e0 + threadIdx.x; e < e1; e += 256) {
      const double v = p[e];
      s = fma(v, v, s);
    }
  }
  s = block_sum(s);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__global__ __launch_bounds__(256) void k_norm(const double* __restrict__ part, uint32_t parts,
                                              float* __restrict__ norm) {
  double s = 0.0;
  for (uint32_t i = threadIdx.x; i < parts; i += 256) s += part[i];
  s = block_sum(s);
  if (threadIdx.x == 0) norm[0] = (float)sqrt(s);
}

// The factor of every element: 1 where the norm is within bounds (and where
// norm + eps is 0), NaN when the norm is.
__device__ __forceinline__ float clip_factor(float norm, float max_norm, float eps) {
  const float den = norm + eps;
  const float f = max_norm / den;
  return den == 0.f ? 1.f : (f >= 1.f ? 1.f : f);
}

__global__ __launch_bounds__(256) void k_scale(Table t, const float* __restrict__ norm, float max_norm,
                                               float eps) {
  const float f = clip_factor(norm[0], max_norm, eps);
  if (f == 1.f) return;
  const uint32_t i = find(t, blockIdx.x);
  const uint64_t e0 = (uint64_t)(blockIdx.x - t.first[i]) * CHUNK;
  const uint64_t e1 = e0 + CHUNK < t.count[i] ? e0 + CHUNK : t.count[i];
  if (t.bf16[i / 32] >> (i % 32) & 1u) {
    bf16_t* p = static_cast<bf16_t*>(t.p[i]);
    for (uint64_t e = e0 + threadIdx.x; e < e1; e += 256) p[e] = from_f32<bf16_t>(to_f32(p[e]) * f);
  } else {
    float* p = static_cast<float*>(t.p[i]);
    for (uint64_t e = e0 + threadIdx.x; e < e1; e += 256) p[e] *= f;
  }
}

// Calls fn(table, chunks) for each launch's worth of tensors.
template <class F>
hipError_t for_tables(const NormArgs& a, F fn) {
  int64_t i = 0;
  while (i < a.tensors) {
    Table t;
    t.tensors = 0;
    for (uint32_t& w : t.bf16) w = 0;
    uint64_t chunks = 0;
    while (i < a.tensors && t.tensors < TABLE) {
      const uint64_t c = (uint64_t)ceil_div(a.counts[i], CHUNK);
      if (chunks && chunks + c > 0x7FFFFFFFull) break;
      if (c) {
        const uint32_t j = t.tensors++;
        t.p[j] = a.ptrs[i];
        t.count[j] = (uint64_t)a.counts[i];
        t.first[j] = (uint32_t)chunks;
        if (a.dtypes[i] == DT_BF16) t.bf16[j / 32] |= 1u << (j % 32);
        chunks += c;
      }
      ++i;
    }
    t.first[t.tensors] = (uint32_t)chunks;
    if (!chunks) continue;
    const hipError_t e = fn(t, (uint32_t)chunks);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

uint64_t all_chunks(int64_t tensors, const int64_t* counts) {
  uint64_t c = 0;
  for (int64_t i = 0; i < tensors; ++i) c += (uint64_t)ceil_div(counts[i], CHUNK);
  return c;
}

}  // namespace

size_t norm_workspace(int64_t tensors, const int64_t* counts) {
  return align256((size_t)all_chunks(tensors, counts) * 8);
}

hipError_t launch_norm(const NormArgs& a, void* ws, hipStream_t s) {
  double* part = static_cast<double*>(ws);
  uint64_t done = 0;
  hipError_t e = for_tables(a, [&](const Table& t, uint32_t chunks) {
    hipLaunchKernelGGL(k_squares, dim3(chunks), dim3(256), 0, s, t, part + done);
    done += chunks;
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_norm, dim3(1), dim3(256), 0, s, part, (uint32_t)done, a.norm);
  e = hipGetLastError();
  if (e != hipSuccess || !a.scale) return e;
  return for_tables(a, [&](const Table& t, uint32_t chunks) {
    hipLaunchKernelGGL(k_scale, dim3(chunks), dim3(256), 0, s, t, a.norm, a.max_norm, a.eps);
    return hipGetLastError();
  });
}

}  // namespace tk
