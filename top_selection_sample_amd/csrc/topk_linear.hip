// The dense product with its epilogue, and the pass that a backward of it
// starts with (the slope of the activation, and the bias gradient).
//
//   y = act(x W^T + b) + residual
//   dz = dy * act'(z);  dx = dz W;  dW = dz^T x;  db = column sums of dz
#include "topk_ops_device.hpp"

namespace tk {

namespace {

// ---------------------------------------------------------------- epilogue
struct Epi {
  const void* bias;
  const void* residual;
  void* c;
  void* pre;
  int64_t ldr, ldc, ldp;
};

// ---------------------------------------------------------------- product
// 64 x 64 outputs per workgroup of 256 threads, 4 x 4 per thread, the summed
// axis in steps of 16 through LDS.
template <class T, int ACT>
__global__ __launch_bounds__(256) void k_gemm_simple(const T* __restrict__ a, const T* __restrict__ b,
                                                     uint32_t m, uint32_t n, uint32_t k,
                                                     int64_t a_row, int64_t a_red, int64_t b_row,
                                                     int64_t b_red, Epi e) {
  __shared__ float sa[16][65], sb[16][65];
  const uint32_t m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
  const uint32_t tr = threadIdx.x / 16, tc = threadIdx.x % 16;
  float acc[4][4] = {};
  for (uint32_t k0 = 0; k0 < k; k0 += 16) {
    for (uint32_t i = threadIdx.x; i < 1024; i += 256) {
      const uint32_t r = i / 16, c = i % 16;
      sa[c][r] = (m0 + r < m && k0 + c < k) ? to_f32(a[(m0 + r) * a_row + (k0 + c) * a_red]) : 0.f;
      sb[c][r] = (n0 + r < n && k0 + c < k) ? to_f32(b[(n0 + r) * b_row + (k0 + c) * b_red]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (uint32_t c = 0; c < 16; ++c) {
      float x[4], y[4];
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) {
        x[i] = sa[c][tr * 4 + i];
        y[i] = sb[c][tc + i * 16];
      }
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i)
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (uint32_t i = 0; i < 4; ++i) {
    const uint32_t r = m0 + tr * 4 + i;
    if (r >= m) continue;
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) {
      const uint32_t c = n0 + tc + j * 16;
      if (c >= n) continue;
      float z = acc[i][j];
      if (e.bias) z += to_f32(static_cast<const T*>(e.bias)[c]);
      if (e.pre) static_cast<T*>(e.pre)[r * e.ldp + c] = from_f32<T>(z);
      float y = act_of<ACT>(z);
      if (e.residual) y += to_f32(static_cast<const T*>(e.residual)[r * e.ldr + c]);
      static_cast<T*>(e.c)[r * e.ldc + c] = from_f32<T>(y);
    }
  }
}

template <class T, int ACT>
hipError_t run_simple(const GemmArgs& g, hipStream_t s) {
  const Epi e{g.bias, g.residual, g.c, g.pre, g.ldr, g.ldc, g.ldp};
  const dim3 grid((uint32_t)ceil_div(g.n, 64), (uint32_t)ceil_div(g.m, 64));
  hipLaunchKernelGGL((k_gemm_simple<T, ACT>), grid, dim3(256), 0, s, static_cast<const T*>(g.a.p),
                     static_cast<const T*>(g.b.p), (uint32_t)g.m, (uint32_t)g.n, (uint32_t)g.k,
                     g.a.trans ? 1 : g.a.ld, g.a.trans ? g.a.ld : 1, g.b.trans ? 1 : g.b.ld,
                     g.b.trans ? g.b.ld : 1, e);
  return hipGetLastError();
}

template <class T>
hipError_t run_act(const GemmArgs& g, hipStream_t s) {
  switch (g.act) {
    case ACT_RELU: return run_simple<T, ACT_RELU>(g, s);
    case ACT_GELU: return run_simple<T, ACT_GELU>(g, s);
    case ACT_SILU: return run_simple<T, ACT_SILU>(g, s);
    default: return run_simple<T, ACT_NONE>(g, s);
  }
}

// ---------------------------------------------------------------- slope pass
// dz = dy * act'(z), and the column sums of dz in 32 bits: a workgroup of
// four waves takes 64 VEC columns and a block of rows; each lane sums its VEC
// columns down the block's rows, the four waves join in LDS, and one partial
// row per block goes to the workspace.  The sums are joined by k_join_rows in
// block order.
constexpr uint32_t SLOPE_ROWS = 64;   // rows per workgroup

template <class T, int ACT, int VEC>
__global__ __launch_bounds__(256) void k_slope(const T* __restrict__ dy, const T* __restrict__ pre,
                                               T* __restrict__ dz, float* __restrict__ part,
                                               uint32_t m, uint32_t n, int64_t ldd, int64_t ldp,
                                               int64_t ldz, uint32_t rows_per) {
  const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  const uint32_t c = (blockIdx.x * 64 + lane) * VEC;
  const uint32_t r0 = blockIdx.y * rows_per;
  const uint32_t r1 = r0 + rows_per < m ? r0 + rows_per : m;
  float sum[VEC] = {};
  if (c < n) {
    for (uint32_t r = r0 + wave; r < r1; r += 4) {
      float v[VEC];
      load_vec<T, VEC>(dy + (int64_t)r * ldd + c, v);
      if constexpr (ACT != ACT_NONE) {
        float z[VEC];
        load_vec<T, VEC>(pre + (int64_t)r * ldp + c, z);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          if constexpr (ACT == ACT_RELU) v[i] = z[i] <= 0.f ? 0.f : v[i];
          else v[i] *= slope_of<ACT>(z[i]);
        }
        if (dz) store_vec<T, VEC>(dz + (int64_t)r * ldz + c, v);
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) sum[i] += v[i];
    }
  }
  if (!part) return;
  __shared__ float join[4][64 * VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) join[wave][lane * VEC + i] = sum[i];
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < 64 * VEC; i += 256) {
    const uint32_t cc = blockIdx.x * 64 * VEC + i;
    if (cc < n)
      part[(size_t)blockIdx.y * n + cc] = (join[0][i] + join[1][i]) + (join[2][i] + join[3][i]);
  }
}

template <class T>
__global__ __launch_bounds__(256) void k_join_rows(const float* __restrict__ part, T* __restrict__ out,
                                                   uint32_t blocks, uint32_t n) {
  const uint32_t c = blockIdx.x * 256 + threadIdx.x;
  if (c >= n) return;
  float s = 0.f;
  for (uint32_t b = 0; b < blocks; ++b) s += part[(size_t)b * n + c];
  out[c] = from_f32<T>(s);
}

// Blocks of rows: 64 rows each, at most 65535 blocks (grid dimension y).
uint32_t slope_rows(int64_t m) {
  const int64_t least = ceil_div(m, 65535);
  return (uint32_t)(least > SLOPE_ROWS ? least : SLOPE_ROWS);
}

bool aligned16(const void* p, int64_t ld, int64_t es) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * es) % 16 == 0;
}

template <class T, int ACT>
hipError_t run_slope(const SlopeArgs& a, void* ws, hipStream_t s) {
  const int64_t es = sizeof(T);
  const uint32_t rows_per = slope_rows(a.m);
  const uint32_t blocks = (uint32_t)ceil_div(a.m, rows_per);
  float* part = a.db ? static_cast<float*>(ws) : nullptr;
  const bool wide = a.n % Vec<T>::N == 0 && aligned16(a.dy, a.ldd, es) &&
                    (!a.pre || aligned16(a.pre, a.ldp, es)) && (!a.dz || aligned16(a.dz, a.ldz, es));
  const T* dy = static_cast<const T*>(a.dy);
  const T* pre = static_cast<const T*>(a.pre);
  T* dz = static_cast<T*>(a.dz);
  if (wide) {
    hipLaunchKernelGGL((k_slope<T, ACT, Vec<T>::N>), dim3((uint32_t)ceil_div(a.n, 64 * Vec<T>::N), blocks),
                       dim3(256), 0, s, dy, pre, dz, part, (uint32_t)a.m, (uint32_t)a.n, a.ldd, a.ldp,
                       a.ldz, rows_per);
  } else {
    hipLaunchKernelGGL((k_slope<T, ACT, 1>), dim3((uint32_t)ceil_div(a.n, 64), blocks), dim3(256), 0, s,
                       dy, pre, dz, part, (uint32_t)a.m, (uint32_t)a.n, a.ldd, a.ldp, a.ldz, rows_per);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.db) return e;
  hipLaunchKernelGGL((k_join_rows<T>), dim3((uint32_t)ceil_div(a.n, 256)), dim3(256), 0, s, part,
                     static_cast<T*>(a.db), blocks, (uint32_t)a.n);
  return hipGetLastError();
}

template <class T>
hipError_t run_slope_act(const SlopeArgs& a, void* ws, hipStream_t s) {
  switch (a.act) {
    case ACT_RELU: return run_slope<T, ACT_RELU>(a, ws, s);
    case ACT_GELU: return run_slope<T, ACT_GELU>(a, ws, s);
    case ACT_SILU: return run_slope<T, ACT_SILU>(a, ws, s);
    default: return run_slope<T, ACT_NONE>(a, ws, s);
  }
}

}  // namespace

size_t gemm_workspace(const GemmArgs&) { return 0; }

hipError_t launch_gemm(const GemmArgs& g, void*, hipStream_t s) {
  if (g.m == 0 || g.n == 0) return hipSuccess;
  return g.dtype == DT_BF16 ? run_act<bf16_t>(g, s) : run_act<float>(g, s);
}

size_t slope_workspace(const SlopeArgs& a) {
  if (!a.db) return 0;
  return align256((size_t)ceil_div(a.m, slope_rows(a.m)) * (size_t)a.n * 4);
}

hipError_t launch_slope(const SlopeArgs& a, void* ws, hipStream_t s) {
  if (a.n == 0 || (a.m == 0 && !a.db)) return hipSuccess;
  if (a.m == 0) {   // no rows: the sums are zero
    if (a.dtype == DT_BF16)
      hipLaunchKernelGGL((k_join_rows<bf16_t>), dim3((uint32_t)ceil_div(a.n, 256)), dim3(256), 0, s,
                         nullptr, static_cast<bf16_t*>(a.db), 0u, (uint32_t)a.n);
    else
      hipLaunchKernelGGL((k_join_rows<float>), dim3((uint32_t)ceil_div(a.n, 256)), dim3(256), 0, s,
                         nullptr, static_cast<float*>(a.db), 0u, (uint32_t)a.n);
    return hipGetLastError();
  }
  return a.dtype == DT_BF16 ? run_slope_act<bf16_t>(a, ws, s) : run_slope_act<float>(a, ws, s);
}

}  // namespace tk
