// The operators on a selection's entries: each entry e has a row r_e, a
// latent j_e and a coefficient.
//
//   by row      out[r] = bias + sum of coef_e src[j_e] over the entries of row r
//   by latent   out[j] = sum of coef_e src[r_e] over the entries of latent j
//   dots        dv_e = <g[r_e], w[j_e]>
#include "topk_ops_device.hpp"

namespace tk {

namespace {

// Row and latent of entry e; false for a padded slot or an index out of range.
__device__ __forceinline__ bool entry_of(const int64_t* __restrict__ idx, uint64_t e, uint64_t rows,
                                         uint64_t k, uint64_t n, bool flat, uint32_t* row,
                                         uint32_t* latent) {
  const int64_t i = idx[e];
  if (i < 0) return false;
  if (flat) {
    const uint64_t r = (uint64_t)i / n;
    if (r >= rows) return false;
    *row = (uint32_t)r;
    *latent = (uint32_t)((uint64_t)i - r * n);
    return true;
  }
  if ((uint64_t)i >= n) return false;
  *row = (uint32_t)(e / k);
  *latent = (uint32_t)i;
  return true;
}

// One workgroup per key; it walks every entry in order and adds those of its
// key, a thread per column.
template <class T>
__global__ __launch_bounds__(256) void k_seg_simple(SegArgs a, uint32_t d, uint64_t keys) {
  const uint64_t key = blockIdx.x;
  const int64_t* idx = a.sel.indices;
  const T* coef = static_cast<const T*>(a.coef);
  const T* gate = static_cast<const T*>(a.gate);
  const T* src = static_cast<const T*>(a.src);
  for (uint32_t c0 = 0; c0 < d || (c0 == 0 && a.coef_sum); c0 += 256) {
    const uint32_t c = c0 + threadIdx.x;
    float sum = 0.f, csum = 0.f;
    for (uint64_t e = 0; e < (uint64_t)a.sel.total; ++e) {
      uint32_t row, latent;
      if (!entry_of(idx, e, a.sel.rows, a.sel.k, a.sel.n, a.sel.flat, &row, &latent)) continue;
      if ((a.by_row ? row : latent) != key) continue;
      float w = to_f32(coef[e]);
      if (gate && !(to_f32(gate[e]) > 0.f)) continue;
      csum += w;
      if (c < d) sum = fmaf(w, to_f32(src[(int64_t)(a.by_row ? latent : row) * a.lds + c]), sum);
    }
    if (c < d) {
      if (a.bias) sum += to_f32(static_cast<const T*>(a.bias)[c]);
      static_cast<T*>(a.out)[(int64_t)key * a.ldo + c] = from_f32<T>(sum);
    }
    if (a.coef_sum && c0 == 0 && threadIdx.x == 0)
      static_cast<T*>(a.coef_sum)[key] = from_f32<T>(csum);
  }
}

template <class T>
__global__ __launch_bounds__(256) void k_dots(DotArgs a, uint32_t d) {
  const uint64_t e = (uint64_t)blockIdx.x * 4 + threadIdx.x / 64;
  const uint32_t lane = threadIdx.x % 64;
  if (e >= (uint64_t)a.sel.total) return;
  uint32_t row, latent;
  float sum = 0.f;
  if (entry_of(a.sel.indices, e, a.sel.rows, a.sel.k, a.sel.n, a.sel.flat, &row, &latent)) {
    const T* g = static_cast<const T*>(a.g) + (int64_t)row * a.ldg;
    const T* w = static_cast<const T*>(a.w) + (int64_t)latent * a.ldw;
    for (uint32_t c = lane; c < d; c += 64) sum = fmaf(to_f32(g[c]), to_f32(w[c]), sum);
  }
  sum = wave_sum(sum);
  if (lane == 0) static_cast<T*>(a.dv)[e] = from_f32<T>(sum);
}

}  // namespace

size_t seg_workspace(const Selection&, int64_t, bool) { return 0; }

hipError_t launch_seg(const SegArgs& a, void*, hipStream_t s) {
  const int64_t keys = a.by_row ? a.sel.rows : a.sel.n;
  if (keys == 0 || (a.d == 0 && !a.coef_sum)) return hipSuccess;
  if (a.sel.dtype == DT_BF16)
    hipLaunchKernelGGL((k_seg_simple<bf16_t>), dim3((uint32_t)keys), dim3(256), 0, s, a, (uint32_t)a.d, (uint64_t)keys);
  else
    hipLaunchKernelGGL((k_seg_simple<float>), dim3((uint32_t)keys), dim3(256), 0, s, a, (uint32_t)a.d, (uint64_t)keys);
  return hipGetLastError();
}

hipError_t launch_dots(const DotArgs& a, hipStream_t s) {
  if (a.sel.total == 0) return hipSuccess;
  const dim3 grid((uint32_t)ceil_div(a.sel.total, 4));
  if (a.sel.dtype == DT_BF16)
    hipLaunchKernelGGL((k_dots<bf16_t>), grid, dim3(256), 0, s, a, (uint32_t)a.d);
  else
    hipLaunchKernelGGL((k_dots<float>), grid, dim3(256), 0, s, a, (uint32_t)a.d);
  return hipGetLastError();
}

}  // namespace tk
