// Internal interface of the operators around the selection (dense product,
// sparse decode, gradient norm): the host checks call these launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace tk {

enum : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_SILU = 3 };

// Rows of a matrix operand are shorter than this, in elements: those of a tile
// (256 of bf16, 128 of f32) then stay below 2^31 bytes, the range of the
// offsets within it.
constexpr int64_t WIDTH_MAX = int64_t(1) << 22;

// One operand of a product, [rows, red] with `red` the summed axis: element
// (r, c) sits at p[r * ld + c], or at p[c * ld + r] when `trans`.
struct Operand {
  const void* p = nullptr;
  int64_t ld = 0;
  bool trans = false;
  bool padded = false;   // not trans: rows go on with zeros up to whole 16 bytes
};

// C[m, n] = epilogue(A[m, k] B[n, k]^T)
struct GemmArgs {
  Operand a, b;
  int64_t m = 0, n = 0, k = 0;
  int dtype = 1;
  int act = ACT_NONE;
  const void* bias = nullptr;       // [n]
  const void* residual = nullptr;   // [m, n], row stride ldr
  int64_t ldr = 0;
  void* c = nullptr;                // [m, n], row stride ldc
  int64_t ldc = 0;
  void* pre = nullptr;              // optional: the pre-activation, row stride ldp
  int64_t ldp = 0;
  int cus = 256;
};

size_t gemm_workspace(const GemmArgs& g);
hipError_t launch_gemm(const GemmArgs& g, void* ws, hipStream_t s);

// dz = dy * act'(pre) into `dz` (null: not wanted), its rows filled up with
// zeros to whole 16 bytes, and its column sums into `db` (null: not wanted).
struct SlopeArgs {
  const void* dy = nullptr;
  int64_t ldd = 0;
  const void* pre = nullptr;
  int64_t ldp = 0;
  int64_t m = 0, n = 0;
  int dtype = 1;
  int act = ACT_NONE;
  void* dz = nullptr;
  int64_t ldz = 0;
  void* db = nullptr;
};

size_t slope_workspace(const SlopeArgs& a);
hipError_t launch_slope(const SlopeArgs& a, void* ws, hipStream_t s);

// out[r] = bias + part[0][r] + part[1][r] + ..., in this order: sums that were
// split, with rows of `ldpart` floats (a multiple of 4).
struct JoinArgs {
  const float* part = nullptr;      // [split][m][ldpart]
  uint32_t split = 0, ldpart = 0;
  int64_t m = 0, n = 0;
  int dtype = 1;
  const void* bias = nullptr;       // [n], or null
  void* out = nullptr;              // [m, n], row stride ldo
  int64_t ldo = 0;
};
hipError_t launch_join(const JoinArgs& a, hipStream_t s);

// The gradients of a product: dx[m, k] = dz[m, n] W[n, k], dw[n, k] = dz^T x,
// db.  `x` and `w` as operands of the product they come from.
struct GradArgs {
  SlopeArgs slope;       // dy, pre, sizes, type, activation and db; the rest is filled in
  int64_t k = 0;
  Operand x, w;
  void* dx = nullptr;    // null: not wanted
  int64_t lddx = 0;
  void* dw = nullptr;
  int64_t lddw = 0;
  int cus = 256;
};

size_t grad_workspace(const GradArgs& a);
hipError_t launch_grad(const GradArgs& a, void* ws, hipStream_t s);

// A selection: `total` entries.  flat: index = row * n + latent; otherwise
// entry e belongs to row e / k and its index is the latent.
struct Selection {
  const void* values = nullptr;
  const int64_t* indices = nullptr;
  int64_t rows = 0, k = 0, n = 0, total = 0;
  int dtype = 1;
  bool flat = false;
};

// out[key] = bias + sum over the entries of `key` of coef * src[other]:
// by_row: key = row, src has a row per latent; otherwise key = latent.
struct SegArgs {
  bool by_row = true;
  const void* src = nullptr;
  int64_t lds = 0;
  const void* bias = nullptr;       // [d], or null
  void* out = nullptr;              // null: not wanted
  int64_t ldo = 0;
  void* coef_sum = nullptr;         // sum of coef per key; null: not wanted
  // by latent only: dots[e] = <src[row_e], other[latent_e]> on the way; null: not wanted
  const void* other = nullptr;
  int64_t ldother = 0;
  void* dots = nullptr;
};

// One or two such sums over the same selection and coefficients.
struct SegCall {
  Selection sel;
  const void* coef = nullptr;       // values, or the gradient of the values
  const void* gate = nullptr;       // entries whose gate value is not > 0 count as 0 (null: none)
  int64_t d = 0;
  int parts = 0;
  SegArgs part[2];
};

// Scratch of a call with a sum by row, by latent, or both.
size_t seg_workspace(const Selection& sel, int64_t d, bool by_row, bool by_latent);
hipError_t launch_seg(const SegCall& a, void* ws, hipStream_t s);

// dv[e] = <g[row_e], w[latent_e]> (0 for padded entries)
struct DotArgs {
  Selection sel;
  const void* g = nullptr;
  int64_t ldg = 0;
  const void* w = nullptr;
  int64_t ldw = 0;
  int64_t d = 0;
  void* dv = nullptr;
};
hipError_t launch_dots(const DotArgs& a, hipStream_t s);

// Global 2-norm of many tensors, and their scaling.
struct NormArgs {
  void* const* ptrs = nullptr;
  const int64_t* counts = nullptr;
  const int32_t* dtypes = nullptr;
  int64_t tensors = 0;
  bool scale = false;
  float max_norm = 0.f, eps = 0.f;
  float* norm = nullptr;
  int cus = 256;
};
size_t norm_workspace(int64_t tensors, const int64_t* counts);
hipError_t launch_norm(const NormArgs& a, void* ws, hipStream_t s);

int device_cus_now();

__host__ __device__ inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace tk
