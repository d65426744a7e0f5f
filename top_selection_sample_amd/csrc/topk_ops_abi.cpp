// C ABI of the operators around the selection: argument checks, workspace
// carving, launches.  Nothing is enqueued before every check has passed.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <utility>
#include <vector>

#include "../../include/topk.h"
#include "topk_launch.hpp"
#include "topk_ops.hpp"

namespace {

constexpr int64_t SIZE_MAX31 = (int64_t(1) << 31) - 1;

bool bad_size(int64_t v) { return v < 0 || v > SIZE_MAX31; }

constexpr int64_t KEYS_MAX = int64_t(1) << 28;    // rows and latents of a selection: two digits of 14 bits

// Elements of a matrix (2^42 of them are more than any device holds): tile and
// workgroup counts then stay within 32 bits.
bool bad_area(int64_t a, int64_t b) { return a > 0 && b > (int64_t(1) << 42) / a; }

bool bad_width(int64_t d) { return d < 0 || d >= tk::WIDTH_MAX; }

int64_t elem(int dtype) { return dtype == TOPK_BF16 ? 2 : 4; }

// A [rows, cols] matrix: its row stride fits, and its address unless it is empty.
bool bad_matrix(const void* p, int64_t ld, int64_t rows, int64_t cols, int dtype) {
  if (bad_size(ld) || (rows > 1 && ld < cols)) return true;
  if (reinterpret_cast<uintptr_t>(p) % (uintptr_t)elem(dtype)) return true;
  return !p && rows > 0 && cols > 0;
}

int check_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return TOPK_OK;
  if (!ws || reinterpret_cast<uintptr_t>(ws) % 256) return TOPK_EINVAL;
  return have < need ? TOPK_EWORKSPACE : TOPK_OK;
}

int status(hipError_t e) { return e == hipSuccess ? TOPK_OK : TOPK_EHIP; }

bool bad_dtype(int dtype) { return dtype != TOPK_F32 && dtype != TOPK_BF16; }

// ---------------------------------------------------------------- linear
int linear_gemm(const topk_linear_args* a, tk::GemmArgs* g) {
  if (!a) return TOPK_EINVAL;
  if (bad_dtype(a->dtype)) return TOPK_EDTYPE;
  if (a->act < TOPK_ACT_NONE || a->act > TOPK_ACT_SILU) return TOPK_EINVAL;
  if (bad_size(a->m) || bad_width(a->n) || bad_width(a->k) || (a->x_trans && bad_width(a->m)) ||
      bad_area(a->m, a->n) || bad_area(a->m, a->k))
    return TOPK_EINVAL;
  const int64_t m = a->m, n = a->n, k = a->k;
  if (a->x_trans ? bad_matrix(a->x, a->ldx, k, m, a->dtype) : bad_matrix(a->x, a->ldx, m, k, a->dtype))
    return TOPK_EINVAL;
  if (a->w_trans ? bad_matrix(a->w, a->ldw, k, n, a->dtype) : bad_matrix(a->w, a->ldw, n, k, a->dtype))
    return TOPK_EINVAL;
  if (bad_matrix(a->y, a->ldy, m, n, a->dtype)) return TOPK_EINVAL;
  if (a->bias && bad_matrix(a->bias, n, 1, n, a->dtype)) return TOPK_EINVAL;
  if (a->residual && bad_matrix(a->residual, a->ldr, m, n, a->dtype)) return TOPK_EINVAL;
  if (a->pre && bad_matrix(a->pre, a->ldp, m, n, a->dtype)) return TOPK_EINVAL;
  // y over its own residual, but with rows elsewhere: one row's result would land on another's residual
  if (a->residual && a->residual == a->y && a->ldr != a->ldy && m > 1 && n > 0) return TOPK_EINVAL;
  g->a = tk::Operand{a->x, a->ldx, a->x_trans != 0};
  g->b = tk::Operand{a->w, a->ldw, a->w_trans != 0};
  g->m = m;
  g->n = n;
  g->k = k;
  g->dtype = a->dtype;
  g->act = a->act;
  g->bias = a->bias;
  g->residual = a->residual;
  g->ldr = a->ldr;
  g->c = a->y;
  g->ldc = a->ldy;
  g->pre = a->pre;
  g->ldp = a->ldp;
  g->cus = tk::device_cus_now();
  return TOPK_OK;
}

int linear_grad(const topk_linear_grad_args* a, tk::GradArgs* g) {
  if (!a) return TOPK_EINVAL;
  if (bad_dtype(a->dtype)) return TOPK_EDTYPE;
  if (a->act < TOPK_ACT_NONE || a->act > TOPK_ACT_SILU) return TOPK_EINVAL;
  if (bad_size(a->m) || bad_width(a->n) || bad_width(a->k) || (a->x_trans && bad_width(a->m)) ||
      bad_area(a->m, a->n) || bad_area(a->m, a->k))
    return TOPK_EINVAL;
  const int64_t m = a->m, n = a->n, k = a->k;
  const int dt = a->dtype;
  if (!a->dx && !a->dw && !a->db) return TOPK_EINVAL;
  if (bad_matrix(a->dy, a->ldd, m, n, dt)) return TOPK_EINVAL;
  if (a->act != TOPK_ACT_NONE && bad_matrix(a->pre, a->ldp, m, n, dt)) return TOPK_EINVAL;
  if (a->dw && (a->x_trans ? bad_matrix(a->x, a->ldx, k, m, dt) : bad_matrix(a->x, a->ldx, m, k, dt)))
    return TOPK_EINVAL;
  if (a->dx && (a->w_trans ? bad_matrix(a->w, a->ldw, k, n, dt) : bad_matrix(a->w, a->ldw, n, k, dt)))
    return TOPK_EINVAL;
  if (a->dx && bad_matrix(a->dx, a->lddx, m, k, dt)) return TOPK_EINVAL;
  if (a->dw && bad_matrix(a->dw, a->lddw, n, k, dt)) return TOPK_EINVAL;
  if (a->db && bad_matrix(a->db, n, 1, n, dt)) return TOPK_EINVAL;
  g->slope.dy = a->dy;
  g->slope.ldd = a->ldd;
  g->slope.pre = a->act != TOPK_ACT_NONE ? a->pre : nullptr;
  g->slope.ldp = a->ldp;
  g->slope.m = m;
  g->slope.n = n;
  g->slope.dtype = dt;
  g->slope.act = a->act;
  g->slope.db = a->db;
  g->k = k;
  g->x = tk::Operand{a->x, a->ldx, a->x_trans != 0};
  g->w = tk::Operand{a->w, a->ldw, a->w_trans != 0};
  g->dx = a->dx;
  g->lddx = a->lddx;
  g->dw = a->dw;
  g->lddw = a->lddw;
  g->cus = tk::device_cus_now();
  return TOPK_OK;
}

// ---------------------------------------------------------------- selection
int to_selection(const topk_selection* in, bool pointers, tk::Selection* s) {
  if (!in) return TOPK_EINVAL;
  if (bad_dtype(in->dtype)) return TOPK_EDTYPE;
  if (bad_size(in->rows) || bad_size(in->k) || bad_size(in->n)) return TOPK_EINVAL;
  if (in->rows >= KEYS_MAX || in->n >= KEYS_MAX) return TOPK_EINVAL;
  const int64_t total = in->flat ? in->k : in->rows * in->k;
  if (total > SIZE_MAX31) return TOPK_EINVAL;   // entries are numbered in 32 bits
  if (pointers && total > 0) {
    if (!in->values || !in->indices) return TOPK_EINVAL;
    if (reinterpret_cast<uintptr_t>(in->values) % (uintptr_t)elem(in->dtype) ||
        reinterpret_cast<uintptr_t>(in->indices) % 8)
      return TOPK_EINVAL;
  }
  s->values = in->values;
  s->indices = in->indices;
  s->rows = in->rows;
  s->k = in->k;
  s->n = in->n;
  s->total = total;
  s->dtype = in->dtype;
  s->flat = in->flat != 0;
  return TOPK_OK;
}

size_t decode_ws(const tk::Selection& s, int64_t d) {
  tk::SlopeArgs sums;
  sums.m = s.rows;
  sums.n = d;
  sums.dtype = s.dtype;
  sums.db = &sums;   // only whether it is wanted counts here
  return std::max(tk::seg_workspace(s, d, true, true), tk::slope_workspace(sums));
}

}  // namespace

namespace tk {

int device_cus_now() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  const int v = cached[dev].load(std::memory_order_relaxed);
  if (v > 0) return v;
  int cus = 0;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0)
    return 256;
  cached[dev].store(cus, std::memory_order_relaxed);
  return cus;
}

}  // namespace tk

extern "C" {

static_assert(sizeof(topk_linear_args) == 128, "topk_linear_args layout is part of the ABI");
static_assert(sizeof(topk_linear_grad_args) == 144, "topk_linear_grad_args layout is part of the ABI");
static_assert(sizeof(topk_selection) == 48, "topk_selection layout is part of the ABI");

int topk_linear_workspace_size(const topk_linear_args* args, size_t* bytes) {
  if (!bytes) return TOPK_EINVAL;
  tk::GemmArgs g;
  const int rc = linear_gemm(args, &g);
  if (rc) return rc;
  *bytes = tk::gemm_workspace(g);
  return TOPK_OK;
}

int topk_linear(const topk_linear_args* args, void* workspace, size_t workspace_bytes, void* stream) {
  tk::GemmArgs g;
  int rc = linear_gemm(args, &g);
  if (rc) return rc;
  rc = check_ws(workspace, workspace_bytes, tk::gemm_workspace(g));
  if (rc) return rc;
  return status(tk::launch_gemm(g, workspace, static_cast<hipStream_t>(stream)));
}

int topk_linear_grad_workspace_size(const topk_linear_grad_args* args, size_t* bytes) {
  if (!bytes) return TOPK_EINVAL;
  tk::GradArgs g;
  const int rc = linear_grad(args, &g);
  if (rc) return rc;
  *bytes = tk::grad_workspace(g);
  return TOPK_OK;
}

int topk_linear_grad(const topk_linear_grad_args* args, void* workspace, size_t workspace_bytes,
                     void* stream) {
  tk::GradArgs g;
  int rc = linear_grad(args, &g);
  if (rc) return rc;
  rc = check_ws(workspace, workspace_bytes, tk::grad_workspace(g));
  if (rc) return rc;
  return status(tk::launch_grad(g, workspace, static_cast<hipStream_t>(stream)));
}

int topk_decode_workspace_size(const topk_selection* sel, int64_t d, size_t* bytes) {
  if (!bytes) return TOPK_EINVAL;
  tk::Selection s;
  const int rc = to_selection(sel, false, &s);
  if (rc) return rc;
  if (bad_width(d)) return TOPK_EINVAL;
  *bytes = decode_ws(s, d);
  return TOPK_OK;
}

int topk_decode(const topk_selection* sel, const void* weight, int64_t ldw, int64_t d,
                const void* bias, void* out, int64_t ldo, void* workspace, size_t workspace_bytes,
                void* stream) {
  tk::SegCall a;
  int rc = to_selection(sel, true, &a.sel);
  if (rc) return rc;
  const int dt = a.sel.dtype;
  if (bad_width(d) || bad_matrix(weight, ldw, a.sel.n, d, dt) || bad_matrix(out, ldo, a.sel.rows, d, dt))
    return TOPK_EINVAL;
  if (bias && bad_matrix(bias, d, 1, d, dt)) return TOPK_EINVAL;
  rc = check_ws(workspace, workspace_bytes, tk::seg_workspace(a.sel, d, true, false));
  if (rc) return rc;
  a.coef = a.sel.values;
  a.d = d;
  a.parts = 1;
  a.part[0].src = weight;
  a.part[0].lds = ldw;
  a.part[0].bias = bias;
  a.part[0].out = out;
  a.part[0].ldo = ldo;
  return status(tk::launch_seg(a, workspace, static_cast<hipStream_t>(stream)));
}

int topk_decode_grad(const topk_selection* sel, const void* weight, int64_t ldw, int64_t d,
                     const void* grad, int64_t ldg, void* dvalues, void* dweight, int64_t lddw,
                     void* dbias, void* workspace, size_t workspace_bytes, void* stream) {
  tk::Selection s;
  int rc = to_selection(sel, true, &s);
  if (rc) return rc;
  const int dt = s.dtype;
  if (bad_width(d) || (!dvalues && !dweight && !dbias)) return TOPK_EINVAL;
  if (bad_matrix(grad, ldg, s.rows, d, dt)) return TOPK_EINVAL;
  if (dvalues && bad_matrix(weight, ldw, s.n, d, dt)) return TOPK_EINVAL;
  if (dvalues && bad_matrix(dvalues, s.total, 1, s.total, dt)) return TOPK_EINVAL;
  if (dweight && bad_matrix(dweight, lddw, s.n, d, dt)) return TOPK_EINVAL;
  if (dbias && bad_matrix(dbias, d, 1, d, dt)) return TOPK_EINVAL;
  tk::SlopeArgs sums;
  sums.dy = grad;
  sums.ldd = ldg;
  sums.m = s.rows;
  sums.n = d;
  sums.dtype = dt;
  sums.db = dbias;
  size_t need = dweight ? tk::seg_workspace(s, d, false, true) : 0;
  if (dbias) need = std::max(need, tk::slope_workspace(sums));
  rc = check_ws(workspace, workspace_bytes, need);
  if (rc) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  hipError_t e = hipSuccess;
  if (dweight) {   // with dvalues on the way
    tk::SegCall a;
    a.sel = s;
    a.coef = s.values;
    a.d = d;
    a.parts = 1;
    a.part[0].by_row = false;
    a.part[0].src = grad;
    a.part[0].lds = ldg;
    a.part[0].out = dweight;
    a.part[0].ldo = lddw;
    a.part[0].other = dvalues ? weight : nullptr;
    a.part[0].ldother = ldw;
    a.part[0].dots = dvalues;
    e = tk::launch_seg(a, workspace, st);
  } else if (dvalues) {
    tk::DotArgs a;
    a.sel = s;
    a.g = grad;
    a.ldg = ldg;
    a.w = weight;
    a.ldw = ldw;
    a.d = d;
    a.dv = dvalues;
    e = tk::launch_dots(a, st);
  }
  if (e == hipSuccess && dbias) e = tk::launch_slope(sums, workspace, st);
  return status(e);
}

int topk_encode_grad(const topk_selection* sel, const void* grad_values, const void* x, int64_t ldx,
                     const void* weight, int64_t ldw, int64_t d, void* dx, int64_t lddx,
                     void* dweight, int64_t lddw, void* dbias, void* workspace,
                     size_t workspace_bytes, void* stream) {
  tk::Selection s;
  int rc = to_selection(sel, true, &s);
  if (rc) return rc;
  const int dt = s.dtype;
  if (bad_width(d) || (!dx && !dweight && !dbias)) return TOPK_EINVAL;
  if (bad_matrix(grad_values, s.total, 1, s.total, dt)) return TOPK_EINVAL;
  if (dx && (bad_matrix(weight, ldw, s.n, d, dt) || bad_matrix(dx, lddx, s.rows, d, dt))) return TOPK_EINVAL;
  if (dweight && (bad_matrix(x, ldx, s.rows, d, dt) || bad_matrix(dweight, lddw, s.n, d, dt)))
    return TOPK_EINVAL;
  if (dbias && bad_matrix(dbias, s.n, 1, s.n, dt)) return TOPK_EINVAL;
  rc = check_ws(workspace, workspace_bytes, tk::seg_workspace(s, d, dx != nullptr, dweight || dbias));
  if (rc) return rc;
  tk::SegCall a;
  a.sel = s;
  a.coef = grad_values;
  a.gate = s.values;
  a.d = d;
  if (dx) {
    tk::SegArgs& p = a.part[a.parts++];
    p.src = weight;
    p.lds = ldw;
    p.out = dx;
    p.ldo = lddx;
  }
  if (dweight || dbias) {
    tk::SegArgs& p = a.part[a.parts++];
    p.by_row = false;
    p.src = x;
    p.lds = ldx;
    p.out = dweight;
    p.ldo = lddw;
    p.coef_sum = dbias;
  }
  return status(tk::launch_seg(a, workspace, static_cast<hipStream_t>(stream)));
}

int topk_grad_norm_workspace_size(int64_t tensors, const int64_t* counts, size_t* bytes) {
  if (!bytes || bad_size(tensors) || (tensors && !counts)) return TOPK_EINVAL;
  for (int64_t i = 0; i < tensors; ++i)
    if (counts[i] < 0 || counts[i] > (int64_t(1) << 40)) return TOPK_EINVAL;
  *bytes = tk::norm_workspace(tensors, counts);
  return TOPK_OK;
}

}  // extern "C"

namespace {

int norm_call(tk::NormArgs& a, void* workspace, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  int rc = topk_grad_norm_workspace_size(a.tensors, a.counts, &need);
  if (rc) return rc;
  if (!a.norm || reinterpret_cast<uintptr_t>(a.norm) % 4 || (a.tensors && (!a.ptrs || !a.dtypes)))
    return TOPK_EINVAL;
  for (int64_t i = 0; i < a.tensors; ++i) {
    if (bad_dtype(a.dtypes[i])) return TOPK_EDTYPE;
    if (reinterpret_cast<uintptr_t>(a.ptrs[i]) % (uintptr_t)elem(a.dtypes[i])) return TOPK_EINVAL;
    if (a.counts[i] && !a.ptrs[i]) return TOPK_EINVAL;
  }
  rc = check_ws(workspace, workspace_bytes, need);
  if (rc) return rc;
  if (a.scale) {   // a tensor listed twice, or two views that share elements, would be scaled twice
    try {
      std::vector<std::pair<uintptr_t, uintptr_t>> span;
      span.reserve((size_t)a.tensors);
      for (int64_t i = 0; i < a.tensors; ++i) {
        const uintptr_t p = reinterpret_cast<uintptr_t>(a.ptrs[i]);
        if (a.counts[i]) span.emplace_back(p, p + (uintptr_t)(a.counts[i] * elem(a.dtypes[i])));
      }
      if (!std::is_sorted(span.begin(), span.end())) std::sort(span.begin(), span.end());
      for (size_t i = 1; i < span.size(); ++i)
        if (span[i].first < span[i - 1].second) return TOPK_EINVAL;
    } catch (...) {
      return TOPK_EINVAL;
    }
  }
  a.cus = tk::device_cus_now();
  return status(tk::launch_norm(a, workspace, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

int topk_grad_norm(const void* const* ptrs, const int64_t* counts, const int32_t* dtypes,
                   int64_t tensors, float* norm, void* workspace, size_t workspace_bytes,
                   void* stream) {
  tk::NormArgs a;
  a.ptrs = const_cast<void* const*>(ptrs);   // only read: nothing is scaled
  a.counts = counts;
  a.dtypes = dtypes;
  a.tensors = tensors;
  a.norm = norm;
  return norm_call(a, workspace, workspace_bytes, stream);
}

int topk_clip_grad_norm(void* const* ptrs, const int64_t* counts, const int32_t* dtypes,
                        int64_t tensors, float max_norm, float eps, float* norm, void* workspace,
                        size_t workspace_bytes, void* stream) {
  if (!(max_norm >= 0.f) || !(eps >= 0.f)) return TOPK_EINVAL;
  tk::NormArgs a;
  a.ptrs = ptrs;
  a.counts = counts;
  a.dtypes = dtypes;
  a.tensors = tensors;
  a.scale = true;
  a.max_norm = max_norm;
  a.eps = eps;
  a.norm = norm;
  return norm_call(a, workspace, workspace_bytes, stream);
}

}  // extern "C"
