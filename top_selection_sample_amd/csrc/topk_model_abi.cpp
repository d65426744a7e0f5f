// C ABI of the operators on a language model's selections: argument checks,
// launches.  Nothing is enqueued before every check has passed.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/topk.h"
#include "topk_model.hpp"
#include "topk_ops.hpp"

namespace {

constexpr int64_t SIZE_MAX31 = (int64_t(1) << 31) - 1;
constexpr int64_t AREA_MAX = int64_t(1) << 42;   // elements: more than any device holds
constexpr int64_t GROUP_MAX = 4096;              // query heads of a key-value head

bool bad_size(int64_t v) { return v < 0 || v > SIZE_MAX31; }
bool bad_area(int64_t a, int64_t b) { return a > 0 && b > AREA_MAX / a; }
bool bad_stride(int64_t v) { return v < 0 || v > AREA_MAX; }
bool bad_dtype(int dtype) { return dtype != TOPK_F32 && dtype != TOPK_BF16; }
int64_t elem(int dtype) { return dtype == TOPK_BF16 ? 2 : 4; }

// An address of elements of `size` bytes; it may be null where there are none.
bool bad_address(const void* p, int64_t size, bool empty = false) {
  return reinterpret_cast<uintptr_t>(p) % (uintptr_t)size || (!p && !empty);
}

// A [rows, cols] matrix whose rows do not overlap.
bool bad_matrix(const void* p, int64_t ld, int64_t rows, int64_t cols, int dtype) {
  return bad_size(ld) || (rows > 1 && ld < cols) || bad_address(p, elem(dtype), rows == 0 || cols == 0);
}

int check_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return TOPK_OK;
  if (!ws || reinterpret_cast<uintptr_t>(ws) % 256) return TOPK_EINVAL;
  return have < need ? TOPK_EWORKSPACE : TOPK_OK;
}

int status(hipError_t e) { return e == hipSuccess ? TOPK_OK : TOPK_EHIP; }

// Rows [0, a) of stride sa hold rows [0, b) of stride sb of `inner` elements
// each: no two of them share an element.
bool overlapping(int64_t a, int64_t sa, int64_t b, int64_t sb, int64_t inner) {
  if (inner == 0 || a == 0 || b == 0) return false;
  if (a == 1) return b > 1 && sb < inner;
  if (b == 1) return sa < inner;
  typedef __int128 Wide;
  if (sb <= sa) return sb < inner || (Wide)sa < (Wide)(b - 1) * sb + inner;
  return sa < inner || (Wide)sb < (Wide)(a - 1) * sa + inner;
}

// The same of three axes, the strides in any order.
bool overlapping3(int64_t a, int64_t sa, int64_t b, int64_t sb, int64_t c, int64_t sc, int64_t inner) {
  if (inner == 0 || a == 0 || b == 0 || c == 0) return false;
  struct Axis {
    int64_t n, s;
  } x[3] = {{a, sa}, {b, sb}, {c, sc}};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (x[j].s > x[j + 1].s) {
        const Axis t = x[j];
        x[j] = x[j + 1];
        x[j + 1] = t;
      }
  __int128 span = inner;
  for (const Axis& v : x) {
    if (v.n == 1) continue;
    if (v.s < span) return true;
    span += (__int128)(v.n - 1) * v.s;
  }
  return false;
}

int check_routing(int64_t tokens, int64_t k) {
  if (bad_size(tokens) || bad_size(k)) return TOPK_EINVAL;
  return tokens > 0 && k > SIZE_MAX31 / tokens ? TOPK_EINVAL : TOPK_OK;   // entries are numbered in 31 bits
}

bool bad_width(int64_t d) { return d < 0 || d >= tk::WIDTH_MAX; }

int check_weights(const void* w, int dtype, int wdtype, bool empty) {
  if (bad_dtype(dtype) || bad_dtype(wdtype)) return TOPK_EDTYPE;
  if (wdtype != dtype && wdtype != TOPK_F32) return TOPK_EDTYPE;
  return bad_address(w, elem(wdtype), empty) ? TOPK_EINVAL : TOPK_OK;
}

int check_combine_grad(const topk_combine_grad_args* a) {
  if (!a) return TOPK_EINVAL;
  const int rc = check_routing(a->tokens, a->k);
  if (rc) return rc;
  const int rw = check_weights(a->weights, a->dtype, a->wdtype, true);   // null: all 1
  if (rw) return rw;
  if (!a->dy && !a->dweights) return TOPK_EINVAL;
  if (bad_size(a->n) || bad_width(a->d) || bad_area(a->n, a->d) || bad_area(a->tokens, a->d)) return TOPK_EINVAL;
  if (bad_matrix(a->grad, a->ldg, a->tokens, a->d, a->dtype)) return TOPK_EINVAL;
  if (a->dweights && (bad_matrix(a->y, a->ldy, a->n, a->d, a->dtype) || bad_address(a->dweights, elem(a->wdtype))))
    return TOPK_EINVAL;
  if (a->dy && bad_matrix(a->dy, a->lddy, a->n, a->d, a->dtype)) return TOPK_EINVAL;
  if (bad_address(a->places, 8, a->tokens * a->k == 0)) return TOPK_EINVAL;
  return TOPK_OK;
}

int check_attend(const topk_attend_args* a, bool pointers) {
  if (!a) return TOPK_EINVAL;
  if (bad_dtype(a->dtype)) return TOPK_EDTYPE;
  if (bad_size(a->batch) || bad_size(a->heads) || bad_size(a->kv_heads) || bad_size(a->n)) return TOPK_EINVAL;
  if (a->d < 0 || a->d > tk::HEAD_MAX || a->kv_heads == 0 || a->heads % a->kv_heads || a->heads / a->kv_heads > GROUP_MAX)
    return TOPK_EINVAL;
  if (bad_area(a->batch, a->heads) || bad_area(a->batch * a->heads, a->d) || bad_area(a->batch * a->kv_heads, a->n) ||
      bad_area(a->batch * a->heads, a->n) || !std::isfinite(a->scale))
    return TOPK_EINVAL;
  for (int64_t s : {a->sqb, a->sqh, a->skb, a->skh, a->skn, a->svb, a->svh, a->svn, a->ssb, a->ssh, a->sob, a->soh})
    if (bad_stride(s)) return TOPK_EINVAL;
  if (a->n > 1 && (a->skn >= tk::STEP_MAX || a->svn >= tk::STEP_MAX)) return TOPK_EINVAL;
  if (overlapping(a->batch, a->sob, a->heads, a->soh, a->d)) return TOPK_EINVAL;
  if (a->scores && overlapping(a->batch, a->ssb, a->kv_heads, a->ssh, a->n)) return TOPK_EINVAL;
  if (!pointers) return TOPK_OK;
  const int64_t e = elem(a->dtype);
  const bool none = a->batch == 0 || a->heads == 0;
  if (bad_address(a->q, e, none || a->d == 0) || bad_address(a->out, e, none || a->d == 0)) return TOPK_EINVAL;
  if (bad_address(a->k, e, none || a->n == 0 || a->d == 0) || bad_address(a->v, e, none || a->n == 0 || a->d == 0)) return TOPK_EINVAL;
  if (bad_address(a->lengths, 8, true) || bad_address(a->scores, 4, true)) return TOPK_EINVAL;
  return TOPK_OK;
}

int check_evict(const topk_evict_args* a, bool pointers) {
  if (!a) return TOPK_EINVAL;
  if (bad_dtype(a->dtype)) return TOPK_EDTYPE;
  if (bad_size(a->batch) || bad_size(a->heads) || bad_size(a->n) || bad_width(a->d) || bad_size(a->budget)) return TOPK_EINVAL;
  if (a->budget < 1 || a->recent < 0 || a->recent > a->budget) return TOPK_EINVAL;
  if (bad_area(a->batch, a->heads) || bad_area(a->batch * a->heads, a->n) || bad_area(a->batch * a->heads, a->budget)) return TOPK_EINVAL;
  for (int64_t s : {a->skb, a->skh, a->skn, a->svb, a->svh, a->svn, a->ssb, a->ssh, a->okb, a->okh, a->okn, a->ovb, a->ovh, a->ovn,
                    a->osb, a->osh})
    if (bad_stride(s)) return TOPK_EINVAL;
  if (overlapping3(a->batch, a->okb, a->heads, a->okh, a->budget, a->okn, a->d) ||
      overlapping3(a->batch, a->ovb, a->heads, a->ovh, a->budget, a->ovn, a->d) ||
      overlapping(a->batch, a->osb, a->heads, a->osh, a->budget))
    return TOPK_EINVAL;
  if (!pointers) return TOPK_OK;
  const int64_t e = elem(a->dtype);
  const bool none = a->batch == 0 || a->heads == 0;
  const bool in = none || a->n == 0;
  if (bad_address(a->k, e, in || a->d == 0) || bad_address(a->v, e, in || a->d == 0) || bad_address(a->scores, 4, in)) return TOPK_EINVAL;
  if (bad_address(a->k_out, e, none || a->d == 0) || bad_address(a->v_out, e, none || a->d == 0) || bad_address(a->scores_out, 4, none))
    return TOPK_EINVAL;
  if (bad_address(a->kept, 8, none) || bad_address(a->lengths_out, 8, none) || bad_address(a->lengths, 8, true)) return TOPK_EINVAL;
  return TOPK_OK;
}

int check_sample(const topk_sample_args* a) {
  if (!a) return TOPK_EINVAL;
  if (bad_dtype(a->dtype)) return TOPK_EDTYPE;
  if (bad_size(a->rows) || a->n < 1 || a->n > tk::VOCABULARY_MAX || bad_area(a->rows, a->n)) return TOPK_EINVAL;
  return TOPK_OK;
}

}  // namespace

extern "C" {

static_assert(sizeof(topk_dispatch_args) == 96, "topk_dispatch_args layout is part of the ABI");
static_assert(sizeof(topk_combine_args) == 88, "topk_combine_args layout is part of the ABI");
static_assert(sizeof(topk_combine_grad_args) == 112, "topk_combine_grad_args layout is part of the ABI");
static_assert(sizeof(topk_attend_args) == 192, "topk_attend_args layout is part of the ABI");
static_assert(sizeof(topk_evict_args) == 256, "topk_evict_args layout is part of the ABI");
static_assert(sizeof(topk_sample_args) == 112, "topk_sample_args layout is part of the ABI");

int topk_dispatch_workspace_size(int64_t tokens, int64_t k, int64_t n_experts, size_t* bytes) {
  if (!bytes || n_experts < 0 || n_experts > tk::EXPERTS_MAX) return TOPK_EINVAL;
  const int rc = check_routing(tokens, k);
  if (rc) return rc;
  *bytes = tk::dispatch_workspace(tokens, k, n_experts);
  return TOPK_OK;
}

int topk_dispatch(const topk_dispatch_args* a, void* workspace, size_t workspace_bytes, void* stream) {
  if (!a) return TOPK_EINVAL;
  if (bad_dtype(a->dtype)) return TOPK_EDTYPE;
  size_t need = 0;
  int rc = topk_dispatch_workspace_size(a->tokens, a->k, a->n_experts, &need);
  if (rc) return rc;
  const int64_t total = a->tokens * a->k;
  if (bad_width(a->d) || bad_area(total, a->d) || bad_area(a->tokens, a->d)) return TOPK_EINVAL;
  if (bad_matrix(a->x, a->ldx, a->tokens, a->d, a->dtype) || bad_matrix(a->rows, a->ldr, total, a->d, a->dtype)) return TOPK_EINVAL;
  if (bad_address(a->experts, 8, total == 0) || bad_address(a->places, 8, total == 0) || bad_address(a->offsets, 8)) return TOPK_EINVAL;
  rc = check_ws(workspace, workspace_bytes, need);
  if (rc) return rc;
  return status(tk::launch_dispatch(*a, workspace, static_cast<hipStream_t>(stream)));
}

int topk_combine(const topk_combine_args* a, void* stream) {
  if (!a) return TOPK_EINVAL;
  int rc = check_routing(a->tokens, a->k);
  if (rc) return rc;
  rc = check_weights(a->weights, a->dtype, a->wdtype, true);
  if (rc) return rc;
  if (bad_size(a->n) || bad_width(a->d) || bad_area(a->n, a->d) || bad_area(a->tokens, a->d)) return TOPK_EINVAL;
  if (bad_matrix(a->y, a->ldy, a->n, a->d, a->dtype) || bad_matrix(a->out, a->ldo, a->tokens, a->d, a->dtype)) return TOPK_EINVAL;
  if (bad_address(a->places, 8, a->tokens * a->k == 0)) return TOPK_EINVAL;
  return status(tk::launch_combine(*a, static_cast<hipStream_t>(stream)));
}

int topk_combine_grad_workspace_size(const topk_combine_grad_args* a, size_t* bytes) {
  if (!bytes) return TOPK_EINVAL;
  const int rc = check_combine_grad(a);
  if (rc) return rc;
  *bytes = tk::combine_grad_workspace(*a);
  return TOPK_OK;
}

int topk_combine_grad(const topk_combine_grad_args* a, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_combine_grad(a);
  if (rc) return rc;
  rc = check_ws(workspace, workspace_bytes, tk::combine_grad_workspace(*a));
  if (rc) return rc;
  return status(tk::launch_combine_grad(*a, workspace, static_cast<hipStream_t>(stream)));
}

int topk_attend_workspace_size(const topk_attend_args* a, size_t* bytes) {
  if (!bytes) return TOPK_EINVAL;
  const int rc = check_attend(a, false);
  if (rc) return rc;
  *bytes = tk::attend_workspace(*a, tk::device_cus_now());
  return TOPK_OK;
}

int topk_attend(const topk_attend_args* a, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_attend(a, true);
  if (rc) return rc;
  const int cus = tk::device_cus_now();
  rc = check_ws(workspace, workspace_bytes, tk::attend_workspace(*a, cus));
  if (rc) return rc;
  return status(tk::launch_attend(*a, workspace, cus, static_cast<hipStream_t>(stream)));
}

int topk_evict_workspace_size(const topk_evict_args* a, size_t* bytes) {
  if (!bytes) return TOPK_EINVAL;
  const int rc = check_evict(a, false);
  if (rc) return rc;
  *bytes = tk::evict_workspace(*a);
  return TOPK_OK;
}

int topk_evict(const topk_evict_args* a, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_evict(a, true);
  if (rc) return rc;
  rc = check_ws(workspace, workspace_bytes, tk::evict_workspace(*a));
  if (rc) return rc;
  return status(tk::launch_evict(*a, workspace, static_cast<hipStream_t>(stream)));
}

int topk_sample_workspace_size(const topk_sample_args* a, size_t* bytes) {
  if (!bytes) return TOPK_EINVAL;
  const int rc = check_sample(a);
  if (rc) return rc;
  *bytes = tk::sample_workspace(*a);
  return TOPK_OK;
}

int topk_sample(const topk_sample_args* a, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_sample(a);
  if (rc) return rc;
  const bool none = a->rows == 0;
  if (bad_matrix(a->logits, a->ld, a->rows, a->n, a->dtype)) return TOPK_EINVAL;
  if (bad_address(a->u, 4, none) || bad_address(a->tokens, 8, none) || bad_address(a->logprobs, 4, none)) return TOPK_EINVAL;
  if (bad_address(a->temperatures, 4, true) || bad_address(a->top_ks, 8, true) || bad_address(a->top_ps, 4, true) ||
      bad_address(a->min_ps, 4, true))
    return TOPK_EINVAL;
  rc = check_ws(workspace, workspace_bytes, tk::sample_workspace(*a));
  if (rc) return rc;
  return status(tk::launch_sample(*a, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
