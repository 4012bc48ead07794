// Host-side argument checks (see moe_ops_host.h).
#include "moe_ops_host.h"

#include <math.h>

namespace moe {
namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// An array of 4-byte elements (int32 or fp32).
bool words_ok(const void* p) { return p != nullptr && aligned(p, 4); }

bool type_ok(int type) { return type == MOE_ACT_F32 || type == MOE_ACT_BF16; }

// A row array: aligned to its element.
bool rows_ok(const void* p, int type) {
  return p != nullptr && aligned(p, type == MOE_ACT_BF16 ? 2 : 4);
}

// Row strides stay far below the sizes at which an offset of rows could
// pass 63 bits.
constexpr int64_t kMaxStride = int64_t{1} << 32;

moe_status check_stride(int64_t stride, int width) {
  if (stride < width) return MOE_ERR_INVALID;
  return stride > kMaxStride ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// Sizes that every call on rows shares: types, counts and the strides of two
// row arrays.
moe_status check_rows(int type, int n_tokens, int top_k, int hidden, int64_t stride_a,
                      int64_t stride_b) {
  if (!type_ok(type)) return MOE_ERR_UNSUPPORTED;
  if (n_tokens < 0 || top_k <= 0 || hidden <= 0) return MOE_ERR_INVALID;
  if (n_tokens > MOE_MAX_TOKENS || top_k > MOE_MAX_TOP_K || hidden > MOE_MAX_DIM)
    return MOE_ERR_UNSUPPORTED;
  moe_status s = check_stride(stride_a, hidden);
  return s != MOE_OK ? s : check_stride(stride_b, hidden);
}

moe_status check_weight(const moe_int8_weight* w) {
  if (w == nullptr) return MOE_ERR_INVALID;
  if (w->n_experts <= 0 || w->rows <= 0 || w->cols <= 0) return MOE_ERR_INVALID;
  if (w->n_experts > MOE_MAX_EXPERTS || w->rows > MOE_MAX_DIM || w->cols > MOE_MAX_DIM ||
      w->cols % 16 != 0)
    return MOE_ERR_UNSUPPORTED;
  if (w->q == nullptr || !aligned(w->q, 16) || !words_ok(w->scale)) return MOE_ERR_INVALID;
  return MOE_OK;
}

}  // namespace

moe_status check_dispatch(const void* x, int type, int64_t x_stride, int n_tokens, int top_k,
                          int hidden, int n_experts, const int32_t* offsets,
                          const int32_t* inv_perm, const void* rows, int64_t rows_stride) {
  moe_status s = check_rows(type, n_tokens, top_k, hidden, x_stride, rows_stride);
  if (s != MOE_OK) return s;
  if (n_experts <= 0) return MOE_ERR_INVALID;
  if (n_experts > MOE_MAX_EXPERTS) return MOE_ERR_UNSUPPORTED;
  if (n_tokens == 0) return MOE_OK;
  if (!rows_ok(x, type) || !rows_ok(rows, type)) return MOE_ERR_INVALID;
  if (!words_ok(offsets) || !words_ok(inv_perm)) return MOE_ERR_INVALID;
  return MOE_OK;
}

moe_status check_combine(const void* rows, int type, int64_t rows_stride, int n_tokens, int top_k,
                         int hidden, const float* topk_w, const int32_t* inv_perm,
                         const void* base, int64_t base_stride, const void* y, int y_type,
                         int64_t y_stride) {
  moe_status s = check_rows(type, n_tokens, top_k, hidden, rows_stride, y_stride);
  if (s != MOE_OK) return s;
  if (!type_ok(y_type)) return MOE_ERR_UNSUPPORTED;
  if (base != nullptr && (s = check_stride(base_stride, hidden)) != MOE_OK) return s;
  if (n_tokens == 0) return MOE_OK;
  if (!rows_ok(rows, type) || !rows_ok(y, y_type)) return MOE_ERR_INVALID;
  if (base != nullptr && !rows_ok(base, y_type)) return MOE_ERR_INVALID;
  if (!aligned(topk_w, 4) || !words_ok(inv_perm)) return MOE_ERR_INVALID;
  return MOE_OK;
}

moe_status check_combine_backward(const void* dy, int y_type, int64_t dy_stride, const void* rows,
                                  int type, int64_t rows_stride, int n_tokens, int top_k,
                                  int hidden, int n_experts, const float* topk_w,
                                  const int32_t* offsets, const int32_t* inv_perm,
                                  const void* drows, int64_t drows_stride, const float* dw) {
  moe_status s = check_dispatch(rows, type, rows_stride, n_tokens, top_k, hidden, n_experts,
                                offsets, inv_perm, drows, drows_stride);
  if (s != MOE_OK) return s;
  if (!type_ok(y_type)) return MOE_ERR_UNSUPPORTED;
  if ((s = check_stride(dy_stride, hidden)) != MOE_OK) return s;
  if (n_tokens == 0) return MOE_OK;
  if (!rows_ok(dy, y_type) || !words_ok(topk_w) || !words_ok(dw)) return MOE_ERR_INVALID;
  return MOE_OK;
}

moe_status check_route_backward(const float* logits, const int32_t* ids, const float* dw,
                                int n_tokens, int n_experts, int top_k, float routed_scale,
                                const float* dlogits, const int32_t* dev_error) {
  if (n_tokens < 0 || n_experts <= 0 || top_k <= 0 || top_k > n_experts) return MOE_ERR_INVALID;
  if (n_experts > MOE_MAX_EXPERTS || top_k > MOE_MAX_TOP_K || n_tokens > MOE_MAX_TOKENS)
    return MOE_ERR_UNSUPPORTED;
  if (!(routed_scale > 0.0f) || !isfinite(routed_scale)) return MOE_ERR_INVALID;
  if (n_tokens > 0 && (!words_ok(logits) || !words_ok(ids) || !words_ok(dw) ||
                       !words_ok(dlogits) || !aligned(dev_error, 4)))
    return MOE_ERR_INVALID;
  return MOE_OK;
}

moe_status check_quantize(const void* x, int x_type, int64_t x_stride, int n_rows, int cols,
                          const int8_t* q, const float* scale) {
  if (!type_ok(x_type)) return MOE_ERR_UNSUPPORTED;
  if (n_rows < 0 || cols <= 0) return MOE_ERR_INVALID;
  if (n_rows > MOE_MAX_TOKENS * MOE_MAX_TOP_K || cols > MOE_MAX_DIM || cols % 16 != 0)
    return MOE_ERR_UNSUPPORTED;
  moe_status s = check_stride(x_stride, cols);
  if (s != MOE_OK || n_rows == 0) return s;
  if (!rows_ok(x, x_type) || q == nullptr || !aligned(q, 16) || !words_ok(scale))
    return MOE_ERR_INVALID;
  return MOE_OK;
}

moe_status check_product(const moe_int8_weight* w, const moe_int8_weight* up, const int8_t* q,
                         const float* scale, int n_slots, const int32_t* offsets,
                         const int32_t* perm, int top_k, const void* out, int out_type,
                         int64_t out_stride) {
  moe_status s = check_weight(w);
  if (s != MOE_OK) return s;
  if (up != nullptr) {
    if ((s = check_weight(up)) != MOE_OK) return s;
    if (up->n_experts != w->n_experts || up->rows != w->rows || up->cols != w->cols)
      return MOE_ERR_INVALID;
  }
  if (!type_ok(out_type)) return MOE_ERR_UNSUPPORTED;
  if (n_slots < 0 || top_k < 0) return MOE_ERR_INVALID;
  if (n_slots > MOE_MAX_TOKENS * MOE_MAX_TOP_K || top_k > MOE_MAX_TOP_K)
    return MOE_ERR_UNSUPPORTED;
  if (offsets == nullptr && (w->n_experts != 1 || top_k != 0)) return MOE_ERR_INVALID;
  if (top_k > 0 && n_slots % top_k != 0) return MOE_ERR_INVALID;
  if ((s = check_stride(out_stride, w->rows)) != MOE_OK || n_slots == 0) return s;
  if (q == nullptr || !aligned(q, 16) || !words_ok(scale) || !rows_ok(out, out_type))
    return MOE_ERR_INVALID;
  if (!aligned(offsets, 4) || (top_k > 0 && !words_ok(perm))) return MOE_ERR_INVALID;
  return MOE_OK;
}

}  // namespace moe
