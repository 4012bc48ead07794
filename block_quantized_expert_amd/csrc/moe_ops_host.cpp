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

// Codes and scale words, or int8 rows.
bool bytes_ok(const void* p) { return p != nullptr && aligned(p, 16); }

// Sizes of a weight whose rows are whole 16-byte words of `block` inputs.
moe_status check_weight_sizes(int n_experts, int rows, int cols, int block) {
  if (n_experts <= 0 || rows <= 0 || cols <= 0) return MOE_ERR_INVALID;
  if (n_experts > MOE_MAX_EXPERTS || rows > MOE_MAX_DIM || cols > MOE_MAX_DIM ||
      cols % block != 0)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_weight(const moe_int8_weight* w) {
  if (w == nullptr) return MOE_ERR_INVALID;
  const moe_status s = check_weight_sizes(w->n_experts, w->rows, w->cols, 16);
  if (s != MOE_OK) return s;
  return bytes_ok(w->q) && words_ok(w->scale) ? MOE_OK : MOE_ERR_INVALID;
}

moe_status check_weight(const moe_mxfp4_weight* w) {
  if (w == nullptr) return MOE_ERR_INVALID;
  const moe_status s = check_weight_sizes(w->n_experts, w->rows, w->cols, 32);
  if (s != MOE_OK) return s;
  return bytes_ok(w->codes) && bytes_ok(w->scales) ? MOE_OK : MOE_ERR_INVALID;
}

// Everything of a product but its operands' arrays.
moe_status check_product_sizes(int n_experts, int rows, int n_slots, const int32_t* offsets,
                               const int32_t* perm, int top_k, const void* out, int out_type,
                               int64_t out_stride) {
  if (!type_ok(out_type)) return MOE_ERR_UNSUPPORTED;
  if (n_slots < 0 || top_k < 0) return MOE_ERR_INVALID;
  if (n_slots > MOE_MAX_TOKENS * MOE_MAX_TOP_K || top_k > MOE_MAX_TOP_K)
    return MOE_ERR_UNSUPPORTED;
  if (offsets == nullptr && (n_experts != 1 || top_k != 0)) return MOE_ERR_INVALID;
  if (top_k > 0 && n_slots % top_k != 0) return MOE_ERR_INVALID;
  const moe_status s = check_stride(out_stride, rows);
  if (s != MOE_OK || n_slots == 0) return s;
  if (!rows_ok(out, out_type) || !aligned(offsets, 4) || (top_k > 0 && !words_ok(perm)))
    return MOE_ERR_INVALID;
  return MOE_OK;
}

// The shape, the rows and the weight of a norm; `block`: hidden's divisor.
moe_status check_norm_rows(const moe_norm_rows* r, int block) {
  if (r == nullptr) return MOE_ERR_INVALID;
  const bool res = r->residual != nullptr;
  if (!type_ok(r->x_type) || !type_ok(r->w_type) || (res && !type_ok(r->res_type)))
    return MOE_ERR_UNSUPPORTED;
  if (r->n_rows < 0 || r->hidden <= 0 || !(r->eps > 0.0f) || !isfinite(r->eps))
    return MOE_ERR_INVALID;
  if (r->n_rows > MOE_MAX_TOKENS * MOE_MAX_TOP_K || r->hidden > MOE_MAX_DIM ||
      r->hidden % block != 0)
    return MOE_ERR_UNSUPPORTED;
  moe_status s = check_stride(r->x_stride, r->hidden);
  if (s != MOE_OK) return s;
  if (res && ((s = check_stride(r->res_stride, r->hidden)) != MOE_OK ||
              (s = check_stride(r->total_stride, r->hidden)) != MOE_OK))
    return s;
  if (r->n_rows == 0) return MOE_OK;
  if (!rows_ok(r->x, r->x_type) || !rows_ok(r->weight, r->w_type)) return MOE_ERR_INVALID;
  if (res && (!rows_ok(r->residual, r->res_type) || !rows_ok(r->total, r->res_type)))
    return MOE_ERR_INVALID;
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
  s = check_product_sizes(w->n_experts, w->rows, n_slots, offsets, perm, top_k, out, out_type,
                          out_stride);
  if (s != MOE_OK || n_slots == 0) return s;
  return bytes_ok(q) && words_ok(scale) ? MOE_OK : MOE_ERR_INVALID;
}

moe_status check_rmsnorm(const moe_norm_rows* rows, const void* y, int y_type, int64_t y_stride) {
  moe_status s = check_norm_rows(rows, 1);
  if (s != MOE_OK) return s;
  if (!type_ok(y_type)) return MOE_ERR_UNSUPPORTED;
  if ((s = check_stride(y_stride, rows->hidden)) != MOE_OK || rows->n_rows == 0) return s;
  return rows_ok(y, y_type) ? MOE_OK : MOE_ERR_INVALID;
}

moe_status check_rmsnorm_int8(const moe_norm_rows* rows, const int8_t* q, const float* scale) {
  const moe_status s = check_norm_rows(rows, 16);
  if (s != MOE_OK || rows->n_rows == 0) return s;
  return bytes_ok(q) && words_ok(scale) ? MOE_OK : MOE_ERR_INVALID;
}

moe_status check_rmsnorm_mxfp4(const moe_norm_rows* rows, const uint8_t* codes,
                               const uint8_t* scales) {
  const moe_status s = check_norm_rows(rows, 32);
  if (s != MOE_OK || rows->n_rows == 0) return s;
  return bytes_ok(codes) && bytes_ok(scales) ? MOE_OK : MOE_ERR_INVALID;
}

int norm_back_groups(int64_t n_rows, int hidden) {
  const int64_t most = norm_back_long(hidden) ? 64 : 256;
  return (int)(n_rows < most ? n_rows : most);
}

size_t norm_inv_bytes(int64_t n_rows, int hidden) {
  return norm_back_long(hidden) ? (size_t)(n_rows + 1) / 2 * 8 : 0;
}

moe_status check_rmsnorm_backward(const void* dy, int dy_type, int64_t dy_stride, const void* s,
                                  int s_type, int64_t s_stride, const void* weight, int w_type,
                                  const void* dtotal, int64_t dtotal_stride, int n_rows,
                                  int hidden, float eps, const void* dx, int64_t dx_stride,
                                  const float* dweight, const void* workspace,
                                  size_t workspace_bytes) {
  moe_norm_rows r{};
  r.n_rows = n_rows;
  r.hidden = hidden;
  r.eps = eps;
  r.x = s;
  r.x_type = s_type;
  r.x_stride = s_stride;
  r.weight = weight;
  r.w_type = w_type;
  moe_status st = check_norm_rows(&r, 1);
  if (st != MOE_OK) return st;
  if (!type_ok(dy_type)) return MOE_ERR_UNSUPPORTED;
  if ((st = check_stride(dy_stride, hidden)) != MOE_OK ||
      (st = check_stride(dx_stride, hidden)) != MOE_OK)
    return st;
  if (dtotal != nullptr && (st = check_stride(dtotal_stride, hidden)) != MOE_OK) return st;
  if (!aligned(dweight, 4)) return MOE_ERR_INVALID;
  if (n_rows == 0) return MOE_OK;
  if (!rows_ok(dy, dy_type) || !rows_ok(dx, s_type)) return MOE_ERR_INVALID;
  if (dtotal != nullptr && !rows_ok(dtotal, s_type)) return MOE_ERR_INVALID;
  if (dweight == nullptr) return MOE_OK;
  if (workspace == nullptr || workspace_bytes < moe_rmsnorm_backward_workspace_bytes(n_rows, hidden))
    return MOE_ERR_WORKSPACE;
  return aligned(workspace, 8) ? MOE_OK : MOE_ERR_INVALID;
}

moe_status check_mxfp4_rows(const void* x, int x_type, int64_t x_stride, int n_rows, int cols,
                            const uint8_t* codes, const uint8_t* scales) {
  if (!type_ok(x_type)) return MOE_ERR_UNSUPPORTED;
  if (n_rows < 0 || cols <= 0) return MOE_ERR_INVALID;
  if (n_rows > MOE_MAX_TOKENS * MOE_MAX_TOP_K || cols > MOE_MAX_DIM || cols % 32 != 0)
    return MOE_ERR_UNSUPPORTED;
  const moe_status s = check_stride(x_stride, cols);
  if (s != MOE_OK || n_rows == 0) return s;
  return rows_ok(x, x_type) && bytes_ok(codes) && bytes_ok(scales) ? MOE_OK : MOE_ERR_INVALID;
}

moe_status check_product_mxfp4(const moe_mxfp4_weight* w, const moe_mxfp4_weight* up,
                               const uint8_t* codes, const uint8_t* scales, int n_slots,
                               const int32_t* offsets, const int32_t* perm, int top_k,
                               const void* out, int out_type, int64_t out_stride) {
  moe_status s = check_weight(w);
  if (s != MOE_OK) return s;
  if (up != nullptr) {
    if ((s = check_weight(up)) != MOE_OK) return s;
    if (up->n_experts != w->n_experts || up->rows != w->rows || up->cols != w->cols)
      return MOE_ERR_INVALID;
  }
  s = check_product_sizes(w->n_experts, w->rows, n_slots, offsets, perm, top_k, out, out_type,
                          out_stride);
  if (s != MOE_OK || n_slots == 0) return s;
  return bytes_ok(codes) && bytes_ok(scales) ? MOE_OK : MOE_ERR_INVALID;
}

}  // namespace moe

extern "C" size_t moe_rmsnorm_backward_workspace_bytes(int n_rows, int hidden) {
  if (n_rows <= 0 || hidden <= 0) return 0;
  return moe::norm_inv_bytes(n_rows, hidden) +
         (size_t)moe::norm_back_groups(n_rows, hidden) * hidden * sizeof(float);
}
