// Host-side argument checks of the entry points of moe_rows.h, moe_int8.h,
// moe_norm.h and moe_mxfp4.h.  Pure host C++, as moe_host.h.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "moe_int8.h"
#include "moe_mxfp4.h"
#include "moe_norm.h"
#include "moe_rows.h"

namespace moe {

moe_status check_dispatch(const void* x, int type, int64_t x_stride, int n_tokens, int top_k,
                          int hidden, int n_experts, const int32_t* offsets,
                          const int32_t* inv_perm, const void* rows, int64_t rows_stride);
// topk_w may be null (weights 1: the gradient of the copy into expert order).
moe_status check_combine(const void* rows, int type, int64_t rows_stride, int n_tokens, int top_k,
                         int hidden, const float* topk_w, const int32_t* inv_perm,
                         const void* base, int64_t base_stride, const void* y, int y_type,
                         int64_t y_stride);
moe_status check_combine_backward(const void* dy, int y_type, int64_t dy_stride, const void* rows,
                                  int type, int64_t rows_stride, int n_tokens, int top_k,
                                  int hidden, int n_experts, const float* topk_w,
                                  const int32_t* offsets, const int32_t* inv_perm,
                                  const void* drows, int64_t drows_stride, const float* dw);
moe_status check_route_backward(const float* logits, const int32_t* ids, const float* dw,
                                int n_tokens, int n_experts, int top_k, float routed_scale,
                                const float* dlogits, const int32_t* dev_error);
moe_status check_quantize(const void* x, int x_type, int64_t x_stride, int n_rows, int cols,
                          const int8_t* q, const float* scale);
// up is NULL for a plain product.
moe_status check_product(const moe_int8_weight* w, const moe_int8_weight* up, const int8_t* q,
                         const float* scale, int n_slots, const int32_t* offsets,
                         const int32_t* perm, int top_k, const void* out, int out_type,
                         int64_t out_stride);
moe_status check_rmsnorm(const moe_norm_rows* rows, const void* y, int y_type, int64_t y_stride);
moe_status check_rmsnorm_int8(const moe_norm_rows* rows, const int8_t* q, const float* scale);
moe_status check_rmsnorm_mxfp4(const moe_norm_rows* rows, const uint8_t* codes,
                               const uint8_t* scales);
moe_status check_rmsnorm_backward(const void* dy, int dy_type, int64_t dy_stride, const void* s,
                                  int s_type, int64_t s_stride, const void* weight, int w_type,
                                  const void* dtotal, int64_t dtotal_stride, int n_rows,
                                  int hidden, float eps, const void* dx, int64_t dx_stride,
                                  const float* dweight, const void* workspace,
                                  size_t workspace_bytes);
// The norm's gradients: rows that do not stay in registers, the most
// workgroups that share the rows (each with a part of dweight), bytes of those
// rows' r in front of the parts.
constexpr int kNormBackCols = 8192;
constexpr bool norm_back_long(int hidden) { return hidden > kNormBackCols || hidden < 8; }
int norm_back_groups(int64_t n_rows, int hidden);
size_t norm_inv_bytes(int64_t n_rows, int hidden);
// Rounding and its inverse alike.
moe_status check_mxfp4_rows(const void* x, int x_type, int64_t x_stride, int n_rows, int cols,
                            const uint8_t* codes, const uint8_t* scales);
// up is NULL for a plain product.
moe_status check_product_mxfp4(const moe_mxfp4_weight* w, const moe_mxfp4_weight* up,
                               const uint8_t* codes, const uint8_t* scales, int n_slots,
                               const int32_t* offsets, const int32_t* perm, int top_k,
                               const void* out, int out_type, int64_t out_stride);

}  // namespace moe
