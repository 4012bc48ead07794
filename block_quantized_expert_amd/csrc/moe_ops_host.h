// Host-side argument checks of the entry points of moe_rows.h and
// moe_int8.h.  Pure host C++, as moe_host.h.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "moe_int8.h"
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

}  // namespace moe
