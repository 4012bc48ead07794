// Host-side argument checks of the entry points of moe_rows.h and
// moe_int8.h.  Pure host C++, as moe_host.h.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "moe_int8.h"
#include "moe_rows.h"

namespace moe {

// Sizes that every call on rows shares: types, counts and the strides of
// its row arrays (0 for an array that the call does not have).
moe_status check_rows(int type, int n_tokens, int top_k, int hidden, int64_t stride_a,
                      int64_t stride_b);
// A row array: null only where there is nothing to read or write, and
// aligned to its element.
bool rows_ptr_ok(const void* p, int type);

moe_status check_dispatch(const void* x, int type, int64_t x_stride, int n_tokens, int top_k,
                          int hidden, int n_experts, const int32_t* offsets,
                          const int32_t* inv_perm, const void* rows, int64_t rows_stride);
moe_status check_combine(const void* rows, int type, int64_t rows_stride, int n_tokens, int top_k,
                         int hidden, const int32_t* inv_perm, const void* base,
                         int64_t base_stride, const void* y, int y_type, int64_t y_stride);
moe_status check_combine_backward(const void* dy, int y_type, int64_t dy_stride, const void* rows,
                                  int type, int64_t rows_stride, int n_tokens, int top_k,
                                  int hidden, int n_experts, const float* topk_w,
                                  const int32_t* offsets, const int32_t* inv_perm,
                                  const void* drows, int64_t drows_stride, const float* dw);
moe_status check_route_backward(const float* logits, const int32_t* ids, const float* dw,
                                int n_tokens, int n_experts, int top_k, float routed_scale,
                                const float* dlogits);
moe_status check_quantize(const void* x, int x_type, int64_t x_stride, int n_rows, int cols,
                          const int8_t* q, const float* scale);
// up is NULL for a plain product.
moe_status check_product(const moe_int8_weight* w, const moe_int8_weight* up, const int8_t* q,
                         const float* scale, int n_slots, const int32_t* offsets,
                         const int32_t* perm, int top_k, const void* out, int out_type,
                         int64_t out_stride);

}  // namespace moe
