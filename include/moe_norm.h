/*
 * moe_norm.h -- the root-mean-square norm in front of a layer, with the
 * residual's addition, outputs in fp32, bf16, int8 (moe_int8.h's rows) or
 * MXFP4 (moe_mxfp4.h's rows), and its gradients.
 *
 * For each row, with j over `hidden` columns:
 *   s_j = x_j + residual_j rounded to the residual's type, which is written to
 *         `total`; without a residual s_j = x_j
 *   r   = 1 / sqrt(sum_j s_j^2 / hidden + eps)
 *   n_j = s_j * r * weight_j
 * The sum is taken in fp64, so neither large values nor the order of the
 * summation show.  n_j is formed in fp64 and rounded to fp32 once where the
 * output is fp32, int8 or MXFP4, so that moe_rmsnorm_int8 and
 * moe_rmsnorm_mxfp4 give bit for bit what moe_quantize_int8 and
 * moe_quantize_mxfp4 give on moe_rmsnorm's fp32 output; for bf16 it is formed
 * in fp32 and rounded once more.
 *
 * Conventions are those of moe.h, and:
 *   - types are moe_act_type.  Strides are in elements from one row to the
 *     next and at least `hidden`; the elements of a row are contiguous and a
 *     row may start at any multiple of its element size.
 *   - hidden is any size in 1..MOE_MAX_DIM (multiples of 16 for int8 and of 32
 *     for MXFP4 outputs); eps is positive and finite.
 *   - outputs do not overlap inputs or one another, except where a call says
 *     that they may.
 *   - a row with an infinity or NaN in s gives what the formulas give: NaN at
 *     that place and 0 or NaN at the others.
 */
#ifndef MOE_NORM_H
#define MOE_NORM_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The rows and the weight of a norm (host memory, read during the call). */
typedef struct {
  int32_t n_rows;
  int32_t hidden;
  float eps;
  const void* x;       /* [n_rows][hidden] of x_type */
  int32_t x_type;
  int64_t x_stride;
  const void* weight;  /* [hidden] of w_type, aligned to its element */
  int32_t w_type;
  const void* residual; /* nullable: [n_rows][hidden] of res_type */
  int32_t res_type;
  int64_t res_stride;
  void* total;          /* out with a residual (unused without): [n_rows][hidden] of
                           res_type.  It may be `residual` itself (same stride). */
  int64_t total_stride;
} moe_norm_rows;

/* y [n_rows][hidden] of y_type, rows y_stride elements apart. */
moe_status moe_rmsnorm(const moe_norm_rows* rows, void* y, int y_type, int64_t y_stride,
                       hipStream_t stream);

/* The norm's rows rounded to int8: q [n_rows][hidden] (16-byte aligned),
 * scale fp32 [n_rows], as moe_quantize_int8 writes them. */
moe_status moe_rmsnorm_int8(const moe_norm_rows* rows, int8_t* q, float* scale,
                            hipStream_t stream);

/* The norm's rows rounded to MXFP4: codes [n_rows][hidden / 2] and scales, as
 * moe_quantize_mxfp4 writes them (16-byte aligned). */
moe_status moe_rmsnorm_mxfp4(const moe_norm_rows* rows, uint8_t* codes, uint8_t* scales,
                             hipStream_t stream);

/*
 * Gradients, from dy = dL/dn, the rows s that were normed (`total`, or x
 * without a residual) and, where `total` is used further on, dtotal = dL/ds
 * by that use.  With g_j = weight_j * dy_j and r recomputed from s:
 *   dx_j      = r g_j - s_j r^3 / hidden * sum_i s_i g_i + dtotal_j,
 *               which is the gradient of x and of the residual alike
 *   dweight_j = sum over the rows of dy_j s_j r
 * The sums along a row are taken in fp64.  Those over rows are fp32 within a
 * wavefront, which adds up a 256th of the rows at most, and fp64 from there on;
 * of more than 8192 columns, or fewer than eight, they are fp64 but for one
 * rounding of each of 64 parts.
 * n_rows, hidden and the types fix their order: a call repeats bit for bit.
 *   dy       [n_rows][hidden] of dy_type.
 *   s        [n_rows][hidden] of s_type.
 *   dtotal   nullable, of s_type.
 *   dx       out, of s_type.  It may be dtotal itself (same stride).
 *   dweight  nullable out, fp32 [hidden]; 0 when there are no rows.
 *   workspace  moe_rmsnorm_backward_workspace_bytes(n_rows, hidden) bytes,
 *            8-byte aligned; not used (and may be null) without dweight.
 *            Calls that may run at the same time need one each.
 */
size_t moe_rmsnorm_backward_workspace_bytes(int n_rows, int hidden);
moe_status moe_rmsnorm_backward(const void* dy, int dy_type, int64_t dy_stride, const void* s,
                                int s_type, int64_t s_stride, const void* weight, int w_type,
                                const void* dtotal, int64_t dtotal_stride, int n_rows, int hidden,
                                float eps, void* dx, int64_t dx_stride, float* dweight,
                                void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_NORM_H */
