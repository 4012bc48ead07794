/*
 * moe_int8.h -- products in 8-bit integers with a scale per token and per
 * channel, dense or grouped by expert.
 *
 * A weight matrix has int8 values and one fp32 scale per output channel
 * (row); activations are rounded to int8 with one fp32 scale per token
 * (moe_quantize_int8).  The product sums int8 x int8 exactly in int32 on the
 * matrix cores and multiplies by both scales in fp32.
 *
 * An INT8 expert layer is moe_quantize_int8 on the tokens, moe_swiglu_int8
 * (gathers each slot's token, gate and up with SwiGLU), moe_quantize_int8 on
 * its output, moe_product_int8 with the down matrices, and moe_combine of
 * moe_rows.h.
 *
 * Conventions are those of moe.h, and:
 *   - `cols` (the length of a reduction) is a multiple of 16 up to
 *     MOE_MAX_DIM, so an int8 row is whole 16-byte words; `rows` (output
 *     channels) is any size up to MOE_MAX_DIM.  int8 arrays are 16-byte
 *     aligned and without gaps between rows; scales, offsets, permutation
 *     and outputs are aligned to their element (MOE_ERR_INVALID otherwise).
 *   - outputs do not overlap inputs.
 *   - -128 is a value like any other: the int32 sum of 65536 products cannot
 *     overflow.
 */
#ifndef MOE_INT8_H
#define MOE_INT8_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Weights of n_experts matrices (1 for a dense one). */
typedef struct {
  int32_t n_experts; /* 1..MOE_MAX_EXPERTS */
  int32_t rows;      /* output channels    */
  int32_t cols;      /* inputs             */
  const int8_t* q;     /* [n_experts][rows][cols], 16-byte aligned */
  const float* scale;  /* [n_experts][rows]                        */
} moe_int8_weight;

/*
 * Rounds each row to int8: with a = max|x_row|,
 *   scale = a / 127 (fp32),  q = 127 x / a rounded to nearest, ties to even,
 * exactly (not from the rounded scale).  A row of zeros gives zeros and scale 0;
 * a row with an infinity or NaN gives zeros and scale NaN, which makes every
 * product of the row NaN.
 *   x      [n_rows][cols], type MOE_ACT_F32 or MOE_ACT_BF16, rows x_stride
 *          elements apart (>= cols), aligned to its element.
 *   q      out int8 [n_rows][cols]; scale out fp32 [n_rows].
 */
moe_status moe_quantize_int8(const void* x, int x_type, int64_t x_stride, int n_rows, int cols,
                             int8_t* q, float* scale, hipStream_t stream);

/*
 * out[p][j] = scale[r] * w.scale[e][j] * sum_k q[r][k] * w.q[e][j][k],
 * rounded once to out_type; the sum takes its two factors in fp32 in the order
 * scale, w.scale.
 *   Dense (offsets NULL): w has one matrix, n_slots rows, r = p.
 *   Grouped: offsets (int32 [n_experts+1], moe_group's) gives the rows
 *     offsets[e] .. offsets[e+1]-1 to expert e.  With top_k == 0 the left
 *     operand is in expert order already (r = p, q has n_slots rows); with
 *     top_k > 0 row p is token perm[p] / top_k of q, which has n_slots /
 *     top_k rows (perm: moe_group's; top_k must divide n_slots).  Rows of
 *     out from offsets[n_experts] on are written as 0.
 *   out    [n_slots][w.rows], rows out_stride elements apart.
 */
moe_status moe_product_int8(const moe_int8_weight* w, const int8_t* q, const float* scale,
                            int n_slots, const int32_t* offsets, const int32_t* perm, int top_k,
                            void* out, int out_type, int64_t out_stride, hipStream_t stream);

/*
 * The gate and up products of the same rows with SwiGLU in their epilogue:
 * out = g / (1 + exp(-g)) * u with g, u as moe_product_int8 would give them
 * in fp32, rounded once to out_type.  gate and up have the same shape.  The
 * other arguments are moe_product_int8's.  Below g = -87, where exp(-g)
 * leaves fp32, out may be 0 (the exact value is below 1.5e-36 |u|).
 */
moe_status moe_swiglu_int8(const moe_int8_weight* gate, const moe_int8_weight* up,
                           const int8_t* q, const float* scale, int n_slots,
                           const int32_t* offsets, const int32_t* perm, int top_k, void* out,
                           int out_type, int64_t out_stride, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_INT8_H */
