/*
 * moe_mxfp4.h -- rounding to MXFP4 and back, and products of MXFP4 rows by
 * MXFP4 weights, dense or grouped by expert.
 *
 * Values are those of moe.h's MOE_W_MXFP4: E2M1 codes, two a byte, in blocks
 * of 32 consecutive columns under one UE8M0 scale byte u, 2^(u-127).  Both
 * operands of a product are MXFP4; the products of their values and of their
 * scales are formed by the matrix cores and summed in fp32.
 *
 * An MXFP4 expert layer is moe_quantize_mxfp4 (or moe_rmsnorm_mxfp4 of
 * moe_norm.h) on the tokens, moe_swiglu_mxfp4 (gathers each slot's token,
 * gate and up with SwiGLU), moe_quantize_mxfp4 on its output,
 * moe_product_mxfp4 with the down matrices, and moe_combine of moe_rows.h.
 *
 * Layout of a matrix [rows][cols]:
 *   codes   uint8 [rows][cols/2], as in moe.h: 16-byte aligned, without gaps.
 *   scales  uint8 [MOE_MXFP4_WORDS(cols)][rows][16], 16-byte aligned: byte i of
 *           word w of a row is the scale of block 16 w + i.  Bytes past block
 *           cols/32 - 1 are 0.  (The words of neighbouring rows lie together,
 *           as a product takes them: 16 blocks of many rows at a time.)
 * Experts follow one another in both.
 *
 * Conventions are those of moe.h, and:
 *   - `cols` is a multiple of 32 up to MOE_MAX_DIM; `rows` (output channels)
 *     is any size up to MOE_MAX_DIM.  offsets, permutation and outputs are
 *     aligned to their element (MOE_ERR_INVALID otherwise).
 *   - outputs do not overlap inputs.
 *   - scale bytes are 2..252, or 255 for a block that is NaN (every product
 *     of its row is then NaN).  Others give unspecified values, in bounds.
 */
#ifndef MOE_MXFP4_H
#define MOE_MXFP4_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 16-byte words of scales in a row. */
#define MOE_MXFP4_WORDS(cols) (((cols) + 511) / 512)

/* Weights of n_experts matrices (1 for a dense one). */
typedef struct {
  int32_t n_experts; /* 1..MOE_MAX_EXPERTS */
  int32_t rows;      /* output channels    */
  int32_t cols;      /* inputs             */
  const uint8_t* codes;  /* [n_experts][rows][cols/2]                      */
  const uint8_t* scales; /* [n_experts][MOE_MXFP4_WORDS(cols)][rows][16]   */
} moe_mxfp4_weight;

/*
 * Rounds each row to MXFP4: a block whose largest magnitude is a has
 *   u = 127 + clamp(floor(log2 a) - 2, -125, 125)
 * and its values over 2^(u-127) go to the nearest E2M1 value, ties to even;
 * magnitudes past 6 go to 6.  A block with an infinity or NaN has codes 0 and u
 * = 255.
 *   x       [n_rows][cols], type MOE_ACT_F32 or MOE_ACT_BF16, rows x_stride
 *           elements apart (>= cols), aligned to its element.
 */
moe_status moe_quantize_mxfp4(const void* x, int x_type, int64_t x_stride, int n_rows, int cols,
                              uint8_t* codes, uint8_t* scales, hipStream_t stream);

/* x = the values of codes and scales, exact in either type; NaN under a scale
 * of 255.  x as in moe_quantize_mxfp4. */
moe_status moe_dequantize_mxfp4(const uint8_t* codes, const uint8_t* scales, int n_rows, int cols,
                                void* x, int x_type, int64_t x_stride, hipStream_t stream);

/*
 * out[p][j] = sum_k a[r][k] * w[e][j][k] of the values a of the left operand
 * (codes, scales) and w of the weights, rounded once to out_type.  The sum is
 * fp32, in an order that the sizes fix.
 *   Dense (offsets NULL): w has one matrix, n_slots rows, r = p.
 *   Grouped: offsets (int32 [n_experts+1], moe_group's) gives the rows
 *     offsets[e] .. offsets[e+1]-1 to expert e.  With top_k == 0 the left
 *     operand is in expert order already (r = p, n_slots rows); with top_k >
 *     0 row p is token perm[p] / top_k of it, which has n_slots / top_k rows
 *     (perm: moe_group's; top_k must divide n_slots).  Rows of out from
 *     offsets[n_experts] on are written as 0.
 *   out    [n_slots][w.rows], rows out_stride elements apart.
 */
moe_status moe_product_mxfp4(const moe_mxfp4_weight* w, const uint8_t* codes,
                             const uint8_t* scales, int n_slots, const int32_t* offsets,
                             const int32_t* perm, int top_k, void* out, int out_type,
                             int64_t out_stride, hipStream_t stream);

/*
 * The gate and up products of the same rows with SwiGLU in their epilogue:
 * out = g / (1 + exp(-g)) * u with g, u as moe_product_mxfp4 would give them
 * in fp32, rounded once to out_type.  gate and up have the same shape.  The
 * other arguments are moe_product_mxfp4's.  Below g = -87, where exp(-g)
 * leaves fp32, out may be 0 (the exact value is below 1.5e-36 |u|).
 */
moe_status moe_swiglu_mxfp4(const moe_mxfp4_weight* gate, const moe_mxfp4_weight* up,
                            const uint8_t* codes, const uint8_t* scales, int n_slots,
                            const int32_t* offsets, const int32_t* perm, int top_k, void* out,
                            int out_type, int64_t out_stride, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_MXFP4_H */
