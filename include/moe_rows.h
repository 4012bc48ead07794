/*
 * moe_rows.h -- rows in expert order, and the gradients of routing.
 *
 * moe.h groups tokens by expert as indices and runs its own experts on them.
 * The calls here move the rows themselves, for experts that the caller runs
 * (any matrix product over contiguous row ranges offsets[e] .. offsets[e+1]),
 * and differentiate the steps around the experts: the copy into expert order,
 * the weighted sum back into token order, and the learned router's weights.
 *
 * Conventions are those of moe.h (device pointers owned by the caller, work
 * enqueued on `stream`, errors before anything is enqueued, nothing
 * allocated, n_tokens == 0 is valid), and:
 *   - slot i of token t has flat index f = t*top_k + i; offsets and inv_perm
 *     are moe_group's.  A slot without an expert has inv_perm -1; an entry
 *     outside [0, n_tokens*top_k) is taken as -1 too.
 *   - `type` is a moe_act_type.  Strides are in elements from one row to the
 *     next and at least `hidden`; the elements of a row are contiguous and
 *     a row may start at any multiple of its element size.  The other arrays
 *     hold 4-byte elements and are aligned to them (MOE_ERR_INVALID
 *     otherwise).
 *   - outputs do not overlap inputs, except where a call says that they may.
 *   - hidden is any size in 1..MOE_MAX_DIM.  Sums are taken in fp32 in slot
 *     order and rounded once to the output's type, so results do not depend
 *     on scheduling.
 *   - every row of an output [n_tokens*top_k][hidden] in expert order is
 *     written; the rows from offsets[n_experts] on, which no slot has, are 0.
 */
#ifndef MOE_ROWS_H
#define MOE_ROWS_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* rows[inv_perm[f]] = x[f / top_k]. */
moe_status moe_dispatch(const void* x, int type, int64_t x_stride, int n_tokens, int top_k,
                        int hidden, int n_experts, const int32_t* offsets,
                        const int32_t* inv_perm, void* rows, int64_t rows_stride,
                        hipStream_t stream);

/* Gradient of moe_dispatch: dx[t] = sum_i drows[inv_perm[t*top_k + i]]; a
 * token without a row gets 0. */
moe_status moe_dispatch_backward(const void* drows, int type, int64_t rows_stride, int n_tokens,
                                 int top_k, int hidden, const int32_t* inv_perm, void* dx,
                                 int64_t dx_stride, hipStream_t stream);

/*
 * y[t] = base[t] + sum_i topk_w[t][i] * rows[inv_perm[t*top_k + i]].
 *   rows    [n_tokens*top_k][hidden] of `type`: the experts' outputs.
 *   topk_w  fp32 [n_tokens][top_k].  A slot without a row is left out, whatever
 *           its weight.
 *   base    nullable, of y_type: the shared expert's output or a residual.  It
 *           may be y itself (same stride).
 *   y       out, of y_type.
 */
moe_status moe_combine(const void* rows, int type, int64_t rows_stride, int n_tokens, int top_k,
                       int hidden, const float* topk_w, const int32_t* inv_perm,
                       const void* base, int64_t base_stride, void* y, int y_type,
                       int64_t y_stride, hipStream_t stream);

/*
 * Gradients of moe_combine, both in one pass over dy and rows:
 *   drows[p]    = topk_w[f] * dy[f / top_k] for p = inv_perm[f], of `type`
 *   dw[t][i]    = <dy[t], rows[inv_perm[t*top_k + i]]>, fp32; 0 for a slot
 *                 without a row
 * (the gradient of base is dy).  The dot product is summed in fp32 in an order
 * that n_tokens, hidden and the types fix, so a call repeats bit for bit, but
 * dw of the same token may differ in its last bits between batches of fewer
 * than 2048 tokens and larger ones.
 */
moe_status moe_combine_backward(const void* dy, int y_type, int64_t dy_stride, const void* rows,
                                int type, int64_t rows_stride, int n_tokens, int top_k,
                                int hidden, int n_experts, const float* topk_w,
                                const int32_t* offsets, const int32_t* inv_perm, void* drows,
                                int64_t drows_stride, float* dw, hipStream_t stream);

/*
 * Gradient of the weights of moe_route (and of moe_route_ex without tail
 * pruning: a selection by groups or with a bias has the same weights; pruned
 * weights see below).  With
 * s_i = sqrt(softplus(l_i)) of the chosen experts, S = sum_j s_j and
 * w_i = routed_scale * s_i / S,
 *   dL/dl_i = routed_scale / S^2 * sum_j s_j (dw_i - dw_j)
 *             * sigmoid(l_i) / (2 s_i),
 * evaluated in fp64 and rounded once; 0 for every expert not chosen.  The
 * selection itself has no gradient.
 *   logits    fp32 [n_tokens][n_experts], the router's.
 *   topk_ids  int32 [n_tokens][top_k], distinct within a token.  An id -1 is
 *             left out of the sums; one outside [-1, n_experts) too, and
 *             sets MOE_DEVERR_EXPERT_ID in *dev_error (nullable).
 *   dw        fp32 [n_tokens][top_k].
 *   dlogits   out fp32 [n_tokens][n_experts], fully overwritten.
 * Logits are finite.  Where all the chosen ones are below -700, S leaves the
 * range of fp64 and the chosen entries are inaccurate or NaN, as the weights
 * are.
 *
 * Tail pruning (keep_max, min_w) rescales: its weights are alpha * w_i on the
 * slots that it keeps, with alpha = sqrt(A / K), A the sum of w_j^2 over all
 * slots and K over the kept ones.  They depend on the dropped slots' logits
 * too, and leaving those out, as the ids -1 that pruning writes would, is not
 * their gradient.  With g the gradient by the pruned weights and
 * G = sum_kept g_j w_j it is this call on the ids of the same routing without
 * pruning, with
 *   dw_i = alpha * (g_i [i kept] + G w_i (1/A - [i kept]/K)).
 */
moe_status moe_route_backward(const float* logits, const int32_t* topk_ids, const float* dw,
                              int n_tokens, int n_experts, int top_k, float routed_scale,
                              float* dlogits, int32_t* dev_error, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_ROWS_H */
