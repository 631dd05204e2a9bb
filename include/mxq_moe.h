/*
 * mxq_moe.h -- C ABI of libmxq, second part: the routed-expert layer around
 * the MXFP4 grouped GEMM of mxq.h.  Router, grouped order of the routed rows,
 * the way there (dispatch) and back (combine), and the experts' activation
 * with its input kept in 8 bits for the backward.
 *
 * The conventions of mxq.h hold here: device pointers owned by the caller, no
 * allocation, no synchronization, host-side checks that return a negative
 * mxq_status before any HIP call, MXQ_OK without a launch for empty problems,
 * dense row-major tensors of any alignment, but for int32 and float arrays
 * (index, rows, weights, bias, offs, ...), which are 4-byte aligned
 * (MXQ_ERR_ALIGN otherwise).  Every result is deterministic: sums have a
 * fixed order and no atomic decides one.  Sums, scores and statistics are
 * held in fp32 or fp64; each output is rounded once, nearest-even.
 *
 * MXQ_ERR_HIP also means a call of more threads than one launch takes (2^32):
 * 64 per token and 512 columns in the row operations, 16 or 64 per token in the
 * router.
 *
 * Words used below
 * ----------------
 *  slot   one of the tokens * top_k routed places: slot t * top_k + j is
 *         token t's j-th expert.
 *  row    a row of the grouped order that the grouped GEMM takes: all slots of
 *         local expert 0 first, then those of expert 1, ... , each expert's
 *         slots in rising slot order; after them, from offs[local - 1] on, the
 *         slots that no local expert serves.  There are tokens * top_k rows.
 *  rows   int32 [tokens, top_k]: rows[t, j] = r >= 0, the slot's row, or
 *         ~r < 0 for a slot that is not served here and whose row r lies
 *         behind the last expert's.  A value outside [~(n-1), n-1], n =
 *         tokens * top_k, is taken for a slot without a row: nothing is read
 *         or written for it.
 */
#ifndef MXQ_MOE_H
#define MXQ_MOE_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MXQ_SCORE_SOFTMAX = 0, MXQ_SCORE_SIGMOID = 1 } mxq_score;

/*
 * moe_route -- experts and weights of each token from its router logits.
 * logits [tokens, experts] of dtype t.  Per token with logits x_e:
 *   s_e = sigmoid(x_e), or the softmax of x over the experts;
 *   key_e = s_e + bias[e] (bias fp32 [experts], NULL = none; it moves the
 *     choice only, not the weights).  Without a bias and with one group the
 *     order of the keys is the order of the logits.
 *   groups > 1: experts form `groups` runs of experts / groups; a group's
 *     value is the sum of its group_best (1 or 2) largest keys, and only the
 *     top_groups groups of largest value are kept.
 *   The top_k experts of largest key are chosen, in falling order.
 *   weights[t, j] = scale * s_j, divided by the sum of the chosen s with
 *     renormalize (0 where sigmoid scores all vanish in fp64, below e^-745).
 * Ties go to the lower group or expert.  Keys are compared as in fp64: where
 * fp32 keys lie too near each other to tell, the token is decided in fp64.
 * An expert whose logit or bias is -inf or NaN is never chosen nor counted in a
 * group's value; one whose logit is -inf or NaN is not counted in a softmax
 * either.  A bias of +inf is a key of +inf: such an expert comes before every
 * other, and a group with one before every group without.  Softmax logits must
 * be below +inf.  A token with token_mask[t] == 0 (uint8 [tokens], NULL = none)
 * chooses none, whatever its logits hold.
 * A place without an expert has index -1 and weight 0.
 * Outputs: weights fp32 and index int32, both [tokens, top_k].
 * Errors: MXQ_ERR_SHAPE (tokens < 0, experts not in 1..1024, top_k not in
 * 1..min(32, experts), groups not in 1..64 or no divisor of experts,
 * top_groups not in 1..groups, group_best not 1 or 2, tokens * experts >=
 * 2^40), MXQ_ERR_DTYPE, MXQ_ERR_FORMAT (score), MXQ_ERR_NULL, MXQ_ERR_ALIAS
 * (an output overlaps another buffer), MXQ_ERR_HIP.
 */
int moe_route(const void* logits, int t, int64_t tokens, int64_t experts, int64_t top_k, int score,
              const float* bias, int64_t groups, int64_t top_groups, int group_best, int renormalize, double scale,
              const uint8_t* token_mask, float* weights, int32_t* index, void* stream);

/*
 * moe_route_bwd -- gradient of moe_route's weights with respect to its logits,
 * for the experts it chose (index as moe_route wrote it; the choice itself has
 * no gradient, nor has the bias).  With g = grad_weights [tokens, top_k] fp32
 * and sums over a token's chosen experts,
 *   u_j = scale * (g_j - sum_i g_i s_i / S) / S, S = sum_i s_i, with
 *         renormalize; u_j = scale * g_j without;
 *   sigmoid: grad_j = u_j s_j (1 - s_j);  softmax: grad_e = s_e (u_e -
 *         sum_i u_i s_i), u = 0 for experts not chosen.
 * grad_logits [tokens, experts] of dtype t is written in full: zeros wherever
 * no gradient arrives, and in every row without a chosen expert.  Index values
 * outside [0, experts) count as places without an expert; the experts of one
 * token must differ.
 * Errors: as moe_route (index, grad_weights and logits must not overlap
 * grad_logits).
 */
int moe_route_bwd(const void* logits, int t, int64_t tokens, int64_t experts, int64_t top_k, int score,
                  int renormalize, double scale, const int32_t* index, const float* grad_weights, void* grad_logits,
                  void* stream);

/*
 * moe_plan -- the grouped order of the slots: a stable counting sort by local
 * expert.  index int32 [tokens, top_k] as moe_route writes it; local experts
 * are first .. first + local - 1, every other value (-1 among them) is a slot
 * that is not served.  Writes offs int32 [local] (cumulative counts: what
 * mxfp4_grouped_mm_fwd takes), rows int32 [tokens, top_k] and slots int32
 * [tokens * top_k] (row r holds slot slots[r], also behind the last expert).
 * workspace: moe_plan_workspace(tokens, top_k, local) bytes, 4-byte aligned
 * (NULL if that is 0); its contents before and after the call mean nothing,
 * and calls that may run at the same time need one each.  With no slot at all
 * offs is still written (zeros).
 * Errors: MXQ_ERR_SHAPE (tokens < 0, top_k < 1, tokens * top_k >= 2^31 - 2^16,
 * local not in 1..1024, first < 0 or first + local >= 2^31, workspace_bytes too
 * small), MXQ_ERR_NULL, MXQ_ERR_ALIGN (workspace), MXQ_ERR_ALIAS, MXQ_ERR_HIP.
 * moe_plan_workspace returns MXQ_ERR_SHAPE for sizes that moe_plan refuses.
 */
int64_t moe_plan_workspace(int64_t tokens, int64_t top_k, int64_t local);
int moe_plan(const int32_t* index, int64_t tokens, int64_t top_k, int64_t first, int64_t local, int32_t* offs,
             int32_t* rows, int32_t* slots, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * moe_dispatch -- rows of tokens into the grouped order: out[rows[t, j]] =
 * x[t], and zeros in the rows of slots that are not served, so that a plan's
 * out is written in full.  x [tokens, hidden], out [tokens * top_k, hidden] of
 * dtype t.
 * moe_dispatch_bwd -- grad_x[t] = sum over the served slots of
 * grad_out[rows[t, j]], in fp32, j rising (moe_combine with weights of 1).
 * Errors: MXQ_ERR_SHAPE (negative sizes, top_k < 1, tokens * top_k >= 2^31 -
 * 2^16, hidden > 2^20), MXQ_ERR_DTYPE, MXQ_ERR_NULL, MXQ_ERR_ALIAS,
 * MXQ_ERR_HIP.
 */
int moe_dispatch(const void* x, int t, int64_t tokens, int64_t hidden, int64_t top_k, const int32_t* rows, void* out,
                 void* stream);
int moe_dispatch_bwd(const void* grad_out, int t, int64_t tokens, int64_t hidden, int64_t top_k, const int32_t* rows,
                     void* grad_x, void* stream);

/*
 * moe_dispatch_quantized -- moe_dispatch with the rows quantized on the way:
 * what quantizing moe_dispatch's output would give, bit for bit, but each
 * token is read and quantized once.  fmt MXQ_FMT_FP8: codes uint8 [rows,
 * hidden] and E8M0 scales uint8 [rows, hidden / 32] as quantize_cache_packed
 * writes them for fp8 and block_size 32 (the operand of
 * mxfp4_grouped_mm_fwd_w4a8); MXQ_FMT_MXFP4: codes [rows, hidden / 2] and
 * scales as quantize_mxfp4 writes them (the operand of
 * mxfp4_grouped_mm_fwd_w4a4).  Inputs must be finite.
 * Errors: as moe_dispatch, and MXQ_ERR_SHAPE (hidden % 32), MXQ_ERR_FORMAT.
 */
int moe_dispatch_quantized(const void* x, int t, int64_t tokens, int64_t hidden, int64_t top_k, const int32_t* rows,
                           int fmt, uint8_t* codes, uint8_t* scales, void* stream);

/*
 * moe_combine -- the rows back to their tokens: out[t] = sum over the served
 * slots of weights[t, j] * y[rows[t, j]], in fp32, j rising; zeros where none
 * is served.  y [tokens * top_k, hidden], out [tokens, hidden] of dtype t,
 * weights fp32 [tokens, top_k] (not read at slots that are not served).
 * moe_combine_bwd -- grad_y[rows[t, j]] = weights[t, j] * grad_out[t] (zeros in
 * the rows of slots that are not served) and grad_weights[t, j] = grad_out[t] .
 * y[rows[t, j]] (0 where not served), fp32 sums.  grad_y or grad_weights may
 * be NULL (not wanted); y is read for grad_weights only, weights for grad_y
 * only.
 * Errors: as moe_dispatch.
 */
int moe_combine(const void* y, int t, int64_t tokens, int64_t hidden, int64_t top_k, const int32_t* rows,
                const float* weights, void* out, void* stream);
int moe_combine_bwd(const void* grad_out, const void* y, int t, int64_t tokens, int64_t hidden, int64_t top_k,
                    const int32_t* rows, const float* weights, void* grad_y, float* grad_weights, void* stream);

/*
 * swiglu_fwd -- h = silu(gate) * up with gate_up [rows, 2 * inter] = [gate |
 * up], h [rows, inter], both of dtype t: silu(g) = g / (1 + exp(-g)), fp32.
 * offs int32 [experts] (device, as the grouped GEMM takes it; NULL = every row)
 * says how many rows count: rows from offs[experts - 1] on are written as
 * zeros and not read.
 * With codes and scales (both or neither) gate_up is kept for the backward in
 * 8 bits: E4M3 codes uint8 [rows, 2 * inter] and one E8M0 scale byte per 32
 * columns, uint8 [rows, 2 * inter / 32], as quantize_cache_packed writes them
 * for fp8 and block_size 32.  Rows that do not count are left as they were.
 * An inf or a NaN in gate or up is one in h, and swiglu_bwd's gradients at its
 * place are inf or NaN too (grad_gate always, grad_up where gate was not
 * finite); the finite values that share its block of 32 columns are lost to the
 * block's scale, and their gradients are not those of their values.
 * swiglu_bwd -- grad_gate_up [rows, 2 * inter] of grad_h [rows, inter]:
 *   grad_gate = grad_h * up * s (1 + gate (1 - s)), grad_up = grad_h * gate *
 *   s, s = sigmoid(gate), fp32, with gate and up read from codes and scales
 *   (gate_up NULL) or from gate_up (codes and scales NULL).  Rows that do not
 *   count get zeros.
 * Errors: MXQ_ERR_SHAPE (negative sizes, inter % 32 != 0, inter > 2^20, rows *
 * inter >= 2^40, experts < 1 with offs), MXQ_ERR_DTYPE, MXQ_ERR_NULL,
 * MXQ_ERR_ALIAS, MXQ_ERR_HIP.
 */
int swiglu_fwd(const void* gate_up, int t, int64_t rows, int64_t inter, const int32_t* offs, int64_t experts, void* h,
               uint8_t* codes, uint8_t* scales, void* stream);
int swiglu_bwd(const void* grad_h, const void* gate_up, const uint8_t* codes, const uint8_t* scales, int t,
               int64_t rows, int64_t inter, const int32_t* offs, int64_t experts, void* grad_gate_up, void* stream);

/*
 * swiglu_quantized -- h as swiglu_fwd writes it, rounded to t, and then quantized
 * on the way out: the operand of the low-bit down product.  What quantizing
 * swiglu_fwd's h would give, bit for bit, without writing h.  fmt, codes and
 * scales as in moe_dispatch_quantized, with inter for hidden; rows that do not
 * count get what a row of zeros gives.  h must be finite.
 * Errors: as swiglu_fwd, and MXQ_ERR_FORMAT.
 */
int swiglu_quantized(const void* gate_up, int t, int64_t rows, int64_t inter, const int32_t* offs, int64_t experts,
                     int fmt, uint8_t* codes, uint8_t* scales, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MXQ_MOE_H */
