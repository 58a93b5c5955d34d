/*
 * fp8mm_moe.h - C ABI of the operators around the grouped (MoE) FP8 GEMMs of
 * fp8mm.h: layer norm, routing of tokens to experts, permutation of token
 * rows into expert order and back, and the gated activation between an
 * expert's two products with its input kept in 8 bits for the backward pass.
 *
 * The conventions of fp8mm.h hold here too: device pointers owned by the
 * caller, argument checks on the host before anything is enqueued, FP8MM_EINVAL
 * / FP8MM_ENOTIMPL / FP8MM_ERUNTIME with fp8mm_last_error(), no allocation, no
 * synchronization, kernels on `stream` only, so that calls can be captured
 * into HIP graphs.  Scratch memory is a caller's workspace whose size a host
 * query gives; its contents do not matter before or after the call.  Results
 * repeat bit for bit: no atomics decide an order of additions.
 *
 * Matrices are row-major with a leading dimension (row stride) in elements.
 * Rows of layer norm, routing, moe_dispatch and moe_combine may have any
 * length and start at any element; fp8_* calls need what the quantizers need
 * (16-byte aligned bases, leading dimensions of whole 16 bytes, columns in
 * groups of 128).  Outputs must not overlap inputs or each other.
 */
#ifndef FP8MM_MOE_H
#define FP8MM_MOE_H

#include "fp8mm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Type of activations and parameters: fp8mm_out_dtype's values. */
typedef fp8mm_out_dtype fp8mm_dtype;

/* ---------------------------------------------------------------------------
 * Layer norm over the last dimension.
 *   mean = sum(x) / C, var = sum((x - mean)^2) / C, rstd = 1 / sqrt(var + eps)
 *   y = (x - mean) rstd weight + bias
 * x, y: [R, C] of `dtype`, row strides ld_x, ld_y >= C.  weight, bias: [C] of
 * `param_dtype`, or NULL (1 and 0).  mean, rstd: float32 [R], or NULL where no
 * backward follows.  eps: finite, >= 0.  1 <= C <= 2^22; R of 0 is
 * allowed.
 * Statistics and sums are float32 with one rounding to `dtype`.
 * ------------------------------------------------------------------------- */
fp8mm_status fp8mm_layer_norm(const void* x, fp8mm_dtype dtype, int64_t R, int64_t C, int64_t ld_x,
                              const void* weight, const void* bias, fp8mm_dtype param_dtype, float eps, void* y,
                              int64_t ld_y, float* mean, float* rstd, hipStream_t stream);

/* Workspace bytes of fp8mm_layer_norm_backward; -1 for arguments out of
 * range.  Host only. */
int64_t fp8mm_layer_norm_backward_workspace(int64_t R, int64_t C);

/* With xh = (x - mean) rstd and a = dy weight:
 *   dx = rstd (a - sum(a) / C - xh sum(a xh) / C)
 *   dweight = sum over rows of dy xh,  dbias = sum over rows of dy
 * dy, x, dx: [R, C] of `dtype`; mean, rstd: as the forward wrote them.  dx,
 * dweight and dbias may each be NULL; dweight and dbias are [C] of
 * `param_dtype`, and zeros for R = 0.  workspace: at least
 * fp8mm_layer_norm_backward_workspace(R, C) bytes, 16-byte aligned (NULL if
 * that is 0 or neither dweight nor dbias is wanted). */
fp8mm_status fp8mm_layer_norm_backward(const void* dy, int64_t ld_dy, const void* x, int64_t ld_x, fp8mm_dtype dtype,
                                       int64_t R, int64_t C, const void* weight, fp8mm_dtype param_dtype,
                                       const float* mean, const float* rstd, void* dx, int64_t ld_dx, void* dweight,
                                       void* dbias, void* workspace, int64_t workspace_bytes, hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Routing of T tokens to k of E experts.
 *   s = softmax(logits) or sigmoid(logits) of a token's row, float32; scores
 *     below 2^-126, where float32 has no normal numbers, count as 0
 *   key = s + bias (bias NULL: key = logit, which orders the same)
 *   groups > 1: the E experts are `groups` runs of E / groups; a group's score
 *     is its largest key, or (FP8MM_GROUP_TOP2) the sum of its two largest
 *     s + bias; only the group_topk best groups take part
 *   ids = the k largest keys, in descending order
 *   weights = s[ids], divided by (their sum + 1e-20) if renormalize, times
 *     scale.  The bias takes part in the choice only.
 * Equal keys and equal groups go to the lower index.  An expert with a logit
 * or a key of -inf is never chosen; a slot for which none is left gets id -1
 * and weight 0 (a row of -inf logits alone: every slot).  A row with a NaN
 * logit or key, or with a +inf logit under softmax, has no defined choice and
 * gets ids 0 .. k-1 with NaN weights.
 *   logits: [T, E] of `dtype`, row stride ld >= E.  bias: float32 [E] or NULL.
 *   ids: int32 [T, k];  weights: float32 [T, k], both dense.
 * 1 <= k <= E; groups divides E, 1 <= group_topk <= groups (groups = 1 without
 * grouping); E <= 1024, k <= 64 and groups <= 64, else FP8MM_ENOTIMPL.
 * ------------------------------------------------------------------------- */
typedef enum { FP8MM_SCORE_SOFTMAX = 0, FP8MM_SCORE_SIGMOID = 1 } fp8mm_score;
typedef enum { FP8MM_GROUP_MAX = 0, FP8MM_GROUP_TOP2 = 1 } fp8mm_group_score;

fp8mm_status fp8mm_moe_route(const void* logits, fp8mm_dtype dtype, int64_t T, int64_t E, int64_t ld,
                             const float* bias, fp8mm_score score, int64_t k, int64_t groups, int64_t group_topk,
                             fp8mm_group_score group_score, int renormalize, float scale, int32_t* ids,
                             float* weights, hipStream_t stream);

/* Gradient of the logits from the gradient of the weights, the choice of ids
 * held fixed (it has no gradient, and neither has the bias):
 *   d_j = scale g_j, or scale (g_j - sum_l g_l s_l / S) / S with S = sum_l s_l +
 *   1e-20 if renormalize;  softmax: s_e (d_e - sum_l s_l d_l);
 *   sigmoid: s_e (1 - s_e) d_e
 * logits, ids, score, renormalize and scale: as in the forward; ids outside
 * [0, E) are empty slots, a token's others differ.  grad_weights: float32 [T, k]; grad_logits: [T, E]
 * of `dtype`, row stride ld_grad >= E, written whole; a row with a NaN logit (or
 * +inf under softmax) gets NaN. */
fp8mm_status fp8mm_moe_route_backward(const float* grad_weights, const void* logits, fp8mm_dtype dtype, int64_t T,
                                      int64_t E, int64_t ld, const int32_t* ids, int64_t k, fp8mm_score score,
                                      int renormalize, float scale, void* grad_logits, int64_t ld_grad,
                                      hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Permutation of token rows into expert order.
 * T k < 2^31 and C < 2^31 throughout, and one launch of at most 2^25 waves, else
 * FP8MM_EINVAL: T ceil(C / 512) waves for bf16 rows, T ceil(C / 256) for fp32
 * rows and T ceil(C / 1024) for codes in dispatch and combine; in combine's
 * backward T k, or T k / 4 for rows of at most 512 (bf16) or 256 (fp32) columns.
 * ------------------------------------------------------------------------- */

/* Workspace bytes of fp8mm_moe_plan for T tokens of k slots over E experts (0
 * for a few thousand slots); -1 for arguments out of range.  Host only. */
int64_t fp8mm_moe_plan_workspace(int64_t T, int64_t k, int64_t E);

/* ids int32 [T, k] -> offsets int32 [E], the experts' cumulative end rows as
 * every grouped call takes them, and row_of_slot int32 [T, k]: slot (t, j)'s
 * row among M = T k, by a stable sort of the slots by expert.  Slots whose id
 * lies outside [0, E) take the rows at and past offsets[E-1], in order, and
 * are written as ~row (a negative number).  T k < 2^31; E >= 1 (E <= 1024,
 * else FP8MM_ENOTIMPL).  workspace: at least fp8mm_moe_plan_workspace bytes,
 * 16-byte aligned (NULL if that is 0). */
fp8mm_status fp8mm_moe_plan(const int32_t* ids, int64_t T, int64_t k, int64_t E, int32_t* offsets,
                            int32_t* row_of_slot, void* workspace, int64_t workspace_bytes, hipStream_t stream);

/* out[row(t, j)] = x[t] for every slot, zeros in the rows of slots without an
 * expert.  x: [T, C] of `dtype`; out: [T k, C]; row_of_slot: int32 [T, k] as
 * fp8mm_moe_plan writes it (rows outside [0, T k) are skipped).  1 <= k <= 64.
 * The backward of a dispatch is fp8mm_moe_combine with weights = NULL. */
fp8mm_status fp8mm_moe_dispatch(const void* x, fp8mm_dtype dtype, int64_t T, int64_t C, int64_t ld_x,
                                const int32_t* row_of_slot, int64_t k, void* out, int64_t ld_out, hipStream_t stream);

/* The same as 1x128 FP8 codes, ready for fp8_scaled_grouped_mm_v2: exactly the
 * codes and scales that fp8_quantize_blockwise with block (1, 128) gives of
 * the dispatched rows, each token quantized once.  x: bf16 [T, C], C % 128 ==
 * 0, ld_x % 8 == 0; q: uint8 [T k, C], ld_q % 16 == 0; scale: float32
 * [C / 128, T k].  Rows of slots without an expert: codes 0, scales 1. */
fp8mm_status fp8_moe_dispatch(const void* x, int64_t T, int64_t C, int64_t ld_x, const int32_t* row_of_slot, int64_t k,
                              uint8_t* q, int64_t ld_q, float* scale, hipStream_t stream);

/* out[t] = sum_j weights[t, j] rows[row(t, j)] over the slots with an expert,
 * added in slot order in float32; a token without any gets zeros.  rows:
 * [T k, C] of `dtype`; weights: float32 [T, k] or NULL (1); out: [T, C]. */
fp8mm_status fp8mm_moe_combine(const void* rows, fp8mm_dtype dtype, int64_t T, int64_t C, int64_t ld_rows,
                               const int32_t* row_of_slot, const float* weights, int64_t k, void* out, int64_t ld_out,
                               hipStream_t stream);

/* grad_rows[row(t, j)] = weights[t, j] grad_out[t] (zeros in the rows of slots
 * without an expert) and grad_weights[t, j] = <grad_out[t], rows[row(t, j)]>
 * (0 for slots without an expert).  grad_out: [T, C], rows and grad_rows:
 * [T k, C], all of `dtype`.  grad_rows or grad_weights may be NULL; rows is
 * needed for grad_weights only. */
fp8mm_status fp8mm_moe_combine_backward(const void* grad_out, int64_t ld_go, const void* rows, int64_t ld_rows,
                                        fp8mm_dtype dtype, int64_t T, int64_t C, const int32_t* row_of_slot,
                                        const float* weights, int64_t k, void* grad_rows, int64_t ld_gr,
                                        float* grad_weights, hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Gated activation with an 8-bit checkpoint:  x = [gate, up] bf16 [R, 2 F],
 * h = gate sigmoid(gate) up, F % 128 == 0, F <= 2^21, R < 2^31 and
 * ceil(R / 32) (F / 128) <= 2^23 (one launch), else FP8MM_EINVAL.
 *   h: bf16 [R, F], or NULL.
 *   h_q, h_scale: the 1x128 codes uint8 [R, F] and scales float32 [F / 128, R]
 *     of the float32 values of h (no bf16 rounding in between), or NULL.
 *   ckpt, ckpt_scale: the 1x128 codes uint8 [R, 2 F] and scales float32
 *     [2 F / 128, R] of x, exactly those of fp8_quantize_blockwise with block
 *     (1, 128): what the backward needs of x in half its bytes; or NULL.
 * Any of the three outputs may be left out.
 * ------------------------------------------------------------------------- */
fp8mm_status fp8_swiglu(const void* x, int64_t R, int64_t F, int64_t ld_x, void* h, int64_t ld_h, uint8_t* h_q,
                        int64_t ld_hq, float* h_scale, uint8_t* ckpt, int64_t ld_ckpt, float* ckpt_scale,
                        hipStream_t stream);

/* Backward from the checkpoint alone, x' = code scale:  with sig =
 * sigmoid(gate'), d_gate = grad_h up' sig (1 + gate' (1 - sig)), d_up = grad_h
 * gate' sig.  grad_h: bf16 [R, F]; grad_x: bf16 [R, 2 F].  h: NULL, or bf16
 * [R, F] that gets gate' sig up' (the input of the second product again, for
 * its weight gradient). */
fp8mm_status fp8_swiglu_backward(const void* grad_h, int64_t ld_gh, const uint8_t* ckpt, int64_t ld_ckpt,
                                 const float* ckpt_scale, int64_t R, int64_t F, void* grad_x, int64_t ld_gx, void* h,
                                 int64_t ld_h, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8MM_MOE_H */
