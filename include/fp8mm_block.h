/*
 * fp8mm_block.h - C ABI of the operators around a block's dense FP8 products
 * and its router: the root-mean-square norm that adds the residual and gives
 * the product's codes, low-rank adapters of many requests beside a shared
 * projection, and the balance loss of a router with its per-expert counts.
 *
 * The conventions of fp8mm_moe.h hold here too: device pointers owned by the
 * caller, argument checks on the host before anything is enqueued, FP8MM_EINVAL
 * / FP8MM_ENOTIMPL / FP8MM_ERUNTIME with fp8mm_last_error(), no allocation, no
 * synchronization, kernels on `stream` only, so that calls can be captured
 * into HIP graphs.  A call launches on the current device, which has to be the
 * stream's and the pointers'.  Scratch memory is a caller's workspace whose size
 * a host query gives; its contents do not matter before or after the call, and
 * two calls that can run at once need one each.  Results repeat bit for bit: no
 * atomics decide an order of additions of floats.
 *
 * Matrices are row-major with a leading dimension (row stride) in elements, from
 * the number of columns to 2^40.  Rows may have any length and start at any
 * element, except where codes are written (see there).  Outputs must not overlap
 * inputs or each other, except where a comment allows it.
 */
#ifndef FP8MM_BLOCK_H
#define FP8MM_BLOCK_H

#include "fp8mm_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * Root-mean-square norm over the last dimension, with the residual's addition
 * in front and the next product's codes behind it, in one pass.
 *   h = x + residual, rounded to `dtype` (residual NULL: h = x)
 *   rstd = 1 / sqrt(sum(h^2) / C + eps)
 *   y = (h rstd) weight
 *   q, scale: the E4M3 codes and scales of y's float32 values (no rounding to
 *     `dtype` in between), as the quantizers define them:
 *     FP8MM_BLOCK_1x128: q [R, C], scale float32 [C / 128, R], amax / 448 (0 -> 1)
 *     FP8MM_ROWWISE: q [R, C], scale float32 [R], amax / 448 + 1e-12
 * x, residual, h, y: [R, C] of `dtype`.  weight: [C] of `param_dtype`, or NULL
 * (1).  rstd: float32 [R], or NULL.  h, y and q may each be NULL (h without a
 * residual is not written at all); `recipe` counts only where q is given.
 * Codes are made of bf16 rows only: q 16-byte aligned, ld_q % 16 == 0, C % 128 ==
 * 0 (FP8MM_BLOCK_1x128) or C % 16 == 0 (FP8MM_ROWWISE).
 * eps: finite, >= 0.  1 <= C <= 2^22, 0 <= R < 2^31.  Sums are float32; a row
 * whose sum of squares, or its mean and eps together, is past float32's range has
 * rstd 0.
 * ------------------------------------------------------------------------- */
fp8mm_status fp8mm_rms_norm(const void* x, int64_t ld_x, const void* residual, int64_t ld_res, fp8mm_dtype dtype,
                            int64_t R, int64_t C, const void* weight, fp8mm_dtype param_dtype, float eps, void* h,
                            int64_t ld_h, void* y, int64_t ld_y, uint8_t* q, int64_t ld_q, float* scale,
                            fp8mm_recipe recipe, float* rstd, hipStream_t stream);

/* Workspace bytes of fp8mm_rms_norm_backward; -1 for arguments out of range.
 * Host only. */
int64_t fp8mm_rms_norm_backward_workspace(int64_t R, int64_t C);

/* With a = dy weight and hr = h rstd:
 *   dx = rstd (a - hr sum(a hr) / C) + grad_h
 *   dweight = sum over rows of dy hr
 * dx is the gradient of x and of the residual alike.  dy, h, grad_h (what arrives
 * at h from behind, or NULL), dx: [R, C] of `dtype`; rstd: as the forward wrote it.
 * dx and dweight ([C] of `param_dtype`, zeros for R = 0) may each be NULL.  dx may
 * be grad_h itself.  workspace: at least fp8mm_rms_norm_backward_workspace(R, C)
 * bytes, 16-byte aligned (NULL if that is 0 or no dweight is wanted). */
fp8mm_status fp8mm_rms_norm_backward(const void* dy, int64_t ld_dy, const void* h, int64_t ld_h, const void* grad_h,
                                     int64_t ld_gh, fp8mm_dtype dtype, int64_t R, int64_t C, const void* weight,
                                     fp8mm_dtype param_dtype, const float* rstd, void* dx, int64_t ld_dx,
                                     void* dweight, void* workspace, int64_t workspace_bytes, hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Balance loss of a router, and the experts' counts.  The batch is S sequences,
 * sequence s the rows [ends[s - 1], ends[s]); rows at and past ends[S - 1] belong
 * to none.  ends NULL: one sequence of all T rows (S = 1).
 *   p = softmax(logits), or sigmoid(logits) divided by its sum over the experts
 *   tokens_s = rows of sequence s that have a logit other than -inf (a row of
 *     -inf alone is padding: no probabilities, no slots, not counted)
 *   counts_se = slots of those rows with id e (ids outside [0, E) are empty)
 *   loss = coeff / S' sum_s sum_e (E counts_se / (k tokens_s)) (sum_t p_te /
 *     tokens_s) over the S' sequences with tokens_s > 0; 0 if there is none
 * logits: [T, E] of `dtype`, row stride ld.  ids: int32 [T, k], dense.  ends: int32
 * [S], ascending, from 0 to T (others give wrong sums, but no access out of range).
 * loss: float32 [1]; counts: int32 [S, E]; tokens: int32 [S].  A NaN logit in a
 * counted row (or +inf under softmax) makes the loss NaN.
 * E <= 1024 and k <= 64, else FP8MM_ENOTIMPL; T k < 2^31, S E < 2^31, S <= 2^20.
 * workspace: at least fp8mm_moe_balance_loss_workspace(T, E, S) bytes, 16-byte
 * aligned (NULL if that is 0, as for one sequence of a few tokens).
 * ------------------------------------------------------------------------- */
int64_t fp8mm_moe_balance_loss_workspace(int64_t T, int64_t E, int64_t S);

fp8mm_status fp8mm_moe_balance_loss(const void* logits, fp8mm_dtype dtype, int64_t T, int64_t E, int64_t ld,
                                    const int32_t* ids, int64_t k, fp8mm_score score, const int32_t* ends, int64_t S,
                                    float coeff, float* loss, int32_t* counts, int32_t* tokens, void* workspace,
                                    int64_t workspace_bytes, hipStream_t stream);

/* Gradient of the logits, the counts held fixed (the choice has no gradient):
 *   d_e = grad_loss coeff E counts_se / (S' k tokens_s^2)
 *   softmax: p_e (d_e - sum_j p_j d_j); sigmoid: that times 1 - sigmoid(logit_e)
 * grad_loss: float32 [1] on the device; counts, tokens: as the forward wrote them.
 * grad_logits: [T, E] of `dtype`, row stride ld_grad, written whole: zeros in rows of
 * no sequence and in padding rows. */
fp8mm_status fp8mm_moe_balance_loss_backward(const float* grad_loss, const void* logits, fp8mm_dtype dtype, int64_t T,
                                             int64_t E, int64_t ld, const int32_t* counts, const int32_t* tokens,
                                             int64_t k, fp8mm_score score, const int32_t* ends, int64_t S, float coeff,
                                             void* grad_logits, int64_t ld_grad, hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Low-rank adapters of many requests beside a shared projection: token t uses
 * adapter a = ids[t], two panels of r rows each,
 *   v[t] = down[a] x[t]                     float32 [r]
 *   out[t] = base[t] + scales[a] up[a]^T v[t]
 * and out[t] = base[t] where ids[t] lies outside [0, n) (base NULL: 0).
 * x: bf16 [T, K]; down: bf16 [n, r, K], up: bf16 [n, r, N], both dense; ids: int32
 * [T], in any order (tokens of one adapter next to each other are the fast case);
 * scales: float32 [n] or NULL (1); base, out: bf16 [T, N].  out may be base itself.
 * v: float32 [splits, T, r rounded up to a multiple of 4] with splits =
 * fp8mm_lora_splits(T, K, n, r): each token's products as that many partial sums over
 * K (their sum is v; zeros behind the rank), which the backward takes; rows of tokens
 * without an adapter are not written.
 * Sums are float32.  v enters the second product as two bf16 numbers, its
 * rounding and the rest, so that it keeps 16 bits (in the gradients of the panels too
 * where they are bf16; all of its bits where they are float32).
 * r <= 256, else FP8MM_ENOTIMPL; 0 <= T < 2^31; 1 <= n < 2^31; 1 <= K, N <= 2^22.
 * ------------------------------------------------------------------------- */
int64_t fp8mm_lora_splits(int64_t T, int64_t K, int64_t n, int64_t r);

fp8mm_status fp8mm_lora(const void* x, int64_t ld_x, int64_t T, int64_t K, const void* down, const void* up, int64_t n,
                        int64_t r, int64_t N, const int32_t* ids, const float* scales, const void* base,
                        int64_t ld_base, void* out, int64_t ld_out, float* v, hipStream_t stream);

/* Workspace bytes of fp8mm_lora_backward; -1 for arguments out of range.  Host
 * only. */
int64_t fp8mm_lora_backward_workspace(int64_t T, int64_t K, int64_t N, int64_t n, int64_t r);

/* With dv[t] = scales[a] up[a] dy[t]:
 *   dx[t] = down[a]^T dv[t]  (0 without an adapter)
 *   ddown[a] = sum over a's tokens of dv[t] x[t]^T
 *   dup[a] = sum over a's tokens of scales[a] v[t] dy[t]^T
 * (base has dy itself for its gradient.)  dy: bf16 [T, N]; x, v: as in the forward;
 * dx: bf16 [T, K]; ddown [n, r, K], dup [n, r, N]: dense, of `grad_dtype`, zeros for
 * an adapter without tokens.  dx, ddown and dup may each be NULL; x is needed for
 * ddown only, v for dup only.  ddown and dup are implemented for n <= 1024
 * (FP8MM_ENOTIMPL).  workspace: at least fp8mm_lora_backward_workspace bytes,
 * 16-byte aligned. */
fp8mm_status fp8mm_lora_backward(const void* dy, int64_t ld_dy, const void* x, int64_t ld_x, int64_t T, int64_t K,
                                 const void* down, const void* up, int64_t n, int64_t r, int64_t N,
                                 const int32_t* ids, const float* scales, const float* v, void* dx, int64_t ld_dx,
                                 void* ddown, void* dup, fp8mm_dtype grad_dtype, void* workspace,
                                 int64_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8MM_BLOCK_H */
