// C ABI of the operators around a block's dense products and its router
// (include/fp8mm_block.h): host-side argument checks and dispatch.  As in the rest of
// the library, nothing allocates, frees or synchronizes, and a call that fails a
// check launches nothing.
#include "fp8mm_block.h"

#include "api_common.hpp"
#include "block_launch.hpp"

using fp8mm::api::aligned16;
using fp8mm::api::fail;
using fp8mm::api::from_hip;
using fp8mm::api::kMaxLd;
using fp8mm::api::ok;

namespace {

constexpr int64_t kMaxInt = (int64_t(1) << 31) - 1;
// workgroups of 256 threads of one launch at most: fewer than 2^32 threads
constexpr int64_t kMaxGroups = (int64_t(1) << 24) - 1;

bool valid_dtype(int d) { return d == FP8MM_OUT_BF16 || d == FP8MM_OUT_FP32; }

bool element_aligned(const void* p, fp8mm_dtype d) {
  return (reinterpret_cast<uintptr_t>(p) & (d == FP8MM_OUT_FP32 ? 3u : 1u)) == 0;
}

fp8mm_status check_ld(int64_t ld, int64_t cols, const char* name) {
  if (ld < cols || ld > (int64_t(1) << 40))
    return fail(FP8MM_EINVAL, "%s (%lld) must be >= %lld and <= 2^40", name, (long long)ld, (long long)cols);
  return FP8MM_OK;
}

fp8mm_status check_workspace(const void* workspace, int64_t bytes, int64_t need) {
  if (need > 0 && (!workspace || bytes < need || !aligned16(workspace)))
    return fail(FP8MM_EINVAL, "workspace must be 16-byte aligned and hold %lld bytes, has %lld", (long long)need,
                (long long)(workspace ? bytes : 0));
  return FP8MM_OK;
}

// Shapes and types shared by the two norm calls.
fp8mm_status check_norm(fp8mm_dtype dtype, fp8mm_dtype param_dtype, int64_t R, int64_t C) {
  if (!valid_dtype(dtype) || !valid_dtype(param_dtype)) return fail(FP8MM_EINVAL, "unknown dtype");
  if (R < 0 || C < 1 || R > kMaxInt || C > kMaxLd)
    return fail(FP8MM_EINVAL, "shape [%lld, %lld]: need 0 <= R < 2^31 and 1 <= C <= 2^22", (long long)R, (long long)C);
  return FP8MM_OK;
}

bool balance_shape(int64_t T, int64_t E, int64_t S) {
  return T >= 0 && T <= kMaxInt && E >= 1 && S >= 1 && S <= (int64_t(1) << 20) && S <= kMaxInt / E;
}

// What the two balance calls share.
fp8mm_status check_balance(fp8mm_dtype dtype, int64_t T, int64_t E, int64_t ld, int64_t k, fp8mm_score score,
                           const int32_t* ends, int64_t S, float coeff) {
  if (!valid_dtype(dtype)) return fail(FP8MM_EINVAL, "unknown dtype");
  if (score != FP8MM_SCORE_SOFTMAX && score != FP8MM_SCORE_SIGMOID) return fail(FP8MM_EINVAL, "unknown score");
  if (!balance_shape(T, E, S))
    return fail(FP8MM_EINVAL, "need 0 <= T < 2^31, E >= 1, 1 <= S <= 2^20 and S E < 2^31");
  if (!ends && S != 1) return fail(FP8MM_EINVAL, "without ends there is one sequence, not %lld", (long long)S);
  if (k < 1 || T > kMaxInt / k) return fail(FP8MM_EINVAL, "need k >= 1 and T k < 2^31");
  if (!(coeff - coeff == 0.0f)) return fail(FP8MM_EINVAL, "coeff must be finite");
  if (E > 1024 || k > 64) return fail(FP8MM_ENOTIMPL, "implemented for E <= 1024 and k <= 64");
  return check_ld(ld, E, "ld");
}

bool lora_shape(int64_t T, int64_t n, int64_t r) {
  return T >= 0 && T <= kMaxInt && n >= 1 && n <= kMaxInt && r >= 1 && r <= fp8mm::kLoraMaxRank;
}
bool lora_columns(int64_t C) { return C >= 1 && C <= kMaxLd; }

// What the two adapter calls share.
fp8mm_status check_lora(int64_t T, int64_t K, int64_t n, int64_t r, int64_t N, const void* down, const void* up,
                        const int32_t* ids) {
  if (T < 0 || T > kMaxInt || n < 1 || n > kMaxInt || r < 1 || !lora_columns(K) || !lora_columns(N))
    return fail(FP8MM_EINVAL, "need 0 <= T < 2^31, 1 <= n < 2^31, r >= 1 and 1 <= K, N <= 2^22");
  if (r > fp8mm::kLoraMaxRank) return fail(FP8MM_ENOTIMPL, "rank (%lld) above %d", (long long)r, fp8mm::kLoraMaxRank);
  if (T > 0 && (!down || !up || !ids)) return fail(FP8MM_EINVAL, "down, up and ids must not be NULL");
  if (!element_aligned(down, FP8MM_OUT_BF16) || !element_aligned(up, FP8MM_OUT_BF16))
    return fail(FP8MM_EINVAL, "pointers must be aligned to their element type");
  const int64_t tiles = (T + 63) / 64, wide = (K > N ? K : N), ranks = (r + 63) / 64;
  if (tiles > 0 && ((wide + 511) / 512 > kMaxGroups / tiles || ranks > kMaxGroups / tiles))
    return fail(FP8MM_EINVAL, "%lld tokens of %lld columns are too many for one launch", (long long)T, (long long)wide);
  return FP8MM_OK;
}

// The parts of the backward's workspace.
int64_t dv_bytes(int64_t T, int64_t N, int64_t n, int64_t r) {
  return 16 * fp8mm::lora_splits(T, N, n, int(r)) * T * ((r + 3) / 4);
}
int64_t partial_bytes(int64_t T, int64_t C, int64_t n, int64_t r) {
  return (fp8mm::lora_outer_workspace(T, C, n, int(r)) + 15) / 16 * 16;
}

}  // namespace

extern "C" {

// ----------------------------------------------------------------- RMS norm

fp8mm_status fp8mm_rms_norm(const void* x, int64_t ld_x, const void* residual, int64_t ld_res, fp8mm_dtype dtype,
                            int64_t R, int64_t C, const void* weight, fp8mm_dtype param_dtype, float eps, void* h,
                            int64_t ld_h, void* y, int64_t ld_y, uint8_t* q, int64_t ld_q, float* scale,
                            fp8mm_recipe recipe, float* rstd, hipStream_t stream) {
  fp8mm_status st = check_norm(dtype, param_dtype, R, C);
  if (st == FP8MM_OK) st = check_ld(ld_x, C, "ld_x");
  if (st == FP8MM_OK && residual) st = check_ld(ld_res, C, "ld_res");
  if (st == FP8MM_OK && residual && h) st = check_ld(ld_h, C, "ld_h");
  if (st == FP8MM_OK && y) st = check_ld(ld_y, C, "ld_y");
  if (st != FP8MM_OK) return st;
  if (!(eps >= 0.0f && eps - eps == 0.0f)) return fail(FP8MM_EINVAL, "eps must be a finite value >= 0");
  if (q) {
    if (recipe != FP8MM_BLOCK_1x128 && recipe != FP8MM_ROWWISE) {
      if (recipe == FP8MM_TENSORWISE || recipe == FP8MM_BLOCK_128x128 || recipe == FP8MM_BLOCK_128x1 ||
          recipe == FP8MM_MXFP8)
        return fail(FP8MM_ENOTIMPL, "codes of a norm are implemented for the 1x128 and rowwise recipes");
      return fail(FP8MM_EINVAL, "unknown recipe");
    }
    if (dtype != FP8MM_OUT_BF16) return fail(FP8MM_ENOTIMPL, "codes are made of bf16 rows only");
    const int64_t group = recipe == FP8MM_ROWWISE ? 16 : 128;
    if (C % group) return fail(FP8MM_EINVAL, "C (%lld) must be a multiple of %lld", (long long)C, (long long)group);
    st = check_ld(ld_q, C, "ld_q");
    if (st != FP8MM_OK) return st;
    if (ld_q % 16 || !aligned16(q)) return fail(FP8MM_EINVAL, "q must be 16-byte aligned, ld_q a multiple of 16");
    if (R > 0 && !scale) return fail(FP8MM_EINVAL, "scale must not be NULL");
    if (!element_aligned(scale, FP8MM_OUT_FP32)) return fail(FP8MM_EINVAL, "scale must be 4-byte aligned");
  }
  if (R == 0) return ok();
  if (!x) return fail(FP8MM_EINVAL, "x must not be NULL");
  if (!element_aligned(x, dtype) || !element_aligned(residual, dtype) || !element_aligned(h, dtype) ||
      !element_aligned(y, dtype) || !element_aligned(weight, param_dtype) || !element_aligned(rstd, FP8MM_OUT_FP32))
    return fail(FP8MM_EINVAL, "pointers must be aligned to their element type");
  if (!y && !q && !rstd && !(residual && h)) return ok();
  fp8mm::RmsProblem p{};
  p.x = x;
  p.residual = residual;
  p.ld_x = ld_x;
  p.ld_res = ld_res;
  p.ld_h = ld_h;
  p.fp32 = dtype == FP8MM_OUT_FP32;
  p.param_fp32 = param_dtype == FP8MM_OUT_FP32;
  p.R = R;
  p.C = C;
  p.weight = weight;
  p.eps = eps;
  p.h = residual ? h : nullptr;
  p.y = y;
  p.ld_y = ld_y;
  p.q = q;
  p.ld_q = ld_q;
  p.scale = scale;
  p.rowwise = recipe == FP8MM_ROWWISE;
  p.rstd = rstd;
  return from_hip(fp8mm::launch_rms_norm(p, stream), "fp8mm_rms_norm");
}

int64_t fp8mm_rms_norm_backward_workspace(int64_t R, int64_t C) {
  if (R < 0 || C < 0 || R > kMaxInt || C > kMaxLd) return -1;
  return fp8mm::rms_backward_workspace(R, C);
}

fp8mm_status fp8mm_rms_norm_backward(const void* dy, int64_t ld_dy, const void* h, int64_t ld_h, const void* grad_h,
                                     int64_t ld_gh, fp8mm_dtype dtype, int64_t R, int64_t C, const void* weight,
                                     fp8mm_dtype param_dtype, const float* rstd, void* dx, int64_t ld_dx,
                                     void* dweight, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  fp8mm_status st = check_norm(dtype, param_dtype, R, C);
  if (st == FP8MM_OK) st = check_ld(ld_dy, C, "ld_dy");
  if (st == FP8MM_OK) st = check_ld(ld_h, C, "ld_h");
  if (st == FP8MM_OK && grad_h) st = check_ld(ld_gh, C, "ld_gh");
  if (st == FP8MM_OK && dx) st = check_ld(ld_dx, C, "ld_dx");
  if (st != FP8MM_OK) return st;
  if (R > 0 && (!dy || !h || !rstd)) return fail(FP8MM_EINVAL, "dy, h and rstd must not be NULL");
  if (!element_aligned(dy, dtype) || !element_aligned(h, dtype) || !element_aligned(grad_h, dtype) ||
      !element_aligned(dx, dtype) || !element_aligned(weight, param_dtype) || !element_aligned(dweight, param_dtype) ||
      !element_aligned(rstd, FP8MM_OUT_FP32))
    return fail(FP8MM_EINVAL, "pointers must be aligned to their element type");
  if (dx && dx == grad_h && ld_dx != ld_gh) return fail(FP8MM_EINVAL, "dx on grad_h needs ld_dx = ld_gh");
  if (!dx && !dweight) return ok();
  if (dweight) {
    st = check_workspace(workspace, workspace_bytes, fp8mm::rms_backward_workspace(R, C));
    if (st != FP8MM_OK) return st;
  }
  fp8mm::RmsProblem p{};
  p.dy = dy;
  p.h_in = h;
  p.grad_h = grad_h;
  p.ld_dy = ld_dy;
  p.ld_h = ld_h;
  p.ld_gh = ld_gh;
  p.fp32 = dtype == FP8MM_OUT_FP32;
  p.param_fp32 = param_dtype == FP8MM_OUT_FP32;
  p.R = R;
  p.C = C;
  p.weight = weight;
  p.rstd = const_cast<float*>(rstd);
  p.dx = dx;
  p.ld_dx = ld_dx;
  p.dweight = dweight;
  p.workspace = static_cast<float*>(workspace);
  return from_hip(fp8mm::launch_rms_norm_backward(p, stream), "fp8mm_rms_norm_backward");
}

// ------------------------------------------------------------- balance loss

int64_t fp8mm_moe_balance_loss_workspace(int64_t T, int64_t E, int64_t S) {
  if (!balance_shape(T, E, S)) return -1;
  return fp8mm::balance_workspace(T, E, S);
}

fp8mm_status fp8mm_moe_balance_loss(const void* logits, fp8mm_dtype dtype, int64_t T, int64_t E, int64_t ld,
                                    const int32_t* ids, int64_t k, fp8mm_score score, const int32_t* ends, int64_t S,
                                    float coeff, float* loss, int32_t* counts, int32_t* tokens, void* workspace,
                                    int64_t workspace_bytes, hipStream_t stream) {
  fp8mm_status st = check_balance(dtype, T, E, ld, k, score, ends, S, coeff);
  if (st != FP8MM_OK) return st;
  if (!loss || !counts || !tokens) return fail(FP8MM_EINVAL, "loss, counts and tokens must not be NULL");
  if (T > 0 && (!logits || !ids)) return fail(FP8MM_EINVAL, "logits and ids must not be NULL");
  if (!element_aligned(logits, dtype)) return fail(FP8MM_EINVAL, "logits must be aligned to their element type");
  st = check_workspace(workspace, workspace_bytes, fp8mm::balance_workspace(T, E, S));
  if (st != FP8MM_OK) return st;
  fp8mm::BalanceProblem p{};
  p.logits = logits;
  p.fp32 = dtype == FP8MM_OUT_FP32;
  p.T = T;
  p.ld = ld;
  p.E = int(E);
  p.k = int(k);
  p.sigmoid = score == FP8MM_SCORE_SIGMOID;
  p.ids = ids;
  p.ends = ends;
  p.S = int(S);
  p.coeff = coeff;
  p.loss = loss;
  p.counts = counts;
  p.tokens = tokens;
  p.workspace = workspace;
  return from_hip(fp8mm::launch_balance(p, stream), "fp8mm_moe_balance_loss");
}

fp8mm_status fp8mm_moe_balance_loss_backward(const float* grad_loss, const void* logits, fp8mm_dtype dtype, int64_t T,
                                             int64_t E, int64_t ld, const int32_t* counts, const int32_t* tokens,
                                             int64_t k, fp8mm_score score, const int32_t* ends, int64_t S, float coeff,
                                             void* grad_logits, int64_t ld_grad, hipStream_t stream) {
  fp8mm_status st = check_balance(dtype, T, E, ld, k, score, ends, S, coeff);
  if (st == FP8MM_OK) st = check_ld(ld_grad, E, "ld_grad");
  if (st != FP8MM_OK) return st;
  if (T == 0) return ok();
  if (!grad_loss || !logits || !counts || !tokens || !grad_logits)
    return fail(FP8MM_EINVAL, "grad_loss, logits, counts, tokens and grad_logits must not be NULL");
  if (!element_aligned(logits, dtype) || !element_aligned(grad_logits, dtype))
    return fail(FP8MM_EINVAL, "pointers must be aligned to their element type");
  fp8mm::BalanceProblem p{};
  p.logits = logits;
  p.fp32 = dtype == FP8MM_OUT_FP32;
  p.T = T;
  p.ld = ld;
  p.E = int(E);
  p.k = int(k);
  p.sigmoid = score == FP8MM_SCORE_SIGMOID;
  p.ends = ends;
  p.S = int(S);
  p.coeff = coeff;
  p.counts = const_cast<int32_t*>(counts);
  p.tokens = const_cast<int32_t*>(tokens);
  p.grad_loss = grad_loss;
  p.grad_logits = grad_logits;
  p.ld_grad = ld_grad;
  return from_hip(fp8mm::launch_balance_backward(p, stream), "fp8mm_moe_balance_loss_backward");
}

// ----------------------------------------------------------------- adapters

int64_t fp8mm_lora_splits(int64_t T, int64_t K, int64_t n, int64_t r) {
  if (!lora_shape(T, n, r) || !lora_columns(K)) return -1;
  return fp8mm::lora_splits(T, K, n, int(r));
}

fp8mm_status fp8mm_lora(const void* x, int64_t ld_x, int64_t T, int64_t K, const void* down, const void* up, int64_t n,
                        int64_t r, int64_t N, const int32_t* ids, const float* scales, const void* base,
                        int64_t ld_base, void* out, int64_t ld_out, float* v, hipStream_t stream) {
  fp8mm_status st = check_lora(T, K, n, r, N, down, up, ids);
  if (st == FP8MM_OK) st = check_ld(ld_x, K, "ld_x");
  if (st == FP8MM_OK && base) st = check_ld(ld_base, N, "ld_base");
  if (st == FP8MM_OK) st = check_ld(ld_out, N, "ld_out");
  if (st != FP8MM_OK) return st;
  if (T == 0) return ok();
  if (!x || !out || !v) return fail(FP8MM_EINVAL, "x, out and v must not be NULL");
  if (!element_aligned(x, FP8MM_OUT_BF16) || !element_aligned(base, FP8MM_OUT_BF16) ||
      !element_aligned(out, FP8MM_OUT_BF16) || !element_aligned(v, FP8MM_OUT_FP32) ||
      !element_aligned(scales, FP8MM_OUT_FP32))
    return fail(FP8MM_EINVAL, "pointers must be aligned to their element type");
  if (base == out && ld_base != ld_out) return fail(FP8MM_EINVAL, "out on base needs ld_out = ld_base");
  fp8mm::LoraProblem p{};
  p.T = T;
  p.C = K;
  p.n = int(n);
  p.r = int(r);
  p.ids = ids;
  p.scales = scales;
  p.panels = static_cast<const uint16_t*>(down);
  p.x = static_cast<const uint16_t*>(x);
  p.ld_x = ld_x;
  p.v = v;
  p.splits = fp8mm::lora_splits(T, K, n, int(r));
  hipError_t e = fp8mm::launch_lora_shrink(p, stream);
  if (e != hipSuccess) return from_hip(e, "fp8mm_lora");
  p.C = N;
  p.panels = static_cast<const uint16_t*>(up);
  p.base = static_cast<const uint16_t*>(base);
  p.ld_base = ld_base;
  p.out = static_cast<uint16_t*>(out);
  p.ld_out = ld_out;
  return from_hip(fp8mm::launch_lora_expand(p, stream), "fp8mm_lora");
}

int64_t fp8mm_lora_backward_workspace(int64_t T, int64_t K, int64_t N, int64_t n, int64_t r) {
  if (!lora_shape(T, n, r) || !lora_columns(K) || !lora_columns(N)) return -1;
  if (n > fp8mm::kLoraMaxAdapters) return dv_bytes(T, N, n, r);
  return dv_bytes(T, N, n, r) + partial_bytes(T, N, n, r) + partial_bytes(T, K, n, r) +
         fp8mm::lora_order_workspace(T, n, int(r));
}

fp8mm_status fp8mm_lora_backward(const void* dy, int64_t ld_dy, const void* x, int64_t ld_x, int64_t T, int64_t K,
                                 const void* down, const void* up, int64_t n, int64_t r, int64_t N,
                                 const int32_t* ids, const float* scales, const float* v, void* dx, int64_t ld_dx,
                                 void* ddown, void* dup, fp8mm_dtype grad_dtype, void* workspace,
                                 int64_t workspace_bytes, hipStream_t stream) {
  if (!valid_dtype(grad_dtype)) return fail(FP8MM_EINVAL, "unknown grad_dtype");
  fp8mm_status st = check_lora(T, K, n, r, N, down, up, ids);
  if (st == FP8MM_OK) st = check_ld(ld_dy, N, "ld_dy");
  if (st == FP8MM_OK && ddown) st = check_ld(ld_x, K, "ld_x");
  if (st == FP8MM_OK && dx) st = check_ld(ld_dx, K, "ld_dx");
  if (st != FP8MM_OK) return st;
  if ((ddown || dup) && n > fp8mm::kLoraMaxAdapters)
    return fail(FP8MM_ENOTIMPL, "gradients of more than %d adapters (%lld)", fp8mm::kLoraMaxAdapters, (long long)n);
  if (T > 0 && !dy) return fail(FP8MM_EINVAL, "dy must not be NULL");
  if (T > 0 && ((ddown && !x) || (dup && !v)))
    return fail(FP8MM_EINVAL, "ddown needs x and dup needs v");
  if (!element_aligned(dy, FP8MM_OUT_BF16) || !element_aligned(x, FP8MM_OUT_BF16) ||
      !element_aligned(dx, FP8MM_OUT_BF16) || !element_aligned(v, FP8MM_OUT_FP32) ||
      !element_aligned(scales, FP8MM_OUT_FP32) || !element_aligned(ddown, grad_dtype) ||
      !element_aligned(dup, grad_dtype))
    return fail(FP8MM_EINVAL, "pointers must be aligned to their element type");
  if ((T == 0 || !dx) && !ddown && !dup) return ok();
  st = check_workspace(workspace, workspace_bytes, fp8mm_lora_backward_workspace(T, K, N, n, r));
  if (st != FP8MM_OK) return st;
  float* dv = static_cast<float*>(workspace);
  const int dv_splits = fp8mm::lora_splits(T, N, n, int(r));
  fp8mm::LoraProblem p{};
  p.T = T;
  p.n = int(n);
  p.r = int(r);
  p.ids = ids;
  p.scales = scales;
  p.grad_fp32 = grad_dtype == FP8MM_OUT_FP32;
  char* at = static_cast<char*>(workspace) + dv_bytes(T, N, n, r);
  const fp8mm::LoraSide sides[2] = {
      {static_cast<const uint16_t*>(dy), ld_dy, N, dup, reinterpret_cast<float*>(at)},
      {static_cast<const uint16_t*>(x), ld_x, K, ddown, reinterpret_cast<float*>(at + partial_bytes(T, N, n, r))}};
  at += partial_bytes(T, N, n, r) + partial_bytes(T, K, n, r);
  hipError_t e = hipSuccess;
  if (dx || ddown) {
    fp8mm::LoraProblem q = p;
    q.C = N;
    q.panels = static_cast<const uint16_t*>(up);
    q.x = static_cast<const uint16_t*>(dy);
    q.ld_x = ld_dy;
    q.v = dv;
    q.splits = dv_splits;
    e = fp8mm::launch_lora_shrink(q, stream);
  }
  fp8mm::LoraOrder o{};
  o.v[0] = dup ? v : nullptr;
  o.splits[0] = fp8mm::lora_splits(T, K, n, int(r));
  o.v[1] = ddown ? dv : nullptr;
  o.splits[1] = dv_splits;
  if (e == hipSuccess && (ddown || dup)) {
    e = fp8mm::launch_lora_order(p, at, o, stream);
    if (e == hipSuccess) e = fp8mm::launch_lora_outer(p, o, sides, stream);
  }
  if (e == hipSuccess && dx) {
    p.C = K;
    p.v = dv;
    p.splits = dv_splits;
    p.panels = static_cast<const uint16_t*>(down);
    p.out = static_cast<uint16_t*>(dx);
    p.ld_out = ld_dx;
    e = fp8mm::launch_lora_expand(p, stream);
  }
  return from_hip(e, "fp8mm_lora_backward");
}

}  // extern "C"
