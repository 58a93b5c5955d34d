// C ABI of the operators around the grouped GEMMs (include/fp8mm_moe.h):
// host-side argument checks and dispatch.  As in the rest of the library,
// nothing allocates, frees or synchronizes, and a call that fails a check
// launches nothing.
#include "fp8mm_moe.h"

#include "api_common.hpp"
#include "moe_launch.hpp"

using fp8mm::api::aligned16;
using fp8mm::api::fail;
using fp8mm::api::from_hip;
using fp8mm::api::kMaxLd;
using fp8mm::api::ok;

namespace {

constexpr int64_t kMaxInt = (int64_t(1) << 31) - 1;
// waves of one launch at most: 64 threads each, fewer than 2^32 threads
constexpr int64_t kMaxWaves = int64_t(1) << 25;

bool valid_dtype(int d) { return d == FP8MM_OUT_BF16 || d == FP8MM_OUT_FP32; }

bool element_aligned(const void* p, fp8mm_dtype d) {
  return (reinterpret_cast<uintptr_t>(p) & (d == FP8MM_OUT_FP32 ? 3u : 1u)) == 0;
}

// Shapes and strides shared by the two layer norm calls.
fp8mm_status check_norm(fp8mm_dtype dtype, fp8mm_dtype param_dtype, int64_t R, int64_t C) {
  if (!valid_dtype(dtype) || !valid_dtype(param_dtype)) return fail(FP8MM_EINVAL, "unknown dtype");
  if (R < 0 || C < 1 || R > kMaxInt || C > kMaxLd)
    return fail(FP8MM_EINVAL, "shape [%lld, %lld]: need 0 <= R < 2^31 and 1 <= C <= 2^22", (long long)R, (long long)C);
  return FP8MM_OK;
}

fp8mm_status check_ld(int64_t ld, int64_t cols, const char* name) {
  if (ld < cols || ld > (int64_t(1) << 40))
    return fail(FP8MM_EINVAL, "%s (%lld) must be >= %lld and <= 2^40", name, (long long)ld, (long long)cols);
  return FP8MM_OK;
}

// `units` waves of each of `n` tokens or slots.
fp8mm_status check_waves(int64_t n, int64_t units, int64_t T, int64_t C) {
  if (n > 0 && units > kMaxWaves / n)
    return fail(FP8MM_EINVAL, "[%lld, %lld] is too large for one launch", (long long)T, (long long)C);
  return FP8MM_OK;
}

fp8mm_status check_permute(fp8mm_dtype dtype, int64_t T, int64_t C, int64_t k, const int32_t* row_of_slot) {
  if (!valid_dtype(dtype)) return fail(FP8MM_EINVAL, "unknown dtype");
  if (T < 0 || C < 0 || k < 1) return fail(FP8MM_EINVAL, "need T >= 0, C >= 0 and k >= 1");
  if (k > fp8mm::kRouteMaxK) return fail(FP8MM_ENOTIMPL, "k (%lld) above %d", (long long)k, fp8mm::kRouteMaxK);
  if (T > kMaxInt / k || C > kMaxInt) return fail(FP8MM_EINVAL, "T k and C must be < 2^31");
  if (T > 0 && !row_of_slot) return fail(FP8MM_EINVAL, "row_of_slot must not be NULL");
  return FP8MM_OK;
}

fp8mm_status check_row_waves(int64_t T, int64_t C, fp8mm_dtype dtype) {
  const int64_t columns = fp8mm::row_columns(dtype == FP8MM_OUT_FP32);
  return check_waves(T, (C + columns - 1) / columns, T, C);
}

}  // namespace

extern "C" {

// --------------------------------------------------------------- layer norm

fp8mm_status fp8mm_layer_norm(const void* x, fp8mm_dtype dtype, int64_t R, int64_t C, int64_t ld_x,
                              const void* weight, const void* bias, fp8mm_dtype param_dtype, float eps, void* y,
                              int64_t ld_y, float* mean, float* rstd, hipStream_t stream) {
  fp8mm_status st = check_norm(dtype, param_dtype, R, C);
  if (st == FP8MM_OK) st = check_ld(ld_x, C, "ld_x");
  if (st == FP8MM_OK) st = check_ld(ld_y, C, "ld_y");
  if (st != FP8MM_OK) return st;
  if (!(eps >= 0.0f && eps - eps == 0.0f)) return fail(FP8MM_EINVAL, "eps must be a finite value >= 0");
  if (R == 0) return ok();
  if (!x || !y) return fail(FP8MM_EINVAL, "x and y must not be NULL");
  if (!element_aligned(x, dtype) || !element_aligned(y, dtype) || !element_aligned(weight, param_dtype) ||
      !element_aligned(bias, param_dtype))
    return fail(FP8MM_EINVAL, "pointers must be aligned to their element type");
  fp8mm::NormProblem p{};
  p.x = x;
  p.out = y;
  p.R = R;
  p.C = C;
  p.ld_x = ld_x;
  p.ld_out = ld_y;
  p.fp32 = dtype == FP8MM_OUT_FP32;
  p.param_fp32 = param_dtype == FP8MM_OUT_FP32;
  p.weight = weight;
  p.bias = bias;
  p.eps = eps;
  p.mean = mean;
  p.rstd = rstd;
  return from_hip(fp8mm::launch_norm(p, stream), "fp8mm_layer_norm");
}

int64_t fp8mm_layer_norm_backward_workspace(int64_t R, int64_t C) {
  if (R < 0 || C < 0 || R > kMaxInt || C > kMaxLd) return -1;
  return fp8mm::norm_backward_workspace(R, C);
}

fp8mm_status fp8mm_layer_norm_backward(const void* dy, int64_t ld_dy, const void* x, int64_t ld_x, fp8mm_dtype dtype,
                                       int64_t R, int64_t C, const void* weight, fp8mm_dtype param_dtype,
                                       const float* mean, const float* rstd, void* dx, int64_t ld_dx, void* dweight,
                                       void* dbias, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  fp8mm_status st = check_norm(dtype, param_dtype, R, C);
  if (st == FP8MM_OK) st = check_ld(ld_dy, C, "ld_dy");
  if (st == FP8MM_OK) st = check_ld(ld_x, C, "ld_x");
  if (st == FP8MM_OK && dx) st = check_ld(ld_dx, C, "ld_dx");
  if (st != FP8MM_OK) return st;
  if (R > 0 && (!dy || !x || !mean || !rstd)) return fail(FP8MM_EINVAL, "dy, x, mean and rstd must not be NULL");
  if (!element_aligned(dy, dtype) || !element_aligned(x, dtype) || !element_aligned(dx, dtype) ||
      !element_aligned(weight, param_dtype) || !element_aligned(dweight, param_dtype) ||
      !element_aligned(dbias, param_dtype))
    return fail(FP8MM_EINVAL, "pointers must be aligned to their element type");
  if (!dx && !dweight && !dbias) return ok();
  const int64_t need = fp8mm::norm_backward_workspace(R, C);
  if ((dweight || dbias) && need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
    return fail(FP8MM_EINVAL, "workspace must be 16-byte aligned and hold %lld bytes, has %lld", (long long)need,
                (long long)(workspace ? workspace_bytes : 0));
  fp8mm::NormProblem p{};
  p.x = x;
  p.dy = dy;
  p.out = dx;
  p.R = R;
  p.C = C;
  p.ld_x = ld_x;
  p.ld_dy = ld_dy;
  p.ld_out = ld_dx;
  p.fp32 = dtype == FP8MM_OUT_FP32;
  p.param_fp32 = param_dtype == FP8MM_OUT_FP32;
  p.weight = weight;
  p.mean = const_cast<float*>(mean);
  p.rstd = const_cast<float*>(rstd);
  p.dweight = dweight;
  p.dbias = dbias;
  p.workspace = static_cast<float*>(workspace);
  return from_hip(fp8mm::launch_norm_backward(p, stream), "fp8mm_layer_norm_backward");
}

// ------------------------------------------------------------------ routing

fp8mm_status fp8mm_moe_route(const void* logits, fp8mm_dtype dtype, int64_t T, int64_t E, int64_t ld,
                             const float* bias, fp8mm_score score, int64_t k, int64_t groups, int64_t group_topk,
                             fp8mm_group_score group_score, int renormalize, float scale, int32_t* ids,
                             float* weights, hipStream_t stream) {
  if (!valid_dtype(dtype)) return fail(FP8MM_EINVAL, "unknown dtype");
  if (score != FP8MM_SCORE_SOFTMAX && score != FP8MM_SCORE_SIGMOID) return fail(FP8MM_EINVAL, "unknown score");
  if (group_score != FP8MM_GROUP_MAX && group_score != FP8MM_GROUP_TOP2)
    return fail(FP8MM_EINVAL, "unknown group_score");
  if (renormalize != 0 && renormalize != 1) return fail(FP8MM_EINVAL, "renormalize must be 0 or 1");
  if (T < 0 || T > kMaxInt || E < 1) return fail(FP8MM_EINVAL, "need 0 <= T < 2^31 and E >= 1");
  if (k < 1 || k > E) return fail(FP8MM_EINVAL, "k (%lld) must be in [1, E = %lld]", (long long)k, (long long)E);
  if (groups < 1 || E % groups != 0)
    return fail(FP8MM_EINVAL, "groups (%lld) must divide E (%lld)", (long long)groups, (long long)E);
  if (group_topk < 1 || group_topk > groups)
    return fail(FP8MM_EINVAL, "group_topk (%lld) must be in [1, groups = %lld]", (long long)group_topk,
                (long long)groups);
  if (!(scale - scale == 0.0f)) return fail(FP8MM_EINVAL, "scale must be finite");
  if (E > fp8mm::kRouteMaxExperts || k > fp8mm::kRouteMaxK || groups > 64)
    return fail(FP8MM_ENOTIMPL, "implemented for E <= %d, k <= %d and groups <= 64", fp8mm::kRouteMaxExperts,
                fp8mm::kRouteMaxK);
  const fp8mm_status st = check_ld(ld, E, "ld");
  if (st != FP8MM_OK) return st;
  if (T == 0) return ok();
  if (!logits || !ids || !weights) return fail(FP8MM_EINVAL, "logits, ids and weights must not be NULL");
  if (!element_aligned(logits, dtype)) return fail(FP8MM_EINVAL, "logits must be aligned to their element type");
  fp8mm::RouteProblem p{};
  p.logits = logits;
  p.fp32 = dtype == FP8MM_OUT_FP32;
  p.T = T;
  p.ld = ld;
  p.E = int(E);
  p.k = int(k);
  p.bias = bias;
  p.sigmoid = score == FP8MM_SCORE_SIGMOID;
  p.groups = int(groups);
  p.group_topk = int(group_topk);
  p.group_top2 = group_score == FP8MM_GROUP_TOP2;
  p.renorm = renormalize != 0;
  p.scale = scale;
  p.ids = ids;
  p.weights = weights;
  return from_hip(fp8mm::launch_route(p, stream), "fp8mm_moe_route");
}

fp8mm_status fp8mm_moe_route_backward(const float* grad_weights, const void* logits, fp8mm_dtype dtype, int64_t T,
                                      int64_t E, int64_t ld, const int32_t* ids, int64_t k, fp8mm_score score,
                                      int renormalize, float scale, void* grad_logits, int64_t ld_grad,
                                      hipStream_t stream) {
  if (!valid_dtype(dtype)) return fail(FP8MM_EINVAL, "unknown dtype");
  if (score != FP8MM_SCORE_SOFTMAX && score != FP8MM_SCORE_SIGMOID) return fail(FP8MM_EINVAL, "unknown score");
  if (renormalize != 0 && renormalize != 1) return fail(FP8MM_EINVAL, "renormalize must be 0 or 1");
  if (T < 0 || T > kMaxInt || E < 1) return fail(FP8MM_EINVAL, "need 0 <= T < 2^31 and E >= 1");
  if (k < 1 || k > E) return fail(FP8MM_EINVAL, "k (%lld) must be in [1, E = %lld]", (long long)k, (long long)E);
  if (!(scale - scale == 0.0f)) return fail(FP8MM_EINVAL, "scale must be finite");
  if (E > fp8mm::kRouteMaxExperts || k > fp8mm::kRouteMaxK)
    return fail(FP8MM_ENOTIMPL, "implemented for E <= %d and k <= %d", fp8mm::kRouteMaxExperts, fp8mm::kRouteMaxK);
  fp8mm_status st = check_ld(ld, E, "ld");
  if (st == FP8MM_OK) st = check_ld(ld_grad, E, "ld_grad");
  if (st != FP8MM_OK) return st;
  if (T == 0) return ok();
  if (!grad_weights || !logits || !ids || !grad_logits) return fail(FP8MM_EINVAL, "null pointer argument");
  if (!element_aligned(logits, dtype) || !element_aligned(grad_logits, dtype))
    return fail(FP8MM_EINVAL, "logits and grad_logits must be aligned to their element type");
  fp8mm::RouteProblem p{};
  p.logits = logits;
  p.fp32 = dtype == FP8MM_OUT_FP32;
  p.T = T;
  p.ld = ld;
  p.E = int(E);
  p.k = int(k);
  p.sigmoid = score == FP8MM_SCORE_SIGMOID;
  p.groups = p.group_topk = 1;
  p.renorm = renormalize != 0;
  p.scale = scale;
  p.ids = const_cast<int32_t*>(ids);
  p.grad_weights = grad_weights;
  p.grad_logits = grad_logits;
  p.ld_grad = ld_grad;
  return from_hip(fp8mm::launch_route_backward(p, stream), "fp8mm_moe_route_backward");
}

// -------------------------------------------------------------- permutation

int64_t fp8mm_moe_plan_workspace(int64_t T, int64_t k, int64_t E) {
  if (T < 0 || k < 0 || E < 0 || E > kMaxInt || (k > 0 && T > kMaxInt / k)) return -1;
  return fp8mm::plan_workspace(T * k, E);
}

fp8mm_status fp8mm_moe_plan(const int32_t* ids, int64_t T, int64_t k, int64_t E, int32_t* offsets,
                            int32_t* row_of_slot, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  if (T < 0 || k < 1 || E < 1) return fail(FP8MM_EINVAL, "need T >= 0, k >= 1 and E >= 1");
  if (T > kMaxInt / k) return fail(FP8MM_EINVAL, "T k must be < 2^31");
  if (E > fp8mm::kRouteMaxExperts)
    return fail(FP8MM_ENOTIMPL, "implemented for E <= %d", fp8mm::kRouteMaxExperts);
  if (!offsets || (T > 0 && (!ids || !row_of_slot))) return fail(FP8MM_EINVAL, "null pointer argument");
  const int64_t need = fp8mm::plan_workspace(T * k, E);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
    return fail(FP8MM_EINVAL, "workspace must be 16-byte aligned and hold %lld bytes, has %lld", (long long)need,
                (long long)(workspace ? workspace_bytes : 0));
  return from_hip(
      fp8mm::launch_plan(ids, T * k, int(E), offsets, row_of_slot, static_cast<int32_t*>(workspace), stream),
      "fp8mm_moe_plan");
}

fp8mm_status fp8mm_moe_dispatch(const void* x, fp8mm_dtype dtype, int64_t T, int64_t C, int64_t ld_x,
                                const int32_t* row_of_slot, int64_t k, void* out, int64_t ld_out, hipStream_t stream) {
  fp8mm_status st = check_permute(dtype, T, C, k, row_of_slot);
  if (st == FP8MM_OK) st = check_row_waves(T, C, dtype);
  if (st == FP8MM_OK) st = check_ld(ld_x, C, "ld_x");
  if (st == FP8MM_OK) st = check_ld(ld_out, C, "ld_out");
  if (st != FP8MM_OK) return st;
  if (T == 0 || C == 0) return ok();
  if (!x || !out) return fail(FP8MM_EINVAL, "x and out must not be NULL");
  if (!element_aligned(x, dtype) || !element_aligned(out, dtype))
    return fail(FP8MM_EINVAL, "x and out must be aligned to their element type");
  fp8mm::PermuteProblem p{};
  p.T = T;
  p.C = C;
  p.k = int(k);
  p.fp32 = dtype == FP8MM_OUT_FP32;
  p.row_of_slot = row_of_slot;
  p.x = x;
  p.ld_x = ld_x;
  p.out = out;
  p.ld_out = ld_out;
  return from_hip(fp8mm::launch_dispatch(p, stream), "fp8mm_moe_dispatch");
}

fp8mm_status fp8_moe_dispatch(const void* x, int64_t T, int64_t C, int64_t ld_x, const int32_t* row_of_slot, int64_t k,
                              uint8_t* q, int64_t ld_q, float* scale, hipStream_t stream) {
  fp8mm_status st = check_permute(FP8MM_OUT_BF16, T, C, k, row_of_slot);
  if (st == FP8MM_OK) st = check_waves(T, (C + fp8mm::kCodeColumns - 1) / fp8mm::kCodeColumns, T, C);
  if (st != FP8MM_OK) return st;
  if (C % 128 != 0) return fail(FP8MM_EINVAL, "C (%lld) must be a multiple of 128", (long long)C);
  if (ld_x < C || ld_x % 8 != 0 || ld_x > kMaxLd)
    return fail(FP8MM_EINVAL, "ld_x (%lld) must be >= C, a multiple of 8 and <= 2^22", (long long)ld_x);
  if (ld_q < C || ld_q % 16 != 0 || ld_q > kMaxLd)
    return fail(FP8MM_EINVAL, "ld_q (%lld) must be >= C, a multiple of 16 and <= 2^22", (long long)ld_q);
  if (T == 0 || C == 0) return ok();
  if (!x || !q || !scale) return fail(FP8MM_EINVAL, "x, q and scale must not be NULL");
  if (!aligned16(x) || !aligned16(q)) return fail(FP8MM_EINVAL, "x and q must be 16-byte aligned");
  fp8mm::PermuteProblem p{};
  p.T = T;
  p.C = C;
  p.k = int(k);
  p.row_of_slot = row_of_slot;
  p.x = x;
  p.ld_x = ld_x;
  p.q = q;
  p.ld_q = ld_q;
  p.scale = scale;
  return from_hip(fp8mm::launch_dispatch_fp8(p, stream), "fp8_moe_dispatch");
}

fp8mm_status fp8mm_moe_combine(const void* rows, fp8mm_dtype dtype, int64_t T, int64_t C, int64_t ld_rows,
                               const int32_t* row_of_slot, const float* weights, int64_t k, void* out, int64_t ld_out,
                               hipStream_t stream) {
  fp8mm_status st = check_permute(dtype, T, C, k, row_of_slot);
  if (st == FP8MM_OK) st = check_row_waves(T, C, dtype);
  if (st == FP8MM_OK) st = check_ld(ld_rows, C, "ld_rows");
  if (st == FP8MM_OK) st = check_ld(ld_out, C, "ld_out");
  if (st != FP8MM_OK) return st;
  if (T == 0 || C == 0) return ok();
  if (!rows || !out) return fail(FP8MM_EINVAL, "rows and out must not be NULL");
  if (!element_aligned(rows, dtype) || !element_aligned(out, dtype))
    return fail(FP8MM_EINVAL, "rows and out must be aligned to their element type");
  fp8mm::PermuteProblem p{};
  p.T = T;
  p.C = C;
  p.k = int(k);
  p.fp32 = dtype == FP8MM_OUT_FP32;
  p.row_of_slot = row_of_slot;
  p.rows = rows;
  p.ld_rows = ld_rows;
  p.weights = weights;
  p.out = out;
  p.ld_out = ld_out;
  return from_hip(fp8mm::launch_combine(p, stream), "fp8mm_moe_combine");
}

fp8mm_status fp8mm_moe_combine_backward(const void* grad_out, int64_t ld_go, const void* rows, int64_t ld_rows,
                                        fp8mm_dtype dtype, int64_t T, int64_t C, const int32_t* row_of_slot,
                                        const float* weights, int64_t k, void* grad_rows, int64_t ld_gr,
                                        float* grad_weights, hipStream_t stream) {
  fp8mm_status st = check_permute(dtype, T, C, k, row_of_slot);
  if (st == FP8MM_OK) {
    const int64_t slots = 64 / fp8mm::slot_lanes(C, dtype == FP8MM_OUT_FP32);    // of a wave
    st = check_waves((T * k + slots - 1) / slots, 1, T * k, C);
  }
  if (st == FP8MM_OK) st = check_ld(ld_go, C, "ld_go");
  if (st == FP8MM_OK && grad_weights) st = check_ld(ld_rows, C, "ld_rows");
  if (st == FP8MM_OK && grad_rows) st = check_ld(ld_gr, C, "ld_gr");
  if (st != FP8MM_OK) return st;
  if (T == 0 || (!grad_rows && !grad_weights)) return ok();
  if (C > 0 && !grad_out) return fail(FP8MM_EINVAL, "grad_out must not be NULL");
  if (C > 0 && grad_weights && !rows) return fail(FP8MM_EINVAL, "rows are needed for grad_weights");
  if (!element_aligned(grad_out, dtype) || !element_aligned(rows, dtype) || !element_aligned(grad_rows, dtype))
    return fail(FP8MM_EINVAL, "pointers must be aligned to their element type");
  fp8mm::PermuteProblem p{};
  p.T = T;
  p.C = C;
  p.k = int(k);
  p.fp32 = dtype == FP8MM_OUT_FP32;
  p.row_of_slot = row_of_slot;
  p.x = grad_out;
  p.ld_x = ld_go;
  p.rows = rows;
  p.ld_rows = ld_rows;
  p.weights = weights;
  p.out = grad_rows;
  p.ld_out = ld_gr;
  p.grad_weights = grad_weights;
  return from_hip(fp8mm::launch_combine_backward(p, stream), "fp8mm_moe_combine_backward");
}

// --------------------------------------------------------- gated activation

static fp8mm_status check_swiglu(int64_t R, int64_t F) {
  if (R < 0 || F < 0 || R > kMaxInt || F > kMaxLd / 2)
    return fail(FP8MM_EINVAL, "need 0 <= R < 2^31 and 0 <= F <= 2^21");
  if (F % 128 != 0) return fail(FP8MM_EINVAL, "F (%lld) must be a multiple of 128", (long long)F);
  if ((R + 31) / 32 * (F / 128) * 4 > kMaxWaves)
    return fail(FP8MM_EINVAL, "[%lld, %lld] is too large for one launch", (long long)R, (long long)F);
  return FP8MM_OK;
}

static fp8mm_status check_rows16(const void* p, int64_t ld, int64_t cols, int64_t unit, const char* name) {
  if (!p) return fail(FP8MM_EINVAL, "%s must not be NULL", name);
  if (!aligned16(p)) return fail(FP8MM_EINVAL, "%s must be 16-byte aligned", name);
  if (ld < cols || ld % unit != 0 || ld > kMaxLd)
    return fail(FP8MM_EINVAL, "leading dimension of %s (%lld) must be >= %lld, a multiple of %lld and <= 2^22", name,
                (long long)ld, (long long)cols, (long long)unit);
  return FP8MM_OK;
}

fp8mm_status fp8_swiglu(const void* x, int64_t R, int64_t F, int64_t ld_x, void* h, int64_t ld_h, uint8_t* h_q,
                        int64_t ld_hq, float* h_scale, uint8_t* ckpt, int64_t ld_ckpt, float* ckpt_scale,
                        hipStream_t stream) {
  fp8mm_status st = check_swiglu(R, F);
  if (st != FP8MM_OK) return st;
  if (R == 0 || F == 0) return ok();
  st = check_rows16(x, ld_x, 2 * F, 8, "x");
  if (st == FP8MM_OK && h) st = check_rows16(h, ld_h, F, 8, "h");
  if (st == FP8MM_OK && h_q) st = check_rows16(h_q, ld_hq, F, 16, "h_q");
  if (st == FP8MM_OK && ckpt) st = check_rows16(ckpt, ld_ckpt, 2 * F, 16, "ckpt");
  if (st != FP8MM_OK) return st;
  if ((h_q && !h_scale) || (ckpt && !ckpt_scale)) return fail(FP8MM_EINVAL, "codes need their scale array");
  fp8mm::SwigluProblem p{};
  p.R = R;
  p.F = F;
  p.x = static_cast<const uint16_t*>(x);
  p.ld_x = ld_x;
  p.h = static_cast<uint16_t*>(h);
  p.ld_h = ld_h;
  p.h_q = h_q;
  p.ld_hq = ld_hq;
  p.h_scale = h_scale;
  p.ckpt = ckpt;
  p.ld_ckpt = ld_ckpt;
  p.ckpt_scale = ckpt_scale;
  return from_hip(fp8mm::launch_swiglu(p, stream), "fp8_swiglu");
}

fp8mm_status fp8_swiglu_backward(const void* grad_h, int64_t ld_gh, const uint8_t* ckpt, int64_t ld_ckpt,
                                 const float* ckpt_scale, int64_t R, int64_t F, void* grad_x, int64_t ld_gx, void* h,
                                 int64_t ld_h, hipStream_t stream) {
  fp8mm_status st = check_swiglu(R, F);
  if (st != FP8MM_OK) return st;
  if (R == 0 || F == 0) return ok();
  st = check_rows16(grad_h, ld_gh, F, 8, "grad_h");
  if (st == FP8MM_OK) st = check_rows16(ckpt, ld_ckpt, 2 * F, 16, "ckpt");
  if (st == FP8MM_OK) st = check_rows16(grad_x, ld_gx, 2 * F, 8, "grad_x");
  if (st == FP8MM_OK && h) st = check_rows16(h, ld_h, F, 8, "h");
  if (st != FP8MM_OK) return st;
  if (!ckpt_scale) return fail(FP8MM_EINVAL, "ckpt_scale must not be NULL");
  fp8mm::SwigluProblem p{};
  p.R = R;
  p.F = F;
  p.h = static_cast<uint16_t*>(h);
  p.ld_h = ld_h;
  p.ckpt = const_cast<uint8_t*>(ckpt);
  p.ld_ckpt = ld_ckpt;
  p.ckpt_scale = const_cast<float*>(ckpt_scale);
  p.grad_h = static_cast<const uint16_t*>(grad_h);
  p.ld_gh = ld_gh;
  p.grad_x = static_cast<uint16_t*>(grad_x);
  p.ld_gx = ld_gx;
  return from_hip(fp8mm::launch_swiglu_backward(p, stream), "fp8_swiglu_backward");
}

}  // extern "C"
