// Launchers of the operators around the grouped GEMMs, shared between their
// C ABI layer and the kernel sources.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8mm {

// ------------------------------------------------------------- layer norm
struct NormProblem {
  const void* x;       // [R, C], row stride ld_x
  const void* dy;      // backward: [R, C], row stride ld_dy
  void* out;           // forward: y; backward: dx (row stride ld_out)
  int64_t R, C;
  int64_t ld_x, ld_dy, ld_out;
  bool fp32;           // x, dy, out are fp32 (else bf16)
  bool param_fp32;     // weight, bias, dweight, dbias are fp32 (else bf16)
  const void* weight;  // [C] or null (1)
  const void* bias;    // [C] or null (0)
  float eps;
  float* mean;         // [R] (forward: null if not wanted)
  float* rstd;
  void* dweight;       // [C] or null
  void* dbias;
  float* workspace;    // backward: norm_backward_workspace bytes
};

hipError_t launch_norm(const NormProblem& p, hipStream_t st);
hipError_t launch_norm_backward(const NormProblem& p, hipStream_t st);
int64_t norm_backward_workspace(int64_t R, int64_t C);

// ---------------------------------------------------------------- routing
struct RouteProblem {
  const void* logits;  // [T, E], row stride ld
  bool fp32;
  int64_t T;
  int64_t ld;
  int E, k;
  const float* bias;   // [E] or null
  bool sigmoid;        // scores: sigmoid, else softmax
  int groups, group_topk;
  bool group_top2;     // group score: sum of the two best, else the best
  bool renorm;
  float scale;
  int32_t* ids;        // [T, k]
  float* weights;      // [T, k]
  // backward
  const float* grad_weights;   // [T, k]
  void* grad_logits;           // [T, E], row stride ld_grad, type of logits
  int64_t ld_grad;
};

constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxK = 64;
// added to the sum of the chosen scores before it divides them
constexpr float kRenormEps = 1e-20f;

hipError_t launch_route(const RouteProblem& p, hipStream_t st);
hipError_t launch_route_backward(const RouteProblem& p, hipStream_t st);

// ------------------------------------------------------------ permutation
// Workspace (bytes) of a plan of n slots over E experts.
int64_t plan_workspace(int64_t n, int64_t E);
hipError_t launch_plan(const int32_t* ids, int64_t n, int E, int32_t* offsets, int32_t* row_of_slot, int32_t* workspace,
                       hipStream_t st);

struct PermuteProblem {
  int64_t T, C;
  int k;
  bool fp32;                     // rows are fp32 (else bf16)
  const int32_t* row_of_slot;    // [T, k]
  const void* x;                 // token-order input [T, C] (dispatch: x; combine backward: grad_out)
  int64_t ld_x;
  const void* rows;              // expert-order input [T k, C] (combine, combine backward)
  int64_t ld_rows;
  const float* weights;          // [T, k] or null (1)
  void* out;                     // dispatch: [T k, C]; combine: [T, C]; combine backward: grad_rows [T k, C]
  int64_t ld_out;
  float* grad_weights;           // combine backward: [T, k] or null
  uint8_t* q;                    // FP8 dispatch: codes [T k, C]
  int64_t ld_q;
  float* scale;                  // FP8 dispatch: [C / 128, T k]
};

// Columns of one token that a wave of dispatch (rows, codes) and of combine covers.
constexpr int64_t kCodeColumns = 1024;
inline int64_t row_columns(bool fp32) { return fp32 ? 256 : 512; }
// Lanes that share a slot in combine's backward.
inline int64_t slot_lanes(int64_t C, bool fp32) { return C > row_columns(fp32) ? 64 : 16; }

hipError_t launch_dispatch(const PermuteProblem& p, hipStream_t st);
hipError_t launch_dispatch_fp8(const PermuteProblem& p, hipStream_t st);
hipError_t launch_combine(const PermuteProblem& p, hipStream_t st);
hipError_t launch_combine_backward(const PermuteProblem& p, hipStream_t st);

// --------------------------------------------------------- gated activation
struct SwigluProblem {
  int64_t R, F;
  const uint16_t* x;        // forward: bf16 [R, 2 F] = gate, up; row stride ld_x
  int64_t ld_x;
  uint16_t* h;              // bf16 [R, F] or null, row stride ld_h
  int64_t ld_h;
  uint8_t* h_q;             // 1x128 codes [R, F] or null, row stride ld_hq
  int64_t ld_hq;
  float* h_scale;           // [F / 128, R]
  uint8_t* ckpt;            // 1x128 codes of x [R, 2 F] (forward: or null), row stride ld_ckpt
  int64_t ld_ckpt;
  float* ckpt_scale;        // [2 F / 128, R]
  const uint16_t* grad_h;   // backward: bf16 [R, F], row stride ld_gh
  int64_t ld_gh;
  uint16_t* grad_x;         // backward: bf16 [R, 2 F], row stride ld_gx
  int64_t ld_gx;
};

hipError_t launch_swiglu(const SwigluProblem& p, hipStream_t st);
hipError_t launch_swiglu_backward(const SwigluProblem& p, hipStream_t st);

}  // namespace fp8mm
