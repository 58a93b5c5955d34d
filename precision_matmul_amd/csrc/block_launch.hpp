// Launchers of the operators around a block's dense products and its router,
// shared between their C ABI layer and the kernel sources.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8mm {

// --------------------------------------------------------------- RMS norm
struct RmsProblem {
  const void* x;         // forward: [R, C]
  const void* residual;  // forward: [R, C] or null
  const void* dy;        // backward: [R, C]
  const void* h_in;      // backward: [R, C]
  const void* grad_h;    // backward: [R, C] or null
  int64_t ld_x, ld_res, ld_dy, ld_h, ld_gh;
  bool fp32;             // rows are fp32 (else bf16)
  bool param_fp32;       // weight and dweight are fp32 (else bf16)
  int64_t R, C;
  const void* weight;    // [C] or null (1)
  float eps;
  void* h;               // forward: x + residual, [R, C] or null (row stride ld_h)
  void* y;               // forward: [R, C] or null
  int64_t ld_y;
  uint8_t* q;            // forward: codes [R, C] or null
  int64_t ld_q;
  float* scale;          // [C / 128, R], or [R] if rowwise
  bool rowwise;
  float* rstd;           // [R] (forward: or null)
  void* dx;              // backward: [R, C] or null
  int64_t ld_dx;
  void* dweight;         // [C] or null
  float* workspace;      // backward: rms_backward_workspace bytes
};

hipError_t launch_rms_norm(const RmsProblem& p, hipStream_t st);
hipError_t launch_rms_norm_backward(const RmsProblem& p, hipStream_t st);
int64_t rms_backward_workspace(int64_t R, int64_t C);

// ----------------------------------------------------------- balance loss
struct BalanceProblem {
  const void* logits;    // [T, E], row stride ld
  bool fp32;
  int64_t T, ld;
  int E, k;
  bool sigmoid;          // probabilities: normalised sigmoid, else softmax
  const int32_t* ids;    // [T, k]
  const int32_t* ends;   // [S] or null (one sequence of T rows)
  int S;
  float coeff;
  float* loss;           // [1]
  int32_t* counts;       // [S, E]
  int32_t* tokens;       // [S]
  void* workspace;       // balance_workspace bytes
  // backward
  const float* grad_loss;
  void* grad_logits;     // [T, E], row stride ld_grad, type of logits
  int64_t ld_grad;
};

int64_t balance_workspace(int64_t T, int64_t E, int64_t S);
hipError_t launch_balance(const BalanceProblem& p, hipStream_t st);
hipError_t launch_balance_backward(const BalanceProblem& p, hipStream_t st);

// --------------------------------------------------------------- adapters
// One product of tokens' rows with the panels of their adapters: v[t] = panel[a]
// x[t] (shrink), out[t] = base[t] + s panel[a]^T v[t] (expand) or panel gradients
// sum_t s v[t] x[t]^T (outer).
struct LoraProblem {
  int64_t T, C;            // rows and columns of x, out
  int n, r;
  const int32_t* ids;      // [T]
  const float* scales;     // [n] or null (1)
  const uint16_t* panels;  // [n, r, C]
  const uint16_t* x;       // shrink, outer: [T, C], row stride ld_x
  int64_t ld_x;
  float* v;                // [splits, T, r rounded up to 4]
  int splits;
  const uint16_t* base;    // expand: [T, C] or null (0)
  int64_t ld_base;
  uint16_t* out;           // expand: [T, C]
  int64_t ld_out;
  bool grad_fp32;          // outer
};

// One panel's gradient.
struct LoraSide {
  const uint16_t* x;       // [T, C], row stride ld_x
  int64_t ld_x, C;
  void* grad;              // [n, r, C], or null: not wanted
  float* partial;          // lora_outer_workspace bytes
};

// Tokens in adapter order, for the gradients: offsets [n], the adapters' cumulative end
// rows, each row's token, and v of both products in that order.
struct LoraOrder {
  const float* v[2];       // as the forward and the backward wrote them, or null
  int splits[2];
  int32_t* offsets;
  int32_t* order;
  uint16_t* sorted[2];
  int64_t ld;
};

constexpr int kLoraMaxRank = 256;
constexpr int kLoraMaxAdapters = 1024;   // of gradients: what a plan takes

int lora_splits(int64_t T, int64_t C, int64_t n, int r);
int64_t lora_outer_workspace(int64_t T, int64_t C, int64_t n, int r);   // bytes
hipError_t launch_lora_shrink(const LoraProblem& p, hipStream_t st);
hipError_t launch_lora_expand(const LoraProblem& p, hipStream_t st);
int64_t lora_order_workspace(int64_t T, int64_t n, int r);              // bytes
// o.v and o.splits are the caller's, the rest is filled in
hipError_t launch_lora_order(const LoraProblem& p, void* workspace, LoraOrder& o, hipStream_t st);
// side i with the i-th v of o
hipError_t launch_lora_outer(const LoraProblem& p, const LoraOrder& o, const LoraSide (&side)[2], hipStream_t st);

}  // namespace fp8mm
