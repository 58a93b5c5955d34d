// Gated activation between an expert's two products, with its input kept in 8
// bits for the backward pass (gfx950).
//
//   x = [gate, up] bf16 [R, 2 F];  sig = 1 / (1 + exp(-gate));  h = gate sig up
//   checkpoint: the 1x128 E4M3 codes and scales of x (bit for bit what the
//     1x128 quantizer writes), half the bytes of x
//   h goes out as bf16, as its own 1x128 codes (quantized from the float32
//     values, not from a bf16 rounding of them), or both
//   backward, from gate' = code s, up' = code s:
//     d_gate = d_h up' sig (1 + gate' (1 - sig)),  d_up = d_h gate' sig
//     and h again, for the weight gradient of the second product
//
// HBM-bound.  A thread holds 16 consecutive columns of one row's gate and up,
// 8 lanes a group of 128; a workgroup holds 32 rows of one column block, so
// that a block's 32 scales are one contiguous 128-byte store ([blocks, R]).
#include "moe_launch.hpp"
#include "ops_common.hpp"
#include "quant_cast.hpp"

namespace fp8mm {
namespace {

using namespace ops;

// 1 / (1 + exp(-x)) from the hardware's exp2 and reciprocal (each within an
// ulp; the product with log2(e) adds |x| 2^-24): results go out in bf16 or E4M3.
__device__ __forceinline__ float fast_sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.4426950408889634f));
}

__device__ __forceinline__ uint4 codes16(const uint2& a, const uint2& b) { return make_uint4(a.x, a.y, b.x, b.y); }

// 1x128 quantization of a thread's 16 bf16 values.
__device__ __forceinline__ void quantize16(const U16x8& v0, const U16x8& v1, uint8_t* q, float* scale, bool first) {
  const uint32_t m = group8_max(max(absmax8(v0), absmax8(v1)));
  const float s = scale_from_amax(bf16_to_f32(uint16_t(m)), 0.0f, false);
  const CastScale cs = make_cast_scale(s);
  *reinterpret_cast<uint4*>(q) = codes16(cast8(v0, cs), cast8(v1, cs));
  if (first) *scale = s;
}

__device__ __forceinline__ uint2 cast8_f32(const float (&x)[8], const CastScale& cs) {
  float y[8];
  const CastScale* c[8] = {&cs, &cs, &cs, &cs, &cs, &cs, &cs, &cs};
  quotients8(x, c, y);
  return make_uint2(pack4(y, x), pack4(y + 4, x + 4));
}

__device__ __forceinline__ void store8_bf16(uint16_t* p, const float (&f)[8]) {
  store_chunk<uint32_t>(reinterpret_cast<uint32_t*>(p), pack<uint16_t>(f));
}

template <bool H, bool HQ, bool CKPT>
__global__ __launch_bounds__(256) void swiglu_kernel(const SwigluProblem p, int blocks) {
  const int t = threadIdx.x;
  const int64_t rb = blockIdx.x / unsigned(blocks);
  const int kb = int(blockIdx.x - rb * blocks);
  const int64_t row = rb * 32 + (t >> 3);
  if (row >= p.R) return;                // whole groups of 8 lanes leave
  const int64_t c = int64_t(kb) * 128 + (t & 7) * 16;
  const bool first = (t & 7) == 0;
  const uint16_t* x = p.x + row * p.ld_x + c;
  const U16x8 g0 = load16(x), g1 = load16(x + 8), u0 = load16(x + p.F), u1 = load16(x + p.F + 8);
  if constexpr (CKPT) {
    uint8_t* q = p.ckpt + row * p.ld_ckpt + c;
    quantize16(g0, g1, q, p.ckpt_scale + int64_t(kb) * p.R + row, first);
    quantize16(u0, u1, q + p.F, p.ckpt_scale + (int64_t(kb) + p.F / 128) * p.R + row, first);
  }
  float g[2][8], u[2][8];
  unpack8(g0, g[0]);
  unpack8(g1, g[1]);
  unpack8(u0, u[0]);
  unpack8(u1, u[1]);
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int i = 0; i < 8; ++i) g[a][i] = g[a][i] * fast_sigmoid(g[a][i]) * u[a][i];
  if constexpr (H) {
    uint16_t* h = p.h + row * p.ld_h + c;
    store8_bf16(h, g[0]);
    store8_bf16(h + 8, g[1]);
  }
  if constexpr (HQ) {
    uint32_t m = 0;                      // |h| orders like its bits; NaN above everything
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(g[a][i]) & 0x7FFFFFFFu);
    m = group8_max(m);
    const float s = scale_from_amax(__uint_as_float(m), 0.0f, false);
    const CastScale cs = make_cast_scale(s);
    *reinterpret_cast<uint4*>(p.h_q + row * p.ld_hq + c) = codes16(cast8_f32(g[0], cs), cast8_f32(g[1], cs));
    if (first) p.h_scale[int64_t(kb) * p.R + row] = s;
  }
}

// 8 codes (two dwords) as floats times s.
__device__ __forceinline__ void decode8(uint32_t lo, uint32_t hi, float s, float (&f)[8]) {
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int v = int(w ? hi : lo);
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(v, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(v, true);
    f[4 * w] = a.x * s;
    f[4 * w + 1] = a.y * s;
    f[4 * w + 2] = b.x * s;
    f[4 * w + 3] = b.y * s;
  }
}

template <bool H>
__global__ __launch_bounds__(256) void swiglu_backward_kernel(const SwigluProblem p, int blocks) {
  const int t = threadIdx.x;
  const int64_t rb = blockIdx.x / unsigned(blocks);
  const int kb = int(blockIdx.x - rb * blocks);
  const int64_t row = rb * 32 + (t >> 3);
  if (row >= p.R) return;
  const int64_t c = int64_t(kb) * 128 + (t & 7) * 16;
  const uint8_t* q = p.ckpt + row * p.ld_ckpt + c;
  const uint4 qg = *reinterpret_cast<const uint4*>(q), qu = *reinterpret_cast<const uint4*>(q + p.F);
  const float sg = p.ckpt_scale[int64_t(kb) * p.R + row];
  const float su = p.ckpt_scale[(int64_t(kb) + p.F / 128) * p.R + row];
  const uint16_t* gh = p.grad_h + row * p.ld_gh + c;
  const U16x8 d0 = load16(gh), d1 = load16(gh + 8);
  uint16_t* gx = p.grad_x + row * p.ld_gx + c;
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    float g[8], u[8], d[8], h[8];
    decode8(a ? qg.z : qg.x, a ? qg.w : qg.y, sg, g);
    decode8(a ? qu.z : qu.x, a ? qu.w : qu.y, su, u);
    unpack8(a ? d1 : d0, d);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float sig = fast_sigmoid(g[i]);
      const float silu = g[i] * sig;
      h[i] = silu * u[i];
      g[i] = d[i] * u[i] * (sig + silu * (1.0f - sig));
      u[i] = d[i] * silu;
    }
    store8_bf16(gx + 8 * a, g);
    store8_bf16(gx + p.F + 8 * a, u);
    if constexpr (H) store8_bf16(p.h + row * p.ld_h + c + 8 * a, h);
  }
}

template <bool H, bool HQ, bool CKPT>
hipError_t run_swiglu(const SwigluProblem& p, hipStream_t st) {
  const int blocks = int(p.F / 128);
  hipLaunchKernelGGL((swiglu_kernel<H, HQ, CKPT>), dim3(unsigned((p.R + 31) / 32 * blocks)), dim3(256), 0, st, p,
                     blocks);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_swiglu(const SwigluProblem& p, hipStream_t st) {
  if (p.R == 0 || p.F == 0) return hipSuccess;
  const int form = (p.h ? 4 : 0) | (p.h_q ? 2 : 0) | (p.ckpt ? 1 : 0);
  switch (form) {
    case 1: return run_swiglu<false, false, true>(p, st);
    case 2: return run_swiglu<false, true, false>(p, st);
    case 3: return run_swiglu<false, true, true>(p, st);
    case 4: return run_swiglu<true, false, false>(p, st);
    case 5: return run_swiglu<true, false, true>(p, st);
    case 6: return run_swiglu<true, true, false>(p, st);
    case 7: return run_swiglu<true, true, true>(p, st);
    default: return hipSuccess;
  }
}

hipError_t launch_swiglu_backward(const SwigluProblem& p, hipStream_t st) {
  if (p.R == 0 || p.F == 0) return hipSuccess;
  const int blocks = int(p.F / 128);
  const dim3 grid(unsigned((p.R + 31) / 32 * blocks));
  if (p.h)
    hipLaunchKernelGGL((swiglu_backward_kernel<true>), grid, dim3(256), 0, st, p, blocks);
  else
    hipLaunchKernelGGL((swiglu_backward_kernel<false>), grid, dim3(256), 0, st, p, blocks);
  return hipGetLastError();
}

}  // namespace fp8mm
