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
// HBM-bound.  8 lanes hold a group of 128 columns of one row's gate and up, lane
// l columns 8 l .. and 64 + 8 l .., so that every load and store of theirs is
// one contiguous piece (16 neighbouring columns a lane leave holes in each
// 16-byte store: the backward took 274 us against 240, and 640 with streaming
// stores, which write the holes' lines twice).  A workgroup holds 32 rows of one
// column block, so that a block's 32 scales are one contiguous 128-byte store
// ([blocks, R]); the column blocks of the same rows follow each other.  Results
// larger than the L2s go out by streaming stores; the forward's input comes in by
// streaming loads where it is larger than twice the L2s.
// 98304 x 1408: forward with codes and checkpoint 181 us, 5.4 TB/s; backward
// with the activation again 233 us, 6.0 TB/s (rows before column blocks 304 us,
// a contiguous range of workgroups an XCD 254, plain stores 240).  Both sides of
// the 32 MiB step, streaming stores against plain ones: backward of 32 MiB of
// results 11.2 against 11.0 us, of 48 MiB 16.2 and 16.3, of 64 MiB 20.9 and 22.6;
// codes and checkpoint of 32 MiB 19.1 and 18.6, of 48 MiB 25.9 and 26.2.
#include "moe_launch.hpp"
#include "ops_common.hpp"
#include "quant_cast.hpp"

namespace fp8mm {
namespace {

using namespace ops;

// 1 / (1 + exp(-x)) from the hardware's exp2 and reciprocal (each within an
// ulp; the product with log2(e) adds |x| 2^-24): for results that go out in bf16.
__device__ __forceinline__ float fast_sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.4426950408889634f));
}

// x / (1 + exp(-x)) as exactly as a float32 quotient, for E4M3 codes that no bf16
// rounding precedes: exp2 corrected by the rounding of its argument (x + t ln 2),
// the quotient by its remainder.  Past 126 ln 2 the result is x, or 0 where
// sig < 2^-126 (NaN at -inf, as inf / inf).  10007 x 1408 with codes and checkpoint
// 21.3 us against 20.1 with fast_sigmoid, whose last bits put some codes on the
// other side of their rounding (1e-4 of the codes' norm in all, 2e-8 with this).
__device__ __forceinline__ float silu(float x) {
  const float t = x * -1.44269504f, e = __builtin_amdgcn_exp2f(t);
  const float rest = fmaf(t, -1.90465421e-9f, fmaf(t, 0.693147182f, x));
  const float d = 1.0f + fmaf(-e, rest, e), inv = __builtin_amdgcn_rcpf(d), q = x * inv;
  return fabsf(x) < 87.3365402f ? fmaf(fmaf(-q, d, x), inv, q) : fmaf(0.5f, fabsf(x), 0.5f * x);
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// A lane's two pieces of 8 codes; of 8 bf16 values.
template <bool NT>
__device__ __forceinline__ void store_codes(uint8_t* p, const uint2& a, const uint2& b) {
  u32x2* at = reinterpret_cast<u32x2*>(p);
  const u32x2 va = {a.x, a.y}, vb = {b.x, b.y};
  if constexpr (NT) {
    __builtin_nontemporal_store(va, at);
    __builtin_nontemporal_store(vb, at + 8);
  } else {
    at[0] = va;
    at[8] = vb;
  }
}

template <bool NT>
__device__ __forceinline__ U16x8 load8_bf16(const uint16_t* p) {
  if constexpr (!NT) return load16(p);
  const Chunk c = load_chunk_nt(p);
  return U16x8{{c.w[0], c.w[1], c.w[2], c.w[3]}};
}

template <bool NT>
__device__ __forceinline__ void store8_bf16(uint16_t* p, const float (&f)[8]) {
  uint32_t* at = reinterpret_cast<uint32_t*>(p);
  NT ? store_chunk_nt(at, pack<uint16_t>(f)) : store_chunk(at, pack<uint16_t>(f));
}

// 1x128 quantization of a lane's 16 bf16 values.
template <bool NT>
__device__ __forceinline__ void quantize16(const U16x8& v0, const U16x8& v1, uint8_t* q, float* scale, bool first) {
  const uint32_t m = group8_max(max(absmax8(v0), absmax8(v1)));
  const float s = scale_from_amax(bf16_to_f32(uint16_t(m)), 0.0f, false);
  const CastScale cs = make_cast_scale(s);
  store_codes<NT>(q, cast8(v0, cs), cast8(v1, cs));
  if (first) *scale = s;
}

__device__ __forceinline__ uint2 cast8_f32(const float (&x)[8], const CastScale& cs) {
  float y[8];
  const CastScale* c[8] = {&cs, &cs, &cs, &cs, &cs, &cs, &cs, &cs};
  quotients8(x, c, y);
  return make_uint2(pack4(y, x), pack4(y + 4, x + 4));
}

template <bool H, bool HQ, bool CKPT, bool LD, bool ST>
__global__ __launch_bounds__(256) void swiglu_kernel(const SwigluProblem p, int blocks) {
  const int t = threadIdx.x;
  const int64_t rb = blockIdx.x / unsigned(blocks);
  const int kb = int(blockIdx.x - rb * blocks);
  const int64_t row = rb * 32 + (t >> 3);
  if (row >= p.R) return;                // whole groups of 8 lanes leave
  const int64_t c = int64_t(kb) * 128 + (t & 7) * 8;
  const bool first = (t & 7) == 0;
  const uint16_t* x = p.x + row * p.ld_x + c;
  const U16x8 g0 = load8_bf16<LD>(x), g1 = load8_bf16<LD>(x + 64);
  const U16x8 u0 = load8_bf16<LD>(x + p.F), u1 = load8_bf16<LD>(x + p.F + 64);
  if constexpr (CKPT) {
    uint8_t* q = p.ckpt + row * p.ld_ckpt + c;
    quantize16<ST>(g0, g1, q, p.ckpt_scale + int64_t(kb) * p.R + row, first);
    quantize16<ST>(u0, u1, q + p.F, p.ckpt_scale + (int64_t(kb) + p.F / 128) * p.R + row, first);
  }
  float g[2][8], u[2][8];
  unpack8(g0, g[0]);
  unpack8(g1, g[1]);
  unpack8(u0, u[0]);
  unpack8(u1, u[1]);
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int i = 0; i < 8; ++i) g[a][i] = (HQ ? silu(g[a][i]) : g[a][i] * fast_sigmoid(g[a][i])) * u[a][i];
  if constexpr (H) {
    uint16_t* h = p.h + row * p.ld_h + c;
    store8_bf16<ST>(h, g[0]);
    store8_bf16<ST>(h + 64, g[1]);
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
    store_codes<ST>(p.h_q + row * p.ld_hq + c, cast8_f32(g[0], cs), cast8_f32(g[1], cs));
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

template <bool H, bool NT>
__global__ __launch_bounds__(256) void swiglu_backward_kernel(const SwigluProblem p, int blocks) {
  const int t = threadIdx.x;
  const int64_t rb = blockIdx.x / unsigned(blocks);
  const int kb = int(blockIdx.x - rb * blocks);
  const int64_t row = rb * 32 + (t >> 3);
  if (row >= p.R) return;
  const int64_t c = int64_t(kb) * 128 + (t & 7) * 8;
  const uint8_t* q = p.ckpt + row * p.ld_ckpt + c;
  const uint2 qg[2] = {*reinterpret_cast<const uint2*>(q), *reinterpret_cast<const uint2*>(q + 64)};
  const uint2 qu[2] = {*reinterpret_cast<const uint2*>(q + p.F), *reinterpret_cast<const uint2*>(q + p.F + 64)};
  const float sg = p.ckpt_scale[int64_t(kb) * p.R + row];
  const float su = p.ckpt_scale[(int64_t(kb) + p.F / 128) * p.R + row];
  const uint16_t* gh = p.grad_h + row * p.ld_gh + c;
  const U16x8 dv[2] = {load16(gh), load16(gh + 64)};
  uint16_t* gx = p.grad_x + row * p.ld_gx + c;
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    float g[8], u[8], d[8], h[8];
    decode8(qg[a].x, qg[a].y, sg, g);
    decode8(qu[a].x, qu[a].y, su, u);
    unpack8(dv[a], d);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float sig = fast_sigmoid(g[i]);
      const float silu = g[i] * sig;
      h[i] = silu * u[i];
      g[i] = d[i] * u[i] * (sig + silu * (1.0f - sig));
      u[i] = d[i] * silu;
    }
    store8_bf16<NT>(gx + 64 * a, g);
    store8_bf16<NT>(gx + p.F + 64 * a, u);
    if constexpr (H) store8_bf16<NT>(p.h + row * p.ld_h + c + 64 * a, h);
  }
}

int64_t workgroups(const SwigluProblem& p) { return (p.R + 31) / 32 * (p.F / 128); }

template <bool H, bool HQ, bool CKPT>
hipError_t run_swiglu(const SwigluProblem& p, hipStream_t st) {
  const auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(unsigned(workgroups(p))), dim3(256), 0, st, p, int(p.F / 128));
    return hipGetLastError();
  };
  constexpr int kOut = (H ? 2 : 0) + (HQ ? 1 : 0) + (CKPT ? 2 : 0);      // bytes written for 4 read
  if (p.R * p.F * 4 > 2 * kL2Bytes) return run(swiglu_kernel<H, HQ, CKPT, true, true>);
  if constexpr (kOut > 2) {      // 2 or less are past the L2s only where the input is past twice them
    if (p.R * p.F * kOut > kL2Bytes) return run(swiglu_kernel<H, HQ, CKPT, false, true>);
  }
  return run(swiglu_kernel<H, HQ, CKPT, false, false>);
}

template <bool H>
hipError_t run_swiglu_backward(const SwigluProblem& p, hipStream_t st) {
  const auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(unsigned(workgroups(p))), dim3(256), 0, st, p, int(p.F / 128));
    return hipGetLastError();
  };
  const int64_t bytes = p.R * p.F * (H ? 6 : 4);
  return bytes > kL2Bytes ? run(swiglu_backward_kernel<H, true>) : run(swiglu_backward_kernel<H, false>);
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
  return p.h ? run_swiglu_backward<true>(p, st) : run_swiglu_backward<false>(p, st);
}

}  // namespace fp8mm
