// Device pieces of the quantizing kernels: 16-byte loads of bf16 values, the
// amax on bf16 bit patterns, the exact quotients and the packed E4M3 codes.
// Shared by the quantizers and by the kernels that quantize what they produce.
#pragma once

#include "fp8_codec.hpp"

namespace fp8mm {

struct alignas(16) U16x8 {
  uint32_t w[4];
};

__device__ __forceinline__ U16x8 load16(const uint16_t* p) {
  return *reinterpret_cast<const U16x8*>(p);
}

// max of |x| over the 8 bf16 values, as a bf16 magnitude bit pattern.
__device__ __forceinline__ uint32_t absmax8(const U16x8& v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = v.w[i] & 0x7FFF7FFFu;
    m = max(m, max(a & 0xFFFFu, a >> 16));
  }
  return m;
}

// Elementwise |x| max of two 8-value vectors, kept as packed magnitudes.
__device__ __forceinline__ void absmax_accum(U16x8& acc, const U16x8& v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = v.w[i] & 0x7FFF7FFFu;
    const uint32_t lo = max(acc.w[i] & 0xFFFFu, a & 0xFFFFu);
    const uint32_t hi = max(acc.w[i] >> 16, a >> 16);
    acc.w[i] = lo | (hi << 16);
  }
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, off, 64));
  return v;
}

// Max over aligned groups of 16 lanes.
__device__ __forceinline__ uint32_t group16_max(uint32_t v) {
#pragma unroll
  for (int off = 8; off >= 1; off >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, off, 64));
  return v;
}

// E4M3 codes of four quotients y = x / s, packed little-endian: round to
// nearest even, saturating to +-448, sign taken from the input x (so that
// -0 and negatives that round to zero give 0x80; the FMA steps of the
// quotient can turn -0 into +0).  The hardware conversion rounds to nearest
// even and agrees with that rule on every float32 of magnitude up to 464;
// clamping larger magnitudes to 448 first (the comparison is false for NaN,
// which stays NaN) extends it to the whole range.
__device__ __forceinline__ float sat448(float y, float x) {
  const float a = __builtin_fabsf(y);
  return __builtin_copysignf(a > 448.0f ? 448.0f : a, x);
}
__device__ __forceinline__ uint32_t pack4(const float* y, const float* x, int stride = 1) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(sat448(y[0], x[0]), sat448(y[stride], x[stride]), 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(sat448(y[2 * stride], x[2 * stride]), sat448(y[3 * stride], x[3 * stride]), w,
                                      true);
  return uint32_t(w);
}

// Quotients fl32(x / s) of 8 values, each with its own cast constants.  The
// exact reciprocal-and-correction path covers every scale >= 2^-90; a wave
// with any smaller scale takes the IEEE division for those values.  The test
// is wave-uniform, so the common case has no per-value branches.
__device__ __forceinline__ void quotients8(const float x[8], const CastScale* const cs[8], float y[8]) {
  bool fast = true;
#pragma unroll
  for (int k = 0; k < 8; ++k) fast = fast && cs[k]->fast;
  if (__all(fast)) {
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = div_by_scale(x[k], cs[k]->s, cs[k]->r);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = cs[k]->fast ? div_by_scale(x[k], cs[k]->s, cs[k]->r) : x[k] / cs[k]->s;
  }
}

__device__ __forceinline__ void unpack8(const U16x8& v, float x[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bits_f32(v.w[i] << 16);
    x[2 * i + 1] = bits_f32(v.w[i] & 0xFFFF0000u);
  }
}

// Encode 8 bf16 values with one scale into 8 codes (little-endian bytes).
__device__ __forceinline__ uint2 cast8(const U16x8& v, const CastScale& cs) {
  float x[8], y[8];
  unpack8(v, x);
  const CastScale* c[8] = {&cs, &cs, &cs, &cs, &cs, &cs, &cs, &cs};
  quotients8(x, c, y);
  return make_uint2(pack4(y, x), pack4(y + 4, x + 4));
}

}  // namespace fp8mm
