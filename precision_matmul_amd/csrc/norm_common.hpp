// Device pieces shared by the norms: a row's sum over the waves that hold it, four
// floats as a chunk.
#pragma once

#include "ops_common.hpp"

namespace fp8mm {
namespace ops {

__device__ __forceinline__ Chunk pack4f(const float* f) {
  return Chunk{{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])}};
}

// Sum of v over the WPR waves that share a row.  `slot` alternates between
// calls, so that one barrier a call is enough.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float (&part)[2][WPR], int slot) {
  v = wave_sum(v);
  if constexpr (WPR == 1) return v;
  if ((threadIdx.x & 63) == 0) part[slot][threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < WPR; ++w) s += part[slot][w];
  return s;
}

}  // namespace ops
}  // namespace fp8mm
