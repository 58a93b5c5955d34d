// Device pieces shared by the norms: a row's sum over the waves that hold it and
// the next row's chunks in flight.
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

// The next row's chunks.  PART: without a path for a row's last elements, for
// which the waves that share a row would all wait where they ask for them: the
// last chunk is loaded whole and shifted, if it has to be, when its turn comes.
template <typename T, bool NT, bool PART>
__device__ __forceinline__ Chunk fetch(const T* row, int64_t c, int64_t C) {
  return PART ? fetch_row<T, NT>(row, c, C) : load_row<T, NT>(row, c, C);
}
template <typename T, bool PART>
__device__ __forceinline__ Chunk settle(const Chunk& v, int64_t c, int64_t C) {
  return PART ? fetched<T>(v, c, C) : v;
}

}  // namespace ops
}  // namespace fp8mm
