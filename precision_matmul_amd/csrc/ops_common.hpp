// Device pieces of the operators around the grouped GEMMs: 16-byte chunks of
// bf16 or fp32 rows, reductions of a wave in the data-parallel primitives
// (no LDS traffic), workgroup order.
//
// bf16 values are uint16_t in memory and float in registers; results go back
// through one round-to-nearest-even conversion.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8mm {
namespace ops {

template <typename T>
constexpr int kVec = 16 / int(sizeof(T));   // elements of a 16-byte chunk

// A chunk in registers.  Memory accesses assume the alignment of one element
// only (rows of odd length start anywhere); the hardware takes the full-width
// access at any address, and an aligned one costs nothing extra.
struct Chunk {
  uint32_t w[4];
};

template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) ChunkAt {
  uint32_t w[4];
};

template <typename T>
__device__ __forceinline__ Chunk load_chunk(const T* p) {
  const ChunkAt<T> c = *reinterpret_cast<const ChunkAt<T>*>(p);
  return Chunk{{c.w[0], c.w[1], c.w[2], c.w[3]}};
}

template <typename T>
__device__ __forceinline__ void store_chunk(T* p, const Chunk& v) {
  *reinterpret_cast<ChunkAt<T>*>(p) = ChunkAt<T>{{v.w[0], v.w[1], v.w[2], v.w[3]}};
}

// The eight L2s together.  A result larger than this is not found there by the
// next kernel: it goes out by streaming stores, which leave the L2s to inputs.
constexpr int64_t kL2Bytes = int64_t(32) << 20;

template <typename T>
__device__ __forceinline__ void store_chunk_nt(T* p, const Chunk& v) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  typedef u32x4 __attribute__((aligned(2))) u32x4_at;
  __builtin_nontemporal_store(u32x4{v.w[0], v.w[1], v.w[2], v.w[3]}, reinterpret_cast<u32x4_at*>(p));
}

// Streaming load, of what is read once and is larger than the L2s.
template <typename T>
__device__ __forceinline__ Chunk load_chunk_nt(const T* p) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  typedef u32x4 __attribute__((aligned(2))) u32x4_at;
  const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_at*>(p));
  return Chunk{{v.x, v.y, v.z, v.w}};
}

// The first n < kVec<T> elements of a row's last chunk, zeros after them.
template <typename T>
__device__ __forceinline__ Chunk load_part(const T* p, int n) {
  Chunk c{{0u, 0u, 0u, 0u}};
  constexpr int per = int(4 / sizeof(T));
#pragma unroll
  for (int i = 0; i < kVec<T>; ++i) {
    if (i < n) {
      uint32_t v;
      if constexpr (sizeof(T) == 2)
        v = p[i];
      else
        v = __float_as_uint(p[i]);
      c.w[i / per] |= v << ((i % per) * 16);
    }
  }
  return c;
}

template <typename T>
__device__ __forceinline__ void store_part(T* p, const Chunk& v, int n) {
#pragma unroll
  for (int i = 0; i < kVec<T>; ++i) {
    if (i < n) {
      if constexpr (sizeof(T) == 2)
        p[i] = uint16_t(v.w[i / 2] >> ((i % 2) * 16));
      else
        p[i] = __uint_as_float(v.w[i]);
    }
  }
}

// Chunk at column c of a row of C elements; zeros past the row.
template <typename T, bool NT = false>
__device__ __forceinline__ Chunk load_row(const T* row, int64_t c, int64_t C) {
  if (c + kVec<T> <= C) return NT ? load_chunk_nt(row + c) : load_chunk(row + c);
  if (c < C) return load_part(row + c, int(C - c));
  return Chunk{{0u, 0u, 0u, 0u}};
}

// The same in two steps, for loads that have to be in flight for a while: the
// chunk, or the row's last whole chunk's worth where it reaches past the end (one
// load either way, for rows of at least a chunk), and, when it is used, what is
// the chunk's own of it.
template <typename T, bool NT = false>
__device__ __forceinline__ Chunk fetch_row(const T* row, int64_t c, int64_t C) {
  if (C < kVec<T>) return load_row(row, c, C);
  if (c >= C) return Chunk{{0u, 0u, 0u, 0u}};
  const T* p = row + min(c, C - kVec<T>);
  return NT ? load_chunk_nt(p) : load_chunk(p);
}

template <typename T>
__device__ __forceinline__ Chunk fetched(const Chunk& v, int64_t c, int64_t C) {
  if (C < kVec<T> || c + kVec<T> <= C || c >= C) return v;
  const int n = int(c + kVec<T> - C) * int(sizeof(T)) * 8;     // bits of the elements past the end
  const uint64_t lo = uint64_t(v.w[1]) << 32 | v.w[0], hi = uint64_t(v.w[3]) << 32 | v.w[2];
  const uint64_t a = n < 64 ? lo >> n | hi << (64 - n) : hi >> (n - 64), b = n < 64 ? hi >> n : 0;
  return Chunk{{uint32_t(a), uint32_t(a >> 32), uint32_t(b), uint32_t(b >> 32)}};
}

template <typename T, bool NT = false>
__device__ __forceinline__ void store_row(T* row, int64_t c, int64_t C, const Chunk& v) {
  if (c + kVec<T> <= C)
    NT ? store_chunk_nt(row + c, v) : store_chunk(row + c, v);
  else if (c < C)
    store_part(row + c, v, int(C - c));
}

template <typename T>
__device__ __forceinline__ void unpack(const Chunk& c, float (&f)[kVec<T>]) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(c.w[i] << 16);
      f[2 * i + 1] = __uint_as_float(c.w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(c.w[i]);
  }
}

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Two floats to packed bf16, nearest even (NaN stays NaN).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const f32x2 v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

__device__ __forceinline__ uint16_t to_bf16(float v) { return uint16_t(pack_bf16(v, v)); }

template <typename T>
__device__ __forceinline__ Chunk pack(const float (&f)[kVec<T>]) {
  Chunk c;
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c.w[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) c.w[i] = __float_as_uint(f[i]);
  }
  return c;
}

template <typename T>
__device__ __forceinline__ float to_float(T v) {
  if constexpr (sizeof(T) == 2)
    return __uint_as_float(uint32_t(v) << 16);
  else
    return v;
}

template <typename T>
__device__ __forceinline__ T from_float(float v) {
  if constexpr (sizeof(T) == 2)
    return to_bf16(v);
  else
    return v;
}

// N consecutive parameters of type P at column c of C, kept in registers as
// they are stored; `none` where there is no parameter vector or the column is
// past its end.
template <typename P, int N>
struct Params {
  struct __attribute__((packed, aligned(sizeof(P)))) At {
    uint32_t w[N * sizeof(P) / 4];
  };
  uint32_t w[N * sizeof(P) / 4];

  __device__ __forceinline__ void load(const P* p, int64_t c, int64_t C, float none) {
    if (p && c + N <= C) {
      const At a = *reinterpret_cast<const At*>(p + c);
#pragma unroll
      for (int i = 0; i < int(N * sizeof(P) / 4); ++i) w[i] = a.w[i];
    } else {
      float f[N];
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = p && c + i < C ? to_float(p[c + i]) : none;
#pragma unroll
      for (int i = 0; i < int(N * sizeof(P) / 4); ++i) {
        if constexpr (sizeof(P) == 2)
          w[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
        else
          w[i] = __float_as_uint(f[i]);
      }
    }
  }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (sizeof(P) == 2)
      return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    else
      return __uint_as_float(w[i]);
  }
};

// ---------------------------------------------------------------- reductions

template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ float dpp(float old, float v) {
  return __uint_as_float(uint32_t(
      __builtin_amdgcn_update_dpp(int(__float_as_uint(old)), int(__float_as_uint(v)), CTRL, ROWS, 0xF, false)));
}

__device__ __forceinline__ float lane_value(float v, int lane) {
  return __uint_as_float(uint32_t(__builtin_amdgcn_readlane(int(__float_as_uint(v)), lane)));
}

// Sum over the 64 lanes, in every lane (a scalar).  Row shifts by 1, 2, 4 and
// 8 sum each row of 16 into its last lane, the two row broadcasts carry the
// row sums on to lane 63: a fixed order, so results repeat bit for bit.
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<0x111>(0.0f, v);
  v += dpp<0x112>(0.0f, v);
  v += dpp<0x114>(0.0f, v);
  v += dpp<0x118>(0.0f, v);
  v += dpp<0x142, 0xA>(0.0f, v);
  v += dpp<0x143, 0xC>(0.0f, v);
  return lane_value(v, 63);
}

// Maximum over the 64 lanes; NaN lanes do not count.
__device__ __forceinline__ float wave_max_f(float v) {
  const float lo = -__builtin_inff();
  v = fmaxf(v, dpp<0x111>(lo, v));
  v = fmaxf(v, dpp<0x112>(lo, v));
  v = fmaxf(v, dpp<0x114>(lo, v));
  v = fmaxf(v, dpp<0x118>(lo, v));
  v = fmaxf(v, dpp<0x142, 0xA>(lo, v));
  v = fmaxf(v, dpp<0x143, 0xC>(lo, v));
  return lane_value(v, 63);
}

// Maximum of unsigned integers over the 64 lanes (a scalar): one instruction a
// step within the rows of 16 (lanes that a shift leaves empty read 0), then the
// rows' maxima in scalars.
__device__ __forceinline__ uint32_t wave_max_u(uint32_t v) {
  v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x111, 0xF, 0xF, true)));
  v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x112, 0xF, 0xF, true)));
  v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x114, 0xF, 0xF, true)));
  v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x118, 0xF, 0xF, true)));
  const int i = int(v);
  return max(max(uint32_t(__builtin_amdgcn_readlane(i, 15)), uint32_t(__builtin_amdgcn_readlane(i, 31))),
             max(uint32_t(__builtin_amdgcn_readlane(i, 47)), uint32_t(__builtin_amdgcn_readlane(i, 63))));
}

// The same within each row of 16 lanes, in all 16: rotations by 8, 4, 2 and 1.
template <int BY>
__device__ __forceinline__ uint32_t row_ror(uint32_t v) {
  return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x120 + BY, 0xF, 0xF, true));
}
__device__ __forceinline__ uint32_t row_max_u(uint32_t v) {
  v = max(v, row_ror<8>(v));
  v = max(v, row_ror<4>(v));
  v = max(v, row_ror<2>(v));
  return max(v, row_ror<1>(v));
}
__device__ __forceinline__ float row_sum_f(float v) {
  v += __uint_as_float(row_ror<8>(__float_as_uint(v)));
  v += __uint_as_float(row_ror<4>(__float_as_uint(v)));
  v += __uint_as_float(row_ror<2>(__float_as_uint(v)));
  return v + __uint_as_float(row_ror<1>(__float_as_uint(v)));
}

// A lane's value as a scalar; a scalar put into one lane.
__device__ __forceinline__ uint32_t read_lane(uint32_t v, int lane) {
  return uint32_t(__builtin_amdgcn_readlane(int(v), lane));
}
// (This compiler has the instruction's intrinsic but no builtin for it.)
extern "C" __device__ int fp8mm_writelane(int value, int lane, int v) __asm("llvm.amdgcn.writelane.i32");
__device__ __forceinline__ uint32_t write_lane(uint32_t value, int lane, uint32_t v) {
  return uint32_t(fp8mm_writelane(int(value), lane, int(v)));
}

// Maximum of unsigned integers over aligned groups of 8 lanes, in all 8.
__device__ __forceinline__ uint32_t group8_max(uint32_t v) {
  v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x141, 0xF, 0xF, false)));   // lane i with 7 - i
  v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x4E, 0xF, 0xF, false)));    // xor 2
  v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0xB1, 0xF, 0xF, false)));    // xor 1
  return v;
}

// ------------------------------------------------------------ workgroup order

// Position of this workgroup when each of the 8 XCDs takes one contiguous
// range of them (workgroup ids go round the XCDs in turn, and each XCD has
// its own L2): neighbouring rows are then written through one L2.  The grid
// is a multiple of 8; positions at or past the work's end do nothing.
__device__ __forceinline__ uint32_t xcd_position() { return blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8; }

inline unsigned xcd_grid(int64_t blocks) { return unsigned((blocks + 7) / 8 * 8); }

}  // namespace ops
}  // namespace fp8mm
