// Low-rank adapters of many requests beside a shared projection, and their gradients
// (gfx950).  With a = ids[t], the adapter of token t, and its panels down, up [r, C]:
//
//   v = down x,  out = base + s up^T v
//   dv = s up dy,  dx = down^T dv,  ddown = sum_t dv x^T,  dup = sum_t s v dy^T
//
// Three products make all of them, because both panels have the rank first: shrink
// (v = panel x), expand (out = base + s panel^T v) and outer (sum_t s v x^T).  The
// rank is small, so all three are HBM-bound: x, base and out pass once, and the panels
// of the adapters in use.
//
// Tokens come in any order.  A workgroup takes 64 neighbouring ones and handles each
// adapter that occurs among them in turn, its tokens gathered into the rows of 16-row
// matrix fragments, so that every token's row is read once.
//
// The matrix instruction (16x16x32 bf16) wants 8 neighbouring values of the summed axis
// in a lane.  shrink sums over columns, which lie so in memory.  expand and outer sum
// over the panel's rows and over tokens: there a lane reads 16 bytes (8 columns) of 8
// rows and transposes the 8 x 8 block in registers, 32 byte permutations for 8 fragments
// of 16 columns, whose columns it numbers so that its own 8 are neighbours again in the
// output (16-byte loads and stores, 256 contiguous bytes of a row).
//
// v is float32 in memory and enters the second product as two bf16 numbers, its rounding
// and the rest, in two instructions: the matrix work is not the bound, and v keeps 16
// bits.
#include "block_launch.hpp"
#include "ops_common.hpp"

namespace fp8mm {
namespace {

using namespace ops;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kTile = 64;          // tokens of a workgroup: one ballot
constexpr int kRankBlock = 64;     // rows of a panel that a workgroup takes at once

__device__ __forceinline__ bf16x8 as_bf16(const Chunk& c) { return __builtin_bit_cast(bf16x8, c); }

__device__ __forceinline__ f32x4 mfma(const bf16x8& a, const bf16x8& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// The tokens of one adapter among a tile's 64: `rows` of them, lane i < rows holds the
// i-th one's place in the tile.
struct Members {
  int rows, place;
};
__device__ __forceinline__ Members members(uint64_t same, int lane) {
  const uint64_t below = (uint64_t(1) << lane) - 1;
  const int rows = __popcll(same);
  const bool in = same >> lane & 1;
  // members to the front, the others behind them: a permutation of the lanes
  const int to = in ? __popcll(same & below) : rows + __popcll(~same & below);
  return Members{rows, __builtin_amdgcn_ds_permute(to * 4, lane)};
}
// The place of member i (of the last one, past it).
__device__ __forceinline__ int place_of(const Members& m, int i) { return __shfl(m.place, min(i, m.rows - 1), 64); }

// Adapter of each lane's token, -1 without one (or no token); runs body(a, members) for
// each that occurs (a < 0 if NONE is true: those without).  With more than one
// workgroup in y, workgroup y handles the adapter of token y, if y is its first.
template <bool NONE, typename Body>
__device__ __forceinline__ void each_adapter(const LoraProblem& p, int64_t t0, const Body& body) {
  const int lane = threadIdx.x & 63;
  const bool in = t0 + lane < p.T;
  int id = in ? p.ids[t0 + lane] : -1;
  if (id < 0 || id >= p.n) id = -1;
  uint64_t todo = __ballot(in && (NONE || id >= 0));
  const bool one = gridDim.y > 1;
  if (one) {
    if (!(todo >> blockIdx.y & 1)) return;
    todo &= ~((uint64_t(1) << blockIdx.y) - 1);
  }
  while (todo) {
    const int first = __builtin_ctzll(todo);
    const int a = __builtin_amdgcn_readlane(id, first);
    const uint64_t same = __ballot(in && id == a);
    if (one && __builtin_ctzll(same) != int(blockIdx.y)) return;
    todo &= ~same;
    body(a, members(same, lane));
    if (one) return;
  }
}

// -------------------------------------------------------------------- shrink

// Partial v of one adapter's tokens over this wave's columns: chunks of 128 columns
// first, first + 4, ... below last.
template <int MF, int RF>
__device__ __forceinline__ void shrink_rows(const LoraProblem& p, int64_t t0, int a, const Members& m, int rank0,
                                            int first, int last, f32x4 (&acc)[MF][RF]) {
  const int lane = threadIdx.x & 63, l15 = lane & 15, g8 = (lane >> 4) * 8;
  const uint16_t* xr[MF];
  const uint16_t* pr[RF];
#pragma unroll
  for (int i = 0; i < MF; ++i) xr[i] = p.x + (t0 + place_of(m, i * 16 + l15)) * p.ld_x;
#pragma unroll
  for (int f = 0; f < RF; ++f)
    pr[f] = p.panels + (int64_t(a) * p.r + min(rank0 + f * 16 + l15, p.r - 1)) * p.C;
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int f = 0; f < RF; ++f) acc[i][f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int c = first; c < last; c += 4) {
    const int64_t k0 = int64_t(c) * 128;
    if (k0 + 128 <= p.C) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int64_t k = k0 + 32 * s + g8;
        Chunk A[MF], B[RF];
#pragma unroll
        for (int i = 0; i < MF; ++i) A[i] = load_chunk(xr[i] + k);
#pragma unroll
        for (int f = 0; f < RF; ++f) B[f] = load_chunk(pr[f] + k);
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
          for (int f = 0; f < RF; ++f) acc[i][f] = mfma(as_bf16(A[i]), as_bf16(B[f]), acc[i][f]);
      }
    } else {
      for (int s = 0; s < 4; ++s) {
        const int64_t k = k0 + 32 * s + g8;
        Chunk A[MF], B[RF];
#pragma unroll
        for (int i = 0; i < MF; ++i) A[i] = load_row(xr[i], k, p.C);
#pragma unroll
        for (int f = 0; f < RF; ++f) B[f] = load_row(pr[f], k, p.C);
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
          for (int f = 0; f < RF; ++f) acc[i][f] = mfma(as_bf16(A[i]), as_bf16(B[f]), acc[i][f]);
      }
    }
  }
}

template <int MF, int RF>
__device__ __forceinline__ void shrink_tile(const LoraProblem& p, int64_t t0, int a, const Members& m, int split,
                                            int rank0, int first, int last, float* red) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  f32x4 acc[MF][RF];
  shrink_rows<MF, RF>(p, t0, a, m, rank0, first + wave, last, acc);
  // the four waves' sums, added in wave order
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int f = 0; f < RF; ++f)
      *reinterpret_cast<f32x4*>(red + ((wave * MF * RF + i * RF + f) * 64 + lane) * 4) = acc[i][f];
  __syncthreads();
  for (int q = wave; q < MF * RF; q += 4) {
    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < 4; ++w) s += *reinterpret_cast<const f32x4*>(red + ((w * MF * RF + q) * 64 + lane) * 4);
    const int j = rank0 + q % RF * 16 + (lane & 15);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = q / RF * 16 + (lane >> 4) * 4 + i;
      const int place = place_of(m, at);
      if (at < m.rows && j < p.r) p.v[(int64_t(split) * p.T + t0 + place) * p.r + j] = s[i];
    }
  }
  __syncthreads();
}

template <int RF>
__global__ __launch_bounds__(256) void lora_shrink_kernel(const LoraProblem p, int rank_blocks) {
  __shared__ __attribute__((aligned(16))) float red[4 * 4 * RF * 64 * 4];
  const int per = p.splits * rank_blocks;
  const int64_t t0 = int64_t(blockIdx.x / per) * kTile;
  const int rest = blockIdx.x % per, split = rest % p.splits, rank0 = rest / p.splits * kRankBlock;
  const int chunks = int((p.C + 127) / 128), each = (chunks + p.splits - 1) / p.splits;
  const int first = split * each, last = min(chunks, first + each);
  each_adapter<false>(p, t0, [&](int a, const Members& m) {
    if (m.rows <= 16)
      shrink_tile<1, RF>(p, t0, a, m, split, rank0, first, last, red);
    else if (m.rows <= 32)
      shrink_tile<2, RF>(p, t0, a, m, split, rank0, first, last, red);
    else
      shrink_tile<4, RF>(p, t0, a, m, split, rank0, first, last, red);
  });
}

// ------------------------------------------------- fragments of rows of columns

// 8 rows of 8 columns (a lane's) to 8 fragments, fragment f the 8 rows of column f.
__device__ __forceinline__ void transpose8(const Chunk (&w)[8], bf16x8 (&b)[8]) {
#pragma unroll
  for (int f = 0; f < 8; ++f) {
    Chunk c;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c.w[i] = __builtin_amdgcn_perm(w[2 * i + 1].w[f / 2], w[2 * i].w[f / 2], f & 1 ? 0x07060302u : 0x05040100u);
    b[f] = as_bf16(c);
  }
}

// 8 float32 values as bf16 and the rest of them as bf16 (0 where the value is past
// bf16's range or not finite).
__device__ __forceinline__ void split8(const float (&v)[8], bf16x8& hi, bf16x8& lo) {
  Chunk h, l;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h.w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    const float a = __uint_as_float(h.w[i] << 16), b = __uint_as_float(h.w[i] & 0xFFFF0000u);
    const float ra = v[2 * i] - a, rb = v[2 * i + 1] - b;
    l.w[i] = pack_bf16(fabsf(a) < __builtin_inff() ? ra : 0.0f, fabsf(b) < __builtin_inff() ? rb : 0.0f);
  }
  hi = as_bf16(h);
  lo = as_bf16(l);
}

// -------------------------------------------------------------------- expand

// v[j0 .. j0 + 8) of a token, its partial sums added, times s; 0 past the rank.
__device__ __forceinline__ void load_v8(const LoraProblem& p, int64_t t, int j0, float s, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  for (int k = 0; k < p.splits; ++k) {
    const float* at = p.v + (int64_t(k) * p.T + t) * p.r + j0;
    if (j0 + 8 <= p.r) {
      float a[4], b[4];
      unpack<float>(load_chunk(at), a);
      unpack<float>(load_chunk(at + 4), b);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += a[i], v[4 + i] += b[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (j0 + i < p.r) v[i] += at[i];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= s;
}

template <int MF>
__device__ __forceinline__ void expand_rows(const LoraProblem& p, int64_t t0, int a, const Members& m, int64_t c) {
  const int lane = threadIdx.x & 63, l15 = lane & 15, g = lane >> 4;
  const float s = p.scales ? p.scales[a] : 1.0f;
  f32x4 acc[MF][8];
  int64_t t[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    t[i] = t0 + place_of(m, i * 16 + l15);
#pragma unroll
    for (int f = 0; f < 8; ++f) acc[i][f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  for (int j = 0; j < p.r; j += 32) {
    Chunk w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = j + g * 8 + i;
      w[i] = row < p.r ? load_row(p.panels + (int64_t(a) * p.r + row) * p.C, c, p.C) : Chunk{{0u, 0u, 0u, 0u}};
    }
    bf16x8 b[8];
    transpose8(w, b);
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      float v[8];
      load_v8(p, t[i], j + g * 8, s, v);
      bf16x8 hi, lo;
      split8(v, hi, lo);
#pragma unroll
      for (int f = 0; f < 8; ++f) acc[i][f] = mfma(lo, b[f], acc[i][f]);
#pragma unroll
      for (int f = 0; f < 8; ++f) acc[i][f] = mfma(hi, b[f], acc[i][f]);
    }
  }
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int at = i * 16 + g * 4 + k;
      const int64_t row = t0 + place_of(m, at);
      if (at < m.rows) {
        float f[8], y[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) y[q] = acc[i][q][k];
        if (p.base) {
          unpack<uint16_t>(load_row(p.base + row * p.ld_base, c, p.C), f);
#pragma unroll
          for (int q = 0; q < 8; ++q) y[q] += f[q];
        }
        store_row(p.out + row * p.ld_out, c, p.C, pack<uint16_t>(y));
      }
    }
}

__global__ __launch_bounds__(256) void lora_expand_kernel(const LoraProblem p, int column_blocks) {
  const int64_t t0 = int64_t(blockIdx.x / column_blocks) * kTile;
  const int lane = threadIdx.x & 63;
  const int64_t first = int64_t(blockIdx.x % column_blocks) * 512 + (threadIdx.x >> 6) * 128;
  if (first >= p.C) return;              // whole waves; nothing below waits for others
  const int64_t c = first + (lane & 15) * 8;
  each_adapter<true>(p, t0, [&](int a, const Members& m) {
    if (a < 0) {                         // no adapter: base alone
      if (p.base == p.out) return;
      for (int i0 = 0; i0 < m.rows; i0 += 4) {
        const int i = i0 + (lane >> 4);
        const int64_t row = t0 + place_of(m, i);
        if (i >= m.rows) continue;
        const Chunk v = p.base ? load_row(p.base + row * p.ld_base, c, p.C) : Chunk{{0u, 0u, 0u, 0u}};
        store_row(p.out + row * p.ld_out, c, p.C, v);
      }
    } else if (m.rows <= 16) {
      expand_rows<1>(p, t0, a, m, c);
    } else if (m.rows <= 32) {
      expand_rows<2>(p, t0, a, m, c);
    } else {
      expand_rows<4>(p, t0, a, m, c);
    }
  });
}

// --------------------------------------------------------------------- outer

// Gradient rows of one adapter's panel: 64 rows of the rank (or fewer) and 128 columns a
// workgroup; its waves take the tokens 64 at a time in turns, skipping those of other
// adapters, and their sums are added in wave order.  Z workgroups share the tokens of
// long batches; their sums go to the workspace and lora_sum_kernel adds them.
template <int RF>
__global__ __launch_bounds__(256) void lora_outer_kernel(const LoraProblem p, int rank_blocks, int column_blocks,
                                                         int Z) {
  __shared__ __attribute__((aligned(16))) float red[2 * RF * 8 * 64 * 4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l15 = lane & 15, g = lane >> 4;
  unsigned at = blockIdx.x;
  const int cb = at % column_blocks;
  at /= column_blocks;
  const int rank0 = at % rank_blocks * kRankBlock;
  at /= rank_blocks;
  const int z = at % Z, a = at / Z;
  const int64_t c = int64_t(cb) * 128 + l15 * 8;
  const int64_t tiles = (p.T + kTile - 1) / kTile, each = (tiles + Z - 1) / Z;
  const int64_t last = min(tiles, (z + 1) * each);
  f32x4 acc[RF][8];
#pragma unroll
  for (int f = 0; f < RF; ++f)
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[f][q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t tile = z * each + wave; tile < last; tile += 4) {
    const int64_t t0 = tile * kTile;
    const uint64_t same = __ballot(t0 + lane < p.T && p.ids[min(t0 + lane, p.T - 1)] == a);
    if (!same) continue;
    const Members m = members(same, lane);
    for (int i0 = 0; i0 < m.rows; i0 += 32) {
      Chunk w[8];
      float v[RF][8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int i1 = i0 + g * 8 + i;
        const int64_t t = t0 + place_of(m, i1);
        const bool in = i1 < m.rows;
        w[i] = in ? load_row(p.x + t * p.ld_x, c, p.C) : Chunk{{0u, 0u, 0u, 0u}};
#pragma unroll
        for (int f = 0; f < RF; ++f) {
          const int j = rank0 + f * 16 + l15;
          v[f][i] = 0.0f;
          if (in && j < p.r)
            for (int k = 0; k < p.splits; ++k) v[f][i] += p.v[(int64_t(k) * p.T + t) * p.r + j];
        }
      }
      bf16x8 b[8];
      transpose8(w, b);
#pragma unroll
      for (int f = 0; f < RF; ++f) {
        bf16x8 hi, lo;
        split8(v[f], hi, lo);
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[f][q] = mfma(lo, b[q], acc[f][q]);
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[f][q] = mfma(hi, b[q], acc[f][q]);
      }
    }
  }
  // the waves' sums, halved twice
#pragma unroll
  for (int half = 2; half >= 1; half >>= 1) {
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int f = 0; f < RF; ++f)
#pragma unroll
        for (int q = 0; q < 8; ++q)
          *reinterpret_cast<f32x4*>(red + (((wave - half) * RF * 8 + f * 8 + q) * 64 + lane) * 4) = acc[f][q];
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int f = 0; f < RF; ++f)
#pragma unroll
        for (int q = 0; q < 8; ++q)
          acc[f][q] += *reinterpret_cast<const f32x4*>(red + ((wave * RF * 8 + f * 8 + q) * 64 + lane) * 4);
    }
    __syncthreads();
  }
  if (wave != 0) return;
  const float s = p.scales ? p.scales[a] : 1.0f;
#pragma unroll
  for (int f = 0; f < RF; ++f)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int j = rank0 + f * 16 + g * 4 + k;
      if (j >= p.r) continue;
      float y[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) y[q] = acc[f][q][k] * s;
      const int64_t row = (int64_t(a) * p.r + j) * p.C;
      if (Z > 1 || p.grad_fp32) {
        float* out = Z > 1 ? p.partial + int64_t(z) * p.n * p.r * p.C + row : static_cast<float*>(p.grad) + row;
        store_row(out, c, p.C, Chunk{{__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]),
                                      __float_as_uint(y[3])}});
        store_row(out, c + 4, p.C, Chunk{{__float_as_uint(y[4]), __float_as_uint(y[5]), __float_as_uint(y[6]),
                                          __float_as_uint(y[7])}});
      } else {
        store_row(static_cast<uint16_t*>(p.grad) + row, c, p.C, pack<uint16_t>(y));
      }
    }
}

// Adds the Z partial gradients in order: four values a thread.
__global__ __launch_bounds__(256) void lora_sum_kernel(const float* partial, int Z, int64_t count, void* grad,
                                                       bool fp32) {
  for (int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4; i < count; i += int64_t(gridDim.x) * 1024) {
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int z = 0; z < Z; ++z) {
      float f[4];
      unpack<float>(load_row(partial + z * count, i, count), f);
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] += f[k];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k < count) {
        if (fp32)
          static_cast<float*>(grad)[i + k] = s[k];
        else
          static_cast<uint16_t*>(grad)[i + k] = to_bf16(s[k]);
      }
  }
}

int64_t tiles_of(int64_t T) { return (T + kTile - 1) / kTile; }
int rank_blocks_of(int r) { return (r + kRankBlock - 1) / kRankBlock; }

// Workgroups of a tile in y: one for each of its tokens where there are few tokens
// (each may have an adapter of its own), else one that takes its adapters in turn.
constexpr int64_t kFewTokens = 256;
unsigned tile_groups(int64_t T) { return unsigned(T <= kFewTokens ? (T < kTile ? T : kTile) : 1); }

// Workgroups that share the tokens of a panel's gradient.
int outer_shares(int64_t T, int64_t C, int64_t n, int r) {
  const int64_t blocks = n * ((C + 127) / 128) * rank_blocks_of(r);
  int64_t z = (512 + blocks - 1) / blocks;
  const int64_t most = T / (16 * n * r);      // partial sums: at most a quarter of x
  if (z > most) z = most;
  return int(z < 1 ? 1 : z > 16 ? 16 : z);
}

}  // namespace

int lora_splits(int64_t T, int64_t C, int64_t n, int r) {
  if (T <= 0) return 1;
  const int64_t adapters = T <= kFewTokens ? (n < kTile ? n : kTile) : 1;
  const int64_t tokens = T < kTile ? T : kTile;
  const int64_t blocks = tiles_of(T) * (adapters < tokens ? adapters : tokens) * rank_blocks_of(r);
  const int64_t quads = (C + 511) / 512;      // a chunk of 128 columns for each wave
  int64_t s = (512 + blocks - 1) / blocks;
  if (s > quads) s = quads;
  return int(s > 16 ? 16 : s);
}

int64_t lora_outer_workspace(int64_t T, int64_t C, int64_t n, int r) {
  const int z = outer_shares(T, C, n, r);
  return z > 1 ? 4 * z * n * r * C : 0;
}

hipError_t launch_lora_shrink(const LoraProblem& p, hipStream_t st) {
  if (p.T == 0) return hipSuccess;
  const int rb = rank_blocks_of(p.r);
  const dim3 grid(unsigned(tiles_of(p.T) * p.splits * rb), tile_groups(p.T));
  if (p.r <= 16)
    hipLaunchKernelGGL((lora_shrink_kernel<1>), grid, dim3(256), 0, st, p, rb);
  else if (p.r <= 32)
    hipLaunchKernelGGL((lora_shrink_kernel<2>), grid, dim3(256), 0, st, p, rb);
  else
    hipLaunchKernelGGL((lora_shrink_kernel<4>), grid, dim3(256), 0, st, p, rb);
  return hipGetLastError();
}

hipError_t launch_lora_expand(const LoraProblem& p, hipStream_t st) {
  if (p.T == 0) return hipSuccess;
  const int cb = int((p.C + 511) / 512);
  hipLaunchKernelGGL(lora_expand_kernel, dim3(unsigned(tiles_of(p.T) * cb), tile_groups(p.T)), dim3(256), 0, st, p, cb);
  return hipGetLastError();
}

hipError_t launch_lora_outer(const LoraProblem& p, hipStream_t st) {
  const int rb = rank_blocks_of(p.r), cb = int((p.C + 127) / 128), Z = outer_shares(p.T, p.C, p.n, p.r);
  const dim3 grid(unsigned(int64_t(p.n) * cb * rb * Z));
  if (p.r <= 16)
    hipLaunchKernelGGL((lora_outer_kernel<1>), grid, dim3(256), 0, st, p, rb, cb, Z);
  else if (p.r <= 32)
    hipLaunchKernelGGL((lora_outer_kernel<2>), grid, dim3(256), 0, st, p, rb, cb, Z);
  else
    hipLaunchKernelGGL((lora_outer_kernel<4>), grid, dim3(256), 0, st, p, rb, cb, Z);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || Z == 1) return e;
  const int64_t count = int64_t(p.n) * p.r * p.C, blocks = (count + 1023) / 1024;
  hipLaunchKernelGGL(lora_sum_kernel, dim3(unsigned(blocks < 4096 ? blocks : 4096)), dim3(256), 0, st, p.partial, Z,
                     count, p.grad, p.grad_fp32);
  return hipGetLastError();
}

}  // namespace fp8mm
