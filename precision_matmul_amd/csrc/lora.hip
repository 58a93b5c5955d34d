// Low-rank adapters of many requests beside a shared projection, and their gradients
// (gfx950).  With a = ids[t], the adapter of token t, and its panels down, up [r, C]:
//
//   v = down x,  out = base + s up^T v
//   dv = s up dy,  dx = down^T dv,  ddown = sum_t dv x^T,  dup = sum_t s v dy^T
//
// Three products make all of them, because both panels have the rank first: shrink
// (v = panel x), expand (out = base + s panel^T v) and outer (sum_t s v x^T).  The
// rank is small, so all three are HBM-bound: x, base and out pass once, and the panels
// of the adapters in use.  Of rank 16, 16640 x 5120 x 8192 takes 36 us of shrink (4.8
// TB/s) and 97 of expand (5.6), both panels' gradients of 16384 x 2048 x 5120 41 us (5.7);
// of rank 64, 4099 x 5120 x 8192 22 and 43 us (1.9 and 3.1: each tile reads as many bytes of
// panel).  Short batches are bound by the latency of a few dependent loads.  (Kernels, three
// sets of operands in turn.  Times of choices between two forms, below, are of one set again
// and again, unless they say otherwise: there shrink of 16640 x 5120 takes 31, of 4099 15.)
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
// v is float32 in memory and enters the second product, and panel gradients in bf16, as two
// bf16 numbers, its rounding and the rest, in two instructions: the matrix work is not the
// bound, and v keeps 16 bits, 8 more than the results.  Panel gradients in float32 take
// three, which hold all of v's bits (backward of 4099 x 5120 x 8192 of rank 64, calls: 180
// us, with two 164; of rank 16, 16384 x 2048 x 5120, 120 and 118.6).
//
// The rest is 0 or of either sign, so that its product with an infinity is NaN, or the
// opposite one, where v's own is an infinity.  Wherever that happens the result is NaN:
// results are looked at before they are stored, and those of a wave that holds a NaN are
// computed again, with the rest's products taken of the finite values alone.  The look
// costs runs of tokens 1 %, and 16384 of 100 adapters in any order, with a few results for
// each look, 4 % (a training step of 1024 x 1024, rank 16, 475 us, 457 without).
#include "block_launch.hpp"
#include "moe_launch.hpp"
#include "ops_common.hpp"

namespace fp8mm {
namespace {

using namespace ops;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kTile = 64;          // tokens of a workgroup: one ballot
constexpr int kRankBlock = 64;     // rows of a panel that a workgroup takes at once
// Batches of up to this many tokens are one tile.  With twice as many, single tokens would
// gain and runs lose, and the host does not see which it has: 600 tokens of 40 adapters,
// 2048 x 2048, 40 us by tiles and 15 adapter by adapter, 1000 tokens of 64 in 5 runs 14 and 47.
constexpr int kFewTokens = 512;

__device__ __forceinline__ bf16x8 as_bf16(const Chunk& c) { return __builtin_bit_cast(bf16x8, c); }

__device__ __forceinline__ f32x4 mfma(const bf16x8& a, const bf16x8& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// A lane's 8 columns from c on, of rows of C.  Where they reach past the end, the lane
// works on the row's last 8 in place of them, so that no load needs a path for a row's
// last elements, for which the wave would wait one by one; it stores only those that are
// its own.  Lanes past the end work on the last 8 too, and store none.  TINY: rows of less
// than 8 columns, which do need that path (in kernels of their own).
template <bool TINY>
struct Columns {
  int64_t at;                      // first column that is loaded
  int skip;                        // leading ones that are other lanes'
  __device__ __forceinline__ Columns(int64_t c, int64_t C) {
    at = TINY ? c : min(c, C - 8);
    skip = int(min(c - at, int64_t(8)));
  }
  template <bool NT = false>
  __device__ __forceinline__ Chunk load(const uint16_t* row, int64_t C) const {
    if constexpr (TINY) return load_row(row, at, C);
    return NT ? load_chunk_nt(row + at) : load_chunk(row + at);
  }
  template <bool NT = false>
  __device__ __forceinline__ void store(uint16_t* row, int64_t C, const Chunk& v) const {
    if constexpr (TINY) {
      store_row(row, at, C, v);
    } else if (skip == 0) {
      NT ? store_chunk_nt(row + at, v) : store_chunk(row + at, v);
    } else {
#pragma unroll
      for (int i = 1; i < 8; ++i)
        if (i >= skip) row[at + i] = uint16_t(v.w[i / 2] >> (i % 2 * 16));
    }
  }
  __device__ __forceinline__ void store(float* row, int64_t C, const float (&f)[8]) const {
    if (!TINY && skip == 0) {
#pragma unroll
      for (int i = 0; i < 8; i += 4)
        store_chunk(row + at + i, Chunk{{__float_as_uint(f[i]), __float_as_uint(f[i + 1]), __float_as_uint(f[i + 2]),
                                         __float_as_uint(f[i + 3])}});
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i >= skip && at + i < C) row[at + i] = f[i];
    }
  }
};

// At most 64 tokens of one adapter: `rows` of them, lane i < rows holds the i-th one.
struct Members {
  int rows, token;
  // Member i (the last one, past it).
  __device__ __forceinline__ int at(int i) const { return __shfl(token, min(i, rows - 1), 64); }
};

// Batches of more than one tile that are taken adapter by adapter: as many adapters as
// make the tokens few for each, so that a panel is read once and not for each tile (256 x
// 5120 x 8192 of 64 adapters, rank 32: 8.4 + 16 us against 18 + 35 by tiles; 512 tokens of
// 33 adapters 10 + 14 against 17 + 23).
__host__ __device__ inline bool few_tokens(int64_t T, int64_t n) {
  return T > kTile && T <= kFewTokens && n > T / 16;
}
// Workgroups of such a batch stand for its tokens, else for the adapters.
__host__ __device__ inline bool by_tokens(const LoraProblem& p) { return p.T < p.n; }

// The adapter of token t, -1 without one (or no token).
__device__ __forceinline__ int adapter_of(const LoraProblem& p, int64_t t) {
  const int id = t < p.T ? p.ids[t] : -1;
  return id >= 0 && id < p.n ? id : -1;
}

// body(a, members) for each adapter among the 64 tokens from t0 on (NONE: and with a =
// -1 for those without one); workgroup y of a tile takes every gridDim.y-th of them.
template <bool NONE, typename Body>
__device__ __forceinline__ void each_adapter(const LoraProblem& p, int64_t t0, const Body& body) {
  const int lane = threadIdx.x & 63;
  const bool in = t0 + lane < p.T;
  const int id = adapter_of(p, t0 + lane);
  const uint64_t below = (uint64_t(1) << lane) - 1;
  uint64_t todo = __ballot(in && (NONE || id >= 0));
  for (unsigned turn = 0; todo; ++turn) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
    const uint64_t same = __ballot(in && id == a);
    todo &= ~same;
    if (turn % gridDim.y != blockIdx.y) continue;
    // members to the front, the others behind them: a permutation of the lanes
    const int rows = __popcll(same);
    const int to = same >> lane & 1 ? __popcll(same & below) : rows + __popcll(~same & below);
    body(a, Members{rows, int(t0) + __builtin_amdgcn_ds_permute(to * 4, lane)});
  }
}

// The same for a batch of few tokens as a whole: workgroup y handles adapter y (the one
// past the last: the tokens without), or, where there are more adapters than tokens, that
// of token y if y is its first token; MOST of its tokens at a time, in turns with the
// gridDim.z - 1 others of the adapter (if most tokens have the same one after all).  `list`
// is the wave's own.
template <bool NONE, int MOST, typename Body>
__device__ __forceinline__ void one_adapter(const LoraProblem& p, uint16_t* list, const Body& body) {
  const int lane = threadIdx.x & 63;
  const bool by_token = by_tokens(p);
  const int a = by_token ? adapter_of(p, blockIdx.y) : int(blockIdx.y) < p.n ? int(blockIdx.y) : -1;
  if (!NONE && a < 0) return;
  int rows = 0, first = -1, id[kFewTokens / kTile];
#pragma unroll
  for (int i = 0; i < kFewTokens / kTile; ++i)
    if (i * kTile < int(p.T)) id[i] = adapter_of(p, i * kTile + lane);
#pragma unroll
  for (int i = 0; i < kFewTokens / kTile; ++i)
    if (i * kTile < int(p.T)) {
      const bool in = i * kTile + lane < p.T && id[i] == a;
      const uint64_t same = __ballot(in);
      if (first < 0 && same) first = i * kTile + __builtin_ctzll(same);
      if (in) list[rows + __popcll(same & ((uint64_t(1) << lane) - 1))] = uint16_t(i * kTile + lane);
      rows += __popcll(same);
    }
  if (by_token && first != int(blockIdx.y)) return;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  for (int i = blockIdx.z * MOST; i < rows; i += gridDim.z * MOST)
    body(a, Members{min(MOST, rows - i), int(list[min(i + lane, rows - 1)])});
}

// Row stride of v: whole 16 bytes, zeros behind the rank.
__host__ __device__ inline int v_columns(int r) { return (r + 3) / 4 * 4; }

// -------------------------------------------------------------------- shrink

// 8 values from p on.  ODD: p may lie between two words, for which a 16-byte load takes
// several times as long: the words that hold them, moved into place at their use.
template <bool ODD>
struct Eight {
  Chunk v;
  uint32_t end[ODD ? 1 : 0];
  __device__ __forceinline__ void load(const uint16_t* p) {
    if constexpr (ODD) {
      struct __attribute__((packed, aligned(4))) Words {
        Chunk c;
      };
      const uintptr_t at = reinterpret_cast<uintptr_t>(p);
      v = reinterpret_cast<const Words*>(at & ~uintptr_t(3))->c;
      end[0] = *reinterpret_cast<const uint32_t*>((at + 14) & ~uintptr_t(3));
    } else {
      v = load_chunk(p);
    }
  }
  // `p`: of the load, or that many bytes from it that their last two bits are the same
  __device__ __forceinline__ bf16x8 get(const uint16_t* p) const {
    if constexpr (!ODD) return as_bf16(v);
    const uint32_t by = (reinterpret_cast<uintptr_t>(p) & 2) * 8;
    Chunk c;
#pragma unroll
    for (int i = 0; i < 4; ++i) c.w[i] = __builtin_amdgcn_alignbit(i < 3 ? v.w[i + 1] : end[0], v.w[i], by);
    return as_bf16(c);
  }
};

// Rows of MF x 16 tokens and RF x 16 panel rows at ST steps of 32 columns from k on.
template <int MF, int RF, int ST, bool ODD>
struct Piece {
  Eight<ODD> A[ST][MF], B[ST][RF];

  __device__ __forceinline__ void load(const uint16_t* const (&xr)[MF], const uint16_t* const (&pr)[RF], int64_t k) {
#pragma unroll
    for (int s = 0; s < ST; ++s) {
#pragma unroll
      for (int i = 0; i < MF; ++i) A[s][i].load(xr[i] + k + 32 * s);
#pragma unroll
      for (int f = 0; f < RF; ++f) B[s][f].load(pr[f] + k + 32 * s);
    }
  }
  __device__ __forceinline__ void add(const uint16_t* const (&xr)[MF], const uint16_t* const (&pr)[RF],
                                      f32x4 (&acc)[MF][RF]) const {
#pragma unroll
    for (int s = 0; s < ST; ++s) {
      bf16x8 b[RF];
#pragma unroll
      for (int f = 0; f < RF; ++f) b[f] = B[s][f].get(pr[f]);
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        const bf16x8 a = A[s][i].get(xr[i]);
#pragma unroll
        for (int f = 0; f < RF; ++f) acc[i][f] = mfma(a, b[f], acc[i][f]);
      }
    }
  }
};

// Steps of 32 columns of a wave's turn; two turns are in registers, one of them in flight.
// 64 columns are whole lines of memory, but with 64 tokens by 64 panel rows the registers
// are for one step (4099 x 5120 of rank 64: 15.2 us, with two steps of 32 tokens, whose
// two halves each read the panel, 19.0).
template <int RF, bool FEW>
constexpr int steps_of = RF == 4 && !FEW ? 1 : 2;

// Partial v of MF x 16 members over the wave's turns first, first + 4, ... below last.
template <int MF, int RF, int ST, bool TINY, bool ODD>
__device__ __forceinline__ void shrink_rows(const LoraProblem& p, int a, const Members& m, int rank0, int first, int last,
                                            f32x4 (&acc)[MF][RF]) {
  const int lane = threadIdx.x & 63, l15 = lane & 15, g8 = (lane >> 4) * 8;
  const uint16_t* xr[MF];
  const uint16_t* pr[RF];
#pragma unroll
  for (int i = 0; i < MF; ++i) xr[i] = p.x + int64_t(m.at(i * 16 + l15)) * p.ld_x;
#pragma unroll
  for (int f = 0; f < RF; ++f)
    pr[f] = p.panels + (int64_t(a) * p.r + min(rank0 + f * 16 + l15, p.r - 1)) * p.C;
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int f = 0; f < RF; ++f) acc[i][f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int whole = min(last, int(p.C / (32 * ST)));
  int c = first;
  Piece<MF, RF, ST, ODD> u, w;
  if (c < whole) u.load(xr, pr, int64_t(c) * (32 * ST) + g8);
  while (c < whole) {
    if (c + 4 < whole) w.load(xr, pr, int64_t(c + 4) * (32 * ST) + g8);
    u.add(xr, pr, acc);
    c += 4;
    if (c >= whole) break;
    if (c + 4 < whole) u.load(xr, pr, int64_t(c + 4) * (32 * ST) + g8);
    w.add(xr, pr, acc);
    c += 4;
  }
  if (c < last) {                        // the row's last columns: zeros past them
#pragma unroll 1
    for (int64_t k = int64_t(c) * (32 * ST) + g8; k < p.C + g8; k += 32) {
      const Columns<TINY> cols(k, p.C);
      const auto own = [&](Chunk v) {    // without the columns of the lane before
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (2 * i + 1 < cols.skip) v.w[i] = 0;
          if (2 * i + 1 == cols.skip) v.w[i] &= 0xFFFF0000u;
        }
        return v;
      };
      Piece<MF, RF, 1, false> end;
#pragma unroll
      for (int i = 0; i < MF; ++i) end.A[0][i].v = own(cols.load(xr[i], p.C));
#pragma unroll
      for (int f = 0; f < RF; ++f) end.B[0][f].v = own(cols.load(pr[f], p.C));
      end.add(xr, pr, acc);
    }
  }
}

// v of up to MF x 16 members; the waves share the columns.
template <int MF, int RF, int ST, bool TINY, bool ODD>
__device__ __forceinline__ void shrink_tile(const LoraProblem& p, int a, const Members& m, int split, int rank0,
                                            int first, int last, float* red) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  f32x4 acc[MF][RF];
  shrink_rows<MF, RF, ST, TINY, ODD>(p, a, m, rank0, first + wave, last, acc);
  // the waves' sums, added in wave order
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
      const int64_t t = m.at(at);
      if (at < m.rows && j < v_columns(p.r)) p.v[(int64_t(split) * p.T + t) * v_columns(p.r) + j] = j < p.r ? s[i] : 0.0f;
    }
  }
  __syncthreads();
}

template <int RF, bool FEW, bool ODD, bool TINY = false>
__global__ __launch_bounds__(256) void lora_shrink_kernel(const LoraProblem p, int rank_blocks) {
  constexpr int ST = steps_of<RF, FEW>, SUMS = 4 * (FEW ? 2 : 4);      // 32 or 64 members' of four waves
  __shared__ __attribute__((aligned(16))) float red[SUMS * RF * 64 * 4];
  __shared__ uint16_t list[4][FEW ? kFewTokens : 1];
  const int per = p.splits * rank_blocks;
  const int rest = blockIdx.x % per, split = rest % p.splits, rank0 = rest / p.splits * kRankBlock;
  constexpr int COLS = 32 * ST;
  const int pieces = int((p.C + COLS - 1) / COLS), each = (pieces + p.splits - 1) / p.splits;
  const int first = split * each, last = min(pieces, first + each);
  const auto body = [&](int a, const Members& m) {
    if (m.rows <= 16)
      shrink_tile<1, RF, ST, TINY, ODD>(p, a, m, split, rank0, first, last, red);
    else if (m.rows <= 32)
      shrink_tile<2, RF, ST, TINY, ODD>(p, a, m, split, rank0, first, last, red);
    else if constexpr (!FEW)
      shrink_tile<4, RF, ST, TINY, ODD>(p, a, m, split, rank0, first, last, red);
  };
  if constexpr (FEW)
    one_adapter<false, 32>(p, list[threadIdx.x >> 6], body);
  else
    each_adapter<false>(p, int64_t(blockIdx.x / per) * kTile, body);
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

// Two float32 values as packed bf16 and the rest of them as packed bf16 (0 where the
// value is not finite).  Values that would round to an infinity take bf16's largest number.
// `last`: what both leave, exactly.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo, uint32_t* last = nullptr) {
  constexpr float MOST = 3.38953139e38f;
  const bool fx = fabsf(x) < __builtin_inff(), fy = fabsf(y) < __builtin_inff();
  hi = pack_bf16(fx ? __builtin_amdgcn_fmed3f(x, -MOST, MOST) : x, fy ? __builtin_amdgcn_fmed3f(y, -MOST, MOST) : y);
  const float a = __uint_as_float(hi << 16), b = __uint_as_float(hi & 0xFFFF0000u);
  const float ra = fx ? x - a : 0.0f, rb = fy ? y - b : 0.0f;
  lo = pack_bf16(ra, rb);
  if (last) *last = pack_bf16(ra - __uint_as_float(lo << 16), rb - __uint_as_float(lo & 0xFFFF0000u));
}

// The finite ones of 8 values, zeros in the place of the others.  (The empty statement keeps
// the compiler from doing this ahead of the loop over rows, for which it spills registers.)
__device__ __forceinline__ bf16x8 finite(const bf16x8& b) {
  Chunk c = __builtin_bit_cast(Chunk, b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    asm volatile("" : "+v"(c.w[i]));
    const uint32_t none = ((c.w[i] & 0x7F807F80u) + 0x00800080u) >> 15 & 0x00010001u;   // exponents of ones
    c.w[i] &= ~(none * 0xFFFFu);
  }
  return as_bf16(c);
}

// t, or NaN where one of 8 packed results is NaN (or above 2^121: as float16 numbers, of which
// one instruction looks at four, those are NaN too).
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ f16x2 watch(f16x2 t, const Chunk& v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) t = __builtin_elementwise_maximum(t, __builtin_bit_cast(f16x2, v.w[i]));
  return t;
}

// -------------------------------------------------------------------- expand

// v of the members (zeros in the rows behind them and in the columns up to ld - 8 behind
// the rank), its partial sums added, times s, as two bf16 numbers each: hi and lo [64][ld].
// QUADS: 4 columns each of a row.  The loads of all rows are in flight together; FEW:
// those of the rows that are there (256 x 5120 x 8192: 22.7 us against 25.2; with the test
// among many rows 4099 x 5120 x 8192 of rank 64 takes 60 against 57.6).
template <int QUADS, bool FEW>
__device__ __forceinline__ void stage_v(const LoraProblem& p, const Members& m, float s, int j0, int ld, uint16_t* hi,
                                        uint16_t* lo) {
  constexpr int ITEMS = kTile * QUADS / 256;
  float v[ITEMS][4];
  const float* at[ITEMS];
  bool in[ITEMS];
  const int64_t next = p.T * v_columns(p.r);
#pragma unroll
  for (int e = 0; e < ITEMS; ++e) {
    if (FEW && e * (256 / QUADS) >= m.rows) continue;   // the same for all threads
    const int i = e * 256 + threadIdx.x, row = i / QUADS, j = j0 + i % QUADS * 4;
    in[e] = row < m.rows && j < p.r;
    at[e] = p.v + int64_t(m.at(row)) * v_columns(p.r) + (j < p.r ? j : 0);
    unpack<float>(load_chunk(at[e]), v[e]);
  }
  // several partial sums' loads together, in arrays: from one value a sum the compiler makes
  // a chain of loads that wait for each other
  const auto add = [&](int k, auto count) {
    constexpr int N = decltype(count)::value;
    Chunk c[N][ITEMS];
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
      for (int e = 0; e < ITEMS; ++e)
        if (!FEW || e * (256 / QUADS) < m.rows) c[u][e] = load_chunk(at[e] + (k + u) * next);
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
      for (int e = 0; e < ITEMS; ++e) {
        if (FEW && e * (256 / QUADS) >= m.rows) continue;
        float f[4];
        unpack<float>(c[u][e], f);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[e][i] += f[i];
      }
  };
  constexpr int MANY = 8 / ITEMS;
  int k = 1;
  for (; k + MANY <= p.splits; k += MANY) add(k, std::integral_constant<int, MANY>{});
  for (; k < p.splits; ++k) add(k, std::integral_constant<int, 1>{});
#pragma unroll
  for (int e = 0; e < ITEMS; ++e) {
    if (FEW && e * (256 / QUADS) >= m.rows) continue;
    const int i = e * 256 + threadIdx.x, to = i / QUADS * ld + j0 + i % QUADS * 4;
    uint32_t h[2], l[2];
    split2(in[e] ? v[e][0] * s : 0.0f, in[e] ? v[e][1] * s : 0.0f, h[0], l[0]);
    split2(in[e] ? v[e][2] * s : 0.0f, in[e] ? v[e][3] * s : 0.0f, h[1], l[1]);
    *reinterpret_cast<uint2*>(hi + to) = make_uint2(h[0], h[1]);
    *reinterpret_cast<uint2*>(lo + to) = make_uint2(l[0], l[1]);
  }
}

// The panel's rows j .. j + 32 at a lane's columns.
template <bool TINY>
__device__ __forceinline__ void load_panel(const LoraProblem& p, int a, int j, const Columns<TINY>& c, Chunk (&w)[8]) {
  const int row = j + (threadIdx.x >> 4 & 3) * 8;
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = c.load(p.panels + (int64_t(a) * p.r + min(row + i, p.r - 1)) * p.C, p.C);
}

// Zeros in the place of rows from the rank on, which repeat the last one.  (Of 0 and v's
// zeros there, but not of an infinity and a zero, the product would be 0.)
__device__ __forceinline__ void clear_rows(const LoraProblem& p, int j, Chunk (&w)[8]) {
  const int rows = p.r - j - int(threadIdx.x >> 4 & 3) * 8;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t keep = i < rows ? 0xFFFFFFFFu : 0u;
#pragma unroll
    for (int k = 0; k < 4; ++k) w[i].w[k] &= keep;
  }
}

// Base of 4 of the members from `row` on.
template <bool NT, bool TINY>
__device__ __forceinline__ void load_base(const LoraProblem& p, const Members& m, int row, const Columns<TINY>& c,
                                          Chunk (&to)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    to[k] = c.template load<NT>(p.base + int64_t(m.at(row + (threadIdx.x >> 4 & 3) * 4 + k)) * p.ld_base, p.C);
}

// Columns c .. c + 8 of every (step / 16)-th 16 of the members' rows from `row` on, with the
// next ones' base in flight (`next` holds the first ones').  KS: steps of 32 rank rows whose
// fragments stay in registers (0: any number, read again for each 16 rows: 4099 x 8192 of
// rank 64 41 us, with two steps kept 33).
template <int KS, bool FEW, bool NT, bool TINY>
__device__ __forceinline__ void expand_rows(const LoraProblem& p, int a, const Members& m, const Columns<TINY>& c, int ld,
                                            const uint16_t* hi, const uint16_t* lo, bf16x8 (&b)[KS ? KS : 1][8],
                                            Chunk (&next)[4], int row, int by) {
  const int lane = threadIdx.x & 63, l15 = lane & 15, g = lane >> 4;
  for (int i = row; i < m.rows; i += by) {
    f32x4 acc[8];
    const auto start = [&](const Chunk (&from)[4]) {     // sums start from base
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float f[8];
        unpack<uint16_t>(p.base ? from[k] : Chunk{{0u, 0u, 0u, 0u}}, f);
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[q][k] = f[q];
      }
    };
    const auto step = [&](int ks, const bf16x8 (&bf)[8], auto rare) {
      const int at = (i + l15) * ld + ks * 32 + g * 8;
      const bf16x8 l = *reinterpret_cast<const bf16x8*>(lo + at), h = *reinterpret_cast<const bf16x8*>(hi + at);
#pragma unroll
      for (int f = 0; f < 8; ++f) acc[f] = mfma(l, decltype(rare)::value ? finite(bf[f]) : bf[f], acc[f]);
#pragma unroll
      for (int f = 0; f < 8; ++f) acc[f] = mfma(h, bf[f], acc[f]);
    };
    const auto product = [&](auto rare) {
      if constexpr (KS > 0) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) step(ks, b[ks], rare);
      } else {
        for (int ks = 0; ks * 32 < p.r; ++ks) {
          Chunk w[8];
          load_panel(p, a, ks * 32, c, w);
          clear_rows(p, ks * 32, w);
          transpose8(w, b[0]);
          step(ks, b[0], rare);
        }
      }
    };
    Chunk y[4];
    const auto results = [&] {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float f[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) f[q] = acc[q][k];
        y[k] = pack<uint16_t>(f);
      }
    };
    start(next);
    if (p.base && i + by < m.rows) load_base<NT>(p, m, i + by, c, next);
    product(std::false_type{});
    results();
    f16x2 seen[2] = {{0, 0}, {0, 0}};
#pragma unroll
    for (int k = 0; k < 4; ++k)          // (rows behind the members hold anything where tokens are few)
      if (!FEW || i + g * 4 + k < m.rows) seen[k % 2] = watch(seen[k % 2], y[k]);
    const f16x2 both = __builtin_elementwise_maximum(seen[0], seen[1]);
    if (__any(__builtin_isunordered(both.x, both.y))) {  // NaN: see above
      Chunk again[4];
      if (p.base) load_base<NT>(p, m, i, c, again);
      start(again);
      product(std::true_type{});
      results();
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int at = i + g * 4 + k;
      const int64_t row = m.at(at);
      if (at < m.rows) c.template store<NT>(p.out + row * p.ld_out, p.C, y[k]);
    }
  }
}

template <int KS, bool FEW, bool NT, bool TINY = false>
__global__ __launch_bounds__(256, KS == 1 ? 3 : 2) void lora_expand_kernel(const LoraProblem p, int column_blocks,
                                                          int column_waves) {
  constexpr int MAX = (KS ? KS * 32 : kLoraMaxRank) + 8;
  __shared__ __attribute__((aligned(16))) uint16_t hi[kTile * MAX], lo[kTile * MAX];
  __shared__ uint16_t list[4][FEW ? kFewTokens : 1];
  const int lane = threadIdx.x & 63, ld = KS ? MAX : (p.r + 31) / 32 * 32 + 8;
  const int wave = threadIdx.x >> 6, row = wave / column_waves * 16, by = 64 / column_waves;
  const int64_t first = (int64_t(blockIdx.x % column_blocks) * column_waves + wave % column_waves) * 128;
  const Columns<TINY> c(first + (lane & 15) * 8, p.C);
  const auto body = [&](int a, const Members& m) {
    const bool idle = first >= p.C || row >= m.rows;     // whole waves, which still stage v
    if (a < 0) {                         // no adapter: base alone
      if (p.base == p.out || first >= p.C) return;
      for (int i0 = row / 4; i0 < m.rows; i0 += by / 4) {
        const int i = i0 + (lane >> 4);
        const int64_t row = m.at(i);
        if (i >= m.rows) continue;
        const Chunk v = p.base ? c.load(p.base + row * p.ld_base, p.C) : Chunk{{0u, 0u, 0u, 0u}};
        c.store(p.out + row * p.ld_out, p.C, v);
      }
      return;
    }
    // all loads first: the panel's, the first base's, v's
    bf16x8 b[KS ? KS : 1][8];
    Chunk w[KS ? KS : 1][8], next[4];
    if (!idle) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) load_panel(p, a, ks * 32, c, w[ks]);
      if (p.base) load_base<NT>(p, m, row, c, next);
    }
    const float s = p.scales ? p.scales[a] : 1.0f;
    if constexpr (KS > 0)
      stage_v<KS * 8, FEW>(p, m, s, 0, ld, hi, lo);
    else
      for (int j = 0; j < p.r; j += 32) stage_v<8, FEW>(p, m, s, j, ld, hi, lo);
    __syncthreads();
    if (!idle) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        clear_rows(p, ks * 32, w[ks]);
        transpose8(w[ks], b[ks]);
      }
      expand_rows<KS, FEW, NT>(p, a, m, c, ld, hi, lo, b, next, row, by);
    }
    __syncthreads();
  };
  if constexpr (FEW)
    one_adapter<true, kTile>(p, list[threadIdx.x >> 6], body);
  else
    each_adapter<true>(p, int64_t(blockIdx.x / column_blocks) * kTile, body);
}

// --------------------------------------------------------------------- outer

// Tokens and their v in adapter order: order[row] = t, and for each of the two (v of the
// forward, dv) its partial sums added, as two bf16 numbers each (three for gradients in
// float32) in hi, lo and last [r][ld], a rank's tokens next to each other.  A thread takes
// four ranks of a token.
__global__ __launch_bounds__(256) void lora_sort_kernel(const LoraProblem p, const int32_t* row_of_token, LoraOrder o) {
  const int64_t t = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (t >= p.T) return;
  const int64_t row = row_of_token[t];
  if (row < 0) return;                   // no adapter
  if (blockIdx.y == 0) o.order[row] = int32_t(t);
  const int j = blockIdx.y * 4;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const float* v = o.v[which];
    if (!v) continue;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k = 0; k < o.splits[which]; k += 4) {       // four loads together
      Chunk c[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        c[u] = load_chunk(v + (min(k + u, o.splits[which] - 1) * p.T + t) * v_columns(p.r) + j);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float f[4];
        unpack<float>(c[u], f);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += k + u < o.splits[which] ? f[e] : 0.0f;
      }
    }
    uint16_t* hi = o.sorted[which] + j * o.ld + row;
    uint16_t* lo = hi + p.r * o.ld;
    uint16_t* last = lo + p.r * o.ld;
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      uint32_t h, l, m;
      split2(s[e], s[e + 1], h, l, &m);
      if (j + e < p.r) hi[e * o.ld] = uint16_t(h), lo[e * o.ld] = uint16_t(l);
      if (j + e + 1 < p.r) hi[(e + 1) * o.ld] = uint16_t(h >> 16), lo[(e + 1) * o.ld] = uint16_t(l >> 16);
      if (p.grad_fp32 && j + e < p.r) last[e * o.ld] = uint16_t(m);
      if (p.grad_fp32 && j + e + 1 < p.r) last[(e + 1) * o.ld] = uint16_t(m >> 16);
    }
  }
}

constexpr int kOuterRows = 32;           // tokens of a turn: one matrix step
__host__ __device__ inline int64_t partial_size(int r, int64_t C) { return (r * C + 3) / 4 * 4; }

// The first n of a lane's 8 values, zeros after them.
__device__ __forceinline__ Chunk first_of(const Chunk& v, int n) {
  Chunk c;
#pragma unroll
  for (int i = 0; i < 4; ++i) c.w[i] = 2 * i + 1 < n ? v.w[i] : 2 * i < n ? v.w[i] & 0xFFFFu : 0u;
  return c;
}

// Panel gradients from tokens in adapter order.  A workgroup takes 512 columns (its
// waves 128 each), 64 rows of the rank (or fewer) and a range z of the rows; for each
// adapter in the range it adds up its rows, 32 at a time, and writes one partial
// gradient.  As z and the adapter only grow from one to the next, z + a names it: no two
// have the same, and lora_sum_kernel finds an adapter's by its rows.  The next turn's
// rows are in flight while this one's are multiplied.
// Both panels' gradients are one launch, the first `blocks` workgroups side 0's.
struct Sides {
  LoraSide side[2];
  int column_blocks[2];
  int64_t per[2];                        // rows of a range
  unsigned blocks;
};

template <int RF, int PARTS, bool TINY = false>
__global__ __launch_bounds__(256) void lora_outer_kernel(const LoraProblem p, const LoraOrder o, const Sides sides,
                                                         int rank_blocks) {
  const int lane = threadIdx.x & 63, l15 = lane & 15, g8 = (lane >> 4) * 8;
  const int which = blockIdx.x >= sides.blocks;
  const unsigned block = blockIdx.x - (which ? sides.blocks : 0);
  const LoraSide& side = sides.side[which];
  const int column_blocks = sides.column_blocks[which];
  const int64_t per = sides.per[which], C = side.C;
  const int cb = block % column_blocks, rest = block / column_blocks;
  const int rank0 = rest % rank_blocks * kRankBlock, z = rest / rank_blocks;
  const int64_t first = int64_t(cb) * 512 + (threadIdx.x >> 6) * 128;
  if (first >= C) return;              // whole waves, which wait for no others
  const Columns<TINY> c(first + l15 * 8, C);
  const int used = o.offsets[p.n - 1];   // rows that have an adapter
  const int z0 = int(min(int64_t(used), z * per)), z1 = int(min(int64_t(used), (z + 1) * per));
  if (z0 >= z1) return;
  int a;
  {
    int low = 0, high = p.n - 1;         // the adapter of row z0: the first that ends past it
    while (low < high) {
      const int mid = (low + high) >> 1;
      if (o.offsets[mid] > z0)
        high = mid;
      else
        low = mid + 1;
    }
    a = low;
  }
  const uint16_t* vr[RF];
#pragma unroll
  for (int f = 0; f < RF; ++f) vr[f] = o.sorted[which] + min(rank0 + f * 16 + l15, p.r - 1) * o.ld + g8;
  const int64_t part = p.r * o.ld;
  for (int begin = z0; begin < z1; ++a) {
    const int end = min(o.offsets[a], z1);
    if (end <= begin) continue;
    f32x4 acc[RF][8];
#pragma unroll
    for (int f = 0; f < RF; ++f)
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[f][q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    Chunk w[8], v[PARTS][RF];
    int token[8];                        // of the next turn
    const auto find = [&](int row0) {    // the last row again, past the end
#pragma unroll
      for (int i = 0; i < 8; ++i) token[i] = o.order[min(row0 + g8 + i, end - 1)];
    };
    const auto ask = [&](int row0) {     // v: up to 31 rows past the end
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = c.load(side.x + int64_t(token[i]) * side.ld_x, C);
#pragma unroll
      for (int f = 0; f < RF; ++f)
#pragma unroll
        for (int k = 0; k < PARTS; ++k) v[k][f] = load_chunk(vr[f] + row0 + k * part);
    };
    bf16x8 b[8], u[PARTS][RF];
    const auto take = [&](int row0) {    // what was asked for
#pragma unroll
      for (int i = 0; i < 8; ++i) {      // zeros past the end
        const uint32_t keep = row0 + g8 + i < end ? 0xFFFFFFFFu : 0u;
#pragma unroll
        for (int k = 0; k < 4; ++k) w[i].w[k] &= keep;
      }
      transpose8(w, b);
#pragma unroll
      for (int f = 0; f < RF; ++f) {
        const int left = end - row0 - g8;          // the next adapter's v are not this one's
#pragma unroll
        for (int k = 0; k < PARTS; ++k) u[k][f] = as_bf16(left < 8 ? first_of(v[k][f], left) : v[k][f]);
      }
    };
    const auto add = [&](auto rare) {
#pragma unroll
      for (int f = 0; f < RF; ++f)
#pragma unroll
        for (int k = PARTS - 1; k >= 0; --k)             // the smallest first
#pragma unroll
          for (int q = 0; q < 8; ++q)
            acc[f][q] = mfma(u[k][f], k && decltype(rare)::value ? finite(b[q]) : b[q], acc[f][q]);
    };
    find(begin);
    ask(begin);
    if (begin + kOuterRows < end) find(begin + kOuterRows);
    for (int row0 = begin; row0 < end; row0 += kOuterRows) {
      take(row0);
      if (row0 + kOuterRows < end) ask(row0 + kOuterRows);
      if (row0 + 2 * kOuterRows < end) find(row0 + 2 * kOuterRows);
      add(std::false_type{});
    }
    float seen[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int f = 0; f < RF; ++f)
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int q = 0; q < 8; ++q) seen[q] = fmaf(acc[f][q][k], 0.0f, seen[q]);
    // NaN (or infinite): as in the second product
    if (__any(((seen[0] + seen[1]) + (seen[2] + seen[3])) + ((seen[4] + seen[5]) + (seen[6] + seen[7])) != 0.0f)) {
#pragma unroll
      for (int f = 0; f < RF; ++f)
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[f][q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
      for (int row0 = begin; row0 < end; row0 += kOuterRows) {
        find(row0);
        ask(row0);
        take(row0);
        add(std::true_type{});
      }
    }
    float* out = side.partial + (z + a) * partial_size(p.r, C);
#pragma unroll
    for (int f = 0; f < RF; ++f)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int j = rank0 + f * 16 + (lane >> 4) * 4 + k;
        if (j >= p.r) continue;
        float y[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) y[q] = acc[f][q][k];
        c.store(out + int64_t(j) * C, C, y);
      }
    begin = end;
  }
}

// Adds an adapter's partial gradients in order, times its scale: four values a thread.
// (Partial gradients start at whole 16 bytes.)
// The first `split` of an adapter's workgroups take side 0.
__global__ __launch_bounds__(256) void lora_sum_kernel(const LoraProblem p, const LoraOrder o, const Sides sides,
                                                       unsigned split, unsigned blocks) {
  const int a = blockIdx.x / blocks;
  const unsigned block = blockIdx.x % blocks;
  const int which = block >= split;
  const LoraSide& side = sides.side[which];
  const int64_t count = int64_t(p.r) * side.C, per = sides.per[which];
  const int64_t first = int64_t(which ? block - split : block) * 256 + threadIdx.x;
  const int64_t step = int64_t(which ? blocks - split : split) * 1024;
  const int begin = a ? o.offsets[a - 1] : 0, end = o.offsets[a];
  const int64_t z0 = begin / per + a, z1 = end > begin ? (end - 1) / per + a + 1 : z0;
  // an adapter without tokens: zeros, whatever its scale
  const float scale = p.scales && end > begin ? p.scales[a] : 1.0f;
  for (int64_t i = first * 4; i < count; i += step) {
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
    for (int64_t z = z0; z < z1; ++z) {
      float f[4];
      unpack<float>(load_chunk(side.partial + z * partial_size(p.r, side.C) + i), f);
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] += f[k];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) s[k] *= scale;
    const Chunk v = Chunk{{__float_as_uint(s[0]), __float_as_uint(s[1]), __float_as_uint(s[2]), __float_as_uint(s[3])}};
    if (p.grad_fp32) {
      store_row(static_cast<float*>(side.grad) + a * count, i, count, v);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + k < count) static_cast<uint16_t*>(side.grad)[a * count + i + k] = to_bf16(s[k]);
    }
  }
}

int64_t tiles_of(int64_t T, int64_t n) { return few_tokens(T, n) ? 1 : (T + kTile - 1) / kTile; }
int rank_blocks_of(int r) { return (r + kRankBlock - 1) / kRankBlock; }

// Workgroups that share a tile's adapters.  Those that find none for them cost little where
// there are few tiles (1453 x 2048 x 2048 of rank 16, in 5 runs, 6.4 us of expand by four
// and 6.8 by two; a call of 6000 x 2048 x 2048 in 5 runs 25 by two and 27 by one), and tiles
// of many adapters gain (20 adapters in any order: 1453 tokens 18 us of expand by four and 29
// by two, 3000 33 by two and 54 by one).
unsigned tile_groups(const LoraProblem& p) {
  const int64_t most = p.T <= kTile ? p.T : p.T <= 512 ? 16 : p.T <= 1024 ? 8 : p.T <= 2048 ? 4 : p.T <= 8192 ? 2 : 1;
  const int64_t all = int64_t(p.n) + 1;       // adapters, and the tokens without one
  return unsigned(all < most ? all : most);
}

// Ranges of rows that share a panel's gradient: a workgroup a compute unit (two: a training
// step of 16384 x 2048 x 5120 210 us against 203).  More of them for short batches pay up to
// some 16 MiB of partial gradients (both of 1453 x 2688 x 128, rank 64: 13 us, with 4 MiB 22).
int64_t outer_ranges(int64_t T, int64_t C, int r) {
  const int64_t blocks = ((C + 511) / 512) * rank_blocks_of(r);
  int64_t z = 256 / blocks;
  // partial gradients: at most a quarter of x's bytes, or 16 MiB
  const int64_t most = T / (16 * r), least = (int64_t(4) << 20) / (r * C);
  z = z < most || z < least ? z : most > least ? most : least;
  const int64_t turns = (T + 2 * kOuterRows - 1) / (2 * kOuterRows);
  z = z < turns ? z : turns;
  return z < 1 ? 1 : z;
}

}  // namespace

// Workgroups that share a tile's columns: as many as run at once, two a compute unit
// (16640 x 5120 of rank 16 31 us with two, 50 with one).
int lora_splits(int64_t T, int64_t C, int64_t n, int r) {
  if (T <= 0) return 1;
  const int64_t adapters = few_tokens(T, n) || T <= kTile ? (n < T ? n : T) : 1;
  const int64_t blocks = tiles_of(T, n) * adapters * rank_blocks_of(r);
  const int64_t turns = (C + 511) / 512;      // a turn or two for each wave
  int64_t s = (512 + blocks - 1) / blocks;
  if (s > turns) s = turns;
  return int(s > 16 ? 16 : s);
}

int64_t lora_outer_workspace(int64_t T, int64_t C, int64_t n, int r) {
  return 4 * (outer_ranges(T, C, r) + n) * partial_size(r, C);
}

// Parts of the order's workspace: rows of tokens, tokens of rows (up to 31 past the last
// are read, but not used), offsets, both v in order, the plan's own.
namespace {
struct OrderBytes {
  int64_t ld, rows, order, offsets, sorted, all;
};
OrderBytes order_bytes(int64_t T, int64_t n, int r) {
  const auto whole = [](int64_t bytes) { return (bytes + 15) / 16 * 16; };
  OrderBytes b;
  b.ld = (T + kOuterRows + 7) / 8 * 8;
  b.rows = whole(4 * T);
  b.order = 4 * b.ld;
  b.offsets = whole(4 * n);
  b.sorted = 3 * 2 * r * b.ld;             // three parts where gradients are float32
  b.all = b.rows + b.order + b.offsets + 2 * b.sorted + plan_workspace(T, n);
  return b;
}
}  // namespace

int64_t lora_order_workspace(int64_t T, int64_t n, int r) { return order_bytes(T, n, r).all; }

hipError_t launch_lora_order(const LoraProblem& p, void* workspace, LoraOrder& o, hipStream_t st) {
  const OrderBytes b = order_bytes(p.T, p.n, p.r);
  char* at = static_cast<char*>(workspace);
  int32_t* row_of_token = reinterpret_cast<int32_t*>(at);
  o.ld = b.ld;
  o.order = reinterpret_cast<int32_t*>(at += b.rows);
  o.offsets = reinterpret_cast<int32_t*>(at += b.order);
  o.sorted[0] = reinterpret_cast<uint16_t*>(at += b.offsets);
  o.sorted[1] = reinterpret_cast<uint16_t*>(at += b.sorted);
  const hipError_t e =
      launch_plan(p.ids, p.T, p.n, o.offsets, row_of_token, reinterpret_cast<int32_t*>(at += b.sorted), st);
  if (e != hipSuccess || p.T == 0) return e;
  hipLaunchKernelGGL(lora_sort_kernel, dim3(unsigned((p.T + 255) / 256), unsigned((p.r + 3) / 4)), dim3(256), 0, st, p,
                     row_of_token, o);
  return hipGetLastError();
}

// Whether a launch goes adapter by adapter.  (Rows of less than 8 columns always go by
// tiles: one kernel for them.)
bool few(const LoraProblem& p) { return few_tokens(p.T, p.n) && p.C >= 8; }
int64_t tiles_of(const LoraProblem& p) { return few(p) ? 1 : (p.T + kTile - 1) / kTile; }

template <bool FEW>
hipError_t run_shrink(const LoraProblem& p, hipStream_t st) {
  const int rb = rank_blocks_of(p.r);
  const dim3 grid(unsigned(tiles_of(p) * p.splits * rb), FEW ? unsigned(by_tokens(p) ? p.T : p.n) : tile_groups(p),
                  FEW ? 2 : 1);
  const auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, p, rb);
    return hipGetLastError();
  };
  if constexpr (!FEW)
    if (p.C < 8) return run(lora_shrink_kernel<4, false, false, true>);
  const auto words = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 4 == 0; };
  if (words(p.x) && words(p.panels) && p.ld_x % 2 == 0 && p.C % 2 == 0) {
    if (p.r <= 16) return run(lora_shrink_kernel<1, FEW, false>);
    return p.r <= 32 ? run(lora_shrink_kernel<2, FEW, false>) : run(lora_shrink_kernel<4, FEW, false>);
  }
  if (p.r <= 16) return run(lora_shrink_kernel<1, FEW, true>);
  return p.r <= 32 ? run(lora_shrink_kernel<2, FEW, true>) : run(lora_shrink_kernel<4, FEW, true>);
}

template <bool FEW, bool NT>
hipError_t run_expand(const LoraProblem& p, hipStream_t st) {
  // Waves side by side, of 128 columns each; the others take every second or fourth 16 rows.
  // Four, for whole stretches of memory (4099 x 8192 34 us, by two waves 50), but fewer where
  // columns are few or workgroups would be (2475 x 384 6.3 us, by four 9.2).
  int cw = 4;
  if (!FEW)
    while (cw > 1 && (p.C <= 64 * cw || tiles_of(p) * ((p.C + 128 * cw - 1) / (128 * cw)) < 128)) cw /= 2;
  const int cb = int((p.C + 128 * cw - 1) / (128 * cw));
  const dim3 grid(unsigned(tiles_of(p) * cb), FEW ? unsigned(by_tokens(p) ? p.T : p.n + 1) : tile_groups(p),
                  FEW ? 2 : 1);
  const auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, p, cb, cw);
    return hipGetLastError();
  };
  if constexpr (!FEW && !NT)
    if (p.C < 8) return run(lora_expand_kernel<0, false, false, true>);
  if (p.r <= 32) return run(lora_expand_kernel<1, FEW, NT>);
  return p.r <= 64 ? run(lora_expand_kernel<2, FEW, NT>) : run(lora_expand_kernel<0, FEW, NT>);
}

hipError_t launch_lora_shrink(const LoraProblem& p, hipStream_t st) {
  if (p.T == 0) return hipSuccess;
  return few(p) ? run_shrink<true>(p, st) : run_shrink<false>(p, st);
}

// Whether expand reads base and writes its result past the caches: where the result is larger
// than the L2s together and of whole lines.  Calls with several sets of operands in turn, so
// that nothing is in the caches from the call before: 4099 x 5120 x 8192 53 us against 57,
// 16640 x 8192 138 and 150, a training step of 16384 x 2048 x 5120 209 and 217; but 7730 x
// 4856, whose rows share lines, 46 against 43.  (The same operands again and again: 7730 x
// 4864 31 against 26.)
bool streams(const LoraProblem& p) {
  return p.C >= 8 && p.T * p.C * 2 > kL2Bytes && p.ld_out % 64 == 0 && reinterpret_cast<uintptr_t>(p.out) % 128 == 0;
}

hipError_t launch_lora_expand(const LoraProblem& p, hipStream_t st) {
  if (p.T == 0) return hipSuccess;
  if (few(p)) return run_expand<true, false>(p, st);
  return streams(p) ? run_expand<false, true>(p, st) : run_expand<false, false>(p, st);
}

hipError_t launch_lora_outer(const LoraProblem& p, const LoraOrder& o, const LoraSide (&side)[2], hipStream_t st) {
  const int rb = rank_blocks_of(p.r);
  Sides sides;
  unsigned blocks[2], sums[2];
  for (int i = 0; i < 2; ++i) {
    sides.side[i] = side[i];
    const int64_t C = side[i].C > 0 ? side[i].C : 1;
    const int64_t Z = outer_ranges(p.T, C, p.r), per = (p.T + Z - 1) / Z;
    sides.column_blocks[i] = int((C + 511) / 512);
    sides.per[i] = per > 0 ? (per + kOuterRows - 1) / kOuterRows * kOuterRows : kOuterRows;
    blocks[i] = side[i].grad ? unsigned(Z * sides.column_blocks[i] * rb) : 0;
    const int64_t fours = (int64_t(p.r) * C + 1023) / 1024;
    sums[i] = side[i].grad ? unsigned(fours < 1024 ? fours : 1024) : 0;
  }
  sides.blocks = blocks[0];
  if (p.T > 0) {
    const auto run = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(blocks[0] + blocks[1]), dim3(256), 0, st, p, o, sides, rb);
      return hipGetLastError();
    };
    const bool tiny = (side[0].grad && side[0].C < 8) || (side[1].grad && side[1].C < 8);
    const auto parts = [&](auto n) {
      constexpr int PARTS = decltype(n)::value;
      return tiny        ? run(lora_outer_kernel<4, PARTS, true>)
             : p.r <= 16 ? run(lora_outer_kernel<1, PARTS>)
             : p.r <= 32 ? run(lora_outer_kernel<2, PARTS>)
                         : run(lora_outer_kernel<4, PARTS>);
    };
    const hipError_t e =
        p.grad_fp32 ? parts(std::integral_constant<int, 3>{}) : parts(std::integral_constant<int, 2>{});
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(lora_sum_kernel, dim3(unsigned(p.n) * (sums[0] + sums[1])), dim3(256), 0, st, p, o, sides, sums[0],
                     sums[0] + sums[1]);
  return hipGetLastError();
}

}  // namespace fp8mm
