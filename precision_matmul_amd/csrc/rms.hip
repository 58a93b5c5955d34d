// Root-mean-square norm over the last dimension with the residual's addition in
// front and the next product's E4M3 codes behind it, forward and backward (gfx950).
//
//   h = x + residual (rounded to the rows' type),  rstd = 1 / sqrt(sum(h^2) / C + eps)
//   y = (h rstd) w;  codes of y: per 128 columns of a row, or per row
//   a = dy w,  hr = h rstd
//   dx = rstd (a - hr sum(a hr) / C) + grad_h,   dw = sum over rows of dy hr
//
// HBM-bound: x and residual (dy, h and grad_h) are read once, h, y and the codes
// (dx) written once: 16640 x 5120 bf16 with residual and 1x128 codes 117 us (5.1 TB/s),
// with rowwise codes 114, backward of 16384 x 2048 47 + 4.7 us (5.7 TB/s in the first
// kernel), 8000 x 5120 60 + 4.8.  A row stays in registers between its sum and its output.
// The norm is that of the rounded h, which is what the residual stream holds and what
// the backward pass reads.  All sums are float32; codes come from float32 values of
// y with no rounding to bf16 in between.
//
// These times are of kernels, three sets of operands in turn; those of choices between two
// forms, below, are of one set again and again, half of which can be in the memory's
// cache, unless they say otherwise.
//
// Lanes past a row's end hold zeros.
#include "block_launch.hpp"
#include "norm_common.hpp"
#include "quant_cast.hpp"

namespace fp8mm {
namespace {

using namespace ops;

constexpr float kRowwiseEps = 1e-12f;   // the rowwise recipe's, as its quantizer's default

enum Form { ROWS = 0, BLOCKS = 1, WHOLE = 2 };   // codes: none, a scale per 128 columns, a scale per row

// A lane's chunk at column c of a row of C >= kVec<T> elements, in two steps: the load, and,
// when it is used, what of it is the lane's own, zeros behind that.  Only a lane's last
// chunk (LAST) can reach past the row; the load is then of the row's last whole chunk, so
// that no branch of the lanes stands between a row's loads, for which they would wait for
// each other.  `first` is the column of the wave's first lane: waves past the end load
// nothing (8000 x 5120 bf16 backward, 10 of 16 waves' chunks in use: 76 us, 85 if they do).
template <typename T, bool NT, bool LAST>
__device__ __forceinline__ Chunk ask_chunk(const T* row, int64_t first, int64_t c, int64_t C) {
  if (LAST && first >= C) return Chunk{{0u, 0u, 0u, 0u}};
  const T* p = row + (LAST ? min(c, C - kVec<T>) : c);
  return NT ? load_chunk_nt(p) : load_chunk(p);
}
template <typename T, bool LAST>
__device__ __forceinline__ Chunk own_chunk(const Chunk& v, int64_t c, int64_t C) {
  if (!LAST) return v;
  if (C % kVec<T> == 0) return c < C ? v : Chunk{{0u, 0u, 0u, 0u}};
  const int n = int(min(max(c + kVec<T> - C, int64_t(0)), int64_t(kVec<T>))) * int(sizeof(T)) * 8;   // bits to drop
  const uint64_t lo = uint64_t(v.w[1]) << 32 | v.w[0], hi = uint64_t(v.w[3]) << 32 | v.w[2];
  const uint64_t a = n == 0 ? lo : n < 64 ? lo >> n | hi << (64 - n) : n < 128 ? hi >> (n - 64) : 0;
  const uint64_t b = n < 64 ? hi >> n : 0;
  return Chunk{{uint32_t(a), uint32_t(a >> 32), uint32_t(b), uint32_t(b >> 32)}};
}

// NIT chunks of a row, STEP columns apart; all but the last are within the row.
template <typename T, bool NT, int NIT>
__device__ __forceinline__ void ask_row(const T* row, int64_t first, int64_t c, int64_t step, int64_t C,
                                        Chunk (&v)[NIT]) {
#pragma unroll
  for (int it = 0; it < NIT; ++it)
    v[it] = it + 1 < NIT ? ask_chunk<T, NT, false>(row, 0, c + it * step, C)
                         : ask_chunk<T, NT, true>(row, first + it * step, c + it * step, C);
}
template <typename T, int NIT>
__device__ __forceinline__ void own_row(const Chunk (&v)[NIT], int64_t c, int64_t step, int64_t C, Chunk (&out)[NIT]) {
#pragma unroll
  for (int it = 0; it < NIT; ++it)
    out[it] = it + 1 < NIT ? v[it] : own_chunk<T, true>(v[it], c + it * step, C);
}

// Column of the wave's first lane in its row, a scalar.
template <int WPR>
__device__ __forceinline__ int64_t wave_column(int vec) {
  return WPR == 1 ? 0 : int64_t(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * 64 * vec;
}

// N parameters at column c of C as float32; `none` without a vector, 0 past its end.
template <int N>
__device__ __forceinline__ void load_weight(const void* weight, bool fp32, int64_t c, int64_t C, float (&w)[N]) {
  if (!weight) {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = 1.0f;
  } else if (fp32) {
    Params<float, N> p;
    p.load(static_cast<const float*>(weight), c, C, 0.0f);
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = p[i];
  } else {
    Params<uint16_t, N> p;
    p.load(static_cast<const uint16_t*>(weight), c, C, 0.0f);
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = p[i];
  }
}

// h = x + residual of one chunk, rounded to the rows' type.
template <typename T>
__device__ __forceinline__ Chunk add_chunks(const Chunk& a, const Chunk& b) {
  float f[kVec<T>], g[kVec<T>];
  unpack<T>(a, f);
  unpack<T>(b, g);
#pragma unroll
  for (int i = 0; i < kVec<T>; ++i) f[i] += g[i];
  return pack<T>(f);
}

template <int N>
__device__ __forceinline__ uint32_t absmax_f32(const float (&f)[N]) {
  uint32_t m = 0;                        // |f| orders like its bits; NaN above everything
#pragma unroll
  for (int i = 0; i < N; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
  return m;
}

// Codes of 8 float32 values, stored.
template <bool NT>
__device__ __forceinline__ void store_codes8(uint8_t* p, const float (&x)[8], const CastScale& cs) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  float y[8];
  const CastScale* c[8] = {&cs, &cs, &cs, &cs, &cs, &cs, &cs, &cs};
  quotients8(x, c, y);
  const u32x2 v = {pack4(y, x), pack4(y + 4, x + 4)};
  if constexpr (NT)
    __builtin_nontemporal_store(v, reinterpret_cast<u32x2*>(p));
  else
    *reinterpret_cast<u32x2*>(p) = v;
}

// Maximum over the WPR waves that share a row; `part` is read until the next call
// with the same slot.
template <int WPR>
__device__ __forceinline__ uint32_t row_max_of(uint32_t v, uint32_t (&part)[2][WPR], int slot) {
  v = wave_max_u(v);
  if constexpr (WPR == 1) return v;
  if ((threadIdx.x & 63) == 0) part[slot][threadIdx.x >> 6] = v;
  __syncthreads();
  uint32_t m = 0;
#pragma unroll
  for (int w = 0; w < WPR; ++w) m = max(m, part[slot][w]);
  return m;
}

// Rows of a workgroup: each XCD has one contiguous range of them, which its
// workgroups take in turns, so that neighbouring rows' scales ([blocks, R]: four
// bytes of each line a row) meet in one L2.
struct Turns {
  int64_t row, end, stride;
};
__device__ __forceinline__ Turns my_rows(int64_t R, int rpb, int wave) {
  const int64_t per = (R + 8 * rpb - 1) / (8 * rpb) * rpb;      // rows of an XCD
  const int64_t begin = int64_t(blockIdx.x % 8) * per;
  return Turns{begin + int64_t(blockIdx.x / 8) * rpb + wave, min(R, begin + per), int64_t(gridDim.x / 8) * rpb};
}

// ---------------------------------------------------------------------------
// Forward, row in registers: WPR waves a row, NIT chunks a lane.  A lane's columns
// are the same in all rows that a workgroup takes, so it keeps its weights in
// registers, and the next row is loaded while this one is reduced and written.  A row has
// a whole wave at least: of 128 bf16 columns 16 of its 64 lanes work (524288 x 128 126 us,
// in three sets of operands; its bytes would take 50).
// ---------------------------------------------------------------------------
template <typename T, int FORM, int WPR, int NIT, bool NT>
__global__ __launch_bounds__(WPR > 4 ? 64 * WPR : 256) void rms_kernel(const RmsProblem p) {
  constexpr int V = kVec<T>;
  constexpr int RPB = WPR == 1 ? 4 : 1;           // rows of a workgroup
  constexpr int64_t STEP = int64_t(WPR) * 64 * V;
  __shared__ float part[2][WPR];
  __shared__ uint32_t top[2][WPR];
  const int in_row = WPR == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int64_t c0 = int64_t(in_row) * V, C = p.C, w0 = wave_column<WPR>(V);
  const T* x = static_cast<const T*>(p.x);
  const T* res = static_cast<const T*>(p.residual);
  float w[NIT][V];
#pragma unroll
  for (int it = 0; it < NIT; ++it) load_weight(p.weight, p.param_fp32, c0 + it * STEP, C, w[it]);
  Turns t = my_rows(p.R, RPB, WPR == 1 ? threadIdx.x >> 6 : 0);
  Chunk nx[NIT], nr[NIT];
  const auto ask = [&](int64_t row) {
    ask_row<T, NT>(x + row * p.ld_x, w0, c0, STEP, C, nx);
    if (res) ask_row<T, NT>(res + row * p.ld_res, w0, c0, STEP, C, nr);
  };
  if (t.row < t.end) ask(t.row);
  int slot = 0;
  for (; t.row < t.end; t.row += t.stride, slot ^= 1) {   // all waves of a row take the same turns
    const int64_t row = t.row;
    Chunk v[NIT];
    own_row<T>(nx, c0, STEP, C, v);
    if (res) {
      Chunk r[NIT];
      own_row<T>(nr, c0, STEP, C, r);
#pragma unroll
      for (int it = 0; it < NIT; ++it) v[it] = add_chunks<T>(v[it], r[it]);
    }
    if (row + t.stride < t.end) ask(row + t.stride);
    float ss = 0.0f;
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
      float f[V];
      unpack<T>(v[it], f);
#pragma unroll
      for (int i = 0; i < V; ++i) ss = fmaf(f[i], f[i], ss);
    }
    if (res && p.h) {
#pragma unroll
      for (int it = 0; it < NIT; ++it)
        store_row<T, NT>(static_cast<T*>(p.h) + row * p.ld_h, c0 + it * STEP, C, v[it]);
    }
    const float rstd = 1.0f / sqrtf(row_sum<WPR>(ss, part, slot) / float(C) + p.eps);
    if (p.rstd && in_row == 0) p.rstd[row] = rstd;
    uint32_t m = 0;
    if constexpr (FORM == WHOLE) {
#pragma unroll
      for (int it = 0; it < NIT; ++it) {
        float f[V];
        unpack<T>(v[it], f);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = f[i] * rstd * w[it][i];
        if (c0 + it * STEP < C) m = max(m, absmax_f32(f));
      }
      m = row_max_of<WPR>(m, top, slot);
    }
    const float whole = scale_from_amax(__uint_as_float(m), kRowwiseEps, true);
    const CastScale row_cs = make_cast_scale(whole);
    if (FORM == WHOLE && in_row == 0) p.scale[row] = whole;
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
      const int64_t c = c0 + it * STEP;
      float f[V];
      unpack<T>(v[it], f);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = f[i] * rstd * w[it][i];
      if (p.y) store_row<T, NT>(static_cast<T*>(p.y) + row * p.ld_y, c, C, pack<T>(f));
      if constexpr (FORM == WHOLE) {
        if (c < C) store_codes8<NT>(p.q + row * p.ld_q + c, f, row_cs);
      } else if constexpr (FORM == BLOCKS) {
        // 16 lanes hold a group of 128 columns; C is whole groups
        const float s = scale_from_amax(__uint_as_float(row_max_u(absmax_f32(f))), 0.0f, false);
        if (c < C) {
          store_codes8<NT>(p.q + row * p.ld_q + c, f, make_cast_scale(s));
          if ((threadIdx.x & 15) == 0) p.scale[c / 128 * p.R + row] = s;
        }
      }
    }
  }
}

// Forward, rows too long for registers: one workgroup a row, which is read again
// (from L2) for each further pass over it.
template <typename T, int FORM>
__global__ __launch_bounds__(256) void rms_long_kernel(const RmsProblem p) {
  constexpr int V = kVec<T>;
  constexpr int64_t STEP = 256 * V;
  __shared__ float part[2][4];
  __shared__ uint32_t top[2][4];
  const int64_t C = p.C;
  int slot = 0;
  for (int64_t row = blockIdx.x; row < p.R; row += gridDim.x, slot ^= 1) {
    const T* x = static_cast<const T*>(p.x) + row * p.ld_x;
    const T* res = p.residual ? static_cast<const T*>(p.residual) + row * p.ld_res : nullptr;
    const auto load = [&](int64_t c) {
      const Chunk v = load_row(x, c, C);
      return res ? add_chunks<T>(v, load_row(res, c, C)) : v;
    };
    float ss = 0.0f;
    for (int64_t c = int64_t(threadIdx.x) * V; c < C; c += STEP) {
      const Chunk v = load(c);
      float f[V];
      unpack<T>(v, f);
#pragma unroll
      for (int i = 0; i < V; ++i) ss = fmaf(f[i], f[i], ss);
      if (res && p.h) store_row(static_cast<T*>(p.h) + row * p.ld_h, c, C, v);
    }
    const float rstd = 1.0f / sqrtf(row_sum<4>(ss, part, slot) / float(C) + p.eps);
    if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
    const auto normed = [&](int64_t c, float (&f)[V]) {
      float w[V];
      unpack<T>(load(c), f);
      load_weight(p.weight, p.param_fp32, c, C, w);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = f[i] * rstd * w[i];
    };
    uint32_t m = 0;
    if constexpr (FORM == WHOLE) {
      for (int64_t c = int64_t(threadIdx.x) * V; c < C; c += STEP) {
        float f[V];
        normed(c, f);
        m = max(m, absmax_f32(f));
      }
      m = row_max_of<4>(m, top, slot);
    }
    const float whole = scale_from_amax(__uint_as_float(m), kRowwiseEps, true);
    const CastScale row_cs = make_cast_scale(whole);
    if (FORM == WHOLE && threadIdx.x == 0) p.scale[row] = whole;
    for (int64_t c = int64_t(threadIdx.x) * V; c < C; c += STEP) {   // whole groups of 16 lanes stay (C % 128 == 0)
      float f[V];
      normed(c, f);
      if (p.y) store_row(static_cast<T*>(p.y) + row * p.ld_y, c, C, pack<T>(f));
      if constexpr (FORM == WHOLE) {
        store_codes8<false>(p.q + row * p.ld_q + c, f, row_cs);
      } else if constexpr (FORM == BLOCKS) {
        const float s = scale_from_amax(__uint_as_float(row_max_u(absmax_f32(f))), 0.0f, false);
        store_codes8<false>(p.q + row * p.ld_q + c, f, make_cast_scale(s));
        if ((threadIdx.x & 15) == 0) p.scale[c / 128 * p.R + row] = s;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Backward, row in registers.  A workgroup takes rows in turns, the next row in
// flight while this one is worked on, and keeps its share of dw in registers over
// all of them; it then writes one partial row of the workspace, [gridDim][C], which
// rms_column_sum_kernel adds up in workgroup order: no atomics, the same bits every
// time.  A row by one wave where that holds it in four chunks a lane, since sums across
// waves wait; longer ones by four or eight waves of two chunks (fp32 above 4096 columns: of
// three or four), bf16 above 8192 by sixteen of two.
// ---------------------------------------------------------------------------
constexpr int kRowWaves = 8;            // waves of a workgroup that takes a row with each

template <typename T, int WPR, int NIT, bool NT>
__global__ __launch_bounds__(64 * (WPR == 1 ? kRowWaves : WPR)) void rms_backward_kernel(const RmsProblem p,
                                                                                         float* partial) {
  constexpr int V = kVec<T>;
  constexpr int RPB = WPR == 1 ? kRowWaves : 1;
  constexpr int64_t STEP = int64_t(WPR) * 64 * V;
  __shared__ float part[2][WPR];
  constexpr int Q = NIT * V / 4;                  // a lane's sums, in fours
  __shared__ float4 acc[WPR == 1 ? kRowWaves / 2 * Q * 64 : 1];
  const int wave = threadIdx.x >> 6;
  const int64_t c0 = int64_t(WPR == 1 ? threadIdx.x & 63 : threadIdx.x) * V, C = p.C, w0 = wave_column<WPR>(V);
  const T* hs = static_cast<const T*>(p.h_in);
  const T* dys = static_cast<const T*>(p.dy);
  const T* ghs = static_cast<const T*>(p.grad_h);
  const float inv_c = 1.0f / float(C);
  float dw[NIT][V], w[NIT][V];
#pragma unroll
  for (int it = 0; it < NIT; ++it) {
#pragma unroll
    for (int i = 0; i < V; ++i) dw[it][i] = 0.0f;
    load_weight(p.weight, p.param_fp32, c0 + it * STEP, C, w[it]);
  }
  const int64_t stride = int64_t(gridDim.x) * RPB;
  int64_t row = int64_t(blockIdx.x) * RPB + (WPR == 1 ? wave : 0);
  Chunk nh[NIT], ng[NIT], ns[NIT];
  float nrstd = 0.0f;
  const auto ask = [&](int64_t at) {
    ask_row<T, NT>(hs + at * p.ld_h, w0, c0, STEP, C, nh);
    ask_row<T, NT>(dys + at * p.ld_dy, w0, c0, STEP, C, ng);
    if (ghs && WPR < 16) ask_row<T, NT>(ghs + at * p.ld_gh, w0, c0, STEP, C, ns);
    nrstd = p.rstd[at];
  };
  if (row < p.R) ask(row);
  for (int slot = 0; row < p.R; row += stride, slot ^= 1) {
    Chunk vh[NIT], vg[NIT], vs[NIT];
    own_row<T>(nh, c0, STEP, C, vh);
    own_row<T>(ng, c0, STEP, C, vg);
    if (ghs && WPR < 16) own_row<T>(ns, c0, STEP, C, vs);
    if (ghs && WPR == 16) ask_row<T, NT>(ghs + row * p.ld_gh, w0, c0, STEP, C, vs);   // for the registers
    const float rstd = nrstd;
    if (row + stride < p.R) ask(row + stride);
    float sah = 0.0f;
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
      float f[V], g[V];
      unpack<T>(vh[it], f);
      unpack<T>(vg[it], g);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float hr = f[i] * rstd;
        sah = fmaf(g[i] * w[it][i], hr, sah);
        dw[it][i] = fmaf(g[i], hr, dw[it][i]);
      }
    }
    sah = row_sum<WPR>(sah, part, slot) * inv_c;
    if (p.dx) {
#pragma unroll
      for (int it = 0; it < NIT; ++it) {
        float f[V], g[V];
        unpack<T>(vh[it], f);
        unpack<T>(vg[it], g);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = rstd * (g[i] * w[it][i] - f[i] * rstd * sah);
        if (ghs) {
          unpack<T>(WPR == 16 && it + 1 == NIT ? own_chunk<T, true>(vs[it], c0 + it * STEP, C) : vs[it], g);
#pragma unroll
          for (int i = 0; i < V; ++i) f[i] += g[i];
        }
        store_row<T, NT>(static_cast<T*>(p.dx) + row * p.ld_dx, c0 + it * STEP, C, pack<T>(f));
      }
    }
  }
  if (!partial) return;
  float* pw = partial + int64_t(blockIdx.x) * C;
  if constexpr (WPR == 1) {
    // the waves' shares, halved three times: the upper half's waves hand theirs
    // to the lower half's
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int half = kRowWaves / 2; half >= 1; half >>= 1) {
      if (wave >= half && wave < 2 * half) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const int it = q * 4 / V, i = q * 4 % V;
          acc[((wave - half) * Q + q) * 64 + lane] =
              make_float4(dw[it][i], dw[it][i + 1], dw[it][i + 2], dw[it][i + 3]);
        }
      }
      __syncthreads();
      if (wave < half) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const int it = q * 4 / V, i = q * 4 % V;
          const float4 a = acc[(wave * Q + q) * 64 + lane];
          dw[it][i] += a.x, dw[it][i + 1] += a.y, dw[it][i + 2] += a.z, dw[it][i + 3] += a.w;
        }
      }
      __syncthreads();
    }
    if (wave != 0) return;
  }
#pragma unroll
  for (int it = 0; it < NIT; ++it)
#pragma unroll
    for (int i = 0; i < V; i += 4) store_row(pw, c0 + it * STEP + i, C, pack4f(&dw[it][i]));
}

// ---------------------------------------------------------------------------
// Backward of few rows in one launch and without a workspace: dw needs no row sums
// (rstd is an input), so the first row_blocks workgroups write dx, a row a wave (WPR
// = 1) or a workgroup, and the others each add up a strip of columns over all rows,
// 64 (WPR = 1) or 16 row slices of it, the slices added in a fixed order.
// ---------------------------------------------------------------------------
template <int WPR>
constexpr int kStripChunks = WPR == 1 ? 4 : 16;

template <typename T, int WPR, int NIT>
__global__ __launch_bounds__(256) void rms_backward_few_kernel(const RmsProblem p, unsigned row_blocks) {
  constexpr int V = kVec<T>;
  constexpr int CL = kStripChunks<WPR>, SLICES = 256 / CL;
  __shared__ float part[SLICES][CL * V];
  __shared__ float sums[2][WPR];
  const int64_t C = p.C;
  const T* hs = static_cast<const T*>(p.h_in);
  const T* dys = static_cast<const T*>(p.dy);
  if (blockIdx.x < row_blocks) {
    constexpr int64_t STEP = int64_t(WPR) * 64 * V;
    const int64_t row = WPR == 1 ? int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6) : blockIdx.x;
    if (row >= p.R) return;                     // WPR = 1: waves of their own; else never
    const int64_t c0 = int64_t(WPR == 1 ? threadIdx.x & 63 : threadIdx.x) * V, w0 = wave_column<WPR>(V);
    Chunk nh[NIT], ng[NIT], ns[NIT], vh[NIT], vg[NIT], vs[NIT];
    float w[NIT][V];
    ask_row<T, false>(hs + row * p.ld_h, w0, c0, STEP, C, nh);
    ask_row<T, false>(dys + row * p.ld_dy, w0, c0, STEP, C, ng);
    if (p.grad_h) ask_row<T, false>(static_cast<const T*>(p.grad_h) + row * p.ld_gh, w0, c0, STEP, C, ns);
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
      vs[it] = Chunk{{0u, 0u, 0u, 0u}};
      load_weight(p.weight, p.param_fp32, c0 + it * STEP, C, w[it]);
    }
    own_row<T>(nh, c0, STEP, C, vh);
    own_row<T>(ng, c0, STEP, C, vg);
    if (p.grad_h) own_row<T>(ns, c0, STEP, C, vs);
    const float rstd = p.rstd[row];
    float sah = 0.0f;
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
      float f[V], g[V];
      unpack<T>(vh[it], f);
      unpack<T>(vg[it], g);
#pragma unroll
      for (int i = 0; i < V; ++i) sah = fmaf(g[i] * w[it][i], f[i] * rstd, sah);
    }
    sah = row_sum<WPR>(sah, sums, 0) / float(C);
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
      float f[V], g[V], s[V];
      unpack<T>(vh[it], f);
      unpack<T>(vg[it], g);
      unpack<T>(vs[it], s);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = rstd * (g[i] * w[it][i] - f[i] * rstd * sah) + s[i];
      store_row(static_cast<T*>(p.dx) + row * p.ld_dx, c0 + it * STEP, C, pack<T>(f));
    }
    return;
  }
  const int chunk = threadIdx.x % CL, slice = threadIdx.x / CL;
  const int64_t strip = int64_t(blockIdx.x - row_blocks) * CL * V;
  const int64_t c = strip + chunk * V;
  float dw[V];
#pragma unroll
  for (int i = 0; i < V; ++i) dw[i] = 0.0f;
#pragma unroll 4
  for (int64_t row = slice; row < p.R; row += SLICES) {
    float f[V], g[V];
    unpack<T>(own_chunk<T, true>(ask_chunk<T, false, true>(hs + row * p.ld_h, 0, c, C), c, C), f);
    unpack<T>(own_chunk<T, true>(ask_chunk<T, false, true>(dys + row * p.ld_dy, 0, c, C), c, C), g);
    const float rstd = p.rstd[row];
#pragma unroll
    for (int i = 0; i < V; ++i) dw[i] = fmaf(g[i], f[i] * rstd, dw[i]);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) part[slice][chunk * V + i] = dw[i];
  __syncthreads();
  // SHARE neighbouring threads add up a column's slices
  constexpr int SHARE = 256 / (CL * V) < SLICES ? 256 / (CL * V) : SLICES;
  static_assert(SHARE >= 1 && (SHARE & (SHARE - 1)) == 0, "a column or more for each thread");
  const int col = threadIdx.x / SHARE, share = threadIdx.x % SHARE;
  if (col >= CL * V) return;
  float s = 0.0f;
#pragma unroll 16
  for (int r = share; r < SLICES; r += SHARE) s += part[r][col];
#pragma unroll
  for (int off = 1; off < SHARE; off <<= 1) s += __shfl_xor(s, off, 64);
  if (share == 0 && strip + col < C) {
    if (p.param_fp32)
      static_cast<float*>(p.dweight)[strip + col] = s;
    else
      static_cast<uint16_t*>(p.dweight)[strip + col] = to_bf16(s);
  }
}

// Backward of rows too long for registers: dx by one workgroup a row ...
template <typename T>
__global__ __launch_bounds__(256) void rms_backward_long_kernel(const RmsProblem p) {
  constexpr int V = kVec<T>;
  __shared__ float part[2][4];
  const int64_t C = p.C;
  int slot = 0;
  for (int64_t row = blockIdx.x; row < p.R; row += gridDim.x, slot ^= 1) {
    const T* h = static_cast<const T*>(p.h_in) + row * p.ld_h;
    const T* dy = static_cast<const T*>(p.dy) + row * p.ld_dy;
    const T* gh = p.grad_h ? static_cast<const T*>(p.grad_h) + row * p.ld_gh : nullptr;
    const float rstd = p.rstd[row];
    float sah = 0.0f;
    for (int64_t c = int64_t(threadIdx.x) * V; c < C; c += 256 * V) {
      float f[V], g[V], w[V];
      unpack<T>(load_row(h, c, C), f);
      unpack<T>(load_row(dy, c, C), g);
      load_weight(p.weight, p.param_fp32, c, C, w);
#pragma unroll
      for (int i = 0; i < V; ++i) sah = fmaf(g[i] * w[i], f[i] * rstd, sah);
    }
    sah = row_sum<4>(sah, part, slot) / float(C);
    for (int64_t c = int64_t(threadIdx.x) * V; c < C; c += 256 * V) {
      float f[V], g[V], w[V];
      unpack<T>(load_row(h, c, C), f);
      unpack<T>(load_row(dy, c, C), g);
      load_weight(p.weight, p.param_fp32, c, C, w);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = rstd * (g[i] * w[i] - f[i] * rstd * sah);
      if (gh) {
        unpack<T>(load_row(gh, c, C), g);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] += g[i];
      }
      store_row(static_cast<T*>(p.dx) + row * p.ld_dx, c, C, pack<T>(f));
    }
  }
}

// ... and the columns' partial sums over rows blockIdx.y, blockIdx.y + gridDim.y,
// ... by one thread a column.
template <typename T>
__global__ __launch_bounds__(256) void rms_columns_kernel(const RmsProblem p, float* partial) {
  const int64_t c = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (c >= p.C) return;
  float dw = 0.0f;
  for (int64_t row = blockIdx.y; row < p.R; row += gridDim.y)
    dw = fmaf(to_float(static_cast<const T*>(p.dy)[row * p.ld_dy + c]),
              to_float(static_cast<const T*>(p.h_in)[row * p.ld_h + c]) * p.rstd[row], dw);
  partial[int64_t(blockIdx.y) * p.C + c] = dw;
}

// Sums the n partial rows of dw: 64 columns and 16 row slices a workgroup, the
// slices added in order.
__global__ __launch_bounds__(1024) void rms_column_sum_kernel(const float* partial, int n, int64_t C, void* dweight,
                                                              bool fp32) {
  __shared__ float part[16][64];
  const int lane = threadIdx.x & 63, slice = threadIdx.x >> 6;
  const int64_t c = int64_t(blockIdx.x) * 64 + lane;
  float s = 0.0f;
  if (c < C) {
#pragma unroll 8
    for (int r = slice; r < n; r += 16) s += partial[int64_t(r) * C + c];
  }
  part[slice][lane] = s;
  __syncthreads();
  if (slice == 0 && c < C) {
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += part[i][lane];
    if (fp32)
      static_cast<float*>(dweight)[c] = s;
    else
      static_cast<uint16_t*>(dweight)[c] = to_bf16(s);
  }
}

constexpr int64_t kForwardGrid = 1024;  // four workgroups a compute unit; whole XCDs
constexpr int kBackwardGrid = 512;      // partial rows at most
constexpr int64_t kRegisterCols = 8192; // longest row that is read once (bf16: twice that)

// Rows that the long rows' kernels take: those, and rows of less than a chunk.
bool long_rows(int64_t C) { return C < 8 || C > kRegisterCols; }
// Backward in one launch: while its columns' sums over all rows, without partial rows, do not
// take longer than the second launch (bf16 512 x 2048 5.7 us, in two launches 7.3 + 3.4; 256 x
// 5120 8.0 and 8.1 + 3.1, but 512 x 5120 21 and 10.4 + 3.9).
bool few_rows(int64_t R, int64_t C) { return R <= (C <= 2048 ? 512 : 256) && !long_rows(C); }

// Long bf16 rows by 16 waves: calls of 4096 x 12288 with a residual 73 us forward and 98
// backward, with grad_h; read twice 93 and 139; the backward with grad_h a row ahead too 109.
// The forward keeps rows in registers.  The backward has 128 of them a lane, and spills 66
// more of its weights, sums and rows into 60 bytes of scratch; its bytes would take 75 us.
template <typename T>
bool by_sixteen(int64_t C) { return sizeof(T) == 2 && C > kRegisterCols && C <= 2 * kRegisterCols; }

// Workgroups of the long rows' kernels, which take further rows in turns past this.
dim3 row_grid(int64_t rows) { return dim3(unsigned(rows < (1 << 20) ? rows : (1 << 20))); }

// Whether rows go past the caches: those larger than the L2s together.  Calls with several
// sets of operands in turn: backward of bf16 16384 x 2048 49.6 us against 53.6, 16384 x 1536
// 39 and 44, fp32 16384 x 1024 51 and 59, codes of 16384 x 2048 43 and 48; about even at the
// border (codes of 16384 x 1152 29 and 27).  The same operands again and again, half of them
// in the memory's cache, gain less, or lose (16384 x 2048 with codes 42 and 37).
bool streams(const RmsProblem& p, size_t size) { return p.R * p.C * int64_t(size) > kL2Bytes; }

// Workgroups of the backward (one partial row each): two a compute unit for rows by four
// waves (bf16 4000 x 2500 20.6 us against 25.5, fp32 16384 x 1280 64 and 73), else one (bf16
// 16384 x 2048 49.8 against 52.9).
int backward_grid(int64_t R, int64_t C, int vec) {
  const int64_t one_wave = 256 * vec;         // rows of up to this many columns: a wave each
  const int64_t rows = C <= one_wave ? kRowWaves : 1;
  const int64_t most = C <= one_wave || C > 2 * one_wave || R < 2048 ? 256 : 512;
  const int64_t blocks = (R + rows - 1) / rows;
  return int(blocks < most ? blocks : most);
}

template <typename T, int FORM, int WPR, int NIT>
hipError_t run_rms(const RmsProblem& p, hipStream_t st) {
  constexpr int RPB = WPR == 1 ? 4 : 1;
  const int64_t blocks = (p.R + RPB - 1) / RPB;
  // six workgroups a compute unit where a lane has one chunk (16384 x 2048 without a
  // residual 25.5 us, with four 29)
  constexpr int64_t MOST = WPR == 4 && NIT == 1 ? 1536 : kForwardGrid;
  const dim3 grid(xcd_grid(blocks < MOST ? blocks : MOST));
  const auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(WPR > 4 ? 64 * WPR : 256), 0, st, p);
    return hipGetLastError();
  };
  return streams(p, sizeof(T)) ? run(rms_kernel<T, FORM, WPR, NIT, true>) : run(rms_kernel<T, FORM, WPR, NIT, false>);
}

template <typename T, int FORM>
hipError_t rms_typed(const RmsProblem& p, hipStream_t st) {
  constexpr int64_t S = 64 * kVec<T>;   // columns of one wave chunk
  if constexpr (sizeof(T) == 2)
    if (by_sixteen<T>(p.C)) return run_rms<T, FORM, 16, 2>(p, st);
  if (long_rows(p.C)) {
    hipLaunchKernelGGL((rms_long_kernel<T, FORM>), row_grid(p.R), dim3(256), 0, st, p);
    return hipGetLastError();
  }
  if (p.C <= S) return run_rms<T, FORM, 1, 1>(p, st);
  if (p.C <= 2 * S) return run_rms<T, FORM, 1, 2>(p, st);
  if (p.C <= 3 * S) return run_rms<T, FORM, 1, 3>(p, st);
  // bf16: four waves a row (16384 x 2048 46.5 us, by single waves 50; 4000 x 2048 with codes
  // 12.5 and 15); fp32: a wave a row
  if (p.C <= 4 * S) return run_rms<T, FORM, sizeof(T) == 2 ? 4 : 1, sizeof(T) == 2 ? 1 : 4>(p, st);
  if (p.C <= 8 * S) return run_rms<T, FORM, 4, 2>(p, st);
  if (p.C <= 12 * S) return run_rms<T, FORM, 4, 3>(p, st);
  if constexpr (sizeof(T) == 2) {   // 16 S is 8192 columns of bf16, 4096 of fp32
    return run_rms<T, FORM, 8, 2>(p, st);
  } else {
    if (p.C <= 16 * S) return run_rms<T, FORM, 4, 4>(p, st);
    if (p.C <= 24 * S) return run_rms<T, FORM, 8, 3>(p, st);
    return run_rms<T, FORM, 8, 4>(p, st);
  }
}

template <typename T, int WPR, int NIT>
hipError_t run_few(const RmsProblem& p, hipStream_t st) {
  const int64_t rows = p.dx ? (WPR == 1 ? (p.R + 3) / 4 : p.R) : 0;
  constexpr int STRIP = kStripChunks<WPR> * kVec<T>;
  const int64_t strips = p.dweight ? (p.C + STRIP - 1) / STRIP : 0;
  hipLaunchKernelGGL((rms_backward_few_kernel<T, WPR, NIT>), dim3(unsigned(rows + strips)), dim3(256), 0, st, p,
                     unsigned(rows));
  return hipGetLastError();
}

// All chunks of a lane but the last are within the row: as many as it takes, no more.
template <typename T>
hipError_t few_typed(const RmsProblem& p, hipStream_t st) {
  constexpr int64_t S = 64 * kVec<T>;
  switch (p.C <= 4 * S ? (p.C + S - 1) / S : 10 + (p.C + 4 * S - 1) / (4 * S)) {
    case 1: return run_few<T, 1, 1>(p, st);
    case 2: return run_few<T, 1, 2>(p, st);
    case 3: return run_few<T, 1, 3>(p, st);
    case 4: return run_few<T, 1, 4>(p, st);
    case 12: return run_few<T, 4, 2>(p, st);
    case 13: return run_few<T, 4, 3>(p, st);
    case 14: return run_few<T, 4, 4>(p, st);
  }
  if constexpr (sizeof(T) == 4) {        // up to 8192 columns
    switch ((p.C + 4 * S - 1) / (4 * S)) {
      case 5: return run_few<T, 4, 5>(p, st);
      case 6: return run_few<T, 4, 6>(p, st);
      case 7: return run_few<T, 4, 7>(p, st);
      case 8: return run_few<T, 4, 8>(p, st);
    }
  }
  return hipErrorInvalidValue;           // no row of kRegisterCols columns or fewer comes here
}

template <typename T, int WPR, int NIT>
hipError_t run_backward(const RmsProblem& p, int grid, float* partial, hipStream_t st) {
  const auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(64 * (WPR == 1 ? kRowWaves : WPR)), 0, st, p, partial);
    return hipGetLastError();
  };
  return streams(p, sizeof(T)) ? run(rms_backward_kernel<T, WPR, NIT, true>) : run(rms_backward_kernel<T, WPR, NIT, false>);
}

template <typename T>
hipError_t backward_typed(const RmsProblem& p, hipStream_t st) {
  constexpr int64_t S = 64 * kVec<T>;
  if (few_rows(p.R, p.C)) return few_typed<T>(p, st);
  const int grid = backward_grid(p.R, p.C, kVec<T>);
  float* partial = p.dweight ? p.workspace : nullptr;
  hipError_t e = hipSuccess;
  if (by_sixteen<T>(p.C)) {
    if constexpr (sizeof(T) == 2) e = run_backward<T, 16, 2>(p, grid, partial, st);
  } else if (long_rows(p.C)) {
    if (p.dx) {
      hipLaunchKernelGGL((rms_backward_long_kernel<T>), row_grid(p.R), dim3(256), 0, st, p);
      e = hipGetLastError();
    }
    if (e == hipSuccess && partial) {
      hipLaunchKernelGGL((rms_columns_kernel<T>), dim3(unsigned((p.C + 255) / 256), grid), dim3(256), 0, st, p,
                         partial);
      e = hipGetLastError();
    }
  } else if (p.C <= S) {
    e = run_backward<T, 1, 1>(p, grid, partial, st);
  } else if (p.C <= 2 * S) {
    e = run_backward<T, 1, 2>(p, grid, partial, st);
  } else if (p.C <= 3 * S) {
    e = run_backward<T, 1, 3>(p, grid, partial, st);
  } else if (p.C <= 4 * S) {
    e = run_backward<T, 1, 4>(p, grid, partial, st);
  } else if (p.C <= 8 * S) {
    e = run_backward<T, 4, 2>(p, grid, partial, st);
  } else if (p.C <= 16 * S) {
    e = run_backward<T, 8, 2>(p, grid, partial, st);
  } else if constexpr (sizeof(T) == 4) {
    e = p.C <= 24 * S ? run_backward<T, 8, 3>(p, grid, partial, st) : run_backward<T, 8, 4>(p, grid, partial, st);
  }
  if (e != hipSuccess || !partial) return e;
  hipLaunchKernelGGL(rms_column_sum_kernel, dim3(unsigned((p.C + 63) / 64)), dim3(1024), 0, st, partial, grid, p.C,
                     p.dweight, p.param_fp32);
  return hipGetLastError();
}

}  // namespace

int64_t rms_backward_workspace(int64_t R, int64_t C) {
  if (few_rows(R, C)) return 0;
  const int64_t n = R < kBackwardGrid ? R : kBackwardGrid;
  return n * C * int64_t(sizeof(float));
}

hipError_t launch_rms_norm(const RmsProblem& p, hipStream_t st) {
  if (p.R == 0) return hipSuccess;
  if (p.fp32) return rms_typed<float, ROWS>(p, st);
  if (!p.q) return rms_typed<uint16_t, ROWS>(p, st);
  return p.rowwise ? rms_typed<uint16_t, WHOLE>(p, st) : rms_typed<uint16_t, BLOCKS>(p, st);
}

hipError_t launch_rms_norm_backward(const RmsProblem& p, hipStream_t st) {
  // no rows: rms_column_sum_kernel over no partial rows writes the zero gradient
  if (p.R == 0) {
    if (!p.dweight) return hipSuccess;
    hipLaunchKernelGGL(rms_column_sum_kernel, dim3(unsigned((p.C + 63) / 64)), dim3(1024), 0, st, nullptr, 0, p.C,
                       p.dweight, p.param_fp32);
    return hipGetLastError();
  }
  return p.fp32 ? backward_typed<float>(p, st) : backward_typed<uint16_t>(p, st);
}

}  // namespace fp8mm
