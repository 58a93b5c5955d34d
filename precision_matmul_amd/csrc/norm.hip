// Layer norm over the last dimension, forward and backward (gfx950).
//
//   mean = sum(x) / C,  var = sum((x - mean)^2) / C,  rstd = 1 / sqrt(var + eps)
//   y  = (x - mean) rstd w + b
//   xh = (x - mean) rstd,  a = dy w
//   dx = rstd (a - sum(a) / C - xh sum(a xh) / C)
//   dw = sum over rows of dy xh,   db = sum over rows of dy
//
// HBM-bound: x (and dy) read once, y (dx) written once.  A row stays in
// registers, as loaded, between its statistics and its output, so the
// variance is the sum of centred squares (two passes over registers, not the
// difference of two large sums).  All sums are float32.
//
// Lanes past a row's end hold x = dy = 0.  The sum of a xh is rstd times the sum of
// a (x - mean), which is 0 there; (x - mean) rstd alone can pass float32's range (a
// row of one large value under a small eps), and 0 times that is NaN.
#include "moe_launch.hpp"
#include "ops_common.hpp"

namespace fp8mm {
namespace {

using namespace ops;

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

// ---------------------------------------------------------------------------
// Forward, row in registers: WPR waves a row, NIT chunks a lane.  A workgroup
// takes rows blockIdx, blockIdx + gridDim, ...; a lane's columns are the same
// in all of them, so it keeps its parameters in registers, and the next row is
// loaded while this one is reduced and written.  Results larger than the L2s
// are read and written by streaming accesses (NT).  16640 x 5120 bf16: 60 us,
// 5.6 TB/s, more than a plain copy reaches.  In us, the other choice in brackets:
//   streaming: 16640 x 5120 60 (plain 66), but where the inputs come from the 256
//   MiB cache of the memory it costs: 9830 x 5120 (96 MiB) 37 (35.5), 16384 x 2048
//   (64 MiB) 32 (25), 8192 x 2048 (32 MiB) 19 (16)
//   eight waves a row above 12 chunks of a wave (16 of fp32): 10000 x 8192 bf16 56
//   (four: 62), 4096 x 4764 fp32 30 (38); 16640 x 5120 60 with four (66)
//   PART where rows end within a chunk and, for results larger than the L2s, at
//   eight waves: 6000 x 6144 fp32 50 (54); four waves 16000 x 5128 bf16 62 without
//   (65); within the L2s 900 x 8192 fp32 14 without (16)
// ---------------------------------------------------------------------------
template <typename T, typename P, int WPR, int NIT, bool NT, bool PART>
__global__ __launch_bounds__(WPR == 8 ? 512 : 256) void norm_kernel(
    const T* __restrict__ x, int64_t R, int64_t C, int64_t ld_x, const P* __restrict__ weight,
    const P* __restrict__ bias, float eps, T* __restrict__ y, int64_t ld_y, float* __restrict__ mean_out,
    float* __restrict__ rstd_out) {
  constexpr int V = kVec<T>;
  constexpr int RPB = WPR == 1 ? 4 : 1;           // rows of a workgroup
  __shared__ float part[2][WPR];
  const int in_row = WPR == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int64_t c0 = int64_t(in_row) * V;
  constexpr int64_t STEP = int64_t(WPR) * 64 * V;
  Params<P, V> w[NIT], b[NIT];
#pragma unroll
  for (int it = 0; it < NIT; ++it) {
    w[it].load(weight, c0 + it * STEP, C, 1.0f);
    b[it].load(bias, c0 + it * STEP, C, 0.0f);
  }
  const int64_t stride = int64_t(gridDim.x) * RPB;
  int64_t row = int64_t(blockIdx.x) * RPB + (WPR == 1 ? threadIdx.x >> 6 : 0);
  Chunk next[NIT];
#pragma unroll
  for (int it = 0; it < NIT; ++it)
    if (row < R) next[it] = fetch<T, NT, PART>(x + row * ld_x, c0 + it * STEP, C);
  for (; row < R; row += stride) {                // all waves of a row take the same turns
    Chunk v[NIT];
#pragma unroll
    for (int it = 0; it < NIT; ++it) v[it] = settle<T, PART>(next[it], c0 + it * STEP, C);
    if (row + stride < R) {
#pragma unroll
      for (int it = 0; it < NIT; ++it) next[it] = fetch<T, NT, PART>(x + (row + stride) * ld_x, c0 + it * STEP, C);
    }
    float s = 0.0f;
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
      float f[V];
      unpack<T>(v[it], f);
#pragma unroll
      for (int i = 0; i < V; ++i) s += f[i];
    }
    const float mean = row_sum<WPR>(s, part, 0) / float(C);
    float ss = 0.0f;
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
      const int64_t c = c0 + it * STEP;
      float f[V];
      unpack<T>(v[it], f);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = f[i] - mean;
        ss += c + i < C ? d * d : 0.0f;
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum<WPR>(ss, part, 1) / float(C) + eps);
    if (in_row == 0) {
      if (mean_out) mean_out[row] = mean;
      if (rstd_out) rstd_out[row] = rstd;
    }
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
      float f[V];
      unpack<T>(v[it], f);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = (f[i] - mean) * rstd * w[it][i] + b[it][i];
      store_row<T, NT>(y + row * ld_y, c0 + it * STEP, C, pack<T>(f));
    }
  }
}

// Forward, rows too long for registers: one workgroup a row, the row read
// three times (from L2 after the first).
template <typename T, typename P>
__global__ __launch_bounds__(256) void norm_long_kernel(const T* __restrict__ x, int64_t R, int64_t C, int64_t ld_x,
                                                        const P* __restrict__ weight, const P* __restrict__ bias,
                                                        float eps, T* __restrict__ y, int64_t ld_y,
                                                        float* __restrict__ mean_out, float* __restrict__ rstd_out) {
  constexpr int V = kVec<T>;
  __shared__ float part[2][4];
  for (int64_t row = blockIdx.x; row < R; row += gridDim.x) {
    const T* xr = x + row * ld_x;
    float s = 0.0f;
    for (int64_t c = int64_t(threadIdx.x) * V; c < C; c += 256 * V) {
      float f[V];
      unpack<T>(load_row(xr, c, C), f);
#pragma unroll
      for (int i = 0; i < V; ++i) s += f[i];
    }
    const float mean = row_sum<4>(s, part, 0) / float(C);
    float ss = 0.0f;
    for (int64_t c = int64_t(threadIdx.x) * V; c < C; c += 256 * V) {
      float f[V];
      unpack<T>(load_row(xr, c, C), f);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = f[i] - mean;
        ss += c + i < C ? d * d : 0.0f;
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum<4>(ss, part, 1) / float(C) + eps);
    if (threadIdx.x == 0) {
      if (mean_out) mean_out[row] = mean;
      if (rstd_out) rstd_out[row] = rstd;
    }
    for (int64_t c = int64_t(threadIdx.x) * V; c < C; c += 256 * V) {
      float f[V];
      Params<P, V> w, b;
      unpack<T>(load_row(xr, c, C), f);
      w.load(weight, c, C, 1.0f);
      b.load(bias, c, C, 0.0f);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = (f[i] - mean) * rstd * w[i] + b[i];
      store_row(y + row * ld_y, c, C, pack<T>(f));
    }
  }
}

// ---------------------------------------------------------------------------
// Backward, row in registers.  A workgroup takes rows in turns like the
// forward's, the next row in flight while this one is worked on, and keeps its
// share of dw and db in registers over all of them; it then writes one partial
// row of the workspace, [2][gridDim][C], which column_sum_kernel adds up in
// workgroup order: no atomics, the same bits every time.  The partial rows are
// traffic of their own (8 gridDim C bytes each way), so there are no more
// workgroups than run at once: 256 of eight waves, with a row each (rows of at most
// 4 chunks of a wave) or sharing one (above 8), and 512 of four waves that share a
// row in between (256 below 2048 rows, where a partial row would stand for one or
// two rows).  16384 x 2048 bf16: 41 us with the column sums, 4.9 TB/s of x, dy and
// dx.  In us, the other choice in brackets:
//   partial rows: 16384 x 2048 41 (512: 55), 16000 x 4096 77 (1024: 93)
//   eight waves a row: 16000 x 6144 101 (four: 106), 2841 x 5127 27 (30), 6000 x
//   6144 fp32 78 (103)
//   PART, wherever rows are shared and stream or end within a chunk: 16000 x 3000
//   62 (85), 16000 x 2056 49 (75), 7534 x 3559 48 (84); within the L2s it costs:
//   1703 x 3000 fp32 22.5 (25 with it)
// Streaming accesses pay above 32 MiB of rows that share waves (4096 x 5120 bf16, 40
// MiB: 32 against 38; 16384 x 2048, 64 MiB: 42.5 against 41) and cost below (3276 x
// 5120, 32 MiB: 28.4 against 27.9; 8192 x 2048 27.0 against 24.2).
// ---------------------------------------------------------------------------
constexpr int kRowWaves = 8;            // waves of a workgroup that takes a row with each

template <typename T, typename P, int WPR, int NIT, bool NT, bool PART>
__global__ __launch_bounds__(64 * (WPR == 1 ? kRowWaves : WPR)) void norm_backward_kernel(
    const T* __restrict__ dy, int64_t ld_dy, const T* __restrict__ x, int64_t ld_x, int64_t R, int64_t C,
    const P* __restrict__ weight, const float* __restrict__ mean_in, const float* __restrict__ rstd_in,
    T* __restrict__ dx, int64_t ld_dx, float* __restrict__ partial) {
  constexpr int V = kVec<T>;
  constexpr int RPB = WPR == 1 ? kRowWaves : 1;
  constexpr int64_t STEP = int64_t(WPR) * 64 * V;
  __shared__ float part[2][2][WPR];
  constexpr int Q = 2 * NIT * V / 4;              // a lane's sums, in fours
  __shared__ float4 acc[WPR == 1 ? kRowWaves / 2 * Q * 64 : 1];
  const int wave = threadIdx.x >> 6;
  const int64_t c0 = int64_t(WPR == 1 ? threadIdx.x & 63 : threadIdx.x) * V;
  const float inv_c = 1.0f / float(C);
  float dw[NIT][V], db[NIT][V];
#pragma unroll
  for (int it = 0; it < NIT; ++it)
#pragma unroll
    for (int i = 0; i < V; ++i) dw[it][i] = db[it][i] = 0.0f;
  Params<P, V> w[NIT];
#pragma unroll
  for (int it = 0; it < NIT; ++it) w[it].load(weight, c0 + it * STEP, C, 1.0f);
  int slot = 0;
  const int64_t stride = int64_t(gridDim.x) * RPB;
  int64_t row = int64_t(blockIdx.x) * RPB + (WPR == 1 ? wave : 0);
  Chunk nx[NIT], ng[NIT];
  float nmean = 0.0f, nrstd = 0.0f;
  if (row < R) {
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
      nx[it] = fetch<T, NT, PART>(x + row * ld_x, c0 + it * STEP, C);
      ng[it] = fetch<T, NT, PART>(dy + row * ld_dy, c0 + it * STEP, C);
    }
    nmean = mean_in[row];
    nrstd = rstd_in[row];
  }
  for (; row < R; row += stride) {
    Chunk vx[NIT], vg[NIT];
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
      vx[it] = settle<T, PART>(nx[it], c0 + it * STEP, C);
      vg[it] = settle<T, PART>(ng[it], c0 + it * STEP, C);
    }
    const float mean = nmean, rstd = nrstd;
    if (row + stride < R) {
#pragma unroll
      for (int it = 0; it < NIT; ++it) {
        nx[it] = fetch<T, NT, PART>(x + (row + stride) * ld_x, c0 + it * STEP, C);
        ng[it] = fetch<T, NT, PART>(dy + (row + stride) * ld_dy, c0 + it * STEP, C);
      }
      nmean = mean_in[row + stride];
      nrstd = rstd_in[row + stride];
    }
    float sa = 0.0f, sax = 0.0f;
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
      float f[V], g[V];
      unpack<T>(vx[it], f);
      unpack<T>(vg[it], g);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float t = f[i] - mean;
        const float a = g[i] * w[it][i];
        sa += a;
        sax += a * t;                             // 0 past the row's end
        dw[it][i] += g[i] * (t * rstd);
        db[it][i] += g[i];
      }
    }
    sa = wave_sum(sa);
    sax = wave_sum(sax);
    if constexpr (WPR > 1) {
      if ((threadIdx.x & 63) == 0) {
        part[slot][0][wave] = sa;
        part[slot][1][wave] = sax;
      }
      __syncthreads();
      sa = sax = 0.0f;
#pragma unroll
      for (int w = 0; w < WPR; ++w) {
        sa += part[slot][0][w];
        sax += part[slot][1][w];
      }
      slot ^= 1;
    }
    sa *= inv_c;
    sax *= rstd * inv_c;
    if (dx) {
#pragma unroll
      for (int it = 0; it < NIT; ++it) {
        float f[V], g[V];
        unpack<T>(vx[it], f);
        unpack<T>(vg[it], g);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float xh = (f[i] - mean) * rstd;
          f[i] = rstd * (g[i] * w[it][i] - sa - xh * sax);
        }
        store_row<T, NT>(dx + row * ld_dx, c0 + it * STEP, C, pack<T>(f));
      }
    }
  }
  if (!partial) return;
  float* pw = partial + int64_t(blockIdx.x) * C;
  float* pb = pw + int64_t(gridDim.x) * C;
  if constexpr (WPR == 1) {
    // the waves' shares, halved three times: the upper half's waves hand theirs
    // to the lower half's
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int half = kRowWaves / 2; half >= 1; half >>= 1) {
      if (wave >= half && wave < 2 * half) {
#pragma unroll
        for (int q = 0; q < Q / 2; ++q) {
          const int it = q * 4 / V, i = q * 4 % V;
          float4* at = acc + (wave - half) * Q * 64 + lane;
          at[q * 64] = make_float4(dw[it][i], dw[it][i + 1], dw[it][i + 2], dw[it][i + 3]);
          at[(Q / 2 + q) * 64] = make_float4(db[it][i], db[it][i + 1], db[it][i + 2], db[it][i + 3]);
        }
      }
      __syncthreads();
      if (wave < half) {
#pragma unroll
        for (int q = 0; q < Q / 2; ++q) {
          const int it = q * 4 / V, i = q * 4 % V;
          const float4* at = acc + wave * Q * 64 + lane;
          const float4 a = at[q * 64], b = at[(Q / 2 + q) * 64];
          dw[it][i] += a.x, dw[it][i + 1] += a.y, dw[it][i + 2] += a.z, dw[it][i + 3] += a.w;
          db[it][i] += b.x, db[it][i + 1] += b.y, db[it][i + 2] += b.z, db[it][i + 3] += b.w;
        }
      }
      __syncthreads();
    }
    if (wave != 0) return;
  }
#pragma unroll
  for (int it = 0; it < NIT; ++it)
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      store_row(pw, c0 + it * STEP + i, C, pack4f(&dw[it][i]));
      store_row(pb, c0 + it * STEP + i, C, pack4f(&db[it][i]));
    }
}

// ---------------------------------------------------------------------------
// Backward of few rows in one launch and without a workspace.  dw and db need
// no row sums (mean and rstd are inputs), so the first row_blocks workgroups
// write dx, a row a wave (WPR = 1) or a workgroup, and the others each add up a
// strip of columns over all rows, 64 (WPR = 1) or 16 row slices of it, the slices
// added in a fixed order.  x and dy come from HBM once and from the L2s the second
// time.  500 x 8192 bf16: 11.5 us against 21.9 in two launches, 455 x 195 10.8
// against 14.6 (the host's part of a call; 23 with strips of 16 chunks); from 1000
// rows on the two launches are the faster form (1000 x 300 14 against 20 us).
// ---------------------------------------------------------------------------
// Chunks of columns of a strip: narrow where rows are short, so that there are
// enough strips.
template <int WPR>
constexpr int kStripChunks = WPR == 1 ? 4 : 16;

template <typename T, typename P, int WPR, int NIT>
__global__ __launch_bounds__(256) void norm_backward_few_kernel(
    const T* __restrict__ dy, int64_t ld_dy, const T* __restrict__ x, int64_t ld_x, int64_t R, int64_t C,
    const P* __restrict__ weight, const float* __restrict__ mean_in, const float* __restrict__ rstd_in,
    T* __restrict__ dx, int64_t ld_dx, P* __restrict__ dweight, P* __restrict__ dbias, unsigned row_blocks) {
  constexpr int V = kVec<T>;
  constexpr int CL = kStripChunks<WPR>, SLICES = 256 / CL;
  __shared__ float part[2][SLICES][CL * V];
  if (blockIdx.x < row_blocks) {
    constexpr int64_t STEP = int64_t(WPR) * 64 * V;
    const int64_t row = WPR == 1 ? int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6) : blockIdx.x;
    if (row >= R) return;                       // WPR = 1: waves of their own; else never
    const int64_t c0 = int64_t(WPR == 1 ? threadIdx.x & 63 : threadIdx.x) * V;
    Chunk vx[NIT], vg[NIT];
    Params<P, V> w[NIT];
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
      vx[it] = load_row(x + row * ld_x, c0 + it * STEP, C);
      vg[it] = load_row(dy + row * ld_dy, c0 + it * STEP, C);
      w[it].load(weight, c0 + it * STEP, C, 1.0f);
    }
    const float mean = mean_in[row], rstd = rstd_in[row];
    float sa = 0.0f, sax = 0.0f;
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
      float f[V], g[V];
      unpack<T>(vx[it], f);
      unpack<T>(vg[it], g);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float a = g[i] * w[it][i];
        sa += a;
        sax += a * (f[i] - mean);                 // 0 past the row's end
      }
    }
    sa = wave_sum(sa);
    sax = wave_sum(sax);
    if constexpr (WPR > 1) {
      const int wave = threadIdx.x >> 6;
      if ((threadIdx.x & 63) == 0) {
        part[0][0][wave] = sa;
        part[1][0][wave] = sax;
      }
      __syncthreads();
      sa = part[0][0][0] + part[0][0][1] + part[0][0][2] + part[0][0][3];
      sax = part[1][0][0] + part[1][0][1] + part[1][0][2] + part[1][0][3];
    }
    sa /= float(C);
    sax = sax * rstd / float(C);
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
      float f[V], g[V];
      unpack<T>(vx[it], f);
      unpack<T>(vg[it], g);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = rstd * (g[i] * w[it][i] - sa - (f[i] - mean) * rstd * sax);
      store_row(dx + row * ld_dx, c0 + it * STEP, C, pack<T>(f));
    }
    return;
  }
  const int chunk = threadIdx.x % CL, slice = threadIdx.x / CL;
  const int64_t strip = int64_t(blockIdx.x - row_blocks) * CL * V;
  const int64_t c = strip + chunk * V;
  float dw[V], db[V];
#pragma unroll
  for (int i = 0; i < V; ++i) dw[i] = db[i] = 0.0f;
#pragma unroll 4
  for (int64_t row = slice; row < R; row += SLICES) {
    float f[V], g[V];
    unpack<T>(load_row(x + row * ld_x, c, C), f);
    unpack<T>(load_row(dy + row * ld_dy, c, C), g);
    const float mean = mean_in[row], rstd = rstd_in[row];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      dw[i] += g[i] * ((f[i] - mean) * rstd);
      db[i] += g[i];
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    part[0][slice][chunk * V + i] = dw[i];
    part[1][slice][chunk * V + i] = db[i];
  }
  __syncthreads();
  // SHARE neighbouring threads add up a column's slices
  constexpr int SHARE = 256 / (2 * CL * V);
  static_assert(SHARE >= 1 && SHARE <= SLICES && (SHARE & (SHARE - 1)) == 0, "a column or more for each thread");
  const int column = threadIdx.x / SHARE, share = threadIdx.x % SHARE;
  const int which = column / (CL * V), col = column - which * CL * V;
  float s = 0.0f;
#pragma unroll 16
  for (int r = share; r < SLICES; r += SHARE) s += part[which][r][col];
#pragma unroll
  for (int off = 1; off < SHARE; off <<= 1) s += __shfl_xor(s, off, 64);
  P* out = which ? dbias : dweight;
  if (share == 0 && out && strip + col < C) out[strip + col] = from_float<P>(s);
}

// Backward of rows too long for registers: dx by one workgroup a row ...
template <typename T, typename P>
__global__ __launch_bounds__(256) void norm_backward_long_kernel(
    const T* __restrict__ dy, int64_t ld_dy, const T* __restrict__ x, int64_t ld_x, int64_t R, int64_t C,
    const P* __restrict__ weight, const float* __restrict__ mean_in, const float* __restrict__ rstd_in,
    T* __restrict__ dx, int64_t ld_dx) {
  constexpr int V = kVec<T>;
  __shared__ float part[2][4];
  for (int64_t row = blockIdx.x; row < R; row += gridDim.x) {
    const float mean = mean_in[row], rstd = rstd_in[row];
    float sa = 0.0f, sax = 0.0f;
    for (int64_t c = int64_t(threadIdx.x) * V; c < C; c += 256 * V) {
      float f[V], g[V];
      Params<P, V> w;
      unpack<T>(load_row(x + row * ld_x, c, C), f);
      unpack<T>(load_row(dy + row * ld_dy, c, C), g);
      w.load(weight, c, C, 1.0f);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        sa += g[i] * w[i];
        sax += g[i] * w[i] * (f[i] - mean);       // 0 past the row's end
      }
    }
    sa = row_sum<4>(sa, part, 0) / float(C);
    sax = row_sum<4>(sax, part, 1) * rstd / float(C);
    for (int64_t c = int64_t(threadIdx.x) * V; c < C; c += 256 * V) {
      float f[V], g[V];
      Params<P, V> w;
      unpack<T>(load_row(x + row * ld_x, c, C), f);
      unpack<T>(load_row(dy + row * ld_dy, c, C), g);
      w.load(weight, c, C, 1.0f);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = rstd * (g[i] * w[i] - sa - (f[i] - mean) * rstd * sax);
      store_row(dx + row * ld_dx, c, C, pack<T>(f));
    }
  }
}

// ... and the columns' partial sums over rows blockIdx.y, blockIdx.y +
// gridDim.y, ... by one thread a column.
template <typename T>
__global__ __launch_bounds__(256) void norm_columns_kernel(const T* __restrict__ dy, int64_t ld_dy,
                                                           const T* __restrict__ x, int64_t ld_x, int64_t R, int64_t C,
                                                           const float* __restrict__ mean_in,
                                                           const float* __restrict__ rstd_in,
                                                           float* __restrict__ partial) {
  const int64_t c = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (c >= C) return;
  float dw = 0.0f, db = 0.0f;
  for (int64_t row = blockIdx.y; row < R; row += gridDim.y) {
    const float g = to_float(dy[row * ld_dy + c]);
    dw += g * ((to_float(x[row * ld_x + c]) - mean_in[row]) * rstd_in[row]);
    db += g;
  }
  partial[int64_t(blockIdx.y) * C + c] = dw;
  partial[(int64_t(gridDim.y) + blockIdx.y) * C + c] = db;
}

// Sums the n partial rows of dw (blockIdx.y 0) or db (1): 64 columns and 16
// row slices a workgroup, the slices added in order.
template <typename P>
__global__ __launch_bounds__(1024) void column_sum_kernel(const float* __restrict__ partial, int n, int64_t C,
                                                          P* __restrict__ dweight, P* __restrict__ dbias) {
  __shared__ float part[16][64];
  P* out = blockIdx.y ? dbias : dweight;
  if (!out) return;
  const float* p = partial + int64_t(blockIdx.y) * n * C;
  const int lane = threadIdx.x & 63, slice = threadIdx.x >> 6;
  const int64_t c = int64_t(blockIdx.x) * 64 + lane;
  float s = 0.0f;
  if (c < C) {
#pragma unroll 8
    for (int r = slice; r < n; r += 16) s += p[int64_t(r) * C + c];
  }
  part[slice][lane] = s;
  __syncthreads();
  if (slice == 0 && c < C) {
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += part[i][lane];
    out[c] = from_float<P>(s);
  }
}

constexpr int64_t kForwardGrid = 1024;  // four workgroups a compute unit
constexpr int kBackwardGrid = 512;      // partial rows at most
constexpr int64_t kRegisterCols = 8192; // longest row kept in registers
constexpr int64_t kFewRows = 512;       // rows at most of the backward in one launch

bool few_rows(int64_t R, int64_t C) { return R <= kFewRows && C <= kRegisterCols; }

// Workgroups of the row kernels, which take further rows in turns past this.
dim3 row_grid(int64_t blocks) { return dim3(unsigned(blocks < (1 << 20) ? blocks : (1 << 20))); }

bool streams(const NormProblem& p, size_t size) { return p.R * p.C * int64_t(size) > kL2Bytes; }

// Workgroups of the backward (one partial row each): as many as run at once.
int backward_grid(int64_t R, int64_t C, int vec) {
  const int64_t one_wave = 256 * vec;         // rows of up to this many columns: a wave each
  const int64_t rows = C <= one_wave ? kRowWaves : 1;
  const int64_t most = C <= one_wave || C > 2 * one_wave || R < 2048 ? 256 : 512;
  const int64_t blocks = (R + rows - 1) / rows;
  return int(blocks < most ? blocks : most);
}

template <typename T, typename P, int WPR, int NIT>
hipError_t run_norm(const NormProblem& p, hipStream_t st) {
  constexpr int RPB = WPR == 1 ? 4 : 1;
  const int64_t blocks = (p.R + RPB - 1) / RPB;
  const dim3 grid(unsigned(blocks < kForwardGrid ? blocks : kForwardGrid));
  const auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(WPR == 8 ? 512 : 256), 0, st, static_cast<const T*>(p.x), p.R, p.C,
                       p.ld_x, static_cast<const P*>(p.weight), static_cast<const P*>(p.bias), p.eps,
                       static_cast<T*>(p.out), p.ld_out, p.mean, p.rstd);
    return hipGetLastError();
  };
  constexpr bool MANY = WPR > 1;
  const bool part = MANY && p.C % kVec<T> != 0;
  if (streams(p, sizeof(T)))
    return part || WPR == 8 ? run(norm_kernel<T, P, WPR, NIT, true, MANY>)
                            : run(norm_kernel<T, P, WPR, NIT, true, false>);
  return part ? run(norm_kernel<T, P, WPR, NIT, false, MANY>) : run(norm_kernel<T, P, WPR, NIT, false, false>);
}

template <typename T, typename P>
hipError_t norm_typed(const NormProblem& p, hipStream_t st) {
  constexpr int64_t S = 64 * kVec<T>;   // columns of one wave chunk
  if (p.C <= S) return run_norm<T, P, 1, 1>(p, st);
  if (p.C <= 2 * S) return run_norm<T, P, 1, 2>(p, st);
  if (p.C <= 4 * S) return run_norm<T, P, 1, 4>(p, st);
  if (p.C <= 8 * S) return run_norm<T, P, 4, 2>(p, st);
  if (p.C <= 12 * S) return run_norm<T, P, 4, 3>(p, st);
  if constexpr (sizeof(T) == 2) {   // 16 S is 8192 columns of bf16, 4096 of fp32
    if (p.C <= 16 * S) return run_norm<T, P, 8, 2>(p, st);
  } else {
    if (p.C <= 16 * S) return run_norm<T, P, 4, 4>(p, st);
    if (p.C <= 24 * S) return run_norm<T, P, 8, 3>(p, st);
    if (p.C <= 32 * S) return run_norm<T, P, 8, 4>(p, st);
  }
  hipLaunchKernelGGL((norm_long_kernel<T, P>), row_grid(p.R), dim3(256), 0, st, static_cast<const T*>(p.x), p.R,
                     p.C, p.ld_x, static_cast<const P*>(p.weight), static_cast<const P*>(p.bias), p.eps,
                     static_cast<T*>(p.out), p.ld_out, p.mean, p.rstd);
  return hipGetLastError();
}

template <typename T, typename P, int WPR, int NIT>
hipError_t run_backward(const NormProblem& p, int grid, float* partial, hipStream_t st) {
  if (few_rows(p.R, p.C)) {
    const int64_t rows = p.out ? (WPR == 1 ? (p.R + 3) / 4 : p.R) : 0;
    constexpr int W = WPR == 1 ? 1 : 4, STRIP = kStripChunks<W> * kVec<T>;
    const int64_t strips = p.dweight || p.dbias ? (p.C + STRIP - 1) / STRIP : 0;
    hipLaunchKernelGGL((norm_backward_few_kernel<T, P, W, NIT * WPR / W>), dim3(unsigned(rows + strips)), dim3(256), 0,
                       st, static_cast<const T*>(p.dy), p.ld_dy, static_cast<const T*>(p.x), p.ld_x, p.R, p.C,
                       static_cast<const P*>(p.weight), p.mean, p.rstd, static_cast<T*>(p.out), p.ld_out,
                       static_cast<P*>(p.dweight), static_cast<P*>(p.dbias), unsigned(rows));
    return hipGetLastError();
  }
  const auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(64 * (WPR == 1 ? kRowWaves : WPR)), 0, st,
                       static_cast<const T*>(p.dy), p.ld_dy, static_cast<const T*>(p.x), p.ld_x, p.R, p.C,
                       static_cast<const P*>(p.weight), p.mean, p.rstd, static_cast<T*>(p.out), p.ld_out, partial);
    return hipGetLastError();
  };
  constexpr bool MANY = WPR > 1;
  if (streams(p, sizeof(T))) return run(norm_backward_kernel<T, P, WPR, NIT, true, MANY>);
  return MANY && p.C % kVec<T> != 0 ? run(norm_backward_kernel<T, P, WPR, NIT, false, MANY>)
                                    : run(norm_backward_kernel<T, P, WPR, NIT, false, false>);
}

template <typename T, typename P>
hipError_t backward_typed(const NormProblem& p, hipStream_t st) {
  constexpr int64_t S = 64 * kVec<T>;
  const int grid = backward_grid(p.R, p.C, kVec<T>);
  float* partial = (p.dweight || p.dbias) && !few_rows(p.R, p.C) ? p.workspace : nullptr;
  hipError_t e = hipSuccess;
  if (p.C <= S) {
    e = run_backward<T, P, 1, 1>(p, grid, partial, st);
  } else if (p.C <= 2 * S) {
    e = run_backward<T, P, 1, 2>(p, grid, partial, st);
  } else if (p.C <= 4 * S) {
    e = run_backward<T, P, 1, 4>(p, grid, partial, st);
  } else if (p.C <= 8 * S) {
    e = run_backward<T, P, 4, 2>(p, grid, partial, st);
  } else if (p.C <= 16 * S) {
    e = run_backward<T, P, 8, 2>(p, grid, partial, st);
  } else if (sizeof(T) == 4 && p.C <= kRegisterCols) {
    if constexpr (sizeof(T) == 4)
      e = p.C <= 24 * S ? run_backward<T, P, 8, 3>(p, grid, partial, st)
                        : run_backward<T, P, 8, 4>(p, grid, partial, st);
  } else {
    if (p.out) {
      hipLaunchKernelGGL((norm_backward_long_kernel<T, P>), row_grid(p.R), dim3(256), 0, st,
                         static_cast<const T*>(p.dy), p.ld_dy, static_cast<const T*>(p.x), p.ld_x, p.R, p.C,
                         static_cast<const P*>(p.weight), p.mean, p.rstd, static_cast<T*>(p.out), p.ld_out);
      e = hipGetLastError();
    }
    if (e == hipSuccess && partial) {
      hipLaunchKernelGGL((norm_columns_kernel<T>), dim3(unsigned((p.C + 255) / 256), grid), dim3(256), 0, st,
                         static_cast<const T*>(p.dy), p.ld_dy, static_cast<const T*>(p.x), p.ld_x, p.R, p.C, p.mean,
                         p.rstd, partial);
      e = hipGetLastError();
    }
  }
  if (e != hipSuccess || !partial) return e;
  hipLaunchKernelGGL((column_sum_kernel<P>), dim3(unsigned((p.C + 63) / 64), 2), dim3(1024), 0, st, partial, grid, p.C,
                     static_cast<P*>(p.dweight), static_cast<P*>(p.dbias));
  return hipGetLastError();
}

}  // namespace

int64_t norm_backward_workspace(int64_t R, int64_t C) {
  if (few_rows(R, C)) return 0;
  const int64_t n = R < kBackwardGrid ? R : kBackwardGrid;
  return 2 * n * C * int64_t(sizeof(float));
}

hipError_t launch_norm(const NormProblem& p, hipStream_t st) {
  if (p.R == 0) return hipSuccess;
  if (p.fp32)
    return p.param_fp32 ? norm_typed<float, float>(p, st) : norm_typed<float, uint16_t>(p, st);
  return p.param_fp32 ? norm_typed<uint16_t, float>(p, st) : norm_typed<uint16_t, uint16_t>(p, st);
}

hipError_t launch_norm_backward(const NormProblem& p, hipStream_t st) {
  // no rows: column_sum_kernel over no partial rows writes the zero gradients
  if (p.R == 0) {
    if (!p.dweight && !p.dbias) return hipSuccess;
    const dim3 grid(unsigned((p.C + 63) / 64), 2);
    if (p.param_fp32)
      hipLaunchKernelGGL((column_sum_kernel<float>), grid, dim3(1024), 0, st, nullptr, 0, p.C,
                         static_cast<float*>(p.dweight), static_cast<float*>(p.dbias));
    else
      hipLaunchKernelGGL((column_sum_kernel<uint16_t>), grid, dim3(1024), 0, st, nullptr, 0, p.C,
                         static_cast<uint16_t*>(p.dweight), static_cast<uint16_t*>(p.dbias));
    return hipGetLastError();
  }
  if (p.fp32)
    return p.param_fp32 ? backward_typed<float, float>(p, st) : backward_typed<float, uint16_t>(p, st);
  return p.param_fp32 ? backward_typed<uint16_t, float>(p, st) : backward_typed<uint16_t, uint16_t>(p, st);
}

}  // namespace fp8mm
