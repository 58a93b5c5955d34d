// Balance loss of a router over packed sequences, with the experts' counts, and its
// gradient (gfx950).
//
//   p = softmax(x), or sigmoid(x) / sum sigmoid(x), of a token's logits
//   n = the sequence's tokens, c_e = their slots with expert e
//   loss = coeff / S' sum over sequences of sum_e (E c_e / (k n)) (sum_t p_te / n)
//   d_e = grad coeff E c_e / (S' k n^2);  dx_e = p_e (d_e - sum_j p_j d_j), for the
//   sigmoid times 1 - sigmoid(x_e)
//
// HBM-bound in principle (the logits read once, their gradient written once), in
// practice a few launches: 16384 x 64 float32 logits are 4 MiB.  The forward needs
// sums over all tokens of a sequence, so it is a pass over the tokens that leaves
// partial sums and a sum over those.  Chunk b of the tokens and sequence s meet in at
// most one run of tokens, and as b and s only grow from run to run, b + s names it:
// its partial row of the workspace, written once, with no search and no atomics.
//
// d_e - sum_j p_j d_j is built from differences of whole counts, c_e - c_r with r the
// token's most probable expert: where p_r is nearly 1, the plain difference would be
// the rounding of two nearly equal numbers.  The sigmoid's scores carry a factor
// exp(-min(max x, 0)) that the normalisation takes out again, so that tokens whose
// scores are all below float32's range have their probabilities too.
#include "block_launch.hpp"
#include "ops_common.hpp"

namespace fp8mm {
namespace {

using namespace ops;

constexpr int kThreads = 256;

// exp(x) for x <= 0: exp2 corrected by the rounding of its argument; 0 below 2^-150.
__device__ __forceinline__ float exp_down(float x) {
  const float t = x * 1.44269504f, e = __builtin_amdgcn_exp2f(t);
  const float rest = fmaf(x, 1.44269504f, -t) + x * 1.92596299e-8f;
  return x < -104.0f ? 0.0f : fmaf(e, rest * 0.693147182f, e);
}

// Four logits at column c of E; -inf past the end.
template <typename T>
__device__ __forceinline__ void load4(const T* row, int c, int E, float (&f)[4]) {
  if (c + 4 <= E) {
    struct __attribute__((packed, aligned(sizeof(T)))) At {
      T v[4];
    };
    const At a = *reinterpret_cast<const At*>(row + c);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = to_float(a.v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = c + i < E ? to_float(row[c + i]) : -__builtin_inff();
  }
}

template <typename T>
__device__ __forceinline__ void store4(T* row, int c, int E, const float (&f)[4]) {
  if (c + 4 <= E) {
    struct __attribute__((packed, aligned(sizeof(T)))) At {
      T v[4];
    };
    *reinterpret_cast<At*>(row + c) =
        At{{from_float<T>(f[0]), from_float<T>(f[1]), from_float<T>(f[2]), from_float<T>(f[3])}};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < E) row[c + i] = from_float<T>(f[i]);
  }
}

// Sum and maximum over the L lanes that share a token, in all of them.
template <int L>
__device__ __forceinline__ float sum_of(float v) {
  return L == 64 ? wave_sum(v) : row_sum_f(v);
}
template <int L>
__device__ __forceinline__ float max_of(float v) {
  if constexpr (L == 64) return wave_max_f(v);
  v = fmaxf(v, __uint_as_float(row_ror<8>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(row_ror<4>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(row_ror<2>(__float_as_uint(v))));
  return fmaxf(v, __uint_as_float(row_ror<1>(__float_as_uint(v))));
}

// Probabilities from logits, in place; false for a row of -inf alone (padding),
// whose probabilities are 0.  A NaN logit (+inf under softmax) makes all NaN.
template <int L, int NQ, bool SIGMOID>
__device__ __forceinline__ bool probabilities(float (&f)[NQ][4]) {
  float m = -__builtin_inff();
#pragma unroll
  for (int q = 0; q < NQ; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, f[q][i] == f[q][i] ? f[q][i] : __builtin_inff());
  m = max_of<L>(m);
  const bool used = m > -__builtin_inff();
  if (SIGMOID || !used) m = used ? fminf(m, 0.0f) : 0.0f;
  float total = 0.0f;
#pragma unroll
  for (int q = 0; q < NQ; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = f[q][i];
      if constexpr (SIGMOID)
        f[q][i] = exp_down(x > 0.0f ? 0.0f : x - m) / (1.0f + exp_down(-fabsf(x)));
      else
        f[q][i] = exp_down(x - m);
      total += f[q][i];
    }
  total = sum_of<L>(total);
  const float inv = used ? 1.0f / total : 0.0f;
#pragma unroll
  for (int q = 0; q < NQ; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) f[q][i] *= inv;
  return used;
}

// The runs that chunk [r0, r1) of the tokens shares with the sequences: body(s, begin,
// end) for each, in order; the first row behind the last of them comes back.
template <typename Body>
__device__ __forceinline__ int64_t each_run(const int32_t* ends, int S, int64_t T, int64_t r0, int64_t r1,
                                            const Body& body) {
  if (!ends) {
    body(0, r0, r1);
    return r1;
  }
  int lo = 0, hi = S;                    // the first sequence that ends past r0
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] > r0)
      hi = mid;
    else
      lo = mid + 1;
  }
  int64_t begin = r0;
  for (int s = lo; s < S && begin < r1; ++s) {
    const int64_t end = min(int64_t(ends[s]), r1);
    if (end > begin) {
      body(s, begin, end);
      begin = end;
    }
  }
  return begin;
}

// Partial sums of a run: P [runs][E4] (sums of probabilities), C [runs][E4] (slots),
// n [runs] (tokens); then a loss for each sequence.
struct Partials {
  float* P;
  int32_t* C;
  int32_t* n;
  float* losses;
  int E4;
  int64_t rows;                          // tokens of a chunk
};

template <typename T, int L, int NQ, bool SIGMOID>
__global__ __launch_bounds__(kThreads) void balance_kernel(const BalanceProblem p, const Partials part) {
  constexpr int SLOTS = kThreads / L;    // tokens at once
  constexpr int COLS = NQ * 4 * L;
  __shared__ float sums[SLOTS][COLS];
  __shared__ int32_t counts[COLS], tokens;
  const int lane = threadIdx.x % L, slot = threadIdx.x / L;
  const int64_t b = blockIdx.x, r0 = b * part.rows, r1 = min(p.T, r0 + part.rows);
  each_run(p.ends, p.S, p.T, r0, r1, [&](int s, int64_t begin, int64_t end) {
    for (int c = threadIdx.x; c < COLS; c += kThreads) counts[c] = 0;
    if (threadIdx.x == 0) tokens = 0;
    __syncthreads();
    float acc[NQ][4];
    int mine = 0;
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[q][i] = 0.0f;
    for (int64_t row = begin + slot; row < end; row += SLOTS) {
      const T* x = static_cast<const T*>(p.logits) + row * p.ld;
      float f[NQ][4];
#pragma unroll
      for (int q = 0; q < NQ; ++q) load4(x, (q * L + lane) * 4, p.E, f[q]);
      if (!probabilities<L, NQ, SIGMOID>(f)) continue;
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[q][i] += f[q][i];
      ++mine;
      for (int j = lane; j < p.k; j += L) {
        const int id = p.ids[row * p.k + j];
        if (id >= 0 && id < p.E) atomicAdd(&counts[id], 1);       // whole numbers: any order
      }
    }
    if (lane == 0 && mine) atomicAdd(&tokens, mine);
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) sums[slot][(q * L + lane) * 4 + i] = acc[q][i];
    __syncthreads();
    const int64_t run = b + s;
    for (int c = threadIdx.x; c < part.E4; c += kThreads) {
      float v = 0.0f;
#pragma unroll
      for (int i = 0; i < SLOTS; ++i) v += sums[i][c];
      part.P[run * part.E4 + c] = v;
      part.C[run * part.E4 + c] = counts[c];
    }
    if (threadIdx.x == 0) part.n[run] = tokens;
    __syncthreads();
  });
}

// Sum over a workgroup of 1024 threads, in every thread, in a fixed order.
__device__ __forceinline__ float block_sum(float v, float (&part)[16]) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) v += part[i];
  return v;
}

// A sequence's counts and loss from its runs' partial sums: four columns a thread, the
// runs shared by 1024 / quads slices.
__global__ __launch_bounds__(1024) void balance_sum_kernel(const BalanceProblem p, const Partials part, int quads) {
  __shared__ float4 sums[1024];
  __shared__ int4 slots[1024];
  __shared__ float sum_part[16];
  const int s = blockIdx.x;
  int64_t begin = s && p.ends ? p.ends[s - 1] : 0, end = p.ends ? p.ends[s] : p.T;
  begin = max(begin, int64_t(0));
  end = min(end, p.T);
  // runs [first, last) of the partial rows
  const int64_t first = begin / part.rows + s, last = end > begin ? (end - 1) / part.rows + s + 1 : first;
  const int q = threadIdx.x % quads, slice = threadIdx.x / quads, slices = 1024 / quads;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  int4 c = make_int4(0, 0, 0, 0);
  if (q * 4 < part.E4) {
#pragma unroll 4
    for (int64_t run = first + slice; run < last; run += slices) {
      const float4 a = *reinterpret_cast<const float4*>(part.P + run * part.E4 + q * 4);
      const int4 d = *reinterpret_cast<const int4*>(part.C + run * part.E4 + q * 4);
      v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
      c.x += d.x, c.y += d.y, c.z += d.z, c.w += d.w;
    }
  }
  sums[threadIdx.x] = v;
  slots[threadIdx.x] = c;
  int n = 0;
  for (int64_t run = first + threadIdx.x; run < last; run += 1024) n += part.n[run];
  __syncthreads();
  float term = 0.0f;
  if (threadIdx.x < part.E4) {
    const int at = threadIdx.x / 4, i = threadIdx.x % 4;
    float P = 0.0f;
    int C = 0;
    for (int k = 0; k < slices; ++k) {
      P += reinterpret_cast<const float*>(&sums[k * quads + at])[i];
      C += reinterpret_cast<const int*>(&slots[k * quads + at])[i];
    }
    if (threadIdx.x < unsigned(p.E)) {
      p.counts[int64_t(s) * p.E + threadIdx.x] = C;
      term = float(C) * P;
    }
  }
  term = block_sum(term, sum_part);
  __shared__ int32_t total;
  if (threadIdx.x == 0) total = 0;
  __syncthreads();
  if (n) atomicAdd(&total, n);
  __syncthreads();
  if (threadIdx.x == 0) {
    p.tokens[s] = total;
    const float inv = 1.0f / float(max(total, 1));
    const float loss = total ? term * inv * (p.coeff * float(p.E) / float(p.k)) * inv : 0.0f;
    if (p.S == 1)
      *p.loss = loss;
    else
      part.losses[s] = loss;
  }
}

// The mean of the sequences' losses over those that have tokens.
__global__ __launch_bounds__(1024) void balance_mean_kernel(const BalanceProblem p, const float* losses) {
  __shared__ float part[16];
  __shared__ int32_t alive;
  if (threadIdx.x == 0) alive = 0;
  __syncthreads();
  float v = 0.0f;
  int n = 0;
  for (int s = threadIdx.x; s < p.S; s += 1024) {
    v += losses[s];
    n += p.tokens[s] > 0;
  }
  if (n) atomicAdd(&alive, n);
  v = block_sum(v, part);
  if (threadIdx.x == 0) *p.loss = alive ? v / float(alive) : 0.0f;
}

template <typename T, int L, int NQ, bool SIGMOID>
__global__ __launch_bounds__(kThreads) void balance_backward_kernel(const BalanceProblem p, int64_t rows) {
  constexpr int SLOTS = kThreads / L;
  const int lane = threadIdx.x % L, slot = threadIdx.x / L;
  const int64_t r0 = int64_t(blockIdx.x) * rows, r1 = min(p.T, r0 + rows);
  int alive = 0;                         // sequences with tokens, counted by every wave for itself
  for (int s = 0; s < p.S; s += 64) {
    const int at = s + int(threadIdx.x & 63);
    alive += __popcll(__ballot(at < p.S && p.tokens[min(at, p.S - 1)] > 0));
  }
  const float whole = *p.grad_loss * p.coeff * float(p.E) / (float(p.k) * float(max(alive, 1)));
  const int64_t done = each_run(p.ends, p.S, p.T, r0, r1, [&](int s, int64_t begin, int64_t end) {
    int c[NQ][4];
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = (q * L + lane) * 4 + i;
        c[q][i] = e < p.E ? p.counts[int64_t(s) * p.E + e] : 0;
      }
    const float inv = 1.0f / float(max(p.tokens[s], 1));
    const float d = whole * inv * inv;
    for (int64_t row = begin + slot; row < end; row += SLOTS) {
      const T* x = static_cast<const T*>(p.logits) + row * p.ld;
      float f[NQ][4], u[NQ][4];
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        load4(x, (q * L + lane) * 4, p.E, f[q]);
        if constexpr (SIGMOID) {         // 1 - sigmoid(x)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            u[q][i] = exp_down(fminf(-f[q][i], 0.0f)) / (1.0f + exp_down(-fabsf(f[q][i])));
        }
      }
      const bool used = probabilities<L, NQ, SIGMOID>(f);
      float top = 0.0f;
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, f[q][i]);
      top = max_of<L>(top);
      int ref = -1;                      // the most probable expert's count (the largest, of equals)
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) ref = f[q][i] == top ? max(ref, c[q][i]) : ref;
      ref = int(L == 64 ? wave_max_u(uint32_t(ref + 1)) : row_max_u(uint32_t(ref + 1))) - 1;
      float mean = 0.0f;
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) mean = fmaf(f[q][i], float(c[q][i] - ref), mean);
      mean = sum_of<L>(mean);
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        float g[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          g[i] = f[q][i] * (float(c[q][i] - ref) - mean) * d;
          if constexpr (SIGMOID) g[i] *= u[q][i];
          if (!used) g[i] = 0.0f;
        }
        store4(static_cast<T*>(p.grad_logits) + row * p.ld_grad, (q * L + lane) * 4, p.E, g);
      }
    }
  });
  const float zeros[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t row = done + slot; row < r1; row += SLOTS)
#pragma unroll
    for (int q = 0; q < NQ; ++q)
      store4(static_cast<T*>(p.grad_logits) + row * p.ld_grad, (q * L + lane) * 4, p.E, zeros);
}

// Tokens of a chunk of the forward: at most 256 chunks, each a few turns.
int64_t chunk_rows(int64_t T) { return T > 256 * 64 ? (T + 255) / 256 : 64; }
int64_t chunks(int64_t T) { return T ? (T + chunk_rows(T) - 1) / chunk_rows(T) : 0; }
int padded(int64_t E) { return int((E + 3) / 4 * 4); }

constexpr int64_t kBackwardRows = 64;    // tokens of a workgroup of the backward at least

template <typename Run>
hipError_t by_experts(int E, const Run& run) {
  if (E <= 64) return run(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
  if (E <= 128) return run(std::integral_constant<int, 16>{}, std::integral_constant<int, 2>{});
  if (E <= 256) return run(std::integral_constant<int, 16>{}, std::integral_constant<int, 4>{});
  if (E <= 512) return run(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
  return run(std::integral_constant<int, 64>{}, std::integral_constant<int, 4>{});
}

template <typename T, bool SIGMOID>
hipError_t forward_typed(const BalanceProblem& p, const Partials& part, hipStream_t st) {
  return by_experts(p.E, [&](auto L, auto NQ) {
    hipLaunchKernelGGL((balance_kernel<T, decltype(L)::value, decltype(NQ)::value, SIGMOID>),
                       dim3(unsigned(chunks(p.T))), dim3(kThreads), 0, st, p, part);
    return hipGetLastError();
  });
}

template <typename T, bool SIGMOID>
hipError_t backward_typed(const BalanceProblem& p, hipStream_t st) {
  const int64_t rows = p.T > kBackwardRows << 20 ? (p.T + (1 << 20) - 1) >> 20 : kBackwardRows;
  return by_experts(p.E, [&](auto L, auto NQ) {
    hipLaunchKernelGGL((balance_backward_kernel<T, decltype(L)::value, decltype(NQ)::value, SIGMOID>),
                       dim3(unsigned((p.T + rows - 1) / rows)), dim3(kThreads), 0, st, p, rows);
    return hipGetLastError();
  });
}

Partials layout(const BalanceProblem& p) {
  const int64_t runs = chunks(p.T) + p.S;
  Partials part;
  part.E4 = padded(p.E);
  part.rows = chunk_rows(p.T);
  part.P = static_cast<float*>(p.workspace);
  part.C = reinterpret_cast<int32_t*>(part.P + runs * part.E4);
  part.n = part.C + runs * part.E4;
  part.losses = reinterpret_cast<float*>(part.n + runs);
  return part;
}

}  // namespace

int64_t balance_workspace(int64_t T, int64_t E, int64_t S) {
  const int64_t runs = chunks(T) + S;
  return 4 * (2 * runs * padded(E) + runs + S);
}

hipError_t launch_balance(const BalanceProblem& p, hipStream_t st) {
  const Partials part = layout(p);
  hipError_t e = hipSuccess;
  if (p.T > 0) {
    if (p.fp32)
      e = p.sigmoid ? forward_typed<float, true>(p, part, st) : forward_typed<float, false>(p, part, st);
    else
      e = p.sigmoid ? forward_typed<uint16_t, true>(p, part, st) : forward_typed<uint16_t, false>(p, part, st);
    if (e != hipSuccess) return e;
  }
  int quads = 1;
  while (quads * 4 < part.E4) quads *= 2;
  hipLaunchKernelGGL(balance_sum_kernel, dim3(unsigned(p.S)), dim3(1024), 0, st, p, part, quads);
  e = hipGetLastError();
  if (e != hipSuccess || p.S == 1) return e;
  hipLaunchKernelGGL(balance_mean_kernel, dim3(1), dim3(1024), 0, st, p, part.losses);
  return hipGetLastError();
}

hipError_t launch_balance_backward(const BalanceProblem& p, hipStream_t st) {
  if (p.T == 0) return hipSuccess;
  if (p.fp32) return p.sigmoid ? backward_typed<float, true>(p, st) : backward_typed<float, false>(p, st);
  return p.sigmoid ? backward_typed<uint16_t, true>(p, st) : backward_typed<uint16_t, false>(p, st);
}

}  // namespace fp8mm
