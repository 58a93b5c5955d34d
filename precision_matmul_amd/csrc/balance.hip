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
// practice a few launches of dependent loads: 16384 x 64 float32 logits are 4 MiB, and
// take 4.9 + 4.1 us forward and 5.2 backward; 16384 x 256 sigmoid scores in 7 sequences 13
// + 4.5 + 2.0 and 14 us.  There a wave has 759 vector instructions in the forward (948 in
// the backward), some 5 (6) us for a SIMD's four, and waits for 57 % (47 %) of its cycles:
// each of a lane's 16 scores has a branch of the lanes around its second exponential, so
// that they run one after the other.  The forward needs sums over all tokens of a sequence,
// so it is a pass over the tokens that leaves partial sums and a sum over those.  Chunk b of
// the tokens and sequence s meet in at most one run of tokens, and as b and s only grow from
// run to run, b + s names it: its partial row of the workspace, written once, with no search
// and no atomics.
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

constexpr int kThreads = 1024;           // of the forward: four waves a SIMD hide each other's chains
constexpr int kBackThreads = 256;

// exp(x) for x <= 0: exp2 corrected by the rounding of its argument; 0 where the result is
// below 2^-126 (the instruction gives no subnormal numbers).
__device__ __forceinline__ float exp_down(float x) {
  const float t = x * 1.44269504f, e = __builtin_amdgcn_exp2f(t);
  const float rest = fmaf(x, 1.44269504f, -t) + x * 1.92596299e-8f;
  return x < -104.0f ? 0.0f : fmaf(e, rest * 0.693147182f, e);
}

// 1 / d of a normal d, within an ulp (d in [1, 2] here): the hardware's and one Newton step.
__device__ __forceinline__ float reciprocal(float d) {
  const float r = __builtin_amdgcn_rcpf(d);
  return fmaf(fmaf(-d, r, 1.0f), r, r);
}

// Logits of a token as they come from memory, four at column c of E each: past the row's
// end its last four (columns, of less than four: its last) in their place.  No branch of
// the lanes and nothing done with them before the turn that uses them, so that all loads
// of a turn are in flight together, beside the turn before.
template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Four {
  T v[4];
};
template <int NQ, typename T>
__device__ __forceinline__ Four<T> ask4(const T* row, int c, int E) {
  if (NQ > 1 || E >= 4) return *reinterpret_cast<const Four<T>*>(row + min(c, E - 4));
  return Four<T>{{row[0], row[min(1, E - 1)], row[E - 1], row[E - 1]}};
}
// Their values; -inf past the end.
template <int NQ, typename T>
__device__ __forceinline__ void settle4(const Four<T>& a, int c, int E, float (&f)[4]) {
  const float none = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = to_float(a.v[i]);
  if (E % 4 == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = c < E ? f[i] : none;
    return;
  }
  const int n = NQ > 1 || E >= 4 ? c - min(c, E - 4) : 0;          // columns that are other lanes'
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (n > k) f[0] = f[1], f[1] = f[2], f[2] = f[3];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = c + i < E ? f[i] : none;
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

// v + v of the lane 16 (32) away.
__device__ __forceinline__ float add_rows(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
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
  // where no row's factor exp(-m) is needed, the sigmoid has one exponential
  const bool plain = SIGMOID && !__any(m < 0.0f);
#pragma unroll
  for (int q = 0; q < NQ; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = f[q][i];
      if constexpr (SIGMOID) {
        const float e = exp_down(-fabsf(x));
        const float top = x > 0.0f ? 1.0f : plain ? e : exp_down(x - m);
        f[q][i] = top * reciprocal(1.0f + e);
      } else {
        f[q][i] = exp_down(x - m);
      }
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

// The first sequence that ends past row r0, by every wave for itself; S if there is none.
// `end` is the wave's lanes' end of the first 64 sequences: one load for few sequences,
// in place of a chain of them.
__device__ __forceinline__ int lane_end(const BalanceProblem& p) {
  const int lane = threadIdx.x & 63;
  return p.ends && lane < p.S ? p.ends[lane] : 0x7FFFFFFF;
}
__device__ __forceinline__ int sequence_of(const BalanceProblem& p, int end, int64_t r0) {
  if (!p.ends) return 0;
  if (p.S <= 64) return __popcll(__ballot(end <= r0));
  int lo = 0, hi = p.S;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (p.ends[mid] > r0)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
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

// A sequence's loss from the sum over its experts of counts times sums.
__device__ __forceinline__ float loss_of(const BalanceProblem& p, float term, int tokens) {
  const float inv = 1.0f / float(max(tokens, 1));
  return tokens ? term * inv * (p.coeff * float(p.E) / float(p.k)) * inv : 0.0f;
}

// The tokens in runs: their probabilities summed over the tokens of each run, their slots
// counted.  L lanes hold a token; a token is loaded before it is known which run it is in.
// ONE: few tokens, a workgroup for each sequence, which then gives its loss itself.
template <typename T, int L, int NQ, bool SIGMOID, bool ONE>
__global__ __launch_bounds__(kThreads) void balance_kernel(const BalanceProblem p, const Partials part) {
  constexpr int SLOTS = kThreads / L;    // tokens of a turn
  constexpr int COLS = NQ * 4 * L, WAVES = kThreads / 64;
  __shared__ float sums[WAVES][COLS];
  __shared__ int32_t counts[COLS], tokens;
  __shared__ float loss_part[16];
  const int lane = threadIdx.x % L, slot = threadIdx.x / L;
  const int64_t b = ONE ? 0 : blockIdx.x;
  const int64_t r0 = !ONE ? b * part.rows : p.ends && blockIdx.x ? max(p.ends[blockIdx.x - 1], 0) : 0;
  const int64_t r1 = !ONE ? min(p.T, r0 + part.rows) : p.ends ? min(int64_t(p.ends[blockIdx.x]), p.T) : p.T;
  float acc[NQ][4];
  int mine = 0;
  const auto clear = [&] {
    for (int c = threadIdx.x; c < COLS; c += kThreads) counts[c] = 0;
    if (threadIdx.x == 0) tokens = 0;
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[q][i] = 0.0f;
    mine = 0;
    __syncthreads();
  };
  // a run's sums: partial row b + s, or (ONE) the loss
  const auto finish = [&](int64_t run) {
    if (lane == 0 && mine) atomicAdd(&tokens, mine);
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v = acc[q][i];
        if constexpr (L == 16) v = add_rows(v);          // the wave's four tokens
        if (L == 64 || (threadIdx.x & 48) == 0) sums[threadIdx.x >> 6][(q * L + lane) * 4 + i] = v;
      }
    __syncthreads();
    float term = 0.0f;
    if (threadIdx.x < part.E4) {         // at most 1024 columns
      const int c = threadIdx.x;
      float v = 0.0f;
#pragma unroll
      for (int i = 0; i < WAVES; ++i) v += sums[i][c];
      if constexpr (ONE) {
        if (c < p.E) {
          p.counts[int64_t(blockIdx.x) * p.E + c] = counts[c];
          term = float(counts[c]) * v;
        }
      } else {
        part.P[run * part.E4 + c] = v;
        part.C[run * part.E4 + c] = counts[c];
      }
    }
    if constexpr (ONE) term = block_sum(term, loss_part);
    if (threadIdx.x == 0) {
      if constexpr (ONE) {
        p.tokens[blockIdx.x] = tokens;
        *(p.S == 1 ? p.loss : part.losses + blockIdx.x) = loss_of(p, term, tokens);
      } else {
        part.n[run] = tokens;
      }
    }
    __syncthreads();
  };
  const auto end_of = [&](int s) { return p.ends ? min(int64_t(p.ends[s]), r1) : r1; };
  Four<T> raw[NQ];                       // the next turn's logits and first ids
  int raw_id;
  const auto ask = [&](int64_t row) {    // past the chunk: its last row, which is not used
    const int64_t at = min(row, r1 - 1);
    const T* x = static_cast<const T*>(p.logits) + at * p.ld;
#pragma unroll
    for (int q = 0; q < NQ; ++q) raw[q] = ask4<NQ>(x, (q * L + lane) * 4, p.E);
    raw_id = p.ids[at * p.k + min(lane, p.k - 1)];
  };
  if (r0 < r1) ask(r0 + slot);
  const int my_end = ONE ? 0 : lane_end(p);
  clear();
  int s = ONE ? 0 : sequence_of(p, my_end, r0);
  int64_t begin = r0, end = ONE ? r1 : s < p.S ? end_of(s) : r0;    // the rest of this run
  for (int64_t turn = r0; turn < r1; turn += SLOTS) {
    const int64_t row = turn + slot, next = min(turn + SLOTS, r1);
    float f[NQ][4];
    const int id0 = lane < p.k ? raw_id : -1;
#pragma unroll
    for (int q = 0; q < NQ; ++q) settle4<NQ>(raw[q], (q * L + lane) * 4, p.E, f[q]);
    if (next < r1) ask(next + slot);
    const bool used = probabilities<L, NQ, SIGMOID>(f) && row < r1;
    while (s < p.S) {
      if (used && row >= begin && row < end) {
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[q][i] += f[q][i];
        ++mine;
        if (id0 >= 0 && id0 < p.E) atomicAdd(&counts[id0], 1);        // whole numbers: any order
        for (int j = lane + L; j < p.k; j += L) {
          const int id = p.ids[row * p.k + j];
          if (id >= 0 && id < p.E) atomicAdd(&counts[id], 1);
        }
      }
      if (ONE || end > next) break;      // goes on in the next turn
      finish(b + s);
      begin = end;
      do {
        ++s;
        end = s < p.S ? end_of(s) : r1;
      } while (s < p.S && end <= begin);
      if (s < p.S) clear();
      if (begin >= next) break;          // the next run starts with the next turn
    }
    if (s >= p.S) return;                // rows behind the last sequence
  }
  if constexpr (ONE) finish(0);
}

// A sequence's counts and loss from its runs' partial sums.  A wave's lanes hold four
// columns each (QL = 1: up to 256 columns, several runs at once where there are fewer;
// else four times four), the 16 waves take the runs in turns.
template <int QL>
__global__ __launch_bounds__(1024) void balance_sum_kernel(const BalanceProblem p, const Partials part, int quads) {
  __shared__ float4 sums[16][QL * 64];
  __shared__ int4 slots[16][QL * 64];
  __shared__ int32_t tokens[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, s = blockIdx.x;
  const int groups = 64 / quads, q = lane % quads, group = lane / quads;
  float4 v[QL];
  int4 c[QL];
  int n = 0;
#pragma unroll
  for (int i = 0; i < QL; ++i) v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f), c[i] = make_int4(0, 0, 0, 0);
  int64_t begin = s && p.ends ? p.ends[s - 1] : 0, end = p.ends ? p.ends[s] : p.T;
  begin = max(begin, int64_t(0));
  end = min(end, p.T);
  // runs [first, last) of the partial rows
  const int first = int(begin / part.rows) + s, last = end > begin ? int((end - 1) / part.rows) + s + 1 : first;
  // no branch in the loop, so that its loads are in flight together: lanes past the columns
  // read the last ones, and all lanes of a run its tokens
#pragma unroll QL == 1 ? 4 : 2
  for (int run = first + wave * groups + group; run < last; run += 16 * groups) {
#pragma unroll
    for (int i = 0; i < QL; ++i) {
      const int64_t at = int64_t(run) * part.E4 + min((i * 64 + q) * 4, part.E4 - 4);
      const float4 a = *reinterpret_cast<const float4*>(part.P + at);
      const int4 d = *reinterpret_cast<const int4*>(part.C + at);
      v[i].x += a.x, v[i].y += a.y, v[i].z += a.z, v[i].w += a.w;
      c[i].x += d.x, c[i].y += d.y, c[i].z += d.z, c[i].w += d.w;
    }
    n += part.n[run];
  }
  for (int off = quads; off < 64; off <<= 1) {   // the lanes' groups (QL = 1)
    v[0].x += __shfl_xor(v[0].x, off, 64), v[0].y += __shfl_xor(v[0].y, off, 64);
    v[0].z += __shfl_xor(v[0].z, off, 64), v[0].w += __shfl_xor(v[0].w, off, 64);
    c[0].x += __shfl_xor(c[0].x, off, 64), c[0].y += __shfl_xor(c[0].y, off, 64);
    c[0].z += __shfl_xor(c[0].z, off, 64), c[0].w += __shfl_xor(c[0].w, off, 64);
    n += __shfl_xor(n, off, 64);
  }
#pragma unroll
  for (int i = 0; i < QL; ++i) sums[wave][i * 64 + lane] = v[i], slots[wave][i * 64 + lane] = c[i];
  if (lane == 0) tokens[wave] = n;
  __syncthreads();
  if (wave != 0) return;
  float term = 0.0f;
  n = 0;
#pragma unroll
  for (int w = 0; w < 16; ++w) n += tokens[w];
#pragma unroll
  for (int i = 0; i < QL; ++i) {
    const int at = (i * 64 + q) * 4;
    if (group != 0 || at >= p.E) continue;
    float P[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    int C[4] = {0, 0, 0, 0};
#pragma unroll 4
    for (int w = 0; w < 16; ++w) {
      const float4 a = sums[w][i * 64 + lane];
      const int4 d = slots[w][i * 64 + lane];
      P[0] += a.x, P[1] += a.y, P[2] += a.z, P[3] += a.w;
      C[0] += d.x, C[1] += d.y, C[2] += d.z, C[3] += d.w;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (at + e >= p.E) continue;
      p.counts[int64_t(s) * p.E + at + e] = C[e];
      term = fmaf(float(C[e]), P[e], term);
    }
  }
  term = wave_sum(term);
  if (lane == 0) {
    p.tokens[s] = n;
    *(p.S == 1 ? p.loss : part.losses + s) = loss_of(p, term, n);
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

// Gradient: L lanes hold a token, loaded a turn ahead; its sequence's counts are loaded
// when they are not those of the lanes' token before.
template <typename T, int L, int NQ, bool SIGMOID>
__global__ __launch_bounds__(kBackThreads) void balance_backward_kernel(const BalanceProblem p, int64_t rows) {
  constexpr int SLOTS = kBackThreads / L;
  const int lane = threadIdx.x % L, slot = threadIdx.x / L, wave_lane = threadIdx.x & 63;
  const int64_t r0 = int64_t(blockIdx.x) * rows, r1 = min(p.T, r0 + rows);
  Four<T> raw[NQ];
  const auto ask = [&](int64_t row) {    // past the chunk: its last row, which is not used
    const T* x = static_cast<const T*>(p.logits) + min(row, r1 - 1) * p.ld;
#pragma unroll
    for (int q = 0; q < NQ; ++q) raw[q] = ask4<NQ>(x, (q * L + lane) * 4, p.E);
  };
  ask(r0 + slot);
  const float grad = *p.grad_loss;
  const int my_tokens = wave_lane < p.S ? p.tokens[wave_lane] : 0;
  const int my_end = lane_end(p);
  int alive = __popcll(__ballot(my_tokens > 0));         // sequences with tokens
  for (int s = 64; s < p.S; s += 64) {
    const int at = s + wave_lane;
    alive += __popcll(__ballot(at < p.S && p.tokens[min(at, p.S - 1)] > 0));
  }
  const float whole = grad * p.coeff * float(p.E) / (float(p.k) * float(max(alive, 1)));
  int c[NQ][4], of = -1;                 // counts of the sequence `of`
  float d = 0.0f;
#pragma unroll
  for (int q = 0; q < NQ; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) c[q][i] = 0;
  for (int64_t turn = r0; turn < r1; turn += SLOTS) {
    const int64_t row = turn + slot;
    float f[NQ][4], u[NQ][4];
#pragma unroll
    for (int q = 0; q < NQ; ++q) settle4<NQ>(raw[q], (q * L + lane) * 4, p.E, f[q]);
    if (turn + SLOTS < r1) ask(row + SLOTS);
    int s = 0;                           // the token's sequence; S behind the last
    if (p.ends && p.S <= 64) {
#pragma unroll
      for (int k = 0; k < 64 / L; ++k) { // the wave's tokens
        const int64_t other = row - slot + (threadIdx.x >> 6) * (64 / L) + k;
        const int before = __popcll(__ballot(my_end <= other));
        s = wave_lane / L == k ? before : s;
      }
    } else if (p.ends) {
      s = sequence_of(p, my_end, row);
    }
    if (__any(s != of)) {
      const int at = min(s, p.S - 1);
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = (q * L + lane) * 4 + i;
          const int count = p.counts[int64_t(at) * p.E + min(e, p.E - 1)];
          c[q][i] = e < p.E ? count : 0;
        }
      const int n = p.S <= 64 ? __shfl(my_tokens, at, 64) : p.tokens[at];
      const float inv = 1.0f / float(max(n, 1));
      d = whole * inv * inv;
      of = s;
    }
    if constexpr (SIGMOID) {             // 1 - sigmoid(x)
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = exp_down(-fabsf(f[q][i]));
          u[q][i] = (f[q][i] > 0.0f ? e : 1.0f) * reciprocal(1.0f + e);
        }
    }
    const bool used = probabilities<L, NQ, SIGMOID>(f) && s < p.S;
    float top = 0.0f;
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, f[q][i]);
    top = max_of<L>(top);
    int ref = -1;                        // the most probable expert's count (the largest, of equals)
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
    if (row >= r1) continue;             // (the wave's other tokens may be there)
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      float g[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        g[i] = f[q][i] * (float(c[q][i] - ref) - mean) * d;
        if constexpr (SIGMOID) g[i] *= u[q][i];
        if (!used) g[i] = 0.0f;          // padding, and rows behind the last sequence
      }
      store4(static_cast<T*>(p.grad_logits) + row * p.ld_grad, (q * L + lane) * 4, p.E, g);
    }
  }
}

// Tokens of a chunk of the forward: at most 256 chunks, each a few turns.
int64_t chunk_rows(int64_t T) { return T > 256 * 64 ? (T + 255) / 256 : 64; }
int64_t chunks(int64_t T) { return T ? (T + chunk_rows(T) - 1) / chunk_rows(T) : 0; }
// Whether a workgroup takes a whole sequence, without partial sums: four turns of tokens (200
// x 64 7.4 us, by chunks 4.8 + 3.3 and a launch), or sequences of few, on average (4000
// tokens in 64 sequences 11 us, by chunks 16 + 5).  Not more: 1000 x 256 in two sequences
// would take 37 us in place of 15, and as much if one sequence has nearly all of the tokens.
bool one_group(int64_t T, int64_t E, int64_t S) { return T <= (E <= 256 ? 256 : 64) || (T <= 1024 && T <= 16 * S); }
int padded(int64_t E) { return int((E + 3) / 4 * 4); }

// Tokens of a workgroup of the backward at least, for 16 or 64 lanes a token: one turn, or
// two (4000 x 256 7.2 us, two turns 9.8; 200 x 800 7.8, four turns 12.6).
constexpr int64_t kBackwardRows[2] = {16, 8};

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
    constexpr int l = decltype(L)::value, nq = decltype(NQ)::value;
    if (one_group(p.T, p.E, p.S))
      hipLaunchKernelGGL((balance_kernel<T, l, nq, SIGMOID, true>), dim3(unsigned(p.S)), dim3(kThreads), 0, st, p, part);
    else
      hipLaunchKernelGGL((balance_kernel<T, l, nq, SIGMOID, false>), dim3(unsigned(chunks(p.T))), dim3(kThreads), 0, st,
                         p, part);
    return hipGetLastError();
  });
}

template <typename T, bool SIGMOID>
hipError_t backward_typed(const BalanceProblem& p, hipStream_t st) {
  const int64_t least = kBackwardRows[p.E > 256], rows = p.T > least << 20 ? (p.T + (1 << 20) - 1) >> 20 : least;
  return by_experts(p.E, [&](auto L, auto NQ) {
    hipLaunchKernelGGL((balance_backward_kernel<T, decltype(L)::value, decltype(NQ)::value, SIGMOID>),
                       dim3(unsigned((p.T + rows - 1) / rows)), dim3(kBackThreads), 0, st, p, rows);
    return hipGetLastError();
  });
}

Partials layout(const BalanceProblem& p) {
  const int64_t runs = one_group(p.T, p.E, p.S) ? 0 : chunks(p.T) + p.S;
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
  if (one_group(T, E, S)) return S == 1 ? 0 : (4 * S + 15) / 16 * 16;
  const int64_t runs = chunks(T) + S;
  return 4 * (2 * runs * padded(E) + runs + S);
}

hipError_t launch_balance(const BalanceProblem& p, hipStream_t st) {
  const Partials part = layout(p);
  hipError_t e;
  if (p.fp32)
    e = p.sigmoid ? forward_typed<float, true>(p, part, st) : forward_typed<float, false>(p, part, st);
  else
    e = p.sigmoid ? forward_typed<uint16_t, true>(p, part, st) : forward_typed<uint16_t, false>(p, part, st);
  if (e != hipSuccess) return e;
  if (!one_group(p.T, p.E, p.S)) {
    int quads = 1;
    while (quads < 64 && quads * 4 < part.E4) quads *= 2;
    if (p.E <= 256)
      hipLaunchKernelGGL((balance_sum_kernel<1>), dim3(unsigned(p.S)), dim3(1024), 0, st, p, part, quads);
    else
      hipLaunchKernelGGL((balance_sum_kernel<4>), dim3(unsigned(p.S)), dim3(1024), 0, st, p, part, quads);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (p.S == 1) return e;
  hipLaunchKernelGGL(balance_mean_kernel, dim3(1), dim3(1024), 0, st, p, part.losses);
  return hipGetLastError();
}

hipError_t launch_balance_backward(const BalanceProblem& p, hipStream_t st) {
  if (p.T == 0) return hipSuccess;
  if (p.fp32) return p.sigmoid ? backward_typed<float, true>(p, st) : backward_typed<float, false>(p, st);
  return p.sigmoid ? backward_typed<uint16_t, true>(p, st) : backward_typed<uint16_t, false>(p, st);
}

}  // namespace fp8mm
