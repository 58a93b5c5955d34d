// Routing of tokens to experts, forward and backward (gfx950).
//
//   s   = softmax(l) or sigmoid(l) over a token's E logits l, in float32
//   key = s + bias (no bias: key = l, the same order without its rounding)
//   groups: each group of E / G experts scores its best key, or the sum of its
//           two best s (+ bias); experts outside the group_topk best groups
//           drop out
//   ids = the k largest keys in descending order, w = s[ids]
//         (/ (sum + 1e-20)) scale
// Equal keys and equal group scores go to the lower index.  An expert whose
// key is -inf (its logit or its bias is) is never chosen: slots without an
// expert get id -1 and weight 0.  A row with a NaN key, or with a +inf logit
// under softmax, has no defined choice: ids 0 .. k-1 with NaN weights, so that
// the fault shows in the token's output.
//
// Everything stays in registers and the logits are read once (T E values against
// T k results), so a large batch is bound by instructions, most of them in the k
// selection rounds: a maximum over lanes, the first lane that has it, the first
// place in that lane.  Two forms: 16 lanes a token, four tokens a wave (E <= 256,
// k <= 16), and one wave a token.  16384 tokens in us, the calls of the other
// form in brackets: 256 experts in 8 groups, sigmoid and bias, k = 8: 12.6 (17.8);
// 256 experts, softmax and bias: 10.8 (15.3); 128 experts 7.7 (11.5); 64 experts,
// k = 6: 7.6 (8.4), about what a call takes the host.  Backward, the kernel alone:
// 64 experts 4.5 (9.2); 256 experts, k = 8, softmax 11.1 (14.3), renormalised 11.0
// (13.4), sigmoid 10.1 (11.2).
#include "moe_launch.hpp"
#include "ops_common.hpp"

namespace fp8mm {
namespace {

using namespace ops;

constexpr float kInf = __builtin_inff();

template <typename T, int N>
__device__ __forceinline__ void load_row_of(const T* row, int e0, int E, float (&x)[N]) {
  struct __attribute__((packed, aligned(sizeof(T)))) At {
    T v[N];
  };
  if (e0 + N <= E) {
    const At a = *reinterpret_cast<const At*>(row + e0);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = to_float(a.v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = e0 + i < E ? to_float(row[e0 + i]) : -kInf;
  }
}

template <typename T, int N>
__device__ __forceinline__ void store_row_of(T* row, int e0, int E, const float (&g)[N]) {
  struct __attribute__((packed, aligned(sizeof(T)))) At {
    T v[N];
  };
  if (e0 + N <= E) {
    At a;
#pragma unroll
    for (int i = 0; i < N; ++i) a.v[i] = from_float<T>(g[i]);
    *reinterpret_cast<At*>(row + e0) = a;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (e0 + i < E) row[e0 + i] = from_float<T>(g[i]);
  }
}

// exp(-a) for a >= 0, to an ulp or two: the hardware's exp2 with the rounding
// error of a log2(e) put back (its part above 2^-24 and log2(e)'s own low part).
// The hardware's exp2 has no subnormal results: from a = 126 ln 2 = 87.3 on the
// result is 0 (float32's own exp is 0 from 104 on).
__device__ __forceinline__ float exp_neg(float a) {
  constexpr float kLog2e = 1.44269502162933349609375f, kLog2eLow = 1.92596299112661746887e-8f;
  a = fminf(a, 104.0f);
  const float t = a * -kLog2e;
  const float low = __builtin_fmaf(a, -kLog2e, -t) - a * kLog2eLow;
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e, low * 0.693147182464599609375f, e);
}

// 1 / d by the hardware's reciprocal and one Newton step; d in [1, 2].
__device__ __forceinline__ float reciprocal(float d) {
  const float r = __builtin_amdgcn_rcpf(d);
  return __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
}

// Floats as unsigned integers of the same order (-0 as +0), so that a wave
// maximum is six fused data-parallel steps; -inf and what is out are at most
// kNone.
constexpr uint32_t kNone = 0x007FFFFFu;

__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);
  return u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float from_ordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}

// Scores of a row: sigmoid(x), or softmax(x) = exp(x - shift) * inv, shift >= x.
// A token's logits lie in 64 lanes, or (ROW) in 16.
template <bool SIGMOID, bool ROW = false>
struct Scores {
  float shift = 0.0f, inv = 1.0f;

  template <int N>
  __device__ __forceinline__ explicit Scores(const float (&x)[N]) {
    if constexpr (!SIGMOID) {
      float m = x[0];
#pragma unroll
      for (int i = 1; i < N; ++i) m = fmaxf(m, x[i]);
      m = ROW ? from_ordered(row_max_u(ordered(m))) : wave_max_f(m);
      shift = m == -kInf ? 0.0f : m;             // a row of -inf alone: every score 0
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i) sum += exp_neg(shift - x[i]);
      sum = ROW ? row_sum_f(sum) : wave_sum(sum);
      inv = sum == 0.0f ? 1.0f : 1.0f / sum;
    }
  }

  __device__ __forceinline__ float operator()(float x) const {
    if constexpr (!SIGMOID) return exp_neg(shift - x) * inv;
    const float e = exp_neg(fabsf(x));
    return (x < 0.0f ? e : 1.0f) * reciprocal(1.0f + e);
  }
};

// The sigmoid and its slope, s (1 - s) as e / (1 + e)^2 with e = exp(-|x|): 1 - s
// has lost its bits where s is near 1 (6 % of it at a logit of 16, all from 17 on).
__device__ __forceinline__ float sigmoid_slope(float x, float& slope) {
  const float e = exp_neg(fabsf(x)), r = reciprocal(1.0f + e);
  slope = e * r * r;
  return (x < 0.0f ? e : 1.0f) * r;
}

// Whether a lane's logits leave its row without a defined choice.
template <bool SIGMOID, int N>
__device__ __forceinline__ bool undefined_logits(const float (&x)[N]) {
  bool bad = false;
#pragma unroll
  for (int i = 0; i < N; ++i) bad |= SIGMOID ? x[i] != x[i] : !(x[i] < kInf);
  return bad;
}

// Group selection: keys of experts outside the chosen groups become -inf.  L
// lanes work on each group: where a group is a power of two of whole lanes,
// those that hold it; else 64 / G rounded down to a power of two, which read its
// values from LDS.  They merge their two best by butterfly and compare the
// group's score with the others', L groups at a time.
struct Groups {
  int count, size;     // groups, experts in each
  int shift;           // L = 1 << shift
  bool whole;          // the L lanes are the group's own
  float inv_size;

  Groups(const RouteProblem& p, int per_lane) : count(p.groups), size(p.E / p.groups), inv_size(1.0f / float(size)) {
    const int lanes = size / per_lane;
    whole = size % per_lane == 0 && (lanes & (lanes - 1)) == 0;
    shift = 31 - __builtin_clz(unsigned(whole ? lanes : 64 / count));
  }
  // e / size: half an expert from the next integer at least, far more than
  // the float product can be off for e < 1024
  __device__ __forceinline__ int of(int e) const { return int((float(e) + 0.5f) * inv_size); }
};

// One butterfly step of (best, second) over lanes that differ in `CTRL`'s bit;
// pairs of lanes already agree below it, so that mirrors serve as well.
template <int CTRL>
__device__ __forceinline__ void merge_dpp(float& best, float& second) {
  const float b = dpp<CTRL>(0.0f, best), s = dpp<CTRL>(0.0f, second);
  second = fmaxf(fmaxf(second, s), fminf(best, b));
  best = fmaxf(best, b);
}

__device__ __forceinline__ void merge_far(float& best, float& second, int off) {
  const float b = __shfl_xor(best, off, 64), s = __shfl_xor(second, off, 64);
  second = fmaxf(fmaxf(second, s), fminf(best, b));
  best = fmaxf(best, b);
}

template <int N>
__device__ __forceinline__ void keep_groups(float (&key)[N], const float (&value)[N], int e0, const Groups& groups,
                                            bool top2, int topk, int E, float* lds) {
  const int lane = threadIdx.x & 63;
  const int L = 1 << groups.shift;
  const int g = lane >> groups.shift;
  float best = -kInf, second = -kInf;
  if (groups.whole) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      second = fmaxf(second, fminf(best, value[i]));
      best = fmaxf(best, value[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (e0 + i < E) lds[e0 + i] = value[i];
    // the wave reads what its own lanes wrote: in order, no barrier needed
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (g < groups.count) {
      for (int j = lane & (L - 1); j < groups.size; j += L) {
        const float v = lds[g * groups.size + j];
        second = fmaxf(second, fminf(best, v));
        best = fmaxf(best, v);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  if (L > 1) merge_dpp<0xB1>(best, second);      // lane ^ 1
  if (L > 2) merge_dpp<0x4E>(best, second);      // lane ^ 2
  if (L > 4) merge_dpp<0x141>(best, second);     // 7 - lane in each 8
  if (L > 8) merge_dpp<0x140>(best, second);     // 15 - lane in each 16
  if (L > 16) merge_far(best, second, 16);
  if (L > 32) merge_far(best, second, 32);
  float score = best;
  if (top2) score = second == -kInf ? best : best + second;
  // rank: groups that come before this one
  const uint64_t mine = (L == 64 ? ~0ull : (1ull << L) - 1) << (g << groups.shift);
  int rank = 0;
  for (int o0 = 0; o0 < groups.count; o0 += L) {
    const int o = o0 + (lane & (L - 1));
    const float other = __shfl(score, o << groups.shift, 64);
    const bool first = (other > score) | ((other == score) & (o < g));
    rank += __popcll(__ballot(first & (o < groups.count)) & mine);
  }
  const bool keep = g < groups.count && rank < topk;
  if (groups.whole) {
#pragma unroll
    for (int i = 0; i < N; ++i) key[i] = keep ? key[i] : -kInf;
  } else {
    const uint64_t kept = __ballot(keep);
#pragma unroll
    for (int i = 0; i < N; ++i) key[i] = (kept >> (groups.of(min(e0 + i, E - 1)) << groups.shift)) & 1 ? key[i] : -kInf;
  }
}

template <int N>
__device__ __forceinline__ void load_logits(const RouteProblem& p, int64_t row, int e0, float (&x)[N]) {
  if (p.fp32)
    load_row_of(static_cast<const float*>(p.logits) + row * p.ld, e0, p.E, x);
  else
    load_row_of(static_cast<const uint16_t*>(p.logits) + row * p.ld, e0, p.E, x);
}

// One wave a token, N = ceil(E / 64) consecutive experts a lane.
template <int N, bool SIGMOID, bool BIAS, bool GROUPS>
__global__ __launch_bounds__(256) void route_kernel(const RouteProblem p, const Groups groups) {
  extern __shared__ float lds_all[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int e0 = lane * N;
  float b[N];
  if constexpr (BIAS) load_row_of(p.bias, e0, p.E, b);
  for (int64_t row = int64_t(blockIdx.x) * 4 + wave; row < p.T; row += int64_t(gridDim.x) * 4) {
    float x[N], key[N];
    load_logits(p, row, e0, x);
    bool bad = undefined_logits<SIGMOID>(x);
    const Scores<SIGMOID> score(x);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      key[i] = x[i];
      if constexpr (BIAS) {
        const float k = score(x[i]) + b[i];
        key[i] = x[i] == -kInf ? -kInf : k;
        bad |= key[i] != key[i];
      }
    }
    if constexpr (GROUPS) {
      float value[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        value[i] = key[i];
        if constexpr (!BIAS) {
          const float s = score(x[i]);
          value[i] = p.group_top2 && x[i] != -kInf ? s : x[i];
        }
      }
      keep_groups(key, value, e0, groups, p.group_top2, p.group_topk, p.E, lds_all + wave * p.E);
    }
    const bool undefined = __ballot(bad) != 0;
    uint32_t u[N];
#pragma unroll
    for (int i = 0; i < N; ++i) u[i] = ordered(key[i]);
    int id = -1;                 // lane j: slot j's expert and its key
    uint32_t best = 0;
    for (int j = 0; j < p.k; ++j) {
      uint32_t local = u[0];
#pragma unroll
      for (int i = 1; i < N; ++i) local = max(local, u[i]);
      const uint32_t m = wave_max_u(local);
      if (m <= kNone) break;
      // the lowest lane with the maximum, and its lowest place with it; all of
      // this in scalars, written back to the one lane that it changes
      const int from = int(__builtin_ctzll(__ballot(local == m) | (1ull << 63)));
      int at = 0;
      if constexpr (N == 1) {
        u[0] = write_lane(0u, from, u[0]);
      } else {
        bool found = false;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const uint32_t v = read_lane(u[i], from);
          const bool here = !found && v == m;
          at = here ? i : at;
          found |= here;
          u[i] = write_lane(here ? 0u : v, from, u[i]);
        }
      }
      id = int(write_lane(uint32_t(from * N + at), j, uint32_t(id)));
      best = write_lane(m, j, best);
    }
    float chosen = from_ordered(best);
    if constexpr (BIAS) {        // the key holds the bias too
      chosen = 0.0f;
      if (id >= 0)
        chosen = p.fp32 ? static_cast<const float*>(p.logits)[row * p.ld + id]
                        : to_float(static_cast<const uint16_t*>(p.logits)[row * p.ld + id]);
    }
    float w = score(chosen);
    w = id < 0 ? 0.0f : w;
    if (p.renorm) w = w / (wave_sum(w) + kRenormEps);
    w *= p.scale;
    if (undefined) {
      id = lane;
      w = __builtin_nanf("");
    }
    if (lane < p.k) {
      p.ids[row * p.k + lane] = id;
      p.weights[row * p.k + lane] = w;
    }
  }
}

// ---------------------------------------------------------------------------
// The same for at most 256 experts and 16 slots, groups (if any) of whole lanes:
// four tokens a wave, 16 lanes each with V consecutive experts, so that the
// rounds' lane steps serve four tokens at once.
// ---------------------------------------------------------------------------
template <int V, bool SIGMOID, bool BIAS, bool GROUPS>
__global__ __launch_bounds__(256) void route16_kernel(const RouteProblem p, const Groups groups) {
  const int lane = threadIdx.x & 63;
  const int l16 = lane & 15, first = lane & 48;
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int e0 = l16 * V;
  float b[V];
  if constexpr (BIAS) load_row_of(p.bias, e0, p.E, b);
  for (int64_t row0 = (int64_t(blockIdx.x) * 4 + wave) * 4; row0 < p.T; row0 += int64_t(gridDim.x) * 16) {
    const int64_t own = row0 + (lane >> 4);
    const int64_t row = min(own, p.T - 1);       // lanes past the last token repeat it and write nothing
    float x[V], key[V];
    load_logits(p, row, e0, x);
    bool bad = undefined_logits<SIGMOID>(x);
    const Scores<SIGMOID, true> score(x);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      key[i] = x[i];
      if constexpr (BIAS) {
        const float k = score(x[i]) + b[i];
        key[i] = x[i] == -kInf ? -kInf : k;
        bad |= key[i] != key[i];
      }
    }
    if constexpr (GROUPS) {
      float best = -kInf, second = -kInf;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float value = key[i];
        if constexpr (!BIAS) {
          const float s = score(x[i]);
          value = p.group_top2 && x[i] != -kInf ? s : x[i];
        }
        second = fmaxf(second, fminf(best, value));
        best = fmaxf(best, value);
      }
      const int L = 1 << groups.shift;
      if (L > 1) merge_dpp<0xB1>(best, second);
      if (L > 2) merge_dpp<0x4E>(best, second);
      if (L > 4) merge_dpp<0x141>(best, second);
      if (L > 8) merge_dpp<0x140>(best, second);
      float value = best;
      if (p.group_top2) value = second == -kInf ? best : best + second;
      const int g = l16 >> groups.shift;
      int rank = 0;
      for (int o = 0; o < groups.count; ++o) {
        const float other = __shfl(value, first + (o << groups.shift), 64);
        rank += (other > value) | ((other == value) & (o < g)) ? 1 : 0;
      }
      const bool keep = rank < p.group_topk;
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = keep ? key[i] : -kInf;
    }
    const bool undefined = row_max_u(bad ? 1u : 0u) != 0;
    uint32_t u[V];
#pragma unroll
    for (int i = 0; i < V; ++i) u[i] = ordered(key[i]);
    int id = -1;                 // lane j of a token: slot j's expert and its key
    uint32_t chosen_key = 0;
    for (int j = 0; j < p.k; ++j) {
      uint32_t local = u[0];
#pragma unroll
      for (int i = 1; i < V; ++i) local = max(local, u[i]);
      const uint32_t m = row_max_u(local);
      if (__ballot(m > kNone) == 0) break;
      // the token's lowest lane with the maximum, and its lowest place with it
      const uint32_t with = uint32_t(__ballot(local == m) >> first) & 0xFFFFu;
      bool take = l16 == __builtin_ctz(with | 0x10000u) && m > kNone;
      uint32_t e = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const bool here = take && u[i] == m;
        e = here ? uint32_t(e0 + i) : e;
        u[i] = here ? 0u : u[i];
        take = take && !here;
      }
      e = row_max_u(e);
      if (l16 == j && m > kNone) {
        id = int(e);
        chosen_key = m;
      }
    }
    float chosen = from_ordered(chosen_key);
    if constexpr (BIAS) {        // the key holds the bias too
      chosen = 0.0f;
      if (id >= 0)
        chosen = p.fp32 ? static_cast<const float*>(p.logits)[row * p.ld + id]
                        : to_float(static_cast<const uint16_t*>(p.logits)[row * p.ld + id]);
    }
    float w = score(chosen);
    w = id < 0 ? 0.0f : w;
    if (p.renorm) w = w / (row_sum_f(w) + kRenormEps);
    w *= p.scale;
    if (undefined) {
      id = l16;
      w = __builtin_nanf("");
    }
    if (l16 < p.k && own < p.T) {
      p.ids[own * p.k + l16] = id;
      p.weights[own * p.k + l16] = w;
    }
  }
}

// Backward.  With d_j the gradient of the chosen score s_j and S = sum_l s_l + 1e-20,
//   d_j = scale g_j                                             (weights as they are)
//   d_j = scale (sum_l s_l (g_j - g_l) + 1e-20 g_j) / S^2       (renormalised)
// the logits get  softmax: s_e (d_e - sum_l s_l d_l),  sigmoid: s_e (1 - s_e) d_e
// (the slope without its subtraction; d_e = 0 for experts not chosen).  The
// differences of the g come before their sum: g_j - sum_l s_l g_l / S, the same
// number, is rounding noise where one slot has nearly all of the weight, and for
// k = 1.  Of sum_l s_l d_l only 1e-20 sum_l s_l g_l scale / S^2 is left when
// renormalised.  In the same way, without renormalisation a chosen expert of a
// softmax gets s_j (d_j rest + sum_l s_l (d_j - d_l)), rest the sum of the scores
// that were not chosen.  The choice itself has no gradient; a row whose choice is
// undefined gets NaN.
template <typename T, int N, bool SIGMOID>
__global__ __launch_bounds__(256) void route_backward_kernel(const RouteProblem p) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int e0 = lane * N;
  for (int64_t row = int64_t(blockIdx.x) * 4 + wave; row < p.T; row += int64_t(gridDim.x) * 4) {
    const T* logits = static_cast<const T*>(p.logits) + row * p.ld;
    const int id = lane < p.k ? p.ids[row * p.k + lane] : -1;
    const bool used = id >= 0 && id < p.E;
    float d = used ? p.grad_weights[row * p.k + lane] : 0.0f;
    const float xj = used ? to_float(logits[id]) : -kInf;
    float x[N];
    load_row_of(logits, e0, p.E, x);
    const Scores<SIGMOID> score(x);
    float sj, slope = 1.0f;
    if constexpr (SIGMOID)
      sj = sigmoid_slope(xj, slope);
    else
      sj = score(xj);
    sj = used ? sj : 0.0f;
    float dot = SIGMOID ? 0.0f : wave_sum(sj * d);
    // d becomes d_j, for a softmax d_j - dot (the sums take every lane); scale comes
    // last, since its rounding would show in the differences
    if (p.renorm || !SIGMOID) {
      float t = 0.0f;
      for (int l = 0; l < p.k; ++l) t += lane_value(sj, l) * (d - lane_value(d, l));
      if (p.renorm) {
        const float total = wave_sum(sj) + kRenormEps;
        dot = kRenormEps * dot / total / total;
        d = (t + kRenormEps * d) / total / total - dot;
      } else {
        uint32_t chosen = 0;
        for (int l = 0; l < p.k; ++l) {
          const uint32_t at = uint32_t(__builtin_amdgcn_readlane(id, l) - e0);
          chosen |= at < uint32_t(N) ? 1u << at : 0u;
        }
        float rest = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) rest += chosen >> i & 1 ? 0.0f : score(x[i]);
        d = t + d * wave_sum(rest);
      }
    }
    d *= p.scale;
    dot *= p.scale;
    if constexpr (SIGMOID) d *= slope;
    const bool undefined = __ballot(undefined_logits<SIGMOID>(x)) != 0;
    float g[N];
#pragma unroll
    for (int i = 0; i < N; ++i) g[i] = 0.0f - dot;
    for (int j = 0; j < p.k; ++j) {
      const int e = __builtin_amdgcn_readlane(used ? id : -1, j);
      const float dj = lane_value(d, j);
#pragma unroll
      for (int i = 0; i < N; ++i) g[i] = e == e0 + i ? dj : g[i];
    }
    T* out = static_cast<T*>(p.grad_logits) + row * p.ld_grad;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (!SIGMOID) g[i] *= score(x[i]);
      g[i] = undefined ? __builtin_nanf("") : g[i];
    }
    store_row_of(out, e0, p.E, g);
  }
}

// sum_l s_l (d_j - d_l) over the 16 lanes of a row: the others' values by rotations.
template <int BY = 15>
__device__ __forceinline__ float row_differences(float s, float d) {
  const float sl = __uint_as_float(row_ror<BY>(__float_as_uint(s)));
  const float dl = __uint_as_float(row_ror<BY>(__float_as_uint(d)));
  if constexpr (BY == 1)
    return sl * (d - dl);
  else
    return row_differences<BY - 1>(s, d) + sl * (d - dl);
}

// The same for at most 256 experts and 16 slots, four tokens a wave (see
// route16_kernel).  Logits (sigmoid) or scores and gradients of single experts
// change lanes through LDS, 16 V values a token.
template <typename T, int V, bool SIGMOID>
__global__ __launch_bounds__(256) void route_backward16_kernel(const RouteProblem p) {
  __shared__ __attribute__((aligned(16))) float lds[16][16 * V];
  const int lane = threadIdx.x & 63;
  const int l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int e0 = l16 * V;
  float* values = lds[threadIdx.x >> 4];
  for (int64_t row0 = (int64_t(blockIdx.x) * 4 + wave) * 4; row0 < p.T; row0 += int64_t(gridDim.x) * 16) {
    const int64_t own = row0 + (lane >> 4);
    const int64_t row = min(own, p.T - 1);       // lanes past the last token repeat it and write nothing
    const int id = l16 < p.k ? p.ids[row * p.k + l16] : -1;
    const bool used = id >= 0 && id < p.E;
    float d = l16 < p.k ? p.grad_weights[row * p.k + l16] : 0.0f;
    d = used ? d : 0.0f;
    float x[V], s[V];
    load_row_of(static_cast<const T*>(p.logits) + row * p.ld, e0, p.E, x);
    const Scores<SIGMOID, true> score(x);
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = SIGMOID ? x[i] : score(x[i]);
    float4* mine = reinterpret_cast<float4*>(values + e0);
#pragma unroll
    for (int i = 0; i < V; i += 4) mine[i / 4] = make_float4(s[i], s[i + 1], s[i + 2], s[i + 3]);
    // a wave's LDS accesses are in order: the fences only keep the compiler's
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    float sj = values[used ? id : 0], slope = 1.0f;
    if constexpr (SIGMOID) sj = sigmoid_slope(sj, slope);
    sj = used ? sj : 0.0f;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    float dot = SIGMOID ? 0.0f : row_sum_f(sj * d);
    // d becomes d_j, for a softmax d_j - dot (the sums take every lane); scale comes
    // last, since its rounding would show in the differences
    if (p.renorm) {
      const float total = row_sum_f(sj) + kRenormEps;
      dot = kRenormEps * dot / total / total;
      d = (row_differences(sj, d) + kRenormEps * d) / total / total - dot;
    } else if constexpr (!SIGMOID) {
      if (used) values[id] = 0.0f;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      float rest = 0.0f;
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float4 v = mine[i / 4];
        rest += v.x + v.y + (v.z + v.w);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      d = row_differences(sj, d) + d * row_sum_f(rest);
    }
    d *= p.scale;
    dot *= p.scale;
    if constexpr (SIGMOID) d *= slope;
    const bool undefined = row_max_u(undefined_logits<SIGMOID>(x) ? 1u : 0u) != 0;
    const float others = 0.0f - dot;
#pragma unroll
    for (int i = 0; i < V; i += 4) mine[i / 4] = make_float4(others, others, others, others);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (used) values[id] = d;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    float g[V];
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 de = mine[i / 4];
      g[i] = de.x, g[i + 1] = de.y, g[i + 2] = de.z, g[i + 3] = de.w;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (!SIGMOID) g[i] *= s[i];
      g[i] = undefined ? __builtin_nanf("") : g[i];
    }
    if (own < p.T) store_row_of(static_cast<T*>(p.grad_logits) + own * p.ld_grad, e0, p.E, g);
  }
}

// Workgroups of four tokens, which take further tokens in turns past this.
dim3 token_grid(int64_t T) {
  const int64_t blocks = (T + 3) / 4;
  return dim3(unsigned(blocks < 4096 ? blocks : 4096));
}

template <int N, bool SIGMOID>
hipError_t run_route(const RouteProblem& p, hipStream_t st) {
  const bool groups = p.group_topk < p.groups;
  const Groups g(p, N);
  const auto run = [&](auto kernel) {
    const size_t lds = groups && !g.whole ? size_t(4) * p.E * sizeof(float) : 0;
    hipLaunchKernelGGL(kernel, token_grid(p.T), dim3(256), lds, st, p, g);
    return hipGetLastError();
  };
  if (p.bias) return groups ? run(route_kernel<N, SIGMOID, true, true>) : run(route_kernel<N, SIGMOID, true, false>);
  return groups ? run(route_kernel<N, SIGMOID, false, true>) : run(route_kernel<N, SIGMOID, false, false>);
}

template <int V, bool SIGMOID>
hipError_t run_route16(const RouteProblem& p, hipStream_t st) {
  const bool groups = p.group_topk < p.groups;
  const Groups g(p, V);
  const auto run = [&](auto kernel) {
    const int64_t blocks = (p.T + 15) / 16;
    hipLaunchKernelGGL(kernel, dim3(unsigned(blocks < 4096 ? blocks : 4096)), dim3(256), 0, st, p, g);
    return hipGetLastError();
  };
  if (p.bias)
    return groups ? run(route16_kernel<V, SIGMOID, true, true>) : run(route16_kernel<V, SIGMOID, true, false>);
  return groups ? run(route16_kernel<V, SIGMOID, false, true>) : run(route16_kernel<V, SIGMOID, false, false>);
}

template <int V, bool SIGMOID>
hipError_t run_route_backward16(const RouteProblem& p, hipStream_t st) {
  const int64_t blocks = (p.T + 15) / 16;
  const dim3 grid(unsigned(blocks < 4096 ? blocks : 4096));
  if (p.fp32)
    hipLaunchKernelGGL((route_backward16_kernel<float, V, SIGMOID>), grid, dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((route_backward16_kernel<uint16_t, V, SIGMOID>), grid, dim3(256), 0, st, p);
  return hipGetLastError();
}

template <int V>
hipError_t route16_of(const RouteProblem& p, bool backward, hipStream_t st) {
  if (backward) return p.sigmoid ? run_route_backward16<V, true>(p, st) : run_route_backward16<V, false>(p, st);
  return p.sigmoid ? run_route16<V, true>(p, st) : run_route16<V, false>(p, st);
}

// Whether the four-tokens form serves: V experts a lane of 16.
bool takes_route16(const RouteProblem& p, int V) {
  return p.E <= 16 * V && p.k <= 16 && (p.group_topk == p.groups || Groups(p, V).whole);
}

template <int N, bool SIGMOID>
hipError_t run_route_backward(const RouteProblem& p, hipStream_t st) {
  if (p.fp32)
    hipLaunchKernelGGL((route_backward_kernel<float, N, SIGMOID>), token_grid(p.T), dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((route_backward_kernel<uint16_t, N, SIGMOID>), token_grid(p.T), dim3(256), 0, st, p);
  return hipGetLastError();
}

template <int N>
hipError_t route_of(const RouteProblem& p, bool backward, hipStream_t st) {
  if (backward) return p.sigmoid ? run_route_backward<N, true>(p, st) : run_route_backward<N, false>(p, st);
  return p.sigmoid ? run_route<N, true>(p, st) : run_route<N, false>(p, st);
}

hipError_t route_any(const RouteProblem& p, bool backward, hipStream_t st) {
  if (p.T == 0) return hipSuccess;
  if (takes_route16(p, 4)) return route16_of<4>(p, backward, st);
  if (takes_route16(p, 8)) return route16_of<8>(p, backward, st);
  if (takes_route16(p, 16)) return route16_of<16>(p, backward, st);
  if (p.E <= 64) return route_of<1>(p, backward, st);
  if (p.E <= 128) return route_of<2>(p, backward, st);
  if (p.E <= 256) return route_of<4>(p, backward, st);
  if (p.E <= 512) return route_of<8>(p, backward, st);
  return route_of<16>(p, backward, st);
}

}  // namespace

hipError_t launch_route(const RouteProblem& p, hipStream_t st) { return route_any(p, false, st); }

hipError_t launch_route_backward(const RouteProblem& p, hipStream_t st) { return route_any(p, true, st); }

}  // namespace fp8mm
