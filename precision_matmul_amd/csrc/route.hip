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
// One wave a token, N = ceil(E / 64) consecutive experts a lane, everything in
// registers.  The logits are read once (T E values against T k results), so a
// large batch is bound by instructions: k selection rounds of a wave maximum
// (six data-parallel steps), a ballot and a lane read.
#include "moe_launch.hpp"
#include "ops_common.hpp"

namespace fp8mm {
namespace {

using namespace ops;

constexpr float kInf = __builtin_inff();

template <typename T, int N>
__device__ __forceinline__ void load_logits(const T* row, int e0, int E, float (&x)[N]) {
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

// Scores of a row: softmax(x) = exp(x - shift) * inv, sigmoid(x).
struct Scores {
  bool sigmoid;
  float shift, inv;
  __device__ __forceinline__ float operator()(float x) const {
    return sigmoid ? 1.0f / (1.0f + expf(-x)) : expf(x - shift) * inv;
  }
};

template <int N>
__device__ __forceinline__ Scores row_scores(const float (&x)[N], bool sigmoid) {
  Scores s{sigmoid, 0.0f, 1.0f};
  if (!sigmoid) {
    float m = x[0];
#pragma unroll
    for (int i = 1; i < N; ++i) m = fmaxf(m, x[i]);
    m = wave_max_f(m);
    s.shift = m == -kInf ? 0.0f : m;           // a row of -inf alone: every score 0
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) sum += expf(x[i] - s.shift);
    sum = wave_sum(sum);
    s.inv = sum == 0.0f ? 1.0f : 1.0f / sum;
  }
  return s;
}

// Group selection: keys of experts outside the chosen groups become -inf.
// L = 64 / G rounded down to a power of two lanes work on each group, reading
// its values from LDS, then merge their two best by butterfly.
template <int N>
__device__ __forceinline__ void keep_groups(float (&key)[N], const float (&value)[N], int e0, const RouteProblem& p,
                                            float* lds) {
  const int lane = threadIdx.x & 63;
  const int gs = p.E / p.groups;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (e0 + i < p.E) lds[e0 + i] = p.group_top2 ? value[i] : key[i];
  // the wave reads what its own lanes wrote: in order, no barrier needed
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  const int shift = 31 - __builtin_clz(unsigned(64 / p.groups));
  const int L = 1 << shift;
  const int g = lane >> shift;
  float best = -kInf, second = -kInf;
  if (g < p.groups) {
    for (int j = lane & (L - 1); j < gs; j += L) {
      const float v = lds[g * gs + j];
      second = fmaxf(second, fminf(best, v));
      best = fmaxf(best, v);
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  for (int off = 1; off < L; off <<= 1) {
    const float b = __shfl_xor(best, off, 64), s = __shfl_xor(second, off, 64);
    second = fmaxf(fmaxf(second, s), fminf(best, b));
    best = fmaxf(best, b);
  }
  float score = best;
  if (p.group_top2 && second != -kInf) score = best + second;
  int rank = 0;
  for (int o = 0; o < p.groups; ++o) {
    const float other = lane_value(score, o << shift);
    rank += other > score || (other == score && o < g) ? 1 : 0;
  }
  const uint64_t kept = __ballot(g < p.groups && rank < p.group_topk);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = e0 + i;
    if (e < p.E && !((kept >> ((e / gs) << shift)) & 1)) key[i] = -kInf;
  }
}

template <typename T, int N, bool BIAS>
__global__ __launch_bounds__(256) void route_kernel(const RouteProblem p) {
  extern __shared__ float lds_all[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e0 = lane * N;
  float b[N];
  if constexpr (BIAS) {
#pragma unroll
    for (int i = 0; i < N; ++i) b[i] = e0 + i < p.E ? p.bias[e0 + i] : 0.0f;
  }
  for (int64_t row = int64_t(blockIdx.x) * 4 + wave; row < p.T; row += int64_t(gridDim.x) * 4) {
    float x[N], key[N];
    load_logits<T, N>(static_cast<const T*>(p.logits) + row * p.ld, e0, p.E, x);
    bool bad = false;
#pragma unroll
    for (int i = 0; i < N; ++i) bad |= x[i] != x[i] || (!p.sigmoid && x[i] == kInf);
    const Scores score = row_scores(x, p.sigmoid);
    const bool by_groups = p.group_topk < p.groups;
    if constexpr (BIAS) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        key[i] = x[i] == -kInf ? -kInf : score(x[i]) + b[i];
        bad |= key[i] != key[i];
      }
      if (by_groups) {
        const float (&value)[N] = key;
        float keep[N];
#pragma unroll
        for (int i = 0; i < N; ++i) keep[i] = value[i];
        keep_groups(key, keep, e0, p, lds_all + wave * p.E);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) key[i] = x[i];
      if (by_groups) {
        float value[N];
#pragma unroll
        for (int i = 0; i < N; ++i) value[i] = p.group_top2 && x[i] != -kInf ? score(x[i]) : -kInf;
        keep_groups(key, value, e0, p, lds_all + wave * p.E);
      }
    }
    const bool none_defined = __ballot(bad) != 0;
    int id = -1;            // lane j: slot j's expert and its logit
    float logit = 0.0f;
    for (int j = 0; j < p.k; ++j) {
      float local = key[0];
#pragma unroll
      for (int i = 1; i < N; ++i) local = fmaxf(local, key[i]);
      const float m = wave_max_f(local);
      if (m == -kInf) break;
      // the lowest lane with the maximum, and its lowest element with it
      const int from = int(__builtin_ctzll(__ballot(local == m) | (1ull << 63)));
      int at = 0;
      float xl = x[0];
      bool found = key[0] == m;
#pragma unroll
      for (int i = 1; i < N; ++i) {
        const bool here = !found && key[i] == m;
        at = here ? i : at;
        if constexpr (BIAS) xl = here ? x[i] : xl;
        found |= here;
      }
      const int e = from * N + __builtin_amdgcn_readlane(at, from);
      const float xe = BIAS ? lane_value(xl, from) : m;
      id = lane == j ? e : id;
      logit = lane == j ? xe : logit;
#pragma unroll
      for (int i = 0; i < N; ++i) key[i] = lane == from && at == i ? -kInf : key[i];
    }
    float w = id < 0 ? 0.0f : score(logit);
    if (p.renorm) w = w / (wave_sum(w) + kRenormEps);
    w *= p.scale;
    if (none_defined) {
      id = lane;
      w = __builtin_nanf("");
    }
    if (lane < p.k) {
      p.ids[row * p.k + lane] = id;
      p.weights[row * p.k + lane] = w;
    }
  }
}

// Backward.  With d_j the gradient of the chosen score s_j,
//   d_j = scale g_j                                     (weights as they are)
//   d_j = scale (g_j - sum_l g_l s_l / S) / S, S = sum_l s_l + 1e-20   (renormalised)
// the logits get  softmax: s_e (d_e - sum_l s_l d_l),  sigmoid: s_e (1 - s_e) d_e
// (d_e = 0 for experts not chosen).  The choice itself has no gradient.
template <typename T, int N>
__global__ __launch_bounds__(256) void route_backward_kernel(const RouteProblem p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e0 = lane * N;
  for (int64_t row = int64_t(blockIdx.x) * 4 + wave; row < p.T; row += int64_t(gridDim.x) * 4) {
    const T* logits = static_cast<const T*>(p.logits) + row * p.ld;
    float x[N];
    load_logits<T, N>(logits, e0, p.E, x);
    const int id = lane < p.k ? p.ids[row * p.k + lane] : -1;
    const bool used = id >= 0 && id < p.E;
    float d = used ? p.grad_weights[row * p.k + lane] * p.scale : 0.0f;
    const float xj = used ? to_float(logits[id]) : -kInf;
    const Scores score = row_scores(x, p.sigmoid);
    const float sj = used ? score(xj) : 0.0f;
    if (p.renorm) {
      // the sums take every lane: outside the choice of d
      const float total = wave_sum(sj) + kRenormEps;
      const float mean = wave_sum(d * sj) / total;
      d = used ? (d - mean) / total : 0.0f;
    }
    const float dot = p.sigmoid ? 0.0f : wave_sum(sj * d);
    float de[N];
#pragma unroll
    for (int i = 0; i < N; ++i) de[i] = 0.0f;
    for (int j = 0; j < p.k; ++j) {
      const int e = __builtin_amdgcn_readlane(id, j);
      const float dj = lane_value(d, j);
#pragma unroll
      for (int i = 0; i < N; ++i) de[i] += e == e0 + i ? dj : 0.0f;
    }
    T* out = static_cast<T*>(p.grad_logits) + row * p.ld_grad;
    float g[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float s = score(x[i]);
      g[i] = p.sigmoid ? s * (1.0f - s) * de[i] : s * (de[i] - dot);
    }
    struct __attribute__((packed, aligned(sizeof(T)))) At {
      T v[N];
    };
    if (e0 + N <= p.E) {
      At a;
#pragma unroll
      for (int i = 0; i < N; ++i) a.v[i] = from_float<T>(g[i]);
      *reinterpret_cast<At*>(out + e0) = a;
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (e0 + i < p.E) out[e0 + i] = from_float<T>(g[i]);
    }
  }
}

// Workgroups of four tokens, which take further tokens in turns past this.
dim3 token_grid(int64_t T) {
  const int64_t blocks = (T + 3) / 4;
  return dim3(unsigned(blocks < (1 << 20) ? blocks : (1 << 20)));
}

template <typename T, int N>
hipError_t run_route(const RouteProblem& p, hipStream_t st) {
  const size_t lds = p.group_topk < p.groups ? size_t(4) * p.E * sizeof(float) : 0;
  if (p.bias)
    hipLaunchKernelGGL((route_kernel<T, N, true>), token_grid(p.T), dim3(256), lds, st, p);
  else
    hipLaunchKernelGGL((route_kernel<T, N, false>), token_grid(p.T), dim3(256), lds, st, p);
  return hipGetLastError();
}

template <typename T, int N>
hipError_t run_route_backward(const RouteProblem& p, hipStream_t st) {
  hipLaunchKernelGGL((route_backward_kernel<T, N>), token_grid(p.T), dim3(256), 0, st, p);
  return hipGetLastError();
}

template <typename T>
hipError_t route_typed(const RouteProblem& p, bool backward, hipStream_t st) {
  if (p.E <= 64) return backward ? run_route_backward<T, 1>(p, st) : run_route<T, 1>(p, st);
  if (p.E <= 128) return backward ? run_route_backward<T, 2>(p, st) : run_route<T, 2>(p, st);
  if (p.E <= 256) return backward ? run_route_backward<T, 4>(p, st) : run_route<T, 4>(p, st);
  if (p.E <= 512) return backward ? run_route_backward<T, 8>(p, st) : run_route<T, 8>(p, st);
  return backward ? run_route_backward<T, 16>(p, st) : run_route<T, 16>(p, st);
}

}  // namespace

hipError_t launch_route(const RouteProblem& p, hipStream_t st) {
  if (p.T == 0) return hipSuccess;
  return p.fp32 ? route_typed<float>(p, false, st) : route_typed<uint16_t>(p, false, st);
}

hipError_t launch_route_backward(const RouteProblem& p, hipStream_t st) {
  if (p.T == 0) return hipSuccess;
  return p.fp32 ? route_typed<float>(p, true, st) : route_typed<uint16_t>(p, true, st);
}

}  // namespace fp8mm
