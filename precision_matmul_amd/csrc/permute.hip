// Token permutation of an expert layer (gfx950): the plan that puts every
// (token, slot) into expert order, the move of token rows there (dispatch, as
// rows or as 1x128 FP8 codes) and the weighted sum back (combine), with its
// backward pass.
//
// Slot n = t k + j of token t goes to the row that a stable sort of the slots
// by expert gives it; slots without an expert (id outside [0, E)) take the
// rows after the last expert's.  row_of_slot holds the row, or ~row for a slot
// without an expert, so that its values are all different rows and the
// dispatch writes every row: zeros (code 0, scale 1) where there is no expert.
#include "moe_launch.hpp"
#include "ops_common.hpp"
#include "quant_cast.hpp"

namespace fp8mm {
namespace {

using namespace ops;

// ---------------------------------------------------------------------------
// Plan: a counting sort.  The slots are cut into chunks; a first launch counts
// each chunk's slots per expert, a second one adds up the counts before each
// chunk and places its slots, 64 at a time in order (a lane's rank among the
// lanes of its wave with the same expert by ballots over the expert's bits).
// Counts are integers and every slot's row is its rank, so the result does not
// depend on the order of the LDS atomics.  One chunk alone needs no first
// launch.  Latency-bound: 8 bytes a slot.  98304 slots, 64 experts: 5 and 6 us;
// 96 slots: 3.5 us (four ids in flight a lane: no faster).
// ---------------------------------------------------------------------------
constexpr int64_t kPlanSingle = 4096;    // slots that one workgroup places alone
constexpr int64_t kPlanChunks = 64;      // chunks at most: the second launch reads all their counts

// A slot's key: its expert, or E without one.
__device__ __forceinline__ int plan_key(int32_t id, int E) { return id >= 0 && id < E ? id : E; }

__global__ __launch_bounds__(1024) void plan_count_kernel(const int32_t* __restrict__ ids, int64_t n, int64_t chunk,
                                                          int E, int* __restrict__ hist) {
  extern __shared__ int cnt[];         // [E + 1]
  for (int e = threadIdx.x; e <= E; e += blockDim.x) cnt[e] = 0;
  __syncthreads();
  const int64_t c0 = int64_t(blockIdx.x) * chunk;
  const int64_t end = min(n, c0 + chunk);
  for (int64_t i = c0 + threadIdx.x; i < end; i += blockDim.x) atomicAdd(&cnt[plan_key(ids[i], E)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += blockDim.x) hist[int64_t(blockIdx.x) * (E + 1) + e] = cnt[e];
}

// W waves a workgroup.  LDS: cnt [W][E + 1] counts, then places, of each wave;
// total and before [E + 1] slots of an expert in all chunks and in the earlier
// ones.
template <int W>
__global__ __launch_bounds__(64 * W) void plan_place_kernel(const int32_t* __restrict__ ids, int64_t n, int64_t chunk,
                                                          int E, int bits, const int* __restrict__ hist,
                                                          int32_t* __restrict__ offsets, int32_t* __restrict__ rows) {
  extern __shared__ int lds[];
  __shared__ int wave_total[W];
  constexpr int threads = 64 * W;
  const int E1 = E + 1;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  int* cnt = lds + wave * E1;
  int* total = lds + W * E1;
  int* before = total + E1;
  for (int i = t; i < (W + 2) * E1; i += threads) lds[i] = 0;
  const int64_t part = chunk / W;
  const int64_t a = min(n, int64_t(blockIdx.x) * chunk + int64_t(wave) * part);
  const int64_t b = min(n, a + part);
  __syncthreads();
  for (int64_t i = a + lane; i < b; i += 64) atomicAdd(&cnt[plan_key(ids[i], E)], 1);
  if (hist) {
    // the chunks dealt out to threads / E1 threads an expert
    const int sets = max(1, threads / E1);
    for (int i = t; i < sets * E1; i += threads) {
      const int set = i / E1, e = i - set * E1;
      int all = 0, early = 0;
#pragma unroll 4
      for (int c = set; c < int(gridDim.x); c += sets) {
        const int h = hist[int64_t(c) * E1 + e];
        all += h;
        early += c < int(blockIdx.x) ? h : 0;
      }
      atomicAdd(&total[e], all);
      atomicAdd(&before[e], early);
    }
  }
  __syncthreads();
  for (int e = t; e < E1; e += threads) {
    int at = before[e];
    // the waves' first places relative to the expert's first row
    int h[W];
#pragma unroll
    for (int w = 0; w < W; ++w) h[w] = lds[w * E1 + e];
#pragma unroll
    for (int w = 0; w < W; ++w) {
      lds[w * E1 + e] = at;
      at += h[w];
    }
    if (!hist) total[e] = at;
  }
  __syncthreads();
  // exclusive scan of total: thread t owns `per` consecutive experts
  const int per = (E1 + threads - 1) / threads;
  const int s0 = min(E1, t * per), s1 = min(E1, s0 + per);
  int sum = 0;
  for (int e = s0; e < s1; ++e) sum += total[e];
  int incl = sum;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int v = __shfl_up(incl, off, 64);
    if (lane >= off) incl += v;
  }
  if (lane == 63) wave_total[wave] = incl;
  __syncthreads();
  int start = incl - sum;
#pragma unroll
  for (int w = 0; w < W; ++w) start += w < wave ? wave_total[w] : 0;
  for (int e = s0; e < s1; ++e) {
    before[e] = start;                 // from here on: the expert's first row
    start += total[e];
    if (blockIdx.x == 0 && e < E) offsets[e] = start;
  }
  __syncthreads();
  for (int64_t i0 = a; i0 < b; i0 += 64) {
    const int64_t i = i0 + lane;
    const bool here = i < b;
    const int key = here ? plan_key(ids[i], E) : 0;
    uint64_t peers = __ballot(here);
    for (int bit = 0; bit < bits; ++bit) {
      const bool set = (key >> bit) & 1;
      const uint64_t with = __ballot(set);
      peers &= set ? with : ~with;
    }
    const uint64_t lower = peers & ((1ull << lane) - 1);
    if (here) {
      const int row = before[key] + cnt[key] + __popcll(lower);
      rows[i] = key == E ? ~row : row;
    }
    // every lane has read its expert's place before its last peer moves it on
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (here && (peers >> lane) == 1) cnt[key] += __popcll(peers);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

// This wave's item: the host keeps items below 2^26 (a launch's threads below
// 2^32), and one item is a wave's, so its arithmetic is scalar and 32-bit.
__device__ __forceinline__ uint32_t wave_item(uint32_t workgroup) {
  return uint32_t(__builtin_amdgcn_readfirstlane(int(workgroup * 4 + (threadIdx.x >> 6))));
}

struct Slot {
  int64_t row;
  bool used;
};

__device__ __forceinline__ Slot slot_row(int32_t v) { return Slot{int64_t(v < 0 ? ~v : v), v >= 0}; }

// ---------------------------------------------------------------------------
// Dispatch: one wave an item of 64 chunks of one token, read once and written
// to the token's k rows.  HBM-bound: (1 + k) rows a token.  16384 x 2048 x 6
// bf16 with the plan: 87 us, 5.4 TB/s (plain stores 100 us); 40 MiB of rows 8.5 us
// against 8.9, 24 MiB the same, but 96 MiB 20.1 against 18.6.
// ---------------------------------------------------------------------------
template <typename T, bool NT>
__global__ __launch_bounds__(256) void dispatch_kernel(const PermuteProblem p, int strips) {
  const int lane = threadIdx.x & 63;
  const uint32_t item = wave_item(blockIdx.x);
  const uint32_t token = item / uint32_t(strips);
  if (token >= p.T) return;
  const int64_t c = (int64_t(item - token * uint32_t(strips)) * 64 + lane) * kVec<T>;
  const int64_t M = p.T * p.k;
  const Chunk v = load_row(static_cast<const T*>(p.x) + int64_t(token) * p.ld_x, c, p.C);
  for (int j = 0; j < p.k; ++j) {
    const Slot s = slot_row(p.row_of_slot[int64_t(token) * p.k + j]);
    if (s.row >= M) continue;
    store_row<T, NT>(static_cast<T*>(p.out) + s.row * p.ld_out, c, p.C, s.used ? v : Chunk{{0u, 0u, 0u, 0u}});
  }
}

// FP8: a wave covers 1024 columns of one token, 16 consecutive ones a lane, 8
// lanes a group of 128; codes and scales as the 1x128 quantizer makes them, each
// token quantized once.  A slot's scales are single floats a whole row of slots
// apart: with a contiguous range of tokens an XCD, neighbouring rows of an
// expert meet in one L2 before they go out.  16384 x 2048 x 6: 41 us, 6.7 TB/s
// of x, codes and scales (plain code stores 53, tokens in launch order 58 with
// the streaming ones); 40 MiB of codes 10.7 us against 11.2, 24 MiB the same.
template <bool NT>
__global__ __launch_bounds__(256) void dispatch_fp8_kernel(const PermuteProblem p, int strips) {
  const int lane = threadIdx.x & 63;
  const uint32_t item = wave_item(xcd_position());
  const uint32_t token = item / uint32_t(strips);
  if (token >= p.T) return;
  const int64_t c = (int64_t(item - token * uint32_t(strips)) * 64 + lane) * 16;
  if (c >= p.C) return;                  // C % 128 == 0: whole groups of 8 lanes leave
  const int64_t M = p.T * p.k;
  const uint16_t* x = static_cast<const uint16_t*>(p.x) + int64_t(token) * p.ld_x + c;
  const U16x8 v0 = load16(x), v1 = load16(x + 8);
  const uint32_t m = group8_max(max(absmax8(v0), absmax8(v1)));
  const float s = scale_from_amax(bf16_to_f32(uint16_t(m)), 0.0f, false);
  const CastScale cs = make_cast_scale(s);
  const uint2 q0 = cast8(v0, cs), q1 = cast8(v1, cs);
  const Chunk q{{q0.x, q0.y, q1.x, q1.y}};
  for (int j = 0; j < p.k; ++j) {
    const Slot slot = slot_row(p.row_of_slot[int64_t(token) * p.k + j]);
    if (slot.row >= M) continue;
    const Chunk codes = slot.used ? q : Chunk{{0u, 0u, 0u, 0u}};
    uint32_t* out = reinterpret_cast<uint32_t*>(p.q + slot.row * p.ld_q + c);
    NT ? store_chunk_nt(out, codes) : store_chunk(out, codes);
    if ((lane & 7) == 0) p.scale[(c / 128) * M + slot.row] = slot.used ? s : 1.0f;
  }
}

// ---------------------------------------------------------------------------
// Combine: one wave an item of 64 chunks of one token; its k rows are added in
// slot order in float32.  HBM-bound: (k + 1) rows a token.  16384 x 2048 x 6: 80
// us, 5.9 TB/s; 4099 x 2048 x 6, 1 of 20 slots empty: 21 us, 5.2 TB/s; 8000 x
// 2375 x 4: 38 us (47 where a row's last elements are loaded one by one).
// ---------------------------------------------------------------------------
template <typename T, bool NT>
__global__ __launch_bounds__(256) void combine_kernel(const PermuteProblem p, int strips) {
  constexpr int V = kVec<T>;
  const int lane = threadIdx.x & 63;
  const uint32_t item = wave_item(blockIdx.x);
  const uint32_t token = item / uint32_t(strips);
  if (token >= p.T) return;
  const int64_t c = (int64_t(item - token * uint32_t(strips)) * 64 + lane) * V;
  const int64_t M = p.T * p.k;
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0f;
#pragma unroll 4
  for (int j = 0; j < p.k; ++j) {
    const Slot s = slot_row(p.row_of_slot[int64_t(token) * p.k + j]);
    if (!s.used || s.row >= M) continue;
    const float w = p.weights ? p.weights[int64_t(token) * p.k + j] : 1.0f;
    float f[V];
    const T* row = static_cast<const T*>(p.rows) + s.row * p.ld_rows;
    unpack<T>(fetched<T>(fetch_row<T, NT>(row, c, p.C), c, p.C), f);
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] += w * f[i];
  }
  store_row(static_cast<T*>(p.out) + int64_t(token) * p.ld_out, c, p.C, pack<T>(acc));
}

// Combine's backward: grad_rows[row] = w g, grad_weights[t, j] = <g, rows[row]>.
// LANES lanes a slot (a wave, or 16 for rows of at most one chunk a lane of a wave),
// U chunks a lane in flight: a token's k slots are neighbours and share its gradient
// through the caches.  HBM-bound: (1 + 2 k) rows a token.  16384 x 2048, k = 6:
// 154 us, 5.7 TB/s.  In us, the other choice in brackets:
//   streaming stores 16384 x 2048 154 (plain 169)
//   16 lanes a slot, rows of at most one chunk of a wave: 16000 x 256, k = 4 13 (a
//   wave 19), 512 columns 24 (25)
//   PART, a row's last chunk loaded whole and shifted: 16000 x 339 24 (30); long
//   rows 34 without (4000 x 2048, 38 with it)
template <typename T, bool LD, bool ST, int LANES, int U, bool PART>
__global__ __launch_bounds__(256) void combine_backward_kernel(const PermuteProblem p) {
  constexpr int V = kVec<T>;
  const int lane = threadIdx.x & (LANES - 1);
  uint32_t slot = wave_item(blockIdx.x) * (64 / LANES);
  if constexpr (LANES < 64) slot += (threadIdx.x & 63) / LANES;
  const int64_t M = p.T * p.k;
  if (slot >= M) return;                 // whole groups of LANES leave
  const uint32_t token = slot / uint32_t(p.k);
  const T* g_row = static_cast<const T*>(p.x) + int64_t(token) * p.ld_x;
  const Slot s = slot_row(p.row_of_slot[slot]);
  const bool inside = s.row < M;
  const float w = p.weights && s.used ? p.weights[slot] : 1.0f;
  const T* r = s.used && inside && p.grad_weights ? static_cast<const T*>(p.rows) + s.row * p.ld_rows : nullptr;
  T* o = inside && p.out ? static_cast<T*>(p.out) + s.row * p.ld_out : nullptr;
  float dot = 0.0f;
  for (int64_t c0 = int64_t(lane) * V; c0 < p.C; c0 += LANES * V * U) {
    Chunk vg[U], vr[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = c0 + u * LANES * V;
      vg[u] = PART ? fetch_row<T, false>(g_row, c, p.C) : load_row(g_row, c, p.C);
      vr[u] = Chunk{{0u, 0u, 0u, 0u}};
      if (r) vr[u] = PART ? fetch_row<T, LD>(r, c, p.C) : load_row<T, LD>(r, c, p.C);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (PART) {
        vg[u] = fetched<T>(vg[u], c0 + u * LANES * V, p.C);
        if (r) vr[u] = fetched<T>(vr[u], c0 + u * LANES * V, p.C);
      }
      float g[V], f[V];
      unpack<T>(vg[u], g);
      unpack<T>(vr[u], f);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (r) dot += g[i] * f[i];
        f[i] = s.used ? w * g[i] : 0.0f;
      }
      if (o) store_row<T, ST>(o, c0 + u * LANES * V, p.C, pack<T>(f));
    }
  }
  dot = LANES == 64 ? wave_sum(dot) : row_sum_f(dot);
  if (p.grad_weights && lane == 0) p.grad_weights[slot] = dot;
}

int64_t rows_bytes(const PermuteProblem& p) { return p.T * p.k * p.C * (p.fp32 ? 4 : 2); }

// Expert-order rows of more than twice the L2s are read by streaming loads:
// combine of 16384 x 2048 x 6 (403 MB) 80 against 92 us, of 134 MB 30 against 34,
// of 100 MB 21.2 against 21.9; of 25 MB 7.1 against 6.8.
bool rows_stream(const PermuteProblem& p) { return rows_bytes(p) > 2 * kL2Bytes; }

int64_t plan_chunk(int64_t n) {
  const int64_t c = n <= kPlanSingle ? n : (n + kPlanChunks - 1) / kPlanChunks;
  return (c + 1023) / 1024 * 1024;
}

}  // namespace

int64_t plan_workspace(int64_t n, int64_t E) {
  if (n <= kPlanSingle) return 0;
  const int64_t chunk = plan_chunk(n);
  return (n + chunk - 1) / chunk * (E + 1) * int64_t(sizeof(int32_t));
}

hipError_t launch_plan(const int32_t* ids, int64_t n, int E, int32_t* offsets, int32_t* row_of_slot,
                       int32_t* workspace, hipStream_t st) {
  const bool single = n <= kPlanSingle;
  const int64_t chunk = n ? plan_chunk(n) : 1024;
  const unsigned chunks = unsigned(n ? (n + chunk - 1) / chunk : 1);
  if (!single) {
    hipLaunchKernelGGL(plan_count_kernel, dim3(chunks), dim3(1024), size_t(E + 1) * 4, st, ids, n, chunk, E, workspace);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int bits = 32 - __builtin_clz(unsigned(E));    // of keys 0 .. E
  const auto place = [&](auto kernel, int W) {
    hipLaunchKernelGGL(kernel, dim3(chunks), dim3(64 * W), size_t(W + 2) * (E + 1) * 4, st, ids, n, chunk, E, bits,
                       single ? nullptr : workspace, offsets, row_of_slot);
    return hipGetLastError();
  };
  // waves that share a chunk: fewer for few slots, and where their counts in
  // LDS would pass 64 KiB
  if (n <= 512) return place(plan_place_kernel<4>, 4);
  return E > 512 ? place(plan_place_kernel<8>, 8) : place(plan_place_kernel<16>, 16);
}

hipError_t launch_dispatch(const PermuteProblem& p, hipStream_t st) {
  if (p.T == 0 || p.C == 0) return hipSuccess;
  const int strips = int((p.C + row_columns(p.fp32) - 1) / row_columns(p.fp32));
  const auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(unsigned((p.T * strips + 3) / 4)), dim3(256), 0, st, p, strips);
    return hipGetLastError();
  };
  const bool nt = rows_bytes(p) > kL2Bytes;
  if (p.fp32) return nt ? run(dispatch_kernel<float, true>) : run(dispatch_kernel<float, false>);
  return nt ? run(dispatch_kernel<uint16_t, true>) : run(dispatch_kernel<uint16_t, false>);
}

hipError_t launch_dispatch_fp8(const PermuteProblem& p, hipStream_t st) {
  if (p.T == 0 || p.C == 0) return hipSuccess;
  const int strips = int((p.C + kCodeColumns - 1) / kCodeColumns);
  const dim3 grid(xcd_grid((p.T * strips + 3) / 4));
  if (p.T * p.k * p.C > kL2Bytes)
    hipLaunchKernelGGL((dispatch_fp8_kernel<true>), grid, dim3(256), 0, st, p, strips);
  else
    hipLaunchKernelGGL((dispatch_fp8_kernel<false>), grid, dim3(256), 0, st, p, strips);
  return hipGetLastError();
}

hipError_t launch_combine(const PermuteProblem& p, hipStream_t st) {
  if (p.T == 0 || p.C == 0) return hipSuccess;
  const int strips = int((p.C + row_columns(p.fp32) - 1) / row_columns(p.fp32));
  const auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(unsigned((p.T * strips + 3) / 4)), dim3(256), 0, st, p, strips);
    return hipGetLastError();
  };
  if (p.fp32) return rows_stream(p) ? run(combine_kernel<float, true>) : run(combine_kernel<float, false>);
  return rows_stream(p) ? run(combine_kernel<uint16_t, true>) : run(combine_kernel<uint16_t, false>);
}

template <typename T, int LANES, int U, bool PART>
static hipError_t run_combine_backward(const PermuteProblem& p, hipStream_t st) {
  const auto run = [&](auto kernel) {
    const int64_t slots = 256 / LANES;   // of a workgroup
    hipLaunchKernelGGL(kernel, dim3(unsigned((p.T * p.k + slots - 1) / slots)), dim3(256), 0, st, p);
    return hipGetLastError();
  };
  if (rows_stream(p)) return run(combine_backward_kernel<T, true, true, LANES, U, PART>);
  return rows_bytes(p) > kL2Bytes ? run(combine_backward_kernel<T, false, true, LANES, U, PART>)
                                  : run(combine_backward_kernel<T, false, false, LANES, U, PART>);
}

template <typename T>
static hipError_t combine_backward_of(const PermuteProblem& p, hipStream_t st) {
  if (slot_lanes(p.C, p.fp32) == 64) return run_combine_backward<T, 64, 4, false>(p, st);
  return p.C % kVec<T> ? run_combine_backward<T, 16, 2, true>(p, st) : run_combine_backward<T, 16, 2, false>(p, st);
}

hipError_t launch_combine_backward(const PermuteProblem& p, hipStream_t st) {
  if (p.T == 0) return hipSuccess;
  return p.fp32 ? combine_backward_of<float>(p, st) : combine_backward_of<uint16_t>(p, st);
}

}  // namespace fp8mm
