// Routing: the choice of k experts by logits, the order of the chosen slots by
// expert, and the choice's gradient.
//
// A warp takes a token, a lane every 32nd expert. Logits become integers of
// the same order (NaN on top, -0 as +0), so the largest is found by one
// reduction over the warp and the lowest expert among equals by another; taken
// ones are struck out and the next round follows. Blocks hold neighbouring
// tokens and count their choices by expert (k_choose); then every block adds up
// what the blocks before it have taken of each expert and places its own slots
// in order (k_order): a stable counting sort, no order left to atomics. Of few
// tokens one block does both. Bound by latencies: 8192 tokens by 16 experts, 2 each, take
// 7.8 us captured (7 and 8 us for the two kernels alone and cold, at 17 and 20 % of the
// issue slots).
#include "block.h"
#include "bulk.cuh"
#include "experts.h"
#include "vec.cuh"

namespace zg {
namespace {

constexpr int kRouteThreads = 1024, kRouteWarps = kRouteThreads / 32;
constexpr uint32_t kLowest = 0x007FFFFFu;  // -inf
constexpr uint32_t kNan = 0xFFFFFFFFu;

__device__ __forceinline__ uint32_t key_of(float v) {
  if (v != v) return kNan;
  const uint32_t b = __float_as_uint(v + 0.0f);  // -0 becomes +0
  return (b & 0x80000000u) != 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) != 0 ? key & 0x7FFFFFFFu : ~key);  // kNan: a NaN
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}

// Exclusive prefix over x[0..n) in shared memory, by the whole block; returns the sum.
__device__ int block_prefix(int32_t* x, int n, int32_t* warps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  int carry = 0;
  for (int at = 0; at < n; at += kRouteThreads) {
    const int i = at + threadIdx.x;
    const int v = i < n ? x[i] : 0;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xFFFFFFFFu, s, o);
      if (lane >= o) s += u;
    }
    if (lane == 31) warps[warp] = s;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < kRouteWarps; ++w) {
      if (w < warp) before += warps[w];
      all += warps[w];
    }
    if (i < n) x[i] = carry + before + s - v;
    carry += all;
    __syncthreads();
  }
  return carry;
}

// The slots [s0, s1) to their rows and the offsets: total[e] choices of each expert in
// all, before[e] of them in blocks before (shared memory; both are overwritten).
__device__ void place_slots(const RouteArgs& a, int64_t s0, int64_t s1, int blocks, int32_t* total, int32_t* before,
                            int32_t* warps) {
  const int E = a.experts;
  const int taken = block_prefix(total, E, warps);
  int32_t* next = before;  // the next row of each expert
  for (int e = threadIdx.x; e < E; e += kRouteThreads) {
    if (blockIdx.x == 0) a.offsets[e] = total[e];
    next[e] += total[e];
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[E] = taken;
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  for (int64_t at = s0; at < s1; at += kRouteThreads) {
    const int64_t slot = at + threadIdx.x;
    const int e = slot < s1 ? a.chosen[slot] : -1;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
    const int rank = __popc(same & ((1u << lane) - 1));
    int row = -1;
    // the warps with slots take their rows one after the other
    const int turns = (int)min((int64_t)kRouteWarps, (s1 - at + 31) / 32);
    for (int w = 0; w < turns; ++w) {
      if (w == warp && e >= 0) row = next[e] + rank;
      __syncwarp();
      if (w == warp && e >= 0 && rank == 0) next[e] += __popc(same);
      __syncthreads();
    }
    if (slot < s1) a.place[slot] = row;
    if (row >= 0) a.source[row] = (int32_t)slot;
  }
  // behind the last row; every block takes a share
  for (int64_t r = taken + (int64_t)blockIdx.x * kRouteThreads + threadIdx.x; r < a.tokens * a.k;
       r += (int64_t)blocks * kRouteThreads)
    a.source[r] = -1;
}

// PER: experts a lane. ALONE: the only block, which places its slots too.
template <typename T, int PER, bool ALONE>
__global__ void __launch_bounds__(kRouteThreads) k_choose(const RouteArgs a, int per_block) {
  griddep_wait();
  griddep_trigger();
  extern __shared__ int32_t count[];  // [experts], twice if ALONE
  for (int e = threadIdx.x; e < (ALONE ? 2 : 1) * a.experts; e += kRouteThreads) count[e] = 0;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const int64_t t0 = (int64_t)blockIdx.x * per_block, t1 = min(t0 + per_block, a.tokens);
  for (int64_t t = t0 + threadIdx.x / 32; t < t1; t += kRouteWarps) {
    const T* row = static_cast<const T*>(a.logits) + t * a.stride;
    uint32_t key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = i * 32 + lane < a.experts ? key_of(DT<T>::to_f32(row[i * 32 + lane])) : 0;
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) best = max(best, key[i]);
    const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, best);
    const float top = value_of(most);
    float total = 0.0f;
    if (!a.normalize) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (key[i] > kLowest) total += expf(value_of(key[i]) - top);
      total = warp_sum(total);
    }
    // lane j keeps the j-th choice
    uint32_t my_key = 0;
    int mine = -1;
    for (int j = 0; j < a.k; ++j) {
      const uint32_t m = j == 0 ? most : __reduce_max_sync(0xFFFFFFFFu, best);
      if (m <= kLowest) break;
      int at = 1 << 30;
#pragma unroll
      for (int i = PER - 1; i >= 0; --i) at = key[i] == m ? i * 32 + lane : at;
      at = __reduce_min_sync(0xFFFFFFFFu, at);
      if (lane == j) {
        my_key = m;
        mine = at;
      }
      best = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (at == i * 32 + lane) key[i] = 0;
        best = max(best, key[i]);
      }
    }
    float w = mine >= 0 ? expf(value_of(my_key) - top) : 0.0f;
    if (a.normalize) total = warp_sum(w);
    if (mine >= 0) {
      w /= total;
      atomicAdd(&count[mine], 1);
    }
    if (lane < a.k) {
      a.weights[t * a.k + lane] = w;
      a.chosen[t * a.k + lane] = mine;
    }
  }
  __syncthreads();
  if constexpr (ALONE) {
    __shared__ int32_t warps[kRouteWarps];
    place_slots(a, 0, a.tokens * a.k, 1, count, count + a.experts, warps);
  } else {
    int32_t* out = a.counts + (int64_t)blockIdx.x * a.experts;
    for (int e = threadIdx.x; e < a.experts; e += kRouteThreads) out[e] = count[e];
  }
}

__global__ void __launch_bounds__(kRouteThreads) k_order(const RouteArgs a, int per_block, int blocks) {
  griddep_wait();
  griddep_trigger();
  extern __shared__ int32_t shared[];
  __shared__ int32_t warps[kRouteWarps];
  int32_t *total = shared, *before = shared + a.experts;
  const int E = a.experts;
  for (int e = threadIdx.x; e < 2 * E; e += kRouteThreads) shared[e] = 0;
  __syncthreads();
  // threads share the blocks' counts of an expert
  const int parts = max(1, kRouteThreads / E);
  for (int i = threadIdx.x; i < E * parts; i += kRouteThreads) {
    const int e = i % E, p = i / E;
    int all = 0, earlier = 0;
#pragma unroll 8
    for (int b = p; b < blocks; b += parts) {
      const int c = a.counts[(int64_t)b * E + e];
      all += c;
      earlier += b < (int)blockIdx.x ? c : 0;
    }
    atomicAdd(&total[e], all);
    atomicAdd(&before[e], earlier);
  }
  __syncthreads();
  const int64_t s0 = (int64_t)blockIdx.x * per_block * a.k;
  place_slots(a, s0, min(s0 + (int64_t)per_block * a.k, a.tokens * a.k), blocks, total, before, warps);
}

__global__ void __launch_bounds__(kRouteThreads) k_no_tokens(int32_t* offsets, int n) {
  griddep_wait();
  griddep_trigger();
  for (int i = threadIdx.x; i < n; i += kRouteThreads) offsets[i] = 0;
}

template <typename T, int PER>
__global__ void __launch_bounds__(256) k_route_backward(const RouteArgs a) {
  griddep_wait();
  griddep_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  if (t >= a.tokens) return;
  int c = -1;
  float g = 0.0f;
  if (lane < a.k) {
    c = a.chosen_in[t * a.k + lane];
    if (c >= 0) g = a.weights_in[t * a.k + lane] * a.dweights[t * a.k + lane];
  }
  const float sum = warp_sum(g);
  float d[PER];
  if (a.normalize) {
    if (c >= 0) g = a.weights_in[t * a.k + lane] * (a.dweights[t * a.k + lane] - sum);
#pragma unroll
    for (int i = 0; i < PER; ++i) d[i] = 0.0f;
  } else {
    const T* row = static_cast<const T*>(a.logits) + t * a.stride;
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const bool in = i * 32 + lane < a.experts;
      d[i] = in ? DT<T>::to_f32(row[i * 32 + lane]) : -INFINITY;
      best = max(best, key_of(d[i]));
    }
    best = __reduce_max_sync(0xFFFFFFFFu, best);
    const float top = value_of(best);
    float total = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      d[i] = d[i] == -INFINITY ? 0.0f : expf(d[i] - top);
      total += d[i];
    }
    total = warp_sum(total);
    const float scale = best > kLowest ? -sum / total : 0.0f;  // a row of -inf: no gradient
#pragma unroll
    for (int i = 0; i < PER; ++i) d[i] *= scale;
  }
  for (int j = 0; j < a.k; ++j) {
    const int cj = __shfl_sync(0xFFFFFFFFu, c, j);
    const float gj = __shfl_sync(0xFFFFFFFFu, g, j);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (cj == i * 32 + lane) d[i] += gj;
  }
  T* out = static_cast<T*>(a.dlogits) + t * a.experts;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (i * 32 + lane < a.experts) out[i * 32 + lane] = DT<T>::from_f32(d[i]);
}

// Up to so many tokens take one block, which saves a launch (3 us of the host).
// Captured, one kernel against two: 33 tokens by 16 experts, 2 each, 4.5 and 5.2 us,
// by 128, 8 each, 8.1 and 8.4; 64 tokens 4.9 and 5.2, 9.9 and 8.3; 128 tokens 7.0 and
// 5.7, 17.3 and 8.4.
constexpr int64_t kFewTokens = 64;

// Tokens a block: a warp's one at least, 152 blocks at most (an SM's one each:
// k_order reads the counts of all of them).
int tokens_per_block(int64_t tokens) {
  if (tokens <= kFewTokens) return (int)tokens;
  const int64_t per = (tokens + 151) / 152;
  return (int)((per + kRouteWarps - 1) / kRouteWarps * kRouteWarps);
}

template <typename T, int PER>
cudaError_t choose(const RouteArgs& a, int per_block, int blocks, cudaStream_t s) {
  return blocks == 1 ? launch_next(k_choose<T, PER, true>, dim3(1), kRouteThreads, a.experts * 8, s, a, per_block)
                     : launch_next(k_choose<T, PER, false>, dim3(blocks), kRouteThreads, a.experts * 4, s, a, per_block);
}
template <typename T, int PER>
cudaError_t backward(const RouteArgs& a, cudaStream_t s) {
  return launch_next(k_route_backward<T, PER>, dim3((unsigned)((a.tokens + 7) / 8)), 256, 0, s, a);
}

#define ZG_BY_EXPERTS(T, call, ...)                                                \
  (a.experts <= 32    ? call<T, 1>(__VA_ARGS__)                                    \
   : a.experts <= 64  ? call<T, 2>(__VA_ARGS__)                                    \
   : a.experts <= 128 ? call<T, 4>(__VA_ARGS__)                                    \
   : a.experts <= 256 ? call<T, 8>(__VA_ARGS__)                                    \
                      : call<T, 32>(__VA_ARGS__))
#define ZG_BY_TYPE(call, ...)                                                      \
  (a.dtype == kF32    ? ZG_BY_EXPERTS(float, call, __VA_ARGS__)                    \
   : a.dtype == kF16  ? ZG_BY_EXPERTS(__half, call, __VA_ARGS__)                   \
                      : ZG_BY_EXPERTS(__nv_bfloat16, call, __VA_ARGS__))

}  // namespace

int64_t route_workspace_bytes(int64_t tokens, int experts, int k) {
  (void)k;
  const int64_t per = tokens_per_block(tokens);
  return per > 0 ? (tokens + per - 1) / per * experts * 4 : 0;
}

cudaError_t launch_route(const RouteArgs& a, cudaStream_t s) {
  if (a.tokens == 0) {
    return launch_next(k_no_tokens, dim3(1), kRouteThreads, 0, s, a.offsets, a.experts + 1);
  }
  const int per = tokens_per_block(a.tokens);
  const int blocks = (int)((a.tokens + per - 1) / per);
  cudaError_t e = ZG_BY_TYPE(choose, a, per, blocks, s);
  if (e != cudaSuccess || blocks == 1) return e;
  return launch_next(k_order, dim3(blocks), kRouteThreads, a.experts * 8, s, a, per, blocks);
}

cudaError_t launch_route_backward(const RouteArgs& a, cudaStream_t s) { return ZG_BY_TYPE(backward, a, s); }

}  // namespace zg
