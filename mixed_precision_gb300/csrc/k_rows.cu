// Rows to their experts and back: gather, the weighted sum back, and its
// gradients.
//
// A warp takes a token: its own row is read once, and its k rows in the experts'
// order are read or written. The places come from the device; a place outside
// the order is passed by. Rows that no slot fills are made zero by the warp of
// their number. Bound by HBM: each row moves once. Gather of 8192 rows of 2048 in bf16
// to two experts each takes 13 us (101 MB: 7.7 TB/s, part of it in the L2 when it ends),
// combine back 25, combine's gradients of 8191 x 1024 in fp16 by 8 43 us (286 MB, 6.7
// TB/s). Few tokens of wide rows leave most SMs idle: 512 of 4096, 8 each, combine in 31 us.
#include "bulk.cuh"
#include "experts.h"
#include "vec.cuh"

namespace zg {
namespace {

constexpr int kRowThreads = 256;

// Elements a lane takes at a time: 8 as 16-byte accesses, or one.
template <typename T, bool VEC>
struct Piece {
  static constexpr int kElems = VEC ? 8 : 1;
  T e[kElems];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC) {
      const Pack8<T> v = load8_raw(p);
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = v.e[i];
    } else {
      e[0] = *p;
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (VEC) {
      Pack8<T> v;
#pragma unroll
      for (int i = 0; i < 8; ++i) v.e[i] = e[i];
      store8_raw(p, v);
    } else {
      *p = e[0];
    }
  }
};

// The rows of the order with the token's slot numbers, where no slot fills them.
template <typename T, bool VEC>
__device__ __forceinline__ void clear_unfilled(const RowsArgs& a, int64_t t, T* out, int lane) {
  using P = Piece<T, VEC>;
  const int64_t r0 = t * a.k;
  for (int j = 0; j < a.k; ++j) {
    if (a.source[r0 + j] >= 0) continue;
    P z;
#pragma unroll
    for (int i = 0; i < P::kElems; ++i) z.e[i] = DT<T>::from_f32(0.0f);
    for (int64_t c = lane * P::kElems; c < a.hidden; c += 32 * P::kElems) z.store(out + (r0 + j) * a.hidden + c);
  }
}

// The token's place for slot j (-1: none), from the lane that holds it.
__device__ __forceinline__ int place_of(int mine, int j) { return __shfl_sync(0xFFFFFFFFu, mine, j); }

__device__ __forceinline__ int load_place(const RowsArgs& a, int64_t t, int lane) {
  const int p = lane < a.k ? a.place[t * a.k + lane] : -1;
  return p < a.tokens * a.k ? p : -1;
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kRowThreads) k_gather(const RowsArgs a) {
  griddep_wait();
  griddep_trigger();
  using P = Piece<T, VEC>;
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * (kRowThreads / 32) + threadIdx.x / 32;
  if (t >= a.tokens) return;
  const int mine = load_place(a, t, lane);
  const T* x = static_cast<const T*>(a.x) + t * a.x_stride;
  T* out = static_cast<T*>(a.out);
  constexpr int kUnroll = 4, kStep = 32 * P::kElems;
  for (int64_t c0 = 0; c0 < a.hidden; c0 += kUnroll * kStep) {
    P v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t c = c0 + u * kStep + lane * P::kElems;
      if (c < a.hidden) v[u].load(x + c);
    }
    for (int j = 0; j < a.k; ++j) {
      const int p = place_of(mine, j);
      if (p < 0) continue;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int64_t c = c0 + u * kStep + lane * P::kElems;
        if (c < a.hidden) v[u].store(out + p * a.hidden + c);
      }
    }
  }
  clear_unfilled<T, VEC>(a, t, out, lane);
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kRowThreads) k_combine(const RowsArgs a) {
  griddep_wait();
  griddep_trigger();
  using P = Piece<T, VEC>;
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * (kRowThreads / 32) + threadIdx.x / 32;
  if (t >= a.tokens) return;
  const int mine = load_place(a, t, lane);
  const float weight = a.weights != nullptr && lane < a.k ? a.weights[t * a.k + lane] : 1.0f;
  const T* y = static_cast<const T*>(a.y);
  T* out = static_cast<T*>(a.out) + t * a.hidden;
  constexpr int kStep = 32 * P::kElems, kAhead = 4;
  for (int64_t c0 = 0; c0 < a.hidden; c0 += kStep) {
    const int64_t c = c0 + lane * P::kElems;
    float sum[P::kElems];
#pragma unroll
    for (int i = 0; i < P::kElems; ++i) sum[i] = 0.0f;
    for (int j0 = 0; j0 < a.k; j0 += kAhead) {
      P v[kAhead];
      int p[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        p[u] = j0 + u < a.k ? place_of(mine, j0 + u) : -1;
        if (p[u] >= 0 && c < a.hidden) v[u].load(y + p[u] * a.y_stride + c);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const float w = __shfl_sync(0xFFFFFFFFu, weight, (j0 + u) & 31);
        if (p[u] < 0) continue;
#pragma unroll
        for (int i = 0; i < P::kElems; ++i) sum[i] += w * DT<T>::to_f32(v[u].e[i]);
      }
    }
    if (c < a.hidden) {
      P r;
#pragma unroll
      for (int i = 0; i < P::kElems; ++i) r.e[i] = DT<T>::from_f32(sum[i]);
      r.store(out + c);
    }
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kRowThreads) k_combine_backward(const RowsArgs a) {
  griddep_wait();
  griddep_trigger();
  using P = Piece<T, VEC>;
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * (kRowThreads / 32) + threadIdx.x / 32;
  if (t >= a.tokens) return;
  const int mine = load_place(a, t, lane);
  const float weight = lane < a.k ? a.weights[t * a.k + lane] : 0.0f;
  const T *x = static_cast<const T*>(a.x) + t * a.x_stride, *y = static_cast<const T*>(a.y);
  T* out = static_cast<T*>(a.out);
  constexpr int kStep = 32 * P::kElems, kSlots = 4;  // slots at a time; x is read again for the next ones
  float result = 0.0f;
  for (int j0 = 0; j0 < a.k; j0 += kSlots) {
    int p[kSlots];
    float w[kSlots], dot[kSlots];
#pragma unroll
    for (int u = 0; u < kSlots; ++u) {
      p[u] = j0 + u < a.k ? place_of(mine, j0 + u) : -1;
      w[u] = __shfl_sync(0xFFFFFFFFu, weight, (j0 + u) & 31);
      dot[u] = 0.0f;
    }
    for (int64_t c = lane * P::kElems; c < a.hidden; c += kStep) {
      P d, v[kSlots];
      d.load(x + c);
#pragma unroll
      for (int u = 0; u < kSlots; ++u)
        if (p[u] >= 0) v[u].load(y + p[u] * a.y_stride + c);
#pragma unroll
      for (int u = 0; u < kSlots; ++u) {
        if (p[u] < 0) continue;
        P r;
#pragma unroll
        for (int i = 0; i < P::kElems; ++i) {
          const float g = DT<T>::to_f32(d.e[i]);
          dot[u] += g * DT<T>::to_f32(v[u].e[i]);
          r.e[i] = DT<T>::from_f32(w[u] * g);
        }
        r.store(out + p[u] * a.hidden + c);
      }
    }
#pragma unroll
    for (int u = 0; u < kSlots; ++u) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot[u] += __shfl_xor_sync(0xFFFFFFFFu, dot[u], o);
      if (lane == j0 + u) result = dot[u];
    }
  }
  if (lane < a.k) a.dweights[t * a.k + lane] = result;
  clear_unfilled<T, VEC>(a, t, out, lane);
}

bool whole_vectors(const RowsArgs& a) {
  return a.hidden % 8 == 0 && a.x_stride % 8 == 0 && a.y_stride % 8 == 0;
}

#define ZG_ROWS(kernel)                                                                             \
  const unsigned blocks = (unsigned)((a.tokens + kRowThreads / 32 - 1) / (kRowThreads / 32));       \
  const bool vec = whole_vectors(a);                                                                \
  auto go = [&](auto* k) { return launch_next(k, dim3(blocks), kRowThreads, 0, s, a); };            \
  if (a.dtype == kF32) return vec ? go(kernel<float, true>) : go(kernel<float, false>);             \
  if (a.dtype == kF16) return vec ? go(kernel<__half, true>) : go(kernel<__half, false>);           \
  return vec ? go(kernel<__nv_bfloat16, true>) : go(kernel<__nv_bfloat16, false>)

}  // namespace

cudaError_t launch_gather(const RowsArgs& a, cudaStream_t s) { ZG_ROWS(k_gather); }
cudaError_t launch_combine(const RowsArgs& a, cudaStream_t s) { ZG_ROWS(k_combine); }
cudaError_t launch_combine_backward(const RowsArgs& a, cudaStream_t s) { ZG_ROWS(k_combine_backward); }

}  // namespace zg
