// Packing activations to 8 bits and restoring them.
//
// pack: for each group of 32 elements along the row, the power of two that
// brings the largest magnitude to 64..127 (found from the exponent bits, no
// logarithm), then round-to-nearest codes. restore: code * scale. A thread
// holds 8 elements, four neighbouring lanes one group. Both are bound by HBM:
// b + 1.03 bytes per element.
#include "act.cuh"
#include "block.h"
#include "vec.cuh"

namespace zg {
namespace {

// 8 elements from column c of a row, zero past its end. VEC: rows and strides
// are whole 16-byte vectors, so a chunk is inside the row or outside it.
template <typename T, bool VEC>
__device__ __forceinline__ void load_chunk(const T* row, int c, int cols, float (&x)[8]) {
  if constexpr (VEC) {
    if (c < cols) {
      load8(row + c, x);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = 0.0f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = c + j < cols ? DT<T>::to_f32(row[c + j]) : 0.0f;
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) k_act_pack(const ActArgs a) {
  const T* x = static_cast<const T*>(a.x);
  const uint32_t per_row = a.pitch / 8;  // chunks of a row, a multiple of 16
  const int64_t total = a.rows * per_row;
  // total is a multiple of 16 chunks but a warp is 32 lanes: the loop bound is
  // rounded up so that whole warps reach the shuffles
  const int64_t bound = (total + 31) / 32 * 32;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < bound; i += gridDim.x * 256ll) {
    const bool live = i < total;
    const int64_t row = live ? i / per_row : 0;
    const int c = live ? static_cast<int>(i - row * per_row) * 8 : a.cols + 8;
    float v[8];
    load_chunk<T, VEC>(x + row * a.stride, c, a.cols, v);
    const uint32_t byte = act_group_byte(v);
    if (live) {
      *reinterpret_cast<uint2*>(a.q + row * a.pitch + c) = act_codes8(v, act_inv_scale(byte));
      if ((threadIdx.x & 3) == 0) a.scales[row * (a.pitch / kActGroup) + c / kActGroup] = byte;
    }
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) k_act_unpack(const ActArgs a) {
  T* out = static_cast<T*>(a.out);
  const uint32_t per_row = (a.cols + 7) / 8;
  const int64_t total = a.rows * per_row;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const int64_t row = i / per_row;
    const int c = static_cast<int>(i - row * per_row) * 8;
    const uint2 q = *reinterpret_cast<const uint2*>(a.q_in + row * a.pitch + c);
    const float s = act_scale(a.scales_in[row * (a.pitch / kActGroup) + c / kActGroup]);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t w = j < 4 ? q.x : q.y;
      v[j] = static_cast<float>(static_cast<int8_t>(w >> 8 * (j & 3))) * s;
    }
    T* o = out + row * a.stride + c;
    if constexpr (VEC) {
      store8(o, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < a.cols) o[j] = DT<T>::from_f32(v[j]);
    }
  }
}

template <typename T>
cudaError_t pack_t(const ActArgs& a, int grid, bool vec, cudaStream_t s) {
  if (vec)
    k_act_pack<T, true><<<grid, 256, 0, s>>>(a);
  else
    k_act_pack<T, false><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename T>
cudaError_t unpack_t(const ActArgs& a, int grid, bool vec, cudaStream_t s) {
  if (vec)
    k_act_unpack<T, true><<<grid, 256, 0, s>>>(a);
  else
    k_act_unpack<T, false><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

int act_grid(int64_t chunks, int sms) {
  const int64_t want = (chunks + 255) / 256;
  return static_cast<int>(want < sms * 8ll ? want : sms * 8ll);
}

}  // namespace

cudaError_t launch_act_pack(const ActArgs& a, int sms, cudaStream_t s) {
  const int grid = act_grid(a.rows * (a.pitch / 8), sms);
  const bool vec = a.cols % 8 == 0 && a.stride % 8 == 0;
  switch (a.dtype) {
    case kF32: return pack_t<float>(a, grid, vec, s);
    case kF16: return pack_t<__half>(a, grid, vec, s);
    default: return pack_t<__nv_bfloat16>(a, grid, vec, s);
  }
}

cudaError_t launch_act_unpack(const ActArgs& a, int sms, cudaStream_t s) {
  const int grid = act_grid(a.rows * ((a.cols + 7) / 8), sms);
  const bool vec = a.cols % 8 == 0 && a.stride % 8 == 0;
  switch (a.dtype) {
    case kF32: return unpack_t<float>(a, grid, vec, s);
    case kF16: return unpack_t<__half>(a, grid, vec, s);
    default: return unpack_t<__nv_bfloat16>(a, grid, vec, s);
  }
}

}  // namespace zg
