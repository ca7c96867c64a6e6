// Packing matrices to e4m3 with a power-of-two scale for each 128 elements
// along the contraction, and restoring them.
//
// A block takes 128 x 128 elements, so it has whole scale blocks along rows and
// along columns: one read of x makes the packed matrix and that of the transpose.
// Along a row, sixteen lanes hold a scale block (8 elements each). Along a
// column, the tile is kept in shared memory and two threads share a column. The
// scale's exponent comes from the bits of the largest magnitude, without a
// logarithm.
#include <cuda_fp8.h>

#include "experts.h"
#include "vec.cuh"

namespace zg {
namespace {

constexpr int kTile = 128;
constexpr int kPackThreads = 256;

// The biased exponent of the least power of two that brings `top` (a finite
// magnitude) to 448 = 1.75 * 2^8 or below; 0 at least.
__device__ __forceinline__ uint32_t scale_byte(float top) {
  const int b = static_cast<int>((__float_as_uint(top) + 0x1FFFFFu) >> 23) - 8;
  return static_cast<uint32_t>(max(b, 0));
}
// 2^-(byte - 127); byte is 247 at most.
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

__device__ __forceinline__ float finite_size(float v) {
  const float s = fabsf(v);
  return s <= 3.4028234664e38f ? s : 0.0f;  // an inf or a NaN has no part in the scale
}

// Two elements as e4m3 codes; an inf or a NaN becomes the NaN code. |x * inv| <= 448.
__device__ __forceinline__ uint32_t codes2(float x, float y, float inv) {
  const float nan = __uint_as_float(0x7FC00000u);
  const float2 v = make_float2(isinf(x) ? nan : x * inv, isinf(y) ? nan : y * inv);
  return __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kPackThreads) k_scaled_pack(const ScaledArgs a) {
  constexpr int kRow = kTile + 2;  // elements between the tile's rows in shared memory
  extern __shared__ uint8_t shared[];
  T* tile = reinterpret_cast<T*>(shared);
  const int64_t r0 = (int64_t)blockIdx.x * kTile, c0 = (int64_t)blockIdx.y * kTile, z = blockIdx.z;
  const T* x = static_cast<const T*>(a.x) + z * a.batch_stride;
  const int part = threadIdx.x & 15, sub = threadIdx.x / 16;
  const int64_t c = c0 + part * 8;
#pragma unroll 4
  for (int i = 0; i < kTile; i += kPackThreads / 16) {
    const int64_t r = r0 + i + sub;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    if (r < a.rows) {
      const T* p = x + r * a.stride + c;
      if constexpr (VEC) {
        if (c < a.cols) load8(p, v);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j < a.cols) v[j] = DT<T>::to_f32(p[j]);
      }
    }
    if (a.qt != nullptr) {
#pragma unroll
      for (int j = 0; j < 8; ++j) tile[(i + sub) * kRow + part * 8 + j] = DT<T>::from_f32(v[j]);
    }
    if (a.q != nullptr) {
      float top = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, finite_size(v[j]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
      const uint32_t byte = scale_byte(top);
      const float inv = inverse_scale(byte);
      const uint32_t lo = codes2(v[0], v[1], inv) | codes2(v[2], v[3], inv) << 16;
      const uint32_t hi = codes2(v[4], v[5], inv) | codes2(v[6], v[7], inv) << 16;
      if (r < a.rows) {
        const int64_t row = z * a.rows + r;
        *reinterpret_cast<uint2*>(a.q + row * a.pitch + c) = make_uint2(lo, hi);
        if (part == 0) a.scales[row * a.scale_pitch + blockIdx.y] = byte;
        // the padding, by the block of the last columns
        const int64_t at = blockIdx.y + 1 + part;
        if (blockIdx.y + 1 == gridDim.y && at < a.scale_pitch) a.scales[row * a.scale_pitch + at] = 127;
      }
    }
  }
  if (a.qt == nullptr) return;
  __syncthreads();
  const int col = threadIdx.x / 2, half = threadIdx.x & 1;
  const T* from = tile + half * 64 * kRow + col;
  float top = 0.0f;
#pragma unroll 16
  for (int i = 0; i < 64; ++i) top = fmaxf(top, finite_size(DT<T>::to_f32(from[i * kRow])));
  top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  if (c0 + col >= a.cols) return;
  const uint32_t byte = scale_byte(top);
  const float inv = inverse_scale(byte);
  const int64_t row = z * a.cols + c0 + col;
  uint8_t* to = a.qt + row * a.pitch_t + r0 + half * 64;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const T* p = from + (g * 16 + k * 4) * kRow;
      w[k] = codes2(DT<T>::to_f32(p[0]), DT<T>::to_f32(p[kRow]), inv) |
             codes2(DT<T>::to_f32(p[2 * kRow]), DT<T>::to_f32(p[3 * kRow]), inv) << 16;
    }
    *reinterpret_cast<uint4*>(to + g * 16) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (half == 0) {
    uint8_t* s = a.scales_t + row * a.scale_pitch_t;
    s[blockIdx.x] = byte;
    if (blockIdx.x + 1 == gridDim.x)
      for (int64_t at = blockIdx.x + 1; at < a.scale_pitch_t; ++at) s[at] = 127;
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kPackThreads) k_scaled_unpack(const ScaledArgs a, int64_t per_row, int64_t total) {
  T* out = static_cast<T*>(a.out);
  for (int64_t i = (int64_t)blockIdx.x * kPackThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kPackThreads) {
    const int64_t row = i / per_row, c = (i - row * per_row) * 8;
    const uint2 q = *reinterpret_cast<const uint2*>(a.q_in + row * a.pitch + c);
    const uint32_t byte = a.scales_in[row * a.scale_pitch + c / kScaledBlock];
    // 2^-127 is a subnormal number; 255 stands for NaN
    const float s = __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7FC00000u : byte << 23);
    float v[8];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const uint32_t w = (p < 2 ? q.x : q.y) >> (p & 1) * 16 & 0xFFFFu;
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)w, __NV_E4M3);
      const float2 f = __half22float2(__half2(h));
      v[2 * p] = f.x * s;
      v[2 * p + 1] = f.y * s;
    }
    T* to = out + row * a.stride + c;
    if constexpr (VEC) {
      Pack8<T> r;
#pragma unroll
      for (int j = 0; j < 8; ++j) r.e[j] = DT<T>::from_f32(v[j]);
      store8_raw(to, r);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < a.cols) to[j] = DT<T>::from_f32(v[j]);
    }
  }
}

template <typename T, bool VEC>
cudaError_t pack(const ScaledArgs& a, cudaStream_t s) {
  const int64_t across = (a.cols + kTile - 1) / kTile, down = (a.rows + kTile - 1) / kTile;
  const int bytes = a.qt != nullptr ? kTile * (kTile + 2) * (int)sizeof(T) : 0;
  if (bytes > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(k_scaled_pack<T, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
  }
  k_scaled_pack<T, VEC><<<dim3((unsigned)down, (unsigned)across, (unsigned)a.batch), kPackThreads, bytes, s>>>(a);
  return cudaGetLastError();
}

template <typename T, bool VEC>
cudaError_t unpack(const ScaledArgs& a, cudaStream_t s) {
  const int64_t per_row = (a.cols + 7) / 8, total = a.rows * per_row;
  const int64_t blocks = (total + kPackThreads - 1) / kPackThreads;
  k_scaled_unpack<T, VEC><<<(unsigned)(blocks < 65536 ? blocks : 65536), kPackThreads, 0, s>>>(a, per_row, total);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_scaled_pack(const ScaledArgs& a, cudaStream_t s) {
  const bool vec = a.cols % 8 == 0 && a.stride % 8 == 0 && a.batch_stride % 8 == 0;
  if (a.dtype == kF32) return vec ? pack<float, true>(a, s) : pack<float, false>(a, s);
  if (a.dtype == kF16) return vec ? pack<__half, true>(a, s) : pack<__half, false>(a, s);
  return vec ? pack<__nv_bfloat16, true>(a, s) : pack<__nv_bfloat16, false>(a, s);
}

cudaError_t launch_scaled_unpack(const ScaledArgs& a, cudaStream_t s) {
  const bool vec = a.cols % 8 == 0 && a.stride % 8 == 0;
  if (a.dtype == kF32) return vec ? unpack<float, true>(a, s) : unpack<float, false>(a, s);
  if (a.dtype == kF16) return vec ? unpack<__half, true>(a, s) : unpack<__half, false>(a, s);
  return vec ? unpack<__nv_bfloat16, true>(a, s) : unpack<__nv_bfloat16, false>(a, s);
}

}  // namespace zg
