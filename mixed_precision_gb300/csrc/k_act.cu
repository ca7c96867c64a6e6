// Packing activations to 8 bits and restoring them.
//
// pack: for each group of 32 elements along the row, the power of two that
// brings the largest magnitude to 64..127 (found from the exponent bits, no
// logarithm), then round-to-nearest codes. restore: code * scale. A thread
// holds 8 elements, four neighbouring lanes one group; four such chunks a thread
// are loaded before the first is used. Both are bound by HBM, b + 1.03 bytes per
// element, pack nearly as much by its instructions (70 % of the issue slots):
// 16384 x 2048 in bf16 packs in 20.1 us (5.05 TB/s), restores in 17.3 us (5.9).
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
      widen8(load8_raw(row + c), x);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = 0.0f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = c + j < cols ? DT<T>::to_f32(row[c + j]) : 0.0f;
  }
}

constexpr int kPer = 4;  // chunks a thread, all loaded before the first is used

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) k_act_pack(const ActArgs a, const Divide per_row, uint32_t total) {
  const T* x = static_cast<const T*>(a.x);
  const uint32_t first = blockIdx.x * (256u * kPer) + threadIdx.x;
  float v[kPer][8];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const uint32_t i = first + k * 256;
    const uint32_t row = i < total ? per_row(i) : 0;
    // past the end: columns outside the row, read as zeros
    const int c = i < total ? static_cast<int>(i - row * per_row.d) * 8 : a.pitch;
    load_chunk<T, VEC>(x + row * a.stride, c, a.cols, v[k]);
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const uint32_t byte = act_group_byte(v[k]);  // whole warps
    const uint32_t i = first + k * 256;
    if (i < total) {  // chunk i of the codes, whose rows have no gaps
      *reinterpret_cast<uint2*>(a.q + i * 8ll) = act_codes8(v[k], act_inv_scale(byte));
      if ((threadIdx.x & 3) == 0) a.scales[i / 4] = byte;
    }
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) k_act_unpack(const ActArgs a, const Divide per_row, uint32_t total) {
  T* out = static_cast<T*>(a.out);
  const uint32_t first = blockIdx.x * (256u * kPer) + threadIdx.x;
  uint2 q[kPer];
  uint32_t b[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const uint32_t i = first + k * 256;
    if (i < total) {
      const uint32_t row = per_row(i), at = row * (a.pitch / 8) + (i - row * per_row.d);
      q[k] = *reinterpret_cast<const uint2*>(a.q_in + at * 8ll);
      b[k] = a.scales_in[at / 4];
    }
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const uint32_t i = first + k * 256;
    if (i >= total) break;
    const uint32_t row = per_row(i);
    const int c = static_cast<int>(i - row * per_row.d) * 8;
    float v[8];
    act_restore8(q[k], act_scale(b[k]), v);
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
cudaError_t pack_t(const ActArgs& a, bool vec, cudaStream_t s) {
  const Divide per_row(a.pitch / 8);
  const uint32_t total = (uint32_t)a.rows * per_row.d, grid = (total + 256 * kPer - 1) / (256 * kPer);
  if (vec)
    k_act_pack<T, true><<<grid, 256, 0, s>>>(a, per_row, total);
  else
    k_act_pack<T, false><<<grid, 256, 0, s>>>(a, per_row, total);
  return cudaGetLastError();
}
template <typename T>
cudaError_t unpack_t(const ActArgs& a, bool vec, cudaStream_t s) {
  const Divide per_row((a.cols + 7) / 8);
  const uint32_t total = (uint32_t)a.rows * per_row.d, grid = (total + 256 * kPer - 1) / (256 * kPer);
  if (vec)
    k_act_unpack<T, true><<<grid, 256, 0, s>>>(a, per_row, total);
  else
    k_act_unpack<T, false><<<grid, 256, 0, s>>>(a, per_row, total);
  return cudaGetLastError();
}

// The kernels count chunks in 31 bits: one launch for up to that many (17 G
// elements), several beyond.
template <typename Launch>
cudaError_t by_rows(ActArgs a, int64_t elem_bytes, Launch launch) {
  const int64_t most = ((int64_t(1) << 31) - 1) / (a.pitch / 8);
  const int64_t rows = a.rows;
  for (int64_t r = 0; r < rows; r += most) {
    a.rows = rows - r < most ? rows - r : most;
    const cudaError_t e = launch(a);
    if (e != cudaSuccess) return e;
    const int64_t step = a.rows * a.stride * elem_bytes, codes = a.rows * a.pitch;
    if (a.x != nullptr) {
      a.x = static_cast<const char*>(a.x) + step;
      a.q += codes;
      a.scales += codes / kActGroup;
    } else {
      a.out = static_cast<char*>(a.out) + step;
      a.q_in += codes;
      a.scales_in += codes / kActGroup;
    }
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_act_pack(const ActArgs& a, cudaStream_t s) {
  const bool vec = a.cols % 8 == 0 && a.stride % 8 == 0;
  return by_rows(a, a.dtype == kF32 ? 4 : 2, [&](const ActArgs& p) {
    switch (p.dtype) {
      case kF32: return pack_t<float>(p, vec, s);
      case kF16: return pack_t<__half>(p, vec, s);
      default: return pack_t<__nv_bfloat16>(p, vec, s);
    }
  });
}

cudaError_t launch_act_unpack(const ActArgs& a, cudaStream_t s) {
  const bool vec = a.cols % 8 == 0 && a.stride % 8 == 0;
  return by_rows(a, a.dtype == kF32 ? 4 : 2, [&](const ActArgs& p) {
    switch (p.dtype) {
      case kF32: return unpack_t<float>(p, vec, s);
      case kF16: return unpack_t<__half>(p, vec, s);
      default: return unpack_t<__nv_bfloat16>(p, vec, s);
    }
  });
}

}  // namespace zg
