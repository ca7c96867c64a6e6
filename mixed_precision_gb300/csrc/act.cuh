// The packed-activation format, shared by every kernel that writes or reads
// it: int8 codes, one biased power-of-two exponent for each 32 elements.
#pragma once

#include <cstdint>

#include "block.h"
#include "vec.cuh"

namespace zg {

// 8 values rounded to T and stored (16-byte aligned; 32 bytes for fp32).
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  Pack8<T> v;
#pragma unroll
  for (int j = 0; j < 8; ++j) v.e[j] = DT<T>::from_f32(x[j]);
  store8_raw(p, v);
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// Scale byte of a group from the bits of its largest magnitude (as integers,
// so a NaN or inf anywhere in the group wins): floor(log2(top)) - 6, biased by
// 127 and at least 0; 255 marks a non-finite group.
__device__ __forceinline__ uint32_t act_scale_byte(uint32_t top_bits) {
  const int e = static_cast<int>(top_bits >> 23);
  return e == 255 ? 255u : static_cast<uint32_t>(max(e - 6, 0));
}

// 2^(127 - byte): what a value is multiplied by to give its code. Exact; 0 for
// a marked group, whose codes do not matter but must be defined.
__device__ __forceinline__ float act_inv_scale(uint32_t byte) {
  return byte == 255 ? 0.0f : __uint_as_float((254u - byte) << 23);
}

// 2^(byte - 127): what a code is multiplied by. Byte 0 is the subnormal
// 2^-127; a marked group restores as NaN.
__device__ __forceinline__ float act_scale(uint32_t byte) {
  const uint32_t bits = byte == 0 ? 0x00400000u : byte == 255 ? 0x7FC00000u : byte << 23;
  return __uint_as_float(bits);
}

// round(x * inv) to nearest even, clamped to +-127. x * inv is below 128 in
// magnitude (or NaN in a marked group, which converts to 0).
__device__ __forceinline__ uint32_t act_code(float x, float inv) {
  const int c = max(-127, min(127, __float2int_rn(x * inv)));
  return static_cast<uint32_t>(c) & 0xFFu;
}

// 8 codes of 8 values.
__device__ __forceinline__ uint2 act_codes8(const float (&x)[8], float inv) {
  uint2 r;
  r.x = act_code(x[0], inv) | act_code(x[1], inv) << 8 | act_code(x[2], inv) << 16 |
        act_code(x[3], inv) << 24;
  r.y = act_code(x[4], inv) | act_code(x[5], inv) << 8 | act_code(x[6], inv) << 16 |
        act_code(x[7], inv) << 24;
  return r;
}

// The scale byte of 8 values held by each of 4 neighbouring lanes (a group of
// 32). All 32 lanes of the warp must call it.
__device__ __forceinline__ uint32_t act_group_byte(const float (&x)[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, abs_bits(x[j]));
  top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
  return act_scale_byte(top);
}

}  // namespace zg
