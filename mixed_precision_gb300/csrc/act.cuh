// The packed-activation format, shared by every kernel that writes or reads
// it: int8 codes, one biased power-of-two exponent for each 32 elements.
#pragma once

#include <cstdint>
#include <type_traits>

#include "block.h"
#include "vec.cuh"

namespace zg {

// Two values rounded to T, the first in the low half.
template <typename T>
__device__ __forceinline__ uint32_t round2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t round2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t round2<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 8 elements as fp32, and 8 values rounded to T. 16-bit types go in pairs: a
// bf16 is the upper half of its fp32, and one instruction rounds two values.
template <typename T>
__device__ __forceinline__ void widen8(const Pack8<T>& v, float (&x)[8]) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(v.e);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = __uint_as_float(w[j] << 16);
      x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = DT<T>::to_f32(v.e[j]);
  }
}
template <typename T>
__device__ __forceinline__ Pack8<T> round8(const float (&x)[8]) {
  Pack8<T> v;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v.e[j] = x[j];
  } else {
    uint32_t* w = reinterpret_cast<uint32_t*>(v.e);
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = round2<T>(x[2 * j], x[2 * j + 1]);
  }
  return v;
}

// 8 values rounded to T and stored (16-byte aligned; 32 bytes for fp32).
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  store8_raw(p, round8<T>(x));
}

// Bytes from a row's codes to those `rows` further on. (A row may be 2^30 bytes:
// two of them leave 32 bits.)
__host__ __device__ constexpr int64_t code_rows(int64_t rows, int pitch) { return rows * pitch; }
static_assert(code_rows(2, 1 << 30) == int64_t(1) << 31, "offsets in 64 bits");

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

// The codes of 8 values: round(x * inv) to nearest even, clamped to +-127. Adding
// 1.5 * 2^23 rounds a small number to a whole one, whose low byte then is its
// two's complement (the conversion instruction runs at an eighth of the rate).
// A marked group (inv = 0) has codes 0.
__device__ __forceinline__ uint2 act_codes8(const float (&x)[8], float inv) {
  uint32_t c[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    c[j] = __float_as_uint(__fadd_rn(fminf(fmaxf(__fmul_rn(x[j], inv), -127.0f), 127.0f), 12582912.0f));
  uint2 r;
  r.x = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
  r.y = __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410);
  return inv == 0.0f ? make_uint2(0, 0) : r;
}

// 8 values restored: code * scale. 2^23 + 128 + code is an fp32 number made by a
// byte move.
__device__ __forceinline__ void act_restore8(uint2 q, float scale, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t w = (j < 4 ? q.x : q.y) ^ 0x80808080u;
    v[j] = __fmul_rn(__fadd_rn(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7650 | (j & 3))), -8388736.0f), scale);
  }
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
