// Packing matrices to e4m3 with a power-of-two scale for each 128 elements
// along the contraction, and restoring them. The scale's exponent comes from the
// bits of the largest magnitude, without a logarithm; infinities and NaN, which have
// no part in it, are looked for in the maxima, and only where there is one is each
// element asked. What counts is that a thread's loads are all under way before it needs
// the first. bf16 8192 x 4096, captured: packed in 15.7 us (6.4 TB/s), the transpose in
// 24, both in 36 (a thread's 32 elements cost it some 450 instructions, and 304 blocks
// at a time their barriers); from cold caches the first takes 18 and restoring 14 (11 captured).
//
// Along rows alone, eight lanes hold a scale block (16 elements each). With the
// transpose, a block of threads takes 128 x 128 elements, so it has whole scale
// blocks both ways and reads x once: a thread holds 4 x 8 of them in registers, and
// the transposed codes change places in shared memory.
#include <type_traits>

#include <cuda_fp8.h>

#include "bulk.cuh"
#include "experts.h"
#include "vec.cuh"

namespace zg {
namespace {

constexpr int kTile = 128;
constexpr int kPackThreads = 256;
constexpr int kPasses = 2;  // rows that a thread of the row kernels takes at once
constexpr int kTileThreads = 512, kTileWarps = kTileThreads / 32;
constexpr int kTileRows = 4;  // x 8 columns a thread

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

// Magnitudes as integers of the same order, in the words that elements lie in (two
// 16-bit ones a word): a word's maximum is one instruction, and infinities and NaN
// come out on top, where one comparison finds them.
template <typename T>
struct Bits {
  static constexpr uint32_t kInf = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
  static __device__ __forceinline__ uint32_t size(uint32_t w) { return w & 0x7FFF7FFFu; }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ uint32_t whole(uint32_t m) { return max(m & 0xFFFFu, m >> 16); }
  static __device__ __forceinline__ float number(uint32_t m) {
    if (std::is_same<T, __half>::value) return __half2float(__ushort_as_half(static_cast<unsigned short>(m)));
    return __uint_as_float(m << 16);
  }
};
template <>
struct Bits<float> {
  static constexpr uint32_t kInf = 0x7F800000u;
  static __device__ __forceinline__ uint32_t size(uint32_t w) { return w & 0x7FFFFFFFu; }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max(a, b); }
  static __device__ __forceinline__ uint32_t whole(uint32_t m) { return m; }
  static __device__ __forceinline__ float number(uint32_t m) { return __uint_as_float(m); }
};

// Two elements as e4m3 codes, |x * inv| <= 448. Without FINITE an inf or a NaN
// becomes the NaN code (with it a NaN could not be).
template <bool FINITE>
__device__ __forceinline__ uint32_t codes2(float x, float y, float inv) {
  const float nan = __uint_as_float(0x7FC00000u);
  const float2 v = FINITE ? make_float2(x * inv, y * inv) : make_float2(isinf(x) ? nan : x * inv, isinf(y) ? nan : y * inv);
  return __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
}

// 8 elements as they are in memory, or zeros where `in` is false. Without VEC only
// the first `cols` of them exist.
template <typename T, bool VEC>
__device__ __forceinline__ Pack8<T> fetch8(const T* p, bool in, int64_t cols) {
  Pack8<T> v;
  if (VEC && in && cols > 0) {
    v = load8_raw(p);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v.e[j] = !VEC && in && j < cols ? p[j] : DT<T>::from_f32(0.0f);
  }
  return v;
}
template <typename T>
__device__ __forceinline__ const uint32_t* words_of(const Pack8<T>& v) {
  return reinterpret_cast<const uint32_t*>(v.e);
}
template <typename T>
constexpr int kWords = 2 * sizeof(T);  // of 8 elements

template <typename T>
__device__ __forceinline__ uint32_t top8(const Pack8<T>& v) {
  uint32_t m = Bits<T>::size(words_of(v)[0]);
#pragma unroll
  for (int k = 1; k < kWords<T>; ++k) m = Bits<T>::larger(m, Bits<T>::size(words_of(v)[k]));
  return m;
}
template <typename T>
__device__ __forceinline__ float finite_top8(const Pack8<T>& v) {
  float top = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = fmaxf(top, finite_size(DT<T>::to_f32(v.e[j])));
  return top;
}
template <typename T, bool FINITE>
__device__ __forceinline__ uint2 codes8(const Pack8<T>& v, float inv) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = codes2<FINITE>(DT<T>::to_f32(v.e[2 * j]), DT<T>::to_f32(v.e[2 * j + 1]), inv);
  return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}
// The largest magnitude of LANES neighbouring lanes: of their words, or of numbers.
template <typename T, int LANES>
__device__ __forceinline__ uint32_t top_words(uint32_t m) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) m = Bits<T>::larger(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  return Bits<T>::whole(m);
}
template <int LANES>
__device__ __forceinline__ float top_numbers(float top) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  return top;
}

// A group of eight lanes' place: the blocks of threads are 2^wide scale blocks across.
struct Place {
  int64_t row;  // of the first pass
  int64_t block;
  int step;     // rows between passes
  __device__ __forceinline__ explicit Place(int wide) {
    const int group = threadIdx.x / 8;
    step = 32 >> wide;
    row = (int64_t)blockIdx.x * (step * kPasses) + (group >> wide);
    block = ((int64_t)blockIdx.y << wide) + (group & ((1 << wide) - 1));
  }
};

template <typename T, bool VEC>
__global__ void __launch_bounds__(kPackThreads, sizeof(T) == 2 ? 5 : 3) k_scaled_pack_rows(const ScaledArgs a, int wide) {
  griddep_wait();
  griddep_trigger();
  const Place at(wide);
  const int64_t z = blockIdx.z, c = at.block * kScaledBlock + (threadIdx.x & 7) * 8;
  const T* x = static_cast<const T*>(a.x) + z * a.batch_stride + c;
  Pack8<T> v[kPasses][2];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int64_t r = at.row + i * at.step;
#pragma unroll
    for (int h = 0; h < 2; ++h) v[i][h] = fetch8<T, VEC>(x + r * a.stride + h * 64, r < a.rows, a.cols - c - h * 64);
  }
  const int64_t blocks = a.pitch / kScaledBlock;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int64_t r = at.row + i * at.step, row = z * a.rows + r;
    const uint32_t top = top_words<T, 8>(Bits<T>::larger(top8(v[i][0]), top8(v[i][1])));
    uint32_t byte;
    uint2 q[2];
    if (__any_sync(0xFFFFFFFFu, top >= Bits<T>::kInf)) {
      byte = scale_byte(top_numbers<8>(fmaxf(finite_top8(v[i][0]), finite_top8(v[i][1]))));
      for (int h = 0; h < 2; ++h) q[h] = codes8<T, false>(v[i][h], inverse_scale(byte));
    } else {
      byte = scale_byte(Bits<T>::number(top));
      for (int h = 0; h < 2; ++h) q[h] = codes8<T, true>(v[i][h], inverse_scale(byte));
    }
    if (r >= a.rows || at.block >= blocks) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) *reinterpret_cast<uint2*>(a.q + row * a.pitch + c + h * 64) = q[h];
    // the last block's lanes write the padding too
    const int64_t s = at.block + (threadIdx.x & 7);
    if (s == at.block || (at.block + 1 == blocks && s < a.scale_pitch))
      a.scales[row * a.scale_pitch + s] = s == at.block ? byte : 127;
  }
}

// The block's codes and scales of 128 x 128 elements; the transposed codes to `turned`.
template <typename T, bool FINITE>
__device__ __forceinline__ void pack_tile(const ScaledArgs& a, const Pack8<T> (&v)[kTileRows], int64_t r0, int64_t c0,
                                          float (&tops)[kTileWarps][kTile], uint32_t* turned) {
  const int part = threadIdx.x & 15, sub = threadIdx.x / 16, warp = threadIdx.x / 32;
  const int64_t c = c0 + part * 8, r = r0 + sub * kTileRows, z = blockIdx.z;
  if (a.q != nullptr) {
#pragma unroll
    for (int i = 0; i < kTileRows; ++i) {
      const float top = FINITE ? Bits<T>::number(top_words<T, 16>(top8(v[i]))) : top_numbers<16>(finite_top8(v[i]));
      const uint32_t byte = scale_byte(top);
      if (r + i >= a.rows) continue;
      const int64_t row = z * a.rows + r + i;
      *reinterpret_cast<uint2*>(a.q + row * a.pitch + c) = codes8<T, FINITE>(v[i], inverse_scale(byte));
      if (part == 0) a.scales[row * a.scale_pitch + blockIdx.y] = byte;
      // the padding, by the block of the last columns
      const int64_t at = blockIdx.y + 1 + part;
      if (blockIdx.y + 1 == gridDim.y && at < a.scale_pitch) a.scales[row * a.scale_pitch + at] = 127;
    }
  }
  // columns: 4 rows here, 8 in the warp, then the warps'
  float column[8];
  if (FINITE) {
#pragma unroll
    for (int k = 0; k < kWords<T>; ++k) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kTileRows; ++i) m = Bits<T>::larger(m, Bits<T>::size(words_of(v[i])[k]));
      m = Bits<T>::larger(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
      if (sizeof(T) == 4) {
        column[k] = Bits<T>::number(m);
      } else {
        column[2 * k] = Bits<T>::number(m & 0xFFFFu);
        column[2 * k + 1] = Bits<T>::number(m >> 16);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < kTileRows; ++i) top = fmaxf(top, finite_size(DT<T>::to_f32(v[i].e[j])));
      column[j] = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16));
    }
  }
  if (sub % 2 == 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) tops[warp][part * 8 + j] = column[j];
  }
  __syncthreads();
  // the scales, a thread a column; the columns' maxima become their inverses
  if (threadIdx.x < kTile) {
    float top = 0.0f;
#pragma unroll
    for (int w = 0; w < kTileWarps; ++w) top = fmaxf(top, tops[w][threadIdx.x]);
    const uint32_t byte = scale_byte(top);
    tops[0][threadIdx.x] = inverse_scale(byte);
    if (c0 + threadIdx.x < a.cols) {
      uint8_t* s = a.scales_t + (z * a.cols + c0 + threadIdx.x) * a.scale_pitch_t;
      s[blockIdx.x] = byte;
      if (blockIdx.x + 1 == gridDim.x)
        for (int64_t at = blockIdx.x + 1; at < a.scale_pitch_t; ++at) s[at] = 127;
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float inv = tops[0][part * 8 + j];
    const uint32_t lo = codes2<FINITE>(DT<T>::to_f32(v[0].e[j]), DT<T>::to_f32(v[1].e[j]), inv);
    const uint32_t hi = codes2<FINITE>(DT<T>::to_f32(v[2].e[j]), DT<T>::to_f32(v[3].e[j]), inv);
    turned[(part * 8 + j) * 32 + (sub ^ part * 2)] = lo | hi << 16;
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kTileThreads, 2) k_scaled_pack(const ScaledArgs a) {
  griddep_wait();
  griddep_trigger();
  __shared__ __align__(16) uint32_t turned[kTile * 32];  // [column][rows as 32 words], word w at w ^ (column / 8 * 2)
  __shared__ float tops[kTileWarps][kTile];
  const int64_t r0 = (int64_t)blockIdx.x * kTile, c0 = (int64_t)blockIdx.y * kTile, z = blockIdx.z;
  const int part = threadIdx.x & 15, sub = threadIdx.x / 16;  // columns part * 8, rows sub * 4 and up
  const int64_t c = c0 + part * 8, r = r0 + sub * kTileRows;
  const T* x = static_cast<const T*>(a.x) + z * a.batch_stride + r * a.stride + c;
  Pack8<T> v[kTileRows];
#pragma unroll
  for (int i = 0; i < kTileRows; ++i) v[i] = fetch8<T, VEC>(x + i * a.stride, r + i < a.rows, a.cols - c);

  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kTileRows; ++i) top = Bits<T>::larger(top, top8(v[i]));
  if (__syncthreads_or(Bits<T>::whole(top) >= Bits<T>::kInf))
    pack_tile<T, false>(a, v, r0, c0, tops, turned);
  else
    pack_tile<T, true>(a, v, r0, c0, tops, turned);
  __syncthreads();
  const int piece = threadIdx.x % 8 * 2;  // of 8 rows, two words
  const uint2* pieces = reinterpret_cast<const uint2*>(turned);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int col = threadIdx.x / 8 + i * (kTileThreads / 8), swap = col / 8;
    const uint2 lo = pieces[col * 16 + (piece ^ swap)], hi = pieces[col * 16 + ((piece + 1) ^ swap)];
    if (c0 + col < a.cols)
      *reinterpret_cast<uint4*>(a.qt + (z * a.cols + c0 + col) * a.pitch_t + r0 + piece * 8) =
          make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
}

// The grid holds 65535 blocks across: wider matrices (the transposes of very many rows)
// take several rounds.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kPackThreads) k_scaled_unpack(const ScaledArgs a, int wide) {
  griddep_wait();
  griddep_trigger();
  const Place at(wide);
  for (int64_t block = at.block; block < a.pitch / kScaledBlock; block += (int64_t)gridDim.y << wide) {
    const int64_t c = block * kScaledBlock + (threadIdx.x & 7) * 8;
    uint2 q[kPasses][2];
    uint32_t byte[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int64_t r = min(at.row + i * at.step, a.rows - 1);
#pragma unroll
      for (int h = 0; h < 2; ++h) q[i][h] = *reinterpret_cast<const uint2*>(a.q_in + r * a.pitch + c + h * 64);
      byte[i] = a.scales_in[r * a.scale_pitch + block];
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int64_t r = at.row + i * at.step;
      if (r >= a.rows) break;
      // 2^-127 is a subnormal number; 255 stands for NaN
      const float s = __uint_as_float(byte[i] == 0 ? 0x00400000u : byte[i] == 255 ? 0x7FC00000u : byte[i] << 23);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        Pack8<T> out;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const uint32_t w = (p < 2 ? q[i][h].x : q[i][h].y) >> (p & 1) * 16 & 0xFFFFu;
          const __half2_raw e = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)w, __NV_E4M3);
          const float2 f = __half22float2(__half2(e));
          out.e[2 * p] = DT<T>::from_f32(f.x * s);
          out.e[2 * p + 1] = DT<T>::from_f32(f.y * s);
        }
        T* to = static_cast<T*>(a.out) + r * a.stride + c + h * 64;
        const int64_t left = a.cols - c - h * 64;
        if constexpr (VEC) {
          if (left > 0) store8_raw(to, out);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < left) to[j] = out.e[j];
        }
      }
    }
  }
}

// The row kernels' grid: as many scale blocks across a block of threads as a row has, up to 32.
struct RowGrid {
  int wide = 0;
  dim3 grid;
  RowGrid(int64_t rows, int64_t blocks, int64_t batch) {
    while (wide < 5 && (1 << wide) < blocks) ++wide;
    const int64_t each = (32 >> wide) * kPasses;
    const int64_t across = (blocks + (1 << wide) - 1) >> wide;
    grid = dim3((unsigned)((rows + each - 1) / each), (unsigned)(across < 65535 ? across : 65535), (unsigned)batch);
  }
};

template <typename T, bool VEC>
cudaError_t pack(const ScaledArgs& a, cudaStream_t s) {
  const int64_t across = a.pitch / kTile, down = (a.rows + kTile - 1) / kTile;
  if (a.qt == nullptr) {
    const RowGrid g(a.rows, across, a.batch);
    return launch_next(k_scaled_pack_rows<T, VEC>, g.grid, kPackThreads, 0, s, a, g.wide);
  }
  return launch_next(k_scaled_pack<T, VEC>, dim3((unsigned)down, (unsigned)across, (unsigned)a.batch), kTileThreads, 0, s, a);
}

template <typename T, bool VEC>
cudaError_t unpack(const ScaledArgs& a, cudaStream_t s) {
  const RowGrid g(a.rows, a.pitch / kScaledBlock, 1);
  return launch_next(k_scaled_unpack<T, VEC>, g.grid, kPackThreads, 0, s, a, g.wide);
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
