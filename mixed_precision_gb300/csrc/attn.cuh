// What the attention kernels share: the keys a row sees, packed fp32 pairs,
// the exponential.
#pragma once

#include <cstdint>
#include <type_traits>

#include "act.cuh"
#include "block.h"
#include "tc.cuh"
#include "vec.cuh"

namespace zg {

constexpr int kTile = 128;                  // query rows and keys of a tile
constexpr int kTileChunk = kTile * 128;     // bytes of 64 head elements x 128 rows
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ int valid_keys(const AttnArgs& a, int64_t b) {
  const int k_len = static_cast<int>(a.k_len);
  return a.lengths == nullptr ? k_len : min(max(a.lengths[b], 0), k_len);
}

// Keys [lo, hi) that query i sees, of `keys` valid ones. (Lengths are at most
// 2^28 and a window at most their sum, so int holds every sum here.)
__device__ __forceinline__ void key_range(const AttnArgs& a, int keys, int i, int& lo, int& hi) {
  const int d = i + static_cast<int>(a.k_len) - static_cast<int>(a.q_len);
  hi = a.causal ? min(keys, d + 1) : keys;
  lo = a.window > 0 ? max(0, d - static_cast<int>(a.window) + 1) : 0;
}

// 16-bit operands in fp16 are kept high in its range, as powers of two that are
// taken out again in fp32: fp16 keeps its 11 bits down to 2^-14 only, and a
// weight below that is part of many small ones, a gradient often below it as a
// whole. bf16 has fp32's range and needs none of this.
//   forward   p = 2^(s - m), at most 2^8 (the maximum m may lag), times 2^7
//   backward  p, at most 1, times 2^14; ds = p (dp - delta) by the power of two
//             that brings its bound below 2^15 (k_attn_bwd.cu)
template <typename T>
constexpr bool kNarrow = std::is_same<T, __half>::value;
__device__ __forceinline__ float power_of_two(int n) { return __uint_as_float((127 + n) << 23); }  // |n| < 127

// 2^x; 0 for -inf, about 2^-22 relative error.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The largest of three values (a NaN among them is passed over).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Bit k: whether column k of 32 lies in [from, to).
__device__ __forceinline__ uint32_t seen_bits(int from, int to) {
  const uint32_t low = from <= 0 ? 0xFFFFFFFFu : from >= 32 ? 0u : 0xFFFFFFFFu << from;
  const uint32_t high = to >= 32 ? 0xFFFFFFFFu : to <= 0 ? 0u : (1u << to) - 1u;
  return low & high;
}
// Values whose bit is not set: `other`. (Testing bits of one word takes a third
// of the instructions of comparing every column with both ends.)
__device__ __forceinline__ void mask_row(uint32_t (&s)[32], uint32_t bits, uint32_t other) {
#pragma unroll
  for (int k = 0; k < 32; ++k) s[k] = bits & 1u << k ? s[k] : other;
}
constexpr uint32_t kMinusInf = 0xFF800000u;

// Registers of a warpgroup's threads, given away and taken (all four warps).
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// A barrier of n threads; id 1 and up.
__device__ __forceinline__ void named_sync(int id, int n) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}

// The 64-wide chunks of a [rows <= 128] x head tile, by one thread.
template <int DP>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, int token, int head, int batch,
                                          uint64_t* bar) {
#pragma unroll
  for (int i = 0; i < DP / 64; ++i) tma_load4(dst + i * kTileChunk, map, i * 64, token, head, batch, bar);
}

// Operand descriptors of a 128-row tile: read along the head (K-major), and
// with its rows as the contraction (MN-major).
__device__ __forceinline__ uint64_t head_desc(uint32_t tile) { return smem_desc(tile, 0, 1024); }
__device__ __forceinline__ uint64_t rows_desc(uint32_t tile) { return smem_desc(tile, kTileChunk, 1024); }

// d = a b^T over the head, DP elements. (Offsets are added to the descriptors'
// address fields, in units of 16 bytes.)
template <int DP>
__device__ __forceinline__ void mma_head(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t one) {
#pragma unroll
  for (int k = 0; k < DP / 16; ++k) {
    const uint32_t off = (k / 4 * kTileChunk + k % 4 * 32) / 16;
    mma_ss(d, a + off, b + off, idesc, k > 0, one);
  }
}

// d [+]= a b over 128 rows: a in TMEM, 16-bit, written by PARTS warps a row, each
// over the front of its own 128 / PARTS fp32 columns.
template <int PARTS>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add, uint32_t one) {
  constexpr int kRun = kTile / 16 / PARTS;  // steps in one warp's part
#pragma unroll
  for (int k = 0; k < kTile / 16; ++k)
    mma_ts(d, a + k / kRun * (kTile / PARTS) + k % kRun * 8, b + k * (2048 / 16), idesc, add || k > 0, one);
}

// A row of a tile to zero; the caller fences.
template <int DP>
__device__ __forceinline__ void zero_row(uint8_t* tile, int row) {
#pragma unroll
  for (int k = 0; k < DP / 8; ++k)
    *reinterpret_cast<uint4*>(tile + k / 8 * kTileChunk + row * 128 + k % 8 * 16) = make_uint4(0, 0, 0, 0);
}

// A thread's part of an output row: N sums from TMEM column addr, times f,
// rounded to T, into a tile at [row][col0] (swizzled as TMA reads it); zeros
// unless `live`, whatever the sums are (0 times a NaN of another row). Rows
// written straight to global memory would touch 32 lines an instruction (3.5 us
// a block); a tile leaves by one bulk store. The whole warp calls it.
template <typename T, int N>
__device__ __forceinline__ void stage_row(uint8_t* tile, int row, int col0, uint32_t addr, float f, bool live) {
  constexpr int kStep = N % 32 == 0 ? 32 : 16;
#pragma unroll 1
  for (int k = 0; k < N; k += kStep) {
    uint32_t o[kStep];
    if constexpr (kStep == 32)
      tmem_ld32(addr + k, o);
    else
      tmem_ld16(addr + k, o);
    tmem_wait_ld();
#pragma unroll
    for (int g = 0; g < kStep / 8; ++g) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = round2<T>(__uint_as_float(o[g * 8 + 2 * e]) * f, __uint_as_float(o[g * 8 + 2 * e + 1]) * f);
      const int piece = (col0 + k) / 8 + g;
      *reinterpret_cast<uint4*>(tile + piece / 8 * kTileChunk + row * 128 + (piece % 8 ^ (row & 7)) * 16) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  if (__any_sync(0xFFFFFFFFu, !live)) {  // seldom
#pragma unroll 1
    for (int piece = col0 / 8; piece < (col0 + N) / 8; ++piece)
      if (!live)
        *reinterpret_cast<uint4*>(tile + piece / 8 * kTileChunk + row * 128 + (piece % 8 ^ (row & 7)) * 16) =
            make_uint4(0, 0, 0, 0);
  }
}

// The 64-wide chunks of a staged tile to the tensor, by one thread.
template <int DP>
__device__ __forceinline__ void store_tile(const CUtensorMap* map, uint32_t src, int dim, int token, int head,
                                           int batch) {
#pragma unroll
  for (int i = 0; i < DP / 64; ++i)
    if (i * 64 < dim) tma_store4(map, src + i * kTileChunk, i * 64, token, head, batch);
  tma_store_done();
}

// Blocks for `pieces` of work: one a multiprocessor, each with its share of the
// pieces, or with key lengths and less than four pieces a multiprocessor one a
// piece. A block that goes on to its next piece overlaps that one's start with
// this one's end, but the shares are fixed, and lengths unknown to the host may
// make them unequal; blocks of one piece start wherever one has ended. With
// random lengths, shares against single pieces:
//   6 x 1021, 12/4 heads of 64, window 256   forward 22.9, 17.8 us; backward 41.6, 38.3
//   2 x 4096, 16/8 heads of 128, causal      forward 62.0, 57.3 us; backward 225, 207
//   16 x 2048, 16/8 heads of 128, causal     forward 188, 191 us
//   32 x 1024, 16/4 heads of 64, causal      forward 119, 131 us
inline unsigned attn_grid(const AttnArgs& a, int64_t pieces, int sms) {
  const bool single = pieces < sms || (a.lengths != nullptr && pieces < 4ll * sms);
  return static_cast<unsigned>(single ? pieces : sms);
}

// Maps of a [batch, token, head, dim] tensor for tiles of 128 tokens x 64.
inline bool attn_map(CUtensorMap* map, const void* base, int dtype, const int64_t s[3], int64_t batch, int64_t len,
                     int heads, int dim) {
  const uint64_t n[4] = {(uint64_t)dim, (uint64_t)len, (uint64_t)heads, (uint64_t)batch};
  const uint64_t b[3] = {(uint64_t)s[1] * 2, (uint64_t)s[2] * 2, (uint64_t)s[0] * 2};
  return make_tensor_map(map, base, dtype, 4, n, b, kTile);
}

}  // namespace zg
