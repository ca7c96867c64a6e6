// Weight gradient from a packed activation: dw[n_out, n_in] = dy^T X, X the
// packed activation restored in dy's type.
//
// On the tensor cores (tcgen05, fp32 sums in TMEM): both operands have the
// contraction (tokens) as their outer dimension, so both are MN-major tiles.
// dy comes by TMA. X goes through registers: sixteen warps read the codes from
// global memory two of their steps ahead, turn each into dy's type (an int8 code and a
// power-of-two scale: exact in bf16) and write the swizzled tile, so the
// 16-bit activation never exists in global memory.
//
// A block makes MT * 128 x BN outputs over a run of tokens. When the outputs
// alone do not fill the machine, a cluster of S blocks shares a tile, each
// over its own run of tokens; each block then sends its sums to the block
// that owns the columns (distributed shared memory), which adds the S parts
// in order. No workspace; the order of every sum is fixed. (Accumulating, an
// unsplit tile is added to dw by one bulk reduction: one addition to each element.)
//
// Bound by the tensor cores: 4096 x 8192 x 8192 in bf16 takes 335 us (1640
// TFLOP/s, 0.95 of what a library product sustains under the power limit). The
// tiles' starts and ends take part of each block's time, but blocks that overlap
// them by going from tile to tile take 338 us. X is restored beside the products.
// An fp32 dw pays for its rounded runs: 520 us.
#include <cmath>
#include <type_traits>

#include "act.cuh"
#include "block.h"
#include "tc.cuh"
#include "vec.cuh"

namespace zg {
namespace {

__device__ unsigned g_wgrad_error;

constexpr int kConvWarps = 16;
constexpr int kParts = kConvWarps / 4;             // warps that share 32 rows of the outputs
constexpr int kWgThreads = (kConvWarps + 2) * 32;  // converters, the TMA warp, the MMA warp
constexpr int kStep = 64;                          // tokens a step
constexpr int kChunk = kStep * 128;                // bytes of 64 columns x 64 tokens
constexpr int kRedRows = 128;

// Steps whose sums stay in one accumulator when dw is fp32. The tensor core
// truncates each addition to the running sum, so its error grows with the
// number of additions in a row, four a step: with terms all of one sign by up to
// 9e-8 of the result each (2048 of them 1.8e-4, 8192 7.5e-4), on normal data by
// less (6.6e-6 after 512). After 16 steps the sums are moved to a second
// accumulator with rounded additions, which keeps the error of one sign at 1.4e-6
// (fp16 dy; 3e-7 with bf16, whose products have fewer bits to lose).
constexpr int kRun = 16;

// A 16-bit dw does without (its tiles may be wider: 335 against 520 us at 4096 x
// 8192 x 8192) until a block's own run of tokens is so long that truncations of one
// sign come to a fifth (fp16) or a tenth (bf16) of the type's rounding: 9e-8 x 4 x
// 256 = 9e-5 of 4.9e-4, 9e-8 x 4 x 1024 = 3.7e-4 of 3.9e-3.
constexpr int64_t kLongRunF16 = 256, kLongRunBF16 = 1024;

// ROUND: with the second accumulator, MT x BN columns further.
template <int MT, int BN, bool ROUND>
struct Tile {
  static constexpr int kABytes = MT * 2 * kChunk, kBBytes = BN / 64 * kChunk;
  static constexpr int kStage = kABytes + kBBytes;
  static constexpr int kStages = 196608 / kStage < 6 ? 196608 / kStage : 6;
  static constexpr int kRed = kRedRows * BN * 4;  // a phase of the cluster's sum
  static constexpr int kSmem = (kStages * kStage > kRed ? kStages * kStage : kRed) + 1024;
  static constexpr int kCols = MT * BN * (ROUND ? 2 : 1);  // TMEM columns
  // The converter warps work in groups on neighbouring steps: a step's chain
  // (wait, convert, fence, arrive) takes longer than its MMAs do in the smaller
  // tiles, so more of them overlap there.
  static constexpr int kGroups = BN == 256 ? 2 : 4;
  static constexpr int kWarpRows = kStep * kGroups / kConvWarps;  // tokens of a step that a warp converts
  // Own steps that a warp's loads run ahead: kGroups steps each, which covers
  // the memory's latency under load.
  static constexpr int kAhead = 2;
  static_assert((kCols & (kCols - 1)) == 0 && kCols <= 512, "a power of two");
};

// Two bf16 products of int8 codes (bytes 2p and 2p+1 of w) and a scale pair.
// 128 + (low seven bits) is a bf16 number made by a byte move; taking away 128
// or, below zero, 256 leaves the code, all exact.
__device__ __forceinline__ uint32_t codes_bf16(uint32_t w, int p, __nv_bfloat162 s) {
  const uint32_t sel = p == 0 ? 0x4140 : 0x4342;
  const uint32_t a = __byte_perm(w & 0x7F7F7F7Fu, 0x43434343u, sel);
  const uint32_t c = __byte_perm(w & 0x80808080u, 0xC3C3C3C3u, sel);
  const __nv_bfloat162 v = __hmul2(__hadd2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                           *reinterpret_cast<const __nv_bfloat162*>(&c)),
                                   s);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 8 codes restored in T; their group's scale byte is byte `at` of w.
template <typename T>
__device__ __forceinline__ uint4 restore8(uint2 q, uint32_t w, int at);

template <>
__device__ __forceinline__ uint4 restore8<__nv_bfloat16>(uint2 q, uint32_t w, int at) {
  // the scale as a bf16 pair: its exponent byte; 0 stands for the subnormal
  // 2^-127, 255 for NaN
  uint32_t b = __byte_perm(w, 0, 0x4040 | at | at << 8) << 7;
  b = max(b, 0x00400040u);
  if (b >= 0x7F807F80u) b = 0x7FC07FC0u;
  const __nv_bfloat162 s = *reinterpret_cast<const __nv_bfloat162*>(&b);
  return make_uint4(codes_bf16(q.x, 0, s), codes_bf16(q.x, 1, s), codes_bf16(q.y, 0, s), codes_bf16(q.y, 1, s));
}

template <>
__device__ __forceinline__ uint4 restore8<__half>(uint2 q, uint32_t scales, int at) {
  // 1024 + (code + 128) is an fp16 number made by a byte move; taking away 1152
  // leaves the code. Its product with the scale may leave fp16's range, so the
  // scale goes in two powers of two of which the first keeps the code exact:
  // one rounding, as if the product had been rounded at once.
  const uint32_t byte = scales >> at * 8 & 0xFFu;
  const int e = static_cast<int>(byte) - 127;
  const int e1 = max(-14, min(8, e)), e2 = max(-24, min(15, e - e1));
  const uint32_t s1 = static_cast<uint32_t>(e1 + 15) << 10;
  const uint32_t s2 = byte == 255 ? 0x7E00u
                      : e2 >= -14 ? static_cast<uint32_t>(e2 + 15) << 10 : 1u << (e2 + 24);
  const uint32_t p1 = s1 | s1 << 16, p2 = s2 | s2 << 16, off = 0xE480E480u;  // -1152
  auto half2_of = [](uint32_t u) { return *reinterpret_cast<const __half2*>(&u); };
  uint4 r;
  uint32_t* o = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const uint32_t w = (p < 2 ? q.x : q.y) ^ 0x80808080u;
    const uint32_t m = __byte_perm(w, 0x64646464u, p & 1 ? 0x4342 : 0x4140);
    const __half2 h = __hmul2(__hmul2(__hadd2(half2_of(m), half2_of(off)), half2_of(p1)), half2_of(p2));
    o[p] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return r;
}

// 8 neighbouring outputs of a row, from column n.
template <typename T>
__device__ __forceinline__ void store_out(const WgradArgs& a, int64_t m, int n, const float (&v)[8]) {
  if (m >= a.n_out || n >= a.n_in) return;
  const int64_t at = m * a.n_in + n;
  if (a.n_in % 8 == 0) {
    if (a.dw_dtype == kF32) {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(a.dw) + at);
      float4 u = make_float4(v[0], v[1], v[2], v[3]), w = make_float4(v[4], v[5], v[6], v[7]);
      if (a.accumulate) {
        const float4 x = p[0], y = p[1];
        u = make_float4(x.x + u.x, x.y + u.y, x.z + u.z, x.w + u.w);
        w = make_float4(y.x + w.x, y.y + w.y, y.z + w.z, y.w + w.w);
      }
      p[0] = u;
      p[1] = w;
    } else {
      store8(static_cast<T*>(a.dw) + at, v);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (n + j >= a.n_in) break;
    if (a.dw_dtype == kF32) {
      float* p = static_cast<float*>(a.dw) + at + j;
      *p = a.accumulate ? *p + v[j] : v[j];
    } else {
      static_cast<T*>(a.dw)[at + j] = DT<T>::from_f32(v[j]);
    }
  }
}

// r += 32 columns of TMEM.
__device__ __forceinline__ void add32(uint32_t addr, uint32_t (&r)[32]) {
  uint32_t t[32];
  tmem_ld32(addr, t);
  tmem_wait_ld();
#pragma unroll
  for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) + __uint_as_float(t[j]));
}

template <typename T, int MT, int BN, bool ROUND>
__global__ void __launch_bounds__(kWgThreads, 1)
    k_wgrad(const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap map_dw, const WgradArgs a,
            int n_tiles, int split, int per_split, bool tiles_out) {
  using C = Tile<MT, BN, ROUND>;
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t full[C::kStages], empty[C::kStages], done, moved;
  __shared__ uint32_t tmem_slot, abort_word;
  // the swizzle is a function of address bits: tiles start on 1024 bytes
  uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  const uint32_t base = smem_u32(smem);
  const int warp = warp_number(), lane = threadIdx.x & 31;
  const int rank = blockIdx.x % split, tile = blockIdx.x / split;
  const int n0 = tile % n_tiles * BN;
  const int64_t m0 = (int64_t)(tile / n_tiles) * (MT * 128);
  const int64_t steps_all = (a.tokens + kStep - 1) / kStep;
  const int64_t first = (int64_t)rank * per_split;
  const int steps = (int)max((int64_t)0, min((int64_t)per_split, steps_all - first));

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1 + kConvWarps / C::kGroups);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&done, 1);
    mbar_init(&moved, kConvWarps);
    abort_word = 0;
    mbar_init_fence();
    tma_prefetch(&map);
  }
  if (warp == kConvWarps + 1) tmem_alloc(&tmem_slot, C::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const Waiter wait{&abort_word, &g_wgrad_error};

  const int row = (warp & 3) * 32 + lane, half = warp / 4 * (BN / kParts);
  const uint32_t mine = tmem + ((uint32_t)(warp & 3) << 21);  // the warp's lanes
  const int runs = ROUND ? (steps + kRun - 1) / kRun : 1;

  if (warp < kConvWarps) {
    // ---- converters: a warp takes kWarpRows tokens of every kGroups-th step, a lane 8 columns of a row
    constexpr int kLanes = BN / 8;        // lanes a row
    constexpr int kRows = 32 / kLanes;    // rows a round
    constexpr int kRounds = C::kWarpRows / kRows;
    constexpr int kTeam = kConvWarps / C::kGroups;
    const int group = warp / kTeam, member = warp % kTeam;
    constexpr int kAhead = C::kAhead;
    const int c = lane % kLanes * 8, r0 = member * C::kWarpRows + lane / kLanes;
    // A row's scales are BN / 32 bytes. The warp's rows of them are one word in
    // each of the first lanes, handed round when used.
    constexpr int kWords = BN / 128;
    const int srow = member * C::kWarpRows + lane / kWords % C::kWarpRows, at = lane / 4 & 3;
    // Columns past the pitch are outputs that nobody stores, tokens past the
    // last meet zeros of dy: both read what is there instead (the last columns,
    // the last token), so no load needs a condition. The last token's own NaN
    // reaches only columns that it makes NaN anyway.
    const int8_t* qp = a.q + min(n0 + c, a.pitch - 8);
    const uint8_t* sp = a.scales + min(n0 + lane % kWords * 128, a.pitch - 128) / kActGroup;
    const int64_t q_row = code_rows(kRows, a.pitch);
    const int s_pitch = a.pitch / kActGroup;
    uint2 q[kAhead][kRounds];
    uint32_t b[kAhead];
    auto fetch = [&](int slot, int step) {
      if (step >= steps) return;
      const int64_t t0 = (first + step) * kStep;
      if (t0 + kStep <= a.tokens) {
        const int8_t* p = qp + code_rows(t0 + r0, a.pitch);
#pragma unroll
        for (int i = 0; i < kRounds; ++i) q[slot][i] = *reinterpret_cast<const uint2*>(p + i * q_row);
        b[slot] = *reinterpret_cast<const uint32_t*>(sp + (t0 + srow) * s_pitch);
      } else {
#pragma unroll
        for (int i = 0; i < kRounds; ++i)
          q[slot][i] =
              *reinterpret_cast<const uint2*>(qp + code_rows(min(t0 + r0 + i * kRows, a.tokens - 1), a.pitch));
        b[slot] = *reinterpret_cast<const uint32_t*>(sp + min(t0 + srow, a.tokens - 1) * s_pitch);
      }
    };
    int place[kRounds];  // of the lane's 16 bytes in a B tile
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      const int r = r0 + k * kRows;
      place[k] = C::kABytes + c / 64 * kChunk + r * 128 + ((c / 8 % 8) ^ (r & 7)) * 16;
    }
    // Add the first accumulator to the second (run 0: copy), rounded.
    auto move = [&](int run) {
      if (!wait(&done, run & 1)) return false;
      tc_fence_after();
#pragma unroll 1
      for (int m = 0; m < MT; ++m)
#pragma unroll 1
        for (int k = m * BN + half; k < m * BN + half + BN / kParts; k += 32) {
          uint32_t r[32];
          tmem_ld32(mine + k, r);
          if (run > 0) add32(mine + MT * BN + k, r);
          tmem_wait_ld();
          tmem_st32(mine + MT * BN + k, r);
        }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&moved);
      return true;
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(i, group + i * C::kGroups);
    bool go = true;
    int run = 0;  // runs moved
    for (int base_step = group; base_step < steps && go; base_step += kAhead * C::kGroups) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int step = base_step + i * C::kGroups;
        if (step >= steps) break;
        // A stage that comes free only after the next run has begun: the run
        // before is moved first, and not before the stages ahead are filled.
        if (ROUND)
          while (go && run + 1 < runs && step >= (run + 1) * kRun + C::kStages) go = move(run++);
        const int s = step % C::kStages;
        if (!go || !(go = wait(&empty[s], (step / C::kStages - 1) & 1))) break;
        uint8_t* stage = smem + s * C::kStage;
#pragma unroll
        for (int k = 0; k < kRounds; ++k) {
          const uint32_t w = __shfl_sync(0xFFFFFFFFu, b[i], k * kRows * kWords + lane / 16);
          *reinterpret_cast<uint4*>(stage + place[k]) = restore8<T>(q[i][k], w, at);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
        fetch(i, step + kAhead * C::kGroups);
      }
    }
    if (ROUND)
      while (go && run + 1 < runs) go = move(run++);
  } else if (warp == kConvWarps) {
    // ---- dy tiles by TMA
    const uint32_t one = elect_one();
    int step = 0;
    for (; step < steps; ++step) {
      const int s = step % C::kStages;
      if (!wait(&empty[s], (step / C::kStages - 1) & 1)) break;
      if (one) {
        mbar_arrive_expect_tx(&full[s], C::kABytes);
#pragma unroll
        for (int i = 0; i < MT * 2; ++i)
          tma_load2(base + s * C::kStage + i * kChunk, &map, (int)m0 + i * 64, (int)((first + step) * kStep), &full[s]);
      }
    }
    if (step < steps)  // gave up: leave the copies in flight time to land
      for (int i = max(0, step - C::kStages); i < step; ++i)
        mbar_wait(&full[i % C::kStages], (i / C::kStages) & 1, kSpinLimit >> 10);
  } else {
    // ---- the tensor cores
    constexpr uint32_t idesc = mma_desc(!std::is_same<T, __half>::value, 128, BN, true, true);
    const uint32_t one = elect_one();
    const uint64_t a_desc = smem_desc(base, kChunk, 1024), b_desc = smem_desc(base + C::kABytes, kChunk, 1024);
#pragma unroll 1
    for (int step = 0; step < steps; ++step) {
      const int s = step % C::kStages;
      if (!wait(&full[s], (step / C::kStages) & 1)) break;
      tc_fence_after();
      const uint32_t at = s * (C::kStage / 16);  // in the descriptors' units of 16 bytes
      const bool go_on = (ROUND ? step % kRun : step) > 0;
#pragma unroll
      for (int k = 0; k < kStep / 16; ++k)
#pragma unroll
        for (int m = 0; m < MT; ++m)
          mma_ss(tmem + m * BN, a_desc + at + (m * 2 * kChunk + k * 2048) / 16, b_desc + at + k * 2048 / 16, idesc,
                 go_on || k > 0, one);
      mma_commit(&empty[s], one);
      if (ROUND && step % kRun == kRun - 1 && step + 1 < steps) {
        mma_commit(&done, one);
        if (!wait(&moved, (step / kRun) & 1)) break;
        tc_fence_after();
      }
    }
    mma_commit(&done, one);
  }
  // Every MMA of the block has finished, and with it every read of the tiles
  // (and every TMA write: each was waited for before its MMAs).
  const bool ok = wait(&done, steps > 0 ? (runs - 1) & 1 : 0);
  tc_fence_after();

  if (split == 1 && tiles_out) {
    // ---- the sums as a swizzled tile in the stages' place, which are done with,
    // and out by bulk stores. Rows written from registers touch 32 lines an
    // instruction: 8 us for a tile of 256 x 256.
    const bool f32 = a.dw_dtype == kF32;
    const int width = f32 ? 32 : 64, rows_bytes = 128 * BN * (f32 ? 4 : 2);  // of 128 rows
    // fp32 sums of 256 x 256 do not fit at once: 128 rows after the other
    const bool again = MT * rows_bytes > C::kStages * C::kStage;
    static_assert(128 * BN * 4 <= C::kStages * C::kStage, "128 rows fit");
#pragma unroll 1
    for (int m = 0; m < MT; ++m) {
      const int region = again ? 0 : m * rows_bytes;
      if (again && m > 0) __syncthreads();  // the rows before have been read
      if (warp < kConvWarps && ok) {
#pragma unroll 1
        for (int c = half; c < half + BN / kParts; c += 32) {
          uint32_t r[32];
          tmem_ld32(mine + m * BN + c, r);
          if (ROUND && runs > 1) add32(mine + (MT + m) * BN + c, r);
          tmem_wait_ld();
          uint8_t* to = smem + region + c / width * (128 * 128) + row * 128;
          if (f32) {
#pragma unroll
            for (int g = 0; g < 8; ++g)
              *reinterpret_cast<uint4*>(to + (g ^ (row & 7)) * 16) =
                  make_uint4(r[4 * g], r[4 * g + 1], r[4 * g + 2], r[4 * g + 3]);
          } else {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = round2<T>(__uint_as_float(r[g * 8 + 2 * e]), __uint_as_float(r[g * 8 + 2 * e + 1]));
              *reinterpret_cast<uint4*>(to + ((c / 32 % 2 * 4 + g) ^ (row & 7)) * 16) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
        fence_async_smem();
      }
      __syncthreads();
      if (warp == kConvWarps && !wait.gave_up() && m0 + m * 128 < a.n_out && elect_one()) {
        for (int c = 0; c < BN / width && n0 + c * width < a.n_in; ++c) {
          const uint32_t from = base + region + c * (128 * 128);
          if (a.accumulate)
            tma_add2(&map_dw, from, n0 + c * width, (int)m0 + m * 128);
          else
            tma_store2(&map_dw, from, n0 + c * width, (int)m0 + m * 128);
        }
        tma_store_done();
      }
    }
  } else if (split == 1) {
    if (warp < kConvWarps && ok) {
#pragma unroll 1
      for (int m = 0; m < MT; ++m)
#pragma unroll 1
        for (int c = 0; c < BN / kParts; c += 32) {
          uint32_t r[32];
          tmem_ld32(mine + m * BN + half + c, r);
          if (ROUND && runs > 1) add32(mine + (MT + m) * BN + half + c, r);
          tmem_wait_ld();
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(r[g * 8 + j]);
            store_out<T>(a, m0 + m * 128 + row, n0 + half + c + g * 8, v);
          }
        }
    }
  } else {
    // ---- the cluster's sum: 128 rows a phase; part p of the columns belongs to
    // block p, which receives [source block][column][row] in its shared memory
    const int part = BN / split;  // columns, 16 at least
#pragma unroll 1
    for (int m = 0; m < MT; ++m) {
      cluster_sync();  // every block's tiles, or last phase's parts, have been read
      if (warp < kConvWarps) {
#pragma unroll 1
        for (int c = half; c < half + BN / kParts; c += 16) {
          uint32_t r[16];
          if (steps > 0 && ok) {
            tmem_ld16(mine + m * BN + c, r);
            if (ROUND && runs > 1) {
              uint32_t t[16];
              tmem_ld16(mine + (MT + m) * BN + c, t);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) + __uint_as_float(t[j]));
            }
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) r[j] = 0;
          }
          const uint32_t to = cluster_map(base + ((rank * part + c % part) * kRedRows + row) * 4, c / part);
#pragma unroll
          for (int j = 0; j < 16; ++j) cluster_store(to + j * kRedRows * 4, __uint_as_float(r[j]));
        }
      }
      cluster_sync();
      if (warp < kConvWarps) {
        const float* in = reinterpret_cast<const float*>(smem);
        for (int c = warp / 4 * 8; c < part; c += 8 * kParts) {
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = in[(c + j) * kRedRows + row];
          for (int s = 1; s < split; ++s)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += in[(s * part + c + j) * kRedRows + row];
          store_out<T>(a, m0 + m * 128 + row, n0 + rank * part + c, v);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kConvWarps + 1) {
    tc_fence_after();
    tmem_free(tmem, C::kCols);
  }
}

// dw of no tokens.
__global__ void __launch_bounds__(256) k_wgrad_zero(const WgradArgs a) {
  const int64_t n = a.n_out * a.n_in;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
    if (a.dw_dtype == kF32)
      static_cast<float*>(a.dw)[i] = 0.0f;
    else
      static_cast<uint16_t*>(a.dw)[i] = 0;
  }
}

struct Plan {
  int mt, bn, split;
};

// The tile and split with the least estimated time, in cycles. Measured with one
// block per SM at 1.9 GHz: a step of 64 tokens takes 1150 cycles in the 256 x 256
// tile, 690 in 256 x 128 and 526 in 128 x 128 (852 and 685 with rounded runs); a
// block's start and end take 15200, 12700 and 10200 (17700, 16900), and a
// cluster's sum 25 more for each 128 outputs. Clusters leave some SMs idle: 148,
// 136 and 120 are used by clusters of 2, 4 and 8. At 8192 x 2048 x 1024 the tile
// of 256 x 128 split in 2 takes 34 us, 128 x 128 without a split 41 us; at
// 4096 x 8192 x 4096 the unsplit 256 x 256 tile takes 185 us, 128 x 128 310 us.
Plan wgrad_plan(int64_t tokens, int64_t n_out, int64_t n_in, bool round, int sms) {
  const int64_t steps = (tokens + kStep - 1) / kStep;
  static const struct {
    int mt, bn;
    double step, ends, step_round, ends_round;  // step_round 0: not built
  } shapes[] = {{2, 256, 1150, 15200, 0, 0}, {2, 128, 690, 12700, 852, 17700}, {1, 128, 526, 10200, 685, 16900}};
  Plan best{1, 128, 1};
  double least = 1e300;
  for (const auto& sh : shapes) {
    const double step = round ? sh.step_round : sh.step, ends = round ? sh.ends_round : sh.ends;
    if (step == 0) continue;
    const double tiles = (double)((n_out + sh.mt * 128 - 1) / (sh.mt * 128)) * ((n_in + sh.bn - 1) / sh.bn);
    for (int split = 1; split <= 8 && split <= steps; split *= 2) {
      const int used = split == 1 ? sms : split == 2 ? sms - 4 : split == 4 ? sms - 16 : sms - 32;
      const double waves = std::ceil(tiles * split / (used > split ? used : split));
      const double t = waves * (ends + (split > 1 ? 25.0 * sh.mt * sh.bn : 0.0) +
                                step * (double)((steps + split - 1) / split));
      if (t < least) {
        least = t;
        best = Plan{sh.mt, sh.bn, split};
      }
    }
  }
  return best;
}

template <typename T, int MT, int BN, bool ROUND>
cudaError_t run(const WgradArgs& a, int split, cudaStream_t s) {
  using C = Tile<MT, BN, ROUND>;
  CUtensorMap map, map_dw{};
  const uint64_t extent[2] = {(uint64_t)a.n_out, (uint64_t)a.tokens}, strides[1] = {(uint64_t)a.dy_stride * 2};
  if (!make_tensor_map(&map, a.dy, a.dtype, 2, extent, strides, kStep)) return cudaErrorInvalidValue;
  // dw's rows have to start on 16 bytes to leave as tiles
  const uint64_t out_extent[2] = {(uint64_t)a.n_in, (uint64_t)a.n_out};
  const uint64_t out_strides[1] = {(uint64_t)a.n_in * (a.dw_dtype == kF32 ? 4 : 2)};
  const bool tiles_out = out_strides[0] % 16 == 0;
  if (tiles_out && !make_tensor_map(&map_dw, a.dw, a.dw_dtype, 2, out_extent, out_strides, 128))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> asked{0};
  cudaError_t e = allow_smem(k_wgrad<T, MT, BN, ROUND>, C::kSmem, asked);
  if (e != cudaSuccess) return e;
  const int n_tiles = (a.n_in + BN - 1) / BN;
  const int64_t m_tiles = (a.n_out + MT * 128 - 1) / (MT * 128);
  const int64_t steps = (a.tokens + kStep - 1) / kStep;
  if (m_tiles * n_tiles * split > 0x7FFFFFFFll || a.tokens > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(m_tiles * n_tiles * split));
  cfg.blockDim = dim3(kWgThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_wgrad<T, MT, BN, ROUND>, map, map_dw, a, n_tiles, split,
                            (int)((steps + split - 1) / split), tiles_out);
}

template <typename T>
cudaError_t wgrad_t(const WgradArgs& a, int sms, cudaStream_t s) {
  // sums of up to kRun steps stay in one accumulator either way
  bool round = a.dw_dtype == kF32 && a.tokens > kRun * kStep;
  Plan p = wgrad_plan(a.tokens, a.n_out, a.n_in, round, sms);
  const int64_t steps = (a.tokens + kStep - 1) / kStep;
  if (!round && (steps + p.split - 1) / p.split > (a.dtype == kF16 ? kLongRunF16 : kLongRunBF16)) {
    round = true;
    p = wgrad_plan(a.tokens, a.n_out, a.n_in, round, sms);
  }
  if (round) return p.mt == 2 ? run<T, 2, 128, true>(a, p.split, s) : run<T, 1, 128, true>(a, p.split, s);
  if (p.bn == 256) return run<T, 2, 256, false>(a, p.split, s);
  return p.mt == 2 ? run<T, 2, 128, false>(a, p.split, s) : run<T, 1, 128, false>(a, p.split, s);
}

}  // namespace

ZG_ERROR_WORD(wgrad_error, g_wgrad_error)

cudaError_t launch_wgrad(const WgradArgs& a, int sms, cudaStream_t s) {
  if (a.tokens == 0) {
    if (a.accumulate) return cudaSuccess;
    k_wgrad_zero<<<sms * 4, 256, 0, s>>>(a);
    return cudaGetLastError();
  }
  return a.dtype == kF16 ? wgrad_t<__half>(a, sms, s) : wgrad_t<__nv_bfloat16>(a, sms, s);
}

}  // namespace zg
