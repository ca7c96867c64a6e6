// Attention backward. With p = exp(scale q.k - lse) on the pairs seen,
//   delta = sum_d do o,  dp = do v^T,  ds = p (dp - delta),
//   dq = scale ds k,  dk = scale ds^T q,  dv = p^T do.
//
// Two kernels, both on the tensor cores with p and ds kept in TMEM:
//   k_attn_dq   pieces of 128 query rows of a head, over their key tiles; it
//               also writes the rows' statistics (-lse in powers of two, -delta).
//   k_attn_dkv  pieces of 128 keys of a key head, over the query tiles of all
//               heads that share it: dk and dv are sums inside one block.
// S and dp are computed in both (seven products a tile pair instead of five).
// In exchange no gradient is added to global memory from two places: no atomic
// adds, no fp32 copy of dq, and every sum has a fixed order.
//
// p and ds become operands of the inputs' type. In fp16 they are scaled, since
// ds may leave its range where dq, dk and dv do not, above and below: p by 2^14,
// and ds by the power of two that brings the bound
//   |dp - delta| <= sum_d |do| max |v| + |delta|
// below 2^15; of a row's own bound for dq, of the largest among the key head's
// rows for dk, whose sums run over rows. A third kernel, before, finds max |v| of
// each key head (finite ones; a row with a non-finite bound is not scaled). The
// factors go into lse's place in the exponent and come out with the sums' scale;
// dk's costs one product a pair. fp16 takes for all this (captured, caches
// flushed) 591 us instead of 576 at 1 x 8192, 157 instead of 150 at 4 x 2048 with
// 16 heads of 64, 51 instead of 46 at 6 x 1021 with a window of 256.
//
// Bound by the tensor cores for heads of 128 (68 and 80 % of their cycles), by
// the softmax warps for heads of 64. Measured in bf16, both kernels, counting
// the five products: 16/8 heads of 128, causal, 1 x 8192 558 us (1230 TFLOP/s),
// 4 x 2048 214 us (800); 16 heads of 64, causal, 4 x 2048 146 us (590).
#include <type_traits>

#include "attn.cuh"

namespace zg {
namespace {

__device__ unsigned g_attn_bwd_error;

// Sixteen softmax warps (four a row of a tile, 32 columns each), the TMA warp,
// the MMA warp. With eight the softmax's chain was longer than the products it
// overlaps (2 x 4096, 16/4 heads of 64: 591 us, with sixteen 459).
constexpr int kParts = 4, kCols = kTile / kParts, kSoftWarps = 4 * kParts, kSoftThreads = kSoftWarps * 32;
constexpr int kTmaWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1, kBwdThreads = (kSoftWarps + 2) * 32;
constexpr int kStats = 2 * kTile;     // floats of a query tile's statistics

// fp16: exponents of the operands' largest value, and of p's scale.
constexpr int kTopExp = 14, kLiftP = 14;
constexpr int kBoundParts = 32;       // max |v| of a key head is found in up to this many parts

// The exponent of the power of two for ds with this bound (its bits): none if it
// is not finite. (A bound other than zero is at least 2^-48.)
__device__ __forceinline__ int ds_lift(uint32_t bound) {
  const int e = static_cast<int>(bound >> 23 & 0xFFu) - 127;
  return e == 128 ? 0 : kTopExp - max(e, -60);
}

// fp16, before the others: the largest finite |v| of each key head's valid keys, in
// a.v_parts parts, and zeros where dq collects the bounds. Reads v once.
__global__ void __launch_bounds__(256) k_attn_bounds(const AttnArgs a, const Divide by_chunks, int64_t work) {
  __shared__ uint32_t tops[8];
  griddep_trigger();
  const int per = static_cast<int>((a.k_len + a.v_parts - 1) / a.v_parts);
  for (int64_t at = blockIdx.x; at < work; at += gridDim.x) {
    const int64_t bc = at / a.v_parts, b = bc / a.kv_heads;
    const int part = static_cast<int>(at - bc * a.v_parts), first = part * per;
    const __half* v = static_cast<const __half*>(a.v) + b * a.vs[0] + first * a.vs[1] + (bc - b * a.kv_heads) * a.vs[2];
    const uint32_t n = max(0, min(per, valid_keys(a, b) - first)) * by_chunks.d;  // chunks of 8 elements
    uint32_t top = 0;  // of two halves
    for (uint32_t i = threadIdx.x; i < n; i += 4 * 256) {
      uint4 u[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t k = min(i + j * 256, n - 1), row = by_chunks(k);
        u[j] = *reinterpret_cast<const uint4*>(v + row * a.vs[1] + (k - row * by_chunks.d) * 8);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t w = (e == 0 ? u[j].x : e == 1 ? u[j].y : e == 2 ? u[j].z : u[j].w) & 0x7FFF7FFFu;
          top = __vmaxu2(top, w & ~__vcmpgeu2(w, 0x7C007C00u));
        }
    }
    top = __reduce_max_sync(0xFFFFFFFFu, max(top & 0xFFFFu, top >> 16));
    if ((threadIdx.x & 31) == 0) tops[threadIdx.x / 32] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 0; w < 8; ++w) top = max(top, tops[w]);
      a.v_top[bc * kBoundParts + part] = __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(top))));
      if (part == 0) a.ds_top[bc] = 0;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// dq
// ---------------------------------------------------------------------------

template <int DP>
struct Dq {
  static constexpr int kTileBytes = DP / 64 * kTileChunk;
  static constexpr int kK = 3, kV = 2;  // slots: a K tile is used again two tiles later than it is first
  // Pieces whose queries are in shared memory: with two, where they fit, the next
  // piece's first products run while this one's result leaves.
  static constexpr int kQ = DP == 64 ? 2 : 1;
  static constexpr int kSmem = (2 * kQ + kK + kV) * kTileBytes + 1024;
  static_assert(kSmem + 1800 <= 227 * 1024, "beside the kernel's own shared memory");
  // TMEM: S twice (ds over it), dp, dq
  static constexpr uint32_t kDp = 256, kDq = 384;
};

// A block takes one piece of work after the other (128 query rows of a head): the
// loads of the next start while the last ends. Pieces with most keys come first;
// every other round runs backwards, so that the rounds' differences even out.
template <typename T, int DP>
__global__ void __launch_bounds__(kBwdThreads, 1)
    k_attn_dq(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_do,
              const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
              const __grid_constant__ CUtensorMap map_dq, const AttnArgs a, int q_tiles, int pieces) {
  using C = Dq<DP>;
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t q_full[C::kQ], q_free[C::kQ], k_full[C::kK], k_empty[C::kK], v_full[C::kV],
      v_empty[C::kV], s_full[2], dp_full, dp_empty, ds_full[2], done, dq_free;
  __shared__ uint32_t tmem_slot, abort_word;
  __shared__ float part[2][kTile];
  // fp16: halves of the sums of |do|, fp32 numbers rounded up to their upper 16
  // bits (32 would be more than the shared memory left beside the tiles)
  __shared__ uint16_t sizes[kNarrow<T> ? 2 : 1][kNarrow<T> ? kTile : 1];
  uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  // queries and do of kQ pieces, then the K and V slots
  const uint32_t q_at = smem_u32(smem), k_at = q_at + 2 * C::kQ * C::kTileBytes,
                 v_at = k_at + C::kK * C::kTileBytes;
  const int warp = warp_number(), lane = threadIdx.x & 31;

  struct Piece {
    int h, b, c, row0, keys, first, n;  // n key tiles from `first`
  };
  auto piece = [&](int round, Piece& p) {
    const int grid = gridDim.x, at = round * grid + (round & 1 ? grid - 1 - (int)blockIdx.x : (int)blockIdx.x);
    if (at >= pieces) return false;
    const int turn = a.by_batch_q(at), bh = at - turn * a.by_batch_q.d;
    p.b = a.by_q_heads(bh);
    p.h = bh - p.b * a.q_heads;
    p.c = a.by_group(p.h);
    p.row0 = (q_tiles - 1 - turn) * kTile;
    p.keys = valid_keys(a, p.b);
    int lo, hi, skip;
    key_range(a, p.keys, p.row0, lo, skip);
    key_range(a, p.keys, min(p.row0 + kTile, (int)a.q_len) - 1, skip, hi);
    p.first = lo / kTile;
    p.n = lo < hi ? (hi + kTile - 1) / kTile - p.first : 0;
    return true;
  };

  // The TMA warp prepares the barriers and starts the first loads before the
  // block's first barrier: TMEM's allocation takes place meanwhile.
  auto load_k = [&](const Piece& p, int j, int at) {  // by one thread; `at`: tiles loaded before
    const int s = at % C::kK;
    mbar_arrive_expect_tx(&k_full[s], C::kTileBytes);
    load_tile<DP>(k_at + s * C::kTileBytes, &map_k, (p.first + j) * kTile, p.c, p.b, &k_full[s]);
  };
  auto load_v = [&](const Piece& p, int j, int at) {
    const int s = at % C::kV;
    mbar_arrive_expect_tx(&v_full[s], C::kTileBytes);
    load_tile<DP>(v_at + s * C::kTileBytes, &map_v, (p.first + j) * kTile, p.c, p.b, &v_full[s]);
  };
  auto load_q = [&](const Piece& p, int s) {
    mbar_arrive_expect_tx(&q_full[s], 2 * C::kTileBytes);
    load_tile<DP>(q_at + 2 * s * C::kTileBytes, &map_q, p.row0, p.h, p.b, &q_full[s]);
    load_tile<DP>(q_at + (2 * s + 1) * C::kTileBytes, &map_do, p.row0, p.h, p.b, &q_full[s]);
  };
  if (warp == kTmaWarp && elect_one()) {
    for (int s = 0; s < C::kQ; ++s) mbar_init(&q_full[s], 1), mbar_init(&q_free[s], 1);
    for (int s = 0; s < C::kK; ++s) mbar_init(&k_full[s], 1), mbar_init(&k_empty[s], 1);
    for (int s = 0; s < C::kV; ++s) mbar_init(&v_full[s], 1), mbar_init(&v_empty[s], 1);
    for (int s = 0; s < 2; ++s) mbar_init(&s_full[s], 1), mbar_init(&ds_full[s], kSoftWarps);
    mbar_init(&dp_full, 1);
    mbar_init(&dp_empty, kSoftWarps);
    mbar_init(&done, 1);
    mbar_init(&dq_free, kSoftWarps);
    abort_word = 0;
    mbar_init_fence();
    Piece p;
    if (piece(0, p) && p.n > 0) {
      load_q(p, 0);
      load_k(p, 0, 0);
      load_v(p, 0, 0);
    }
  }
  if (warp == kMmaWarp) {
    if (lane == 0) tma_prefetch(&map_dq);
    __syncwarp();
    tmem_alloc(&tmem_slot, 512);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const Waiter wait{&abort_word, &g_attn_bwd_error};

  griddep_trigger();
  Piece p;
  if (warp == kTmaWarp) {
    const uint32_t one = elect_one();
    bool go = true;
    for (int round = 0, at = 0, live = 0; go && piece(round, p); at += p.n, ++round) {
      if (p.n == 0) continue;
      const int s = live % C::kQ;
      auto next_q = [&] {  // the place is free once the piece before in it has left
        go = wait(&q_free[s], (live / C::kQ - 1) & 1);
        if (go && one && round > 0) load_q(p, s);
      };
      if (C::kQ > 1) next_q();
      for (int j = round == 0 ? 1 : 0; go && j < p.n; ++j) {
        const int t = at + j;
        if (!(go = wait(&k_empty[t % C::kK], (t / C::kK - 1) & 1))) break;
        if (one) load_k(p, j, t);
        if (!(go = wait(&v_empty[t % C::kV], (t / C::kV - 1) & 1))) break;
        if (one) load_v(p, j, t);
        if (C::kQ == 1 && j == 0) next_q();  // the first key tile does not wait for it
      }
      ++live;
    }
    if (!go)  // gave up: leave the copies in flight time to land
      for (int i = 0; i < 64; ++i) mbar_try_wait(&q_free[0], 0) && mbar_try_wait(&q_free[0], 1);
  } else if (warp == kMmaWarp) {
    constexpr bool bf16 = !std::is_same<T, __half>::value;
    constexpr uint32_t by_head = mma_desc(bf16, kTile, kTile, false, false);
    constexpr uint32_t by_rows = mma_desc(bf16, kTile, DP, false, true);
    constexpr uint32_t kStep = C::kTileBytes / 16;
    const uint32_t one = elect_one();
    const uint64_t k_desc = head_desc(k_at), v_desc = head_desc(v_at), k_rows = rows_desc(k_at);
    uint64_t q_desc = 0, do_desc = 0;
    // t: key tiles since the block's start
    auto make_s = [&](int t) {
      if (!wait(&k_full[t % C::kK], (t / C::kK) & 1)) return false;
      tc_fence_after();
      mma_head<DP>(tmem + (t & 1) * kTile, q_desc, k_desc + t % C::kK * kStep, by_head, one);
      mma_commit(&s_full[t & 1], one);
      return true;
    };
    auto make_dp = [&](int t) {
      if (!wait(&v_full[t % C::kV], (t / C::kV) & 1)) return false;
      tc_fence_after();
      mma_head<DP>(tmem + C::kDp, do_desc, v_desc + t % C::kV * kStep, by_head, one);
      mma_commit(&dp_full, one);
      mma_commit(&v_empty[t % C::kV], one);
      return true;
    };
    bool go = true;
    for (int round = 0, at = 0, live = 0; go && piece(round, p); at += p.n, ++round) {
      if (p.n == 0) continue;
      const int s = live % C::kQ;
      q_desc = head_desc(q_at + 2 * s * C::kTileBytes);
      do_desc = q_desc + kStep;
      // the S and dp of the piece before have been read: its last ds was waited for
      go = wait(&q_full[s], (live / C::kQ) & 1) && make_s(at) && make_dp(at) && (p.n < 2 || make_s(at + 1));
#pragma unroll 1
      for (int j = 0; go && j < p.n; ++j) {
        const int t = at + j;
        // the next dp as soon as this one has been read, then dq from this ds
        if (!(go = wait(&dp_empty, t & 1))) break;
        tc_fence_after();
        if (j + 1 < p.n && !(go = make_dp(t + 1))) break;
        if (!(go = wait(&ds_full[t & 1], (t / 2) & 1))) break;
        if (j == 0 && live > 0 && !(go = wait(&dq_free, (live - 1) & 1))) break;
        tc_fence_after();
        mma_rows<kParts>(tmem + C::kDq, tmem + (t & 1) * kTile, k_rows + t % C::kK * kStep, by_rows, j > 0, one);
        mma_commit(&k_empty[t % C::kK], one);
        if (j + 2 < p.n) go = make_s(t + 2);
      }
      mma_commit(&done, one);
      ++live;
    }
  } else {
    // ---- a thread a quarter of a row: columns [32 part, 32 part + 32) of each tile
    const int quarter = warp / 4, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const float scale2 = a.scale * kLog2e;
    const uint64_t scale_pair = pair(scale2, scale2);
    // A wait that gives up ends the waits of every later piece too; the barriers
    // of the softmax warps are passed all the same, so none is left in one.
    bool ok = true;
#pragma unroll 1
    for (int round = 0, at = 0, live = 0; piece(round, p); at += p.n, ++round) {
      const int i = p.row0 + row;
      const bool in = i < a.q_len;
      const int64_t head = p.b * (int64_t)a.q_heads + p.h;
      float delta = 0.0f, size = 0.0f;
      if (in && quarter < 2) {  // half the head each
        const T* o = static_cast<const T*>(a.o_in) + p.b * a.os[0] + (int64_t)i * a.os[1] + p.h * a.os[2];
        const T* g = static_cast<const T*>(a.dout) + p.b * a.dos[0] + (int64_t)i * a.dos[1] + p.h * a.dos[2];
        for (int d = quarter * (DP / 2); d < min(a.head_dim, (quarter + 1) * (DP / 2)); d += 8) {
          float x[8], y[8];
          widen8(load8_raw(o + d), x);
          widen8(load8_raw(g + d), y);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            delta = fmaf(x[e], y[e], delta);
            if constexpr (kNarrow<T>) size += fabsf(y[e]);
          }
        }
      }
      // a row that sees nothing (or is none) gets p = 2^-inf = 0 everywhere
      const float lse = in ? a.lse_in[head * a.q_len + i] : -INFINITY;
      if (quarter < 2) {
        part[quarter][row] = delta;
        if constexpr (kNarrow<T>)
          sizes[quarter][row] = static_cast<uint16_t>(min((__float_as_uint(size) >> 16) + 1, 0x7FFFu));
      }
      named_sync(1, kSoftThreads);
      const float minus_delta = -(part[0][row] + part[1][row]),
                  minus_lse = lse == -INFINITY ? -INFINITY : -lse * kLog2e;
      int lift = 0;  // of ds
      if constexpr (kNarrow<T>) {
        const int64_t bc = p.b * (int64_t)a.kv_heads + p.c;
        if (round == 0) griddep_wait();  // for max |v|; nothing has been written before
        const uint32_t v_top =
            __reduce_max_sync(0xFFFFFFFFu, lane < a.v_parts ? __ldcg(&a.v_top[bc * kBoundParts + lane]) : 0u);
        size = __uint_as_float(sizes[0][row] << 16) + __uint_as_float(sizes[1][row] << 16);
        const uint32_t bound = __float_as_uint(fmaf(size, __uint_as_float(v_top), fabsf(minus_delta)));
        lift = ds_lift(bound);
        if (quarter == 0) {
          const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, in && bound < 0x7F800000u ? bound : 0u);
          if (lane == 0) atomicMax(&a.ds_top[bc], most);  // the same in any order
        }
      }
      if (quarter == 0) {
        float* st = a.stats + (head * q_tiles + p.row0 / kTile) * kStats + row;
        st[0] = kNarrow<T> ? minus_lse + kLiftP : minus_lse;
        st[kTile] = minus_delta;
      }
      if (p.n == 0) {  // no key is seen; no place in shared memory is its own
        if (in) {
          T* dq = static_cast<T*>(a.dq) + p.b * a.dqs[0] + (int64_t)i * a.dqs[1] + p.h * a.dqs[2];
          for (int d = quarter * (DP / kParts); d < min(a.head_dim, (quarter + 1) * (DP / kParts)); d += 8)
            *reinterpret_cast<uint4*>(dq + d) = make_uint4(0, 0, 0, 0);
        }
        named_sync(1, kSoftThreads);  // the halves' sums have been read
        continue;
      }
      int lo, hi;
      key_range(a, p.keys, i, lo, hi);
      const float minus = kNarrow<T> ? minus_lse + static_cast<float>(lift) : minus_lse;  // p is only a factor of ds here
      const uint64_t lse_pair = pair(minus, minus), delta_pair = pair(minus_delta, minus_delta);
#pragma unroll 1
      for (int j = 0; ok && j < p.n; ++j) {
        const int t = at + j;
        const uint32_t s_at = tmem + lanes + (t & 1) * kTile + quarter * kCols;
        if (!(ok = wait(&s_full[t & 1], (t / 2) & 1))) break;
        tc_fence_after();
        uint32_t e[kCols];
        tmem_ld32(s_at, e);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < kCols; k += 2) {
          float x, y;
          unpair(fma2(pair(__uint_as_float(e[k]), __uint_as_float(e[k + 1])), scale_pair, lse_pair), x, y);
          e[k] = __float_as_uint(exp2_fast(x));
          e[k + 1] = __float_as_uint(exp2_fast(y));
        }
        if (!(ok = wait(&dp_full, t & 1))) break;
        tc_fence_after();
        uint32_t dp[kCols];
        tmem_ld32(tmem + lanes + C::kDp + quarter * kCols, dp);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&dp_empty);
#pragma unroll
        for (int k = 0; k < kCols; k += 2) {
          float x, y;
          unpair(mul2(pair(__uint_as_float(e[k]), __uint_as_float(e[k + 1])),
                      add2(pair(__uint_as_float(dp[k]), __uint_as_float(dp[k + 1])), delta_pair)),
                 x, y);
          e[k] = __float_as_uint(x);
          e[k + 1] = __float_as_uint(y);
        }
        const int key0 = (p.first + j) * kTile + quarter * kCols, from = lo - key0, to = hi - key0;
        if (__any_sync(0xFFFFFFFFu, from > 0 || to < kCols))  // whatever p and dp are there
          mask_row(e, seen_bits(from, to), 0u);
        uint32_t w[kCols / 2];
#pragma unroll
        for (int k = 0; k < kCols; k += 2) w[k / 2] = round2<T>(__uint_as_float(e[k]), __uint_as_float(e[k + 1]));
        tmem_st16(s_at, w);
        // keys past the length: their ds is zero, and so must be what it meets
        if (quarter == 0 && p.keys < a.k_len && (p.first + j + 1) * kTile > p.keys) {
          if ((p.first + j) * kTile + row >= p.keys) zero_row<DP>(smem + (2 * C::kQ + t % C::kK) * C::kTileBytes, row);
          fence_async_smem();
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ds_full[t & 1]);
      }
      ok = ok && wait(&done, live & 1);
      tc_fence_after();
      // the tile leaves from the place of its queries, which are done with
      constexpr int kOut = DP / kParts;
      const int slot = live % C::kQ, place = 2 * slot * C::kTileBytes;
      stage_row<T, kOut>(smem + place, row, quarter * kOut, tmem + lanes + C::kDq + quarter * kOut,
                         kNarrow<T> ? a.scale * power_of_two(-lift) : a.scale, lo < hi);
      fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&dq_free);
      named_sync(1, kSoftThreads);
      if (warp == 0) {
        if (elect_one()) {
          if (!wait.gave_up()) store_tile<DP>(&map_dq, q_at + place, a.head_dim, p.row0, p.h, p.b);
          mbar_arrive(&q_free[slot]);
        }
        __syncwarp();
      }
      ++live;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// dk, dv
// ---------------------------------------------------------------------------

template <int DP>
struct Dkv {
  static constexpr int kTileBytes = DP / 64 * kTileChunk;
  static constexpr int kSlots = 2;  // of q and do each
  static constexpr int kSmem = (2 + 2 * kSlots) * kTileBytes + kSlots * kStats * 4 + 1024;
  // TMEM: S^T (p^T over it), dp^T (ds^T over it), dv, dk
  static constexpr uint32_t kDp = 128, kDv = 256, kDk = 384;
};

// As k_attn_dq, a block takes one piece after the other (128 keys of a key head).
// The next piece's keys and values load after the last products that read
// these; its first S and dp run while dk and dv leave through the places of the
// last query tile.
template <typename T, int DP>
__global__ void __launch_bounds__(kBwdThreads, 1)
    k_attn_dkv(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_do,
               const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
               const __grid_constant__ CUtensorMap map_dk, const __grid_constant__ CUtensorMap map_dv,
               const AttnArgs a, int q_tiles, int pieces) {
  using C = Dkv<DP>;
  constexpr int kS = C::kSlots;
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t kv_full, kv_free, q_full[kS], q_empty[kS], do_full[kS], do_empty[kS], s_full,
      dp_full, p_full, ds_full, done, sums_free, out_free[2];
  __shared__ uint32_t tmem_slot, abort_word;
  uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  const uint32_t k_at = smem_u32(smem), v_at = k_at + C::kTileBytes, q_at = v_at + C::kTileBytes,
                 do_at = q_at + kS * C::kTileBytes;
  float* stats = reinterpret_cast<float*>(smem + (2 + 2 * kS) * C::kTileBytes);
  const int warp = warp_number(), lane = threadIdx.x & 31;

  struct Piece {
    int b, c, key0, keys, first, span, n;  // query tiles first ... first + span of each head: n items
  };
  const int off = (int)(a.k_len - a.q_len);
  auto piece = [&](int round, Piece& p) {
    const int grid = gridDim.x, at = round * grid + (round & 1 ? grid - 1 - (int)blockIdx.x : (int)blockIdx.x);
    if (at >= pieces) return false;
    const int kt = a.by_batch_kv(at), bc = at - kt * a.by_batch_kv.d;  // most queries first
    p.b = a.by_kv_heads(bc);
    p.c = bc - p.b * a.kv_heads;
    p.keys = valid_keys(a, p.b);
    p.key0 = kt * kTile;
    // query tiles [first, last) that see one of the tile's valid keys
    int last = q_tiles;
    p.first = a.causal ? max(0, p.key0 - off) / kTile : 0;
    if (a.window > 0) {
      const int end = min(p.key0 + kTile, p.keys) - 1 - off + (int)a.window;  // queries before this
      last = min(last, end <= 0 ? 0 : (end + kTile - 1) / kTile);
    }
    p.span = p.key0 < p.keys ? max(0, last - p.first) : 0;
    p.n = p.span * a.group;
    return true;
  };

  // item i: query tile first + i % span of the group's head i / span; `at`: items before
  auto load_q = [&](const Piece& p, int i, int at) {  // with the tile's statistics; by one thread
    const int s = (at + i) % kS, g = i / p.span, h = p.c * a.group + g, qt = p.first + i - g * p.span;
    mbar_arrive_expect_tx(&q_full[s], C::kTileBytes + kStats * 4);
    load_tile<DP>(q_at + s * C::kTileBytes, &map_q, qt * kTile, h, p.b, &q_full[s]);
    bulk_g2s(stats + s * kStats, a.stats + ((p.b * (int64_t)a.q_heads + h) * q_tiles + qt) * kStats, kStats * 4,
             &q_full[s]);
  };
  auto load_do = [&](const Piece& p, int i, int at) {
    const int s = (at + i) % kS, g = i / p.span, h = p.c * a.group + g, qt = p.first + i - g * p.span;
    mbar_arrive_expect_tx(&do_full[s], C::kTileBytes);
    load_tile<DP>(do_at + s * C::kTileBytes, &map_do, qt * kTile, h, p.b, &do_full[s]);
  };
  auto load_kv = [&](const Piece& p) {
    mbar_arrive_expect_tx(&kv_full, 2 * C::kTileBytes);
    load_tile<DP>(k_at, &map_k, p.key0, p.c, p.b, &kv_full);
    load_tile<DP>(v_at, &map_v, p.key0, p.c, p.b, &kv_full);
  };
  if (warp == kTmaWarp && elect_one()) {
    mbar_init(&kv_full, 1);
    mbar_init(&kv_free, 1);
    for (int s = 0; s < kS; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 1);
      mbar_init(&do_full[s], 1);
      mbar_init(&do_empty[s], 1);
    }
    mbar_init(&s_full, 1);
    mbar_init(&dp_full, 1);
    mbar_init(&p_full, kSoftWarps);
    mbar_init(&ds_full, kSoftWarps);
    mbar_init(&done, 1);
    mbar_init(&sums_free, kSoftWarps);
    for (int d = 0; d < 2; ++d) mbar_init(&out_free[d], 2);
    abort_word = 0;
    mbar_init_fence();
    Piece p;
    const int early = piece(0, p) ? min(p.n, kS) : 0;
    if (early > 0) load_kv(p);
    for (int i = 0; i < early; ++i) load_do(p, i, 0);
    // The statistics are the kernel's before, which may still be running. Every
    // block waits for it, so that this kernel does not end before that one.
    griddep_wait();
    for (int i = 0; i < early; ++i) load_q(p, i, 0);
  }
  if (warp == kMmaWarp) {
    if (lane == 0) {
      tma_prefetch(&map_dk);
      tma_prefetch(&map_dv);
    }
    __syncwarp();
    tmem_alloc(&tmem_slot, 512);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const Waiter wait{&abort_word, &g_attn_bwd_error};

  // `at` items and `live` pieces before, counted over the pieces with items
  Piece p;
  if (warp == kTmaWarp) {
    const uint32_t one = elect_one();
    bool go = true;
    for (int round = 0, at = 0, live = 0; go && piece(round, p); at += p.n, ++round) {
      if (p.n == 0) continue;
      if (round > 0 && (go = wait(&kv_free, (live - 1) & 1)) && one) load_kv(p);
      for (int i = 0; go && i < max(p.n, 2); ++i) {
        // the second item's place is the one that the piece before leaves through
        if (i == 1 && live > 0 && !(go = wait(&out_free[(live - 1) & 1], (live - 1) / 2 & 1))) break;
        if (i == p.n) break;
        if (round == 0 && i < kS) continue;
        const int s = (at + i) % kS, turn = ((at + i) / kS - 1) & 1;
        if (!(go = wait(&q_empty[s], turn))) break;
        if (one) load_q(p, i, at);
        if (!(go = wait(&do_empty[s], turn))) break;
        if (one) load_do(p, i, at);
      }
      ++live;
    }
    if (!go)  // gave up: leave the copies in flight time to land
      for (int i = 0; i < 64; ++i) mbar_try_wait(&kv_free, 0) && mbar_try_wait(&kv_free, 1);
  } else if (warp == kMmaWarp) {
    constexpr bool bf16 = !std::is_same<T, __half>::value;
    constexpr uint32_t by_head = mma_desc(bf16, kTile, kTile, false, false);
    constexpr uint32_t by_rows = mma_desc(bf16, kTile, DP, false, true);
    constexpr uint32_t kStep = C::kTileBytes / 16;
    const uint32_t one = elect_one();
    const uint64_t q_desc = head_desc(q_at), do_desc = head_desc(do_at), k_desc = head_desc(k_at),
                   v_desc = head_desc(v_at), q_rows = rows_desc(q_at), do_rows = rows_desc(do_at);
    auto make_s = [&](int t) {  // t: items since the block's start
      if (!wait(&q_full[t % kS], (t / kS) & 1)) return false;
      tc_fence_after();
      mma_head<DP>(tmem, k_desc, q_desc + t % kS * kStep, by_head, one);
      mma_commit(&s_full, one);
      return true;
    };
    auto make_dp = [&](int t, bool last) {
      if (!wait(&do_full[t % kS], (t / kS) & 1)) return false;
      tc_fence_after();
      mma_head<DP>(tmem + C::kDp, v_desc, do_desc + t % kS * kStep, by_head, one);
      mma_commit(&dp_full, one);
      if (last) mma_commit(&kv_free, one);
      return true;
    };
    bool go = true;
    for (int round = 0, at = 0, live = 0; go && piece(round, p); at += p.n, ++round) {
      if (p.n == 0) continue;
      // While the warps make p the tensor core makes dk and the next dp, while
      // they make ds it makes dv and the next S. (The S and dp of the piece before
      // have been read: its last ds was waited for.)
      go = wait(&kv_full, live & 1) && make_s(at) && make_dp(at, p.n == 1);
#pragma unroll 1
      for (int i = 0; go && i < p.n; ++i) {
        const int t = at + i, s = t % kS;
        if (!(go = wait(&p_full, t & 1))) break;
        if (i == 0 && live > 0 && !(go = wait(&sums_free, (live - 1) & 1))) break;
        tc_fence_after();
        mma_rows<kParts>(tmem + C::kDv, tmem, do_rows + s * kStep, by_rows, i > 0, one);
        mma_commit(&do_empty[s], one);
        if (i + 1 < p.n && !(go = make_s(t + 1))) break;
        if (!(go = wait(&ds_full, t & 1))) break;
        tc_fence_after();
        mma_rows<kParts>(tmem + C::kDk, tmem + C::kDp, q_rows + s * kStep, by_rows, i > 0, one);
        mma_commit(&q_empty[s], one);
        if (i + 1 < p.n && !(go = make_dp(t + 1, i + 2 == p.n))) break;
      }
      mma_commit(&done, one);
      ++live;
    }
  } else {
    // ---- a thread a quarter of a key's row: columns (queries) [32 quarter, ...)
    const int quarter = warp / 4, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21, s_at = tmem + lanes + quarter * kCols, dp_at = s_at + C::kDp;
    const float scale2 = a.scale * kLog2e;
    const uint64_t scale_pair = pair(scale2, scale2);
    // The first eight warps store dk, the others dv, half a row a thread.
    const int second = quarter / 2, col0 = (quarter & 1) * (DP / 2);
    bool ok = true;
#pragma unroll 1
    for (int round = 0, at = 0, live = 0; piece(round, p); at += p.n, ++round) {
      const int key = p.key0 + row;
      if (p.n == 0) {  // seen by no query
        const int64_t* step = second ? a.dvs : a.dks;
        T* out = static_cast<T*>(second ? a.dv : a.dk) + p.b * step[0] + (int64_t)key * step[1] + p.c * step[2];
        if (key < a.k_len)
          for (int d = col0; d < min(a.head_dim, col0 + DP / 2); d += 8)
            *reinterpret_cast<uint4*>(out + d) = make_uint4(0, 0, 0, 0);
        continue;
      }
      // queries [lo, hi) that see the key
      int lo = a.causal ? max(0, key - off) : 0;
      int hi = a.window > 0 ? min((int)a.q_len, key - off + (int)a.window) : (int)a.q_len;
      if (key >= p.keys) hi = lo = 0;
      // p is 2^kLiftP times itself: what is missing to the lift of ds
      const int lift = kNarrow<T> ? ds_lift(__ldcg(&a.ds_top[p.b * (int64_t)a.kv_heads + p.c])) : 0;
      const float rest = kNarrow<T> ? power_of_two(lift - kLiftP) : 1.0f;
      const uint64_t rest_pair = pair(rest, rest);
#pragma unroll 1
      for (int i = 0, qt = 0; ok && i < p.n; ++i, qt = qt + 1 == p.span ? 0 : qt + 1) {
        const int t = at + i, s = t % kS, q0 = (p.first + qt) * kTile + quarter * kCols;
        // the statistics came with the query tile
        if (!(ok = wait(&q_full[s], (t / kS) & 1) && wait(&s_full, t & 1))) break;
        tc_fence_after();
        const uint64_t* lse = reinterpret_cast<const uint64_t*>(stats + s * kStats + quarter * kCols);
        const uint64_t* delta = lse + kTile / 2;
        uint32_t e[kCols], w[kCols / 2];
        tmem_ld32(s_at, e);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < kCols; k += 2) {
          float x, y;
          unpair(fma2(pair(__uint_as_float(e[k]), __uint_as_float(e[k + 1])), scale_pair, lse[k / 2]), x, y);
          e[k] = __float_as_uint(exp2_fast(x));
          e[k + 1] = __float_as_uint(exp2_fast(y));
        }
        const int from = lo - q0, to = hi - q0;
        const bool mask = __any_sync(0xFFFFFFFFu, from > 0 || to < kCols);
        if (mask) mask_row(e, seen_bits(from, to), 0u);
#pragma unroll
        for (int k = 0; k < kCols; k += 2) w[k / 2] = round2<T>(__uint_as_float(e[k]), __uint_as_float(e[k + 1]));
        tmem_st16(s_at, w);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full);
        if (!(ok = wait(&dp_full, t & 1))) break;
        tc_fence_after();
        uint32_t dp[kCols];
        tmem_ld32(dp_at, dp);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < kCols; k += 2) {
          float x, y;
          uint64_t d = add2(pair(__uint_as_float(dp[k]), __uint_as_float(dp[k + 1])), delta[k / 2]);
          if constexpr (kNarrow<T>) d = mul2(d, rest_pair);
          unpair(mul2(pair(__uint_as_float(e[k]), __uint_as_float(e[k + 1])), d), x, y);
          e[k] = __float_as_uint(x);
          e[k + 1] = __float_as_uint(y);
        }
        if (mask) mask_row(e, seen_bits(from, to), 0u);  // 0 times whatever dp is there
#pragma unroll
        for (int k = 0; k < kCols; k += 2) w[k / 2] = round2<T>(__uint_as_float(e[k]), __uint_as_float(e[k + 1]));
        tmem_st16(dp_at, w);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ds_full);
      }
      ok = ok && wait(&done, live & 1);
      tc_fence_after();
      // from the last item's places, which are done with
      const int slot = 2 + second * kS + (at + p.n - 1) % kS;
      stage_row<T, DP / 2>(smem + slot * C::kTileBytes, row, col0, tmem + lanes + (second ? C::kDv : C::kDk) + col0,
                           (second ? 1.0f : a.scale) * (kNarrow<T> ? power_of_two(second ? -kLiftP : -lift) : 1.0f),
                           lo < hi);
      fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sums_free);
      named_sync(1 + second, kSoftThreads / 2);
      if ((warp & 7) == 0) {
        if (elect_one()) {
          if (!wait.gave_up())
            store_tile<DP>(second ? &map_dv : &map_dk, k_at + slot * C::kTileBytes, a.head_dim, p.key0, p.c, p.b);
          mbar_arrive(&out_free[live & 1]);
        }
        __syncwarp();
      }
      ++live;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

int64_t tiles(int64_t len) { return (len + kTile - 1) / kTile; }

template <typename T, int DP>
cudaError_t run(const AttnArgs& a, int sms, cudaStream_t s) {
  CUtensorMap q, g, k, v, dq, dk, dv;
  // a side without rows is never loaded, but its maps still have to be valid
  const bool qs = a.q_len > 0, ks = a.k_len > 0;
  const int64_t q_len = qs ? a.q_len : 1, k_len = ks ? a.k_len : 1;
  if (!attn_map(&q, qs ? a.q : a.k, a.dtype, a.qs, a.batch, q_len, a.q_heads, a.head_dim) ||
      !attn_map(&g, qs ? a.dout : a.k, a.dtype, a.dos, a.batch, q_len, a.q_heads, a.head_dim) ||
      !attn_map(&k, ks ? a.k : a.q, a.dtype, a.ks, a.batch, k_len, a.kv_heads, a.head_dim) ||
      !attn_map(&v, ks ? a.v : a.q, a.dtype, a.vs, a.batch, k_len, a.kv_heads, a.head_dim) ||
      !attn_map(&dq, qs ? a.dq : a.dk, a.dtype, a.dqs, a.batch, q_len, a.q_heads, a.head_dim) ||
      !attn_map(&dk, ks ? a.dk : a.dq, a.dtype, a.dks, a.batch, k_len, a.kv_heads, a.head_dim) ||
      !attn_map(&dv, ks ? a.dv : a.dq, a.dtype, a.dvs, a.batch, k_len, a.kv_heads, a.head_dim))
    return cudaErrorInvalidValue;
  const int64_t q_blocks = tiles(a.q_len) * a.batch * a.q_heads, k_blocks = tiles(a.k_len) * a.batch * a.kv_heads;
  if (q_blocks > 0x70000000ll || k_blocks > 0x70000000ll) return cudaErrorInvalidConfiguration;
  static std::atomic<uint64_t> asked_dq{0}, asked_dkv{0};
  cudaError_t e = allow_smem(k_attn_dq<T, DP>, Dq<DP>::kSmem, asked_dq);
  if (e != cudaSuccess) return e;
  e = allow_smem(k_attn_dkv<T, DP>, Dkv<DP>::kSmem, asked_dkv);
  if (e != cudaSuccess) return e;
  const int q_tiles = (int)tiles(a.q_len);
  // Shares for dq also where attn_grid would take single blocks (lengths, less than
  // four pieces a multiprocessor): a block's next loads then start early, and there
  // are heads x batch pieces of each size to even out. dq, dk and dv with random
  // lengths, dq in shares against single blocks, 12/4 heads, window 256, 6 x 1021:
  // of 64 38.5, 40.5 us, of 128 64.8, 67.6; 16/8 heads, causal: 8 x 512 of 64 39.0,
  // 40.8, 4 x 512 of 128 35.2, 35.6, 3 x 1024 of 128 56.0, 56.9; no mask, 4 x 1024 82.0,
  // 82.1. With lengths, dk and dv are the other way round (attn_grid).
  // Each kernel's blocks start while the last of the one before run, and wait for
  // it where they need its results.
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kBwdThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  if (q_blocks > 0) {
    if (a.v_parts > 0) {
      const int64_t work = a.batch * a.kv_heads * a.v_parts;
      k_attn_bounds<<<(unsigned)(work < sms * 8ll ? work : sms * 8ll), 256, 0, s>>>(a, Divide(a.head_dim / 8), work);
      e = cudaGetLastError();
      if (e != cudaSuccess) return e;
      cfg.numAttrs = 1;
    }
    cfg.gridDim = dim3((unsigned)(q_blocks < sms ? q_blocks : sms));
    cfg.dynamicSmemBytes = Dq<DP>::kSmem;
    e = cudaLaunchKernelEx(&cfg, k_attn_dq<T, DP>, q, g, k, v, dq, a, q_tiles, (int)q_blocks);
    if (e != cudaSuccess) return e;
  }
  if (k_blocks == 0) return cudaSuccess;
  cfg.gridDim = dim3(attn_grid(a, k_blocks, sms));
  cfg.dynamicSmemBytes = Dkv<DP>::kSmem;
  cfg.numAttrs = q_blocks > 0 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k_attn_dkv<T, DP>, q, g, k, v, dk, dv, a, q_tiles, (int)k_blocks);
}

template <typename T>
cudaError_t backward_t(const AttnArgs& a, int sms, cudaStream_t s) {
  return a.head_dim <= 64 ? run<T, 64>(a, sms, s) : run<T, 128>(a, sms, s);
}

}  // namespace

ZG_ERROR_WORD(attn_bwd_error, g_attn_bwd_error)

int64_t attention_backward_bytes(const AttnArgs& a) {
  const int64_t bounds = a.dtype == kF16 ? a.batch * a.kv_heads * (kBoundParts + 1) : 0;
  return (a.batch * a.q_heads * tiles(a.q_len) * kStats + bounds) * 4;
}

cudaError_t launch_attention_backward(const AttnArgs& args, int sms, cudaStream_t s) {
  AttnArgs a = args;
  if (a.dtype != kF16) return backward_t<__nv_bfloat16>(a, sms, s);
  a.v_top = reinterpret_cast<uint32_t*>(a.stats + a.batch * a.q_heads * tiles(a.q_len) * kStats);
  a.ds_top = a.v_top + a.batch * a.kv_heads * kBoundParts;
  a.v_parts = static_cast<int>(tiles(a.k_len) < kBoundParts ? tiles(a.k_len) : kBoundParts);
  return backward_t<__half>(a, sms, s);
}

}  // namespace zg
