// Attention forward: o = softmax(scale q k^T) v and the rows' log-sum-exp.
//
// A piece of work is two tiles of 128 query rows that share their keys: tiles
// of the query heads of one key head, counted tile by tile and head by head,
// so with two heads a group both tiles are the same rows of two heads. Keys
// and values pass once through shared memory (TMA) in tiles of 128.
//   S_t = Q_t K^T      tcgen05, S in TMEM (fp32)
//   P_t = 2^(c S_t - c m)   two threads a row, 64 keys each; P_t (16 bits) over
//                      S_t in TMEM
//   O_t += P_t V       tcgen05, P from TMEM, O in TMEM
// The two tiles alternate: while eight warps turn S_0 into P_0 the tensor core
// works for tile 1, and the other way round. The row's maximum m is kept as it
// was until it grows by more than 8 in the exponent of two: P stays below 2^8
// (in fp16 it is held 2^7 higher: weights down to 2^-21 of the largest keep all
// their bits, the error of smaller ones is 2^-32 of it), sums and O are fp32, and O is rescaled rarely (once or twice a row on ordinary
// data) instead of in every tile. The first tile's maximum is taken alone, so
// that tile is not worked on twice.
//
// What bounds it is the chain from one S through the softmax to the next; two
// threads a row instead of one shorten it (1 x 8192, 16/8 heads of 128, no mask:
// 450 us with one, 400 with two). Measured in bf16, 16/8 heads of 128, causal:
// 1 x 8192 187 us (1470 TFLOP/s), 4 x 2048 65 us (1050); blocks that end with
// each piece took 196 and 75 us. 16 heads of 64, 4 x 2048: 62 us (550), where a
// pair's products are half as long but the softmax is not.
//
// Keys past a batch entry's length: their S is replaced by -inf, and their
// rows of V (whatever they hold) by zeros in shared memory.
#include <type_traits>

#include "attn.cuh"

namespace zg {
namespace {

__device__ unsigned g_attn_fwd_error;

// Four softmax groups of four warps (tile, half of the keys), then a group of
// which one warp issues the TMA loads and one the MMAs. The groups' registers
// add up to the launch's: 512 x 104 + 128 x 64 = 640 x 96.
constexpr int kFwdThreads = 20 * 32, kTmaWarp = 16, kMmaWarp = 17;
constexpr int kSoftmaxRegs = 104, kOtherRegs = 64;
// How far the maximum may lag, as an exponent of two. In fp16 p and its sums are
// lifted by what then is left below the largest number, 2^16. (A lag of 3 and a
// lift of 12: 1 x 8192 192 to 209 us, 4 x 2048 70 to 76, for more rescaling.)
constexpr float kStale = 8.0f;
template <typename T>
constexpr float kLift = kNarrow<T> ? 15.0f - kStale : 0.0f;

template <int DP>
struct Fwd {
  static constexpr int kTileBytes = DP / 64 * kTileChunk;
  static constexpr int kSlots = DP == 128 ? 4 : 8;  // keys and values in turn
  static constexpr int kSmem = (2 + kSlots) * kTileBytes + 1024;
  static constexpr uint32_t kO = 256;  // TMEM: S_0, S_1 at 0, 128; O_0, O_1 from here, DP columns each
};

// A block takes one piece of work after the other: while a piece's result leaves,
// the next one's keys and values arrive, and its first products start as soon as
// its queries are there. Pieces with most keys come first; every other round runs
// backwards, so that the rounds' differences even out. Pieces that see no key
// touch no barrier and no shared memory: slots and phases count the others.
template <typename T, int DP>
__global__ void __launch_bounds__(kFwdThreads, 1)
    k_attn_fwd(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
               const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o, const AttnArgs a,
               int units, int pairs, int pieces) {
  using C = Fwd<DP>;
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t q_full[2], q_free[2], kv_full[C::kSlots], kv_empty[C::kSlots], s_full[2], p_full[2],
      o_full[2], o_free[2];
  __shared__ uint32_t tmem_slot, abort_word;
  __shared__ float tops[2][2][2][kTile];  // [turn][tile][half][row]: maxima, in the end sums
  uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  const uint32_t base = smem_u32(smem), ring = base + 2 * C::kTileBytes;
  const int warp = warp_number(), lane = threadIdx.x & 31;

  struct Piece {
    int b, c, u, tiles, keys, first, n;  // query tiles (units) u ... and n key tiles from `first`
  };
  auto piece = [&](int round, Piece& w) {
    const int grid = gridDim.x, at = round * grid + (round & 1 ? grid - 1 - (int)blockIdx.x : (int)blockIdx.x);
    if (at >= pieces) return false;
    const int turn = a.by_batch_kv(at), bh = at - turn * a.by_batch_kv.d;
    w.b = a.by_kv_heads(bh);
    w.c = bh - w.b * a.kv_heads;
    w.u = 2 * (pairs - 1 - turn);
    w.tiles = min(2, units - w.u);
    w.keys = valid_keys(a, w.b);
    int last = 0;  // key tiles [first, last) that one of the query tiles sees
    w.first = 0x7FFFFFFF;
    for (int t = 0; t < w.tiles; ++t) {
      const int row0 = a.by_group(w.u + t) * kTile, row1 = min(row0 + kTile, (int)a.q_len) - 1;
      int lo, hi, skip;
      key_range(a, w.keys, row0, lo, skip);
      key_range(a, w.keys, row1, skip, hi);
      if (lo < hi) {
        w.first = min(w.first, lo / kTile);
        last = max(last, (hi + kTile - 1) / kTile);
      }
    }
    w.n = max(0, last - w.first);
    return true;
  };

  // The TMA warp prepares the barriers and starts the first loads before the
  // block's first barrier: TMEM's allocation takes place meanwhile.
  auto load = [&](const Piece& w, int i, int at) {  // K and V tiles in turn, by one thread; `at`: loads before
    const int s = (at + i) % C::kSlots;
    mbar_arrive_expect_tx(&kv_full[s], C::kTileBytes);
    load_tile<DP>(ring + s * C::kTileBytes, i & 1 ? &map_v : &map_k, (w.first + i / 2) * kTile, w.c, w.b, &kv_full[s]);
  };
  auto load_q = [&](const Piece& w, int t) {
    mbar_arrive_expect_tx(&q_full[t], C::kTileBytes);
    load_tile<DP>(base + t * C::kTileBytes, &map_q, a.by_group(w.u + t) * kTile, w.c * a.group + a.by_group.mod(w.u + t),
                  w.b, &q_full[t]);
  };
  if (warp == kTmaWarp && elect_one()) {
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 1);
      mbar_init(&q_free[t], 1);
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 8);
      mbar_init(&o_full[t], 1);
      mbar_init(&o_free[t], 8);
    }
    abort_word = 0;
    mbar_init_fence();
    Piece w;
    if (piece(0, w) && w.n > 0) {
      for (int t = 0; t < w.tiles; ++t) load_q(w, t);
      for (int i = 0; i < min(2 * w.n, C::kSlots); ++i) load(w, i, 0);
    }
  }
  if (warp == kMmaWarp) {
    if (lane == 0) tma_prefetch(&map_o);
    __syncwarp();
    tmem_alloc(&tmem_slot, 512);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const Waiter wait{&abort_word, &g_attn_fwd_error};

  if (warp >= kTmaWarp) fewer_registers<kOtherRegs>();
  else more_registers<kSoftmaxRegs>();
  // Counted over the pieces with keys: `at` K and V tiles, done[t] pieces of
  // query tile t, steps[t] its key tiles.
  Piece w;
  if (warp == kTmaWarp) {
    const uint32_t one = elect_one();
    int done[2] = {0, 0}, at = 0;
    bool go = true;
    for (int round = 0; go && piece(round, w); ++round) {
      if (w.n == 0) continue;
      const int early = min(2 * w.n, C::kSlots);
      for (int i = round == 0 ? early : 0; go && i < 2 * w.n; ++i) {
        if (!(go = wait(&kv_empty[(at + i) % C::kSlots], ((at + i) / C::kSlots - 1) & 1))) break;
        if (one) load(w, i, at);
        if (i != early - 1) continue;
        // the queries' places are free once the results before have left
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (t < w.tiles && go && (go = wait(&q_free[t], (done[t] - 1) & 1)) && one) load_q(w, t);
      }
      at += 2 * w.n;
      ++done[0];
      done[1] += w.tiles - 1;
    }
    if (!go)  // gave up: leave the copies in flight time to land
      for (int i = 0; i < 64; ++i) mbar_try_wait(&q_free[0], 0) && mbar_try_wait(&q_free[0], 1);
  } else if (warp == kMmaWarp) {
    // ---- the tensor cores
    constexpr bool bf16 = !std::is_same<T, __half>::value;
    constexpr uint32_t by_head = mma_desc(bf16, kTile, kTile, false, false);
    constexpr uint32_t by_rows = mma_desc(bf16, kTile, DP, false, true);
    const uint32_t one = elect_one();
    const uint64_t q_desc = head_desc(base), k_desc = head_desc(ring), v_desc = rows_desc(ring);
    auto slot = [&](int i) { return static_cast<uint32_t>(i % C::kSlots * (C::kTileBytes / 16)); };
    auto arrived = [&](int i) {
      const bool ok = wait(&kv_full[i % C::kSlots], (i / C::kSlots) & 1);
      tc_fence_after();
      return ok;
    };
    auto make_s = [&](int t, int i) {
      mma_head<DP>(tmem + t * kTile, q_desc + t * (C::kTileBytes / 16), k_desc + slot(i), by_head, one);
      mma_commit(&s_full[t], one);
    };
    uint32_t done[2] = {0, 0}, steps[2] = {0, 0};
    int at = 0;
    bool go = true;
    for (int round = 0; go && piece(round, w); ++round) {
      if (w.n == 0) continue;
      go = arrived(at);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (t >= w.tiles || !go) break;
        if (!(go = wait(&q_full[t], done[t] & 1))) break;
        tc_fence_after();
        make_s(t, at);
      }
      if (go) mma_commit(&kv_empty[at % C::kSlots], one);
#pragma unroll 1
      for (int j = 0; go && j < w.n; ++j) {
        const int kn = at + 2 * j + 2, v = at + 2 * j + 1;
        const bool more = j + 1 < w.n;
        go = arrived(v);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (t >= w.tiles || !go) break;
          if (!(go = wait(&p_full[t], (steps[t] + j) & 1))) break;
          if (j == 0 && done[t] > 0 && !(go = wait(&o_free[t], (done[t] - 1) & 1))) break;
          tc_fence_after();
          mma_rows<2>(tmem + C::kO + t * DP, tmem + t * kTile, v_desc + slot(v), by_rows, j > 0, one);
          if (t == w.tiles - 1) mma_commit(&kv_empty[v % C::kSlots], one);
          if (!more) {
            mma_commit(&o_full[t], one);
            continue;
          }
          if (t == 0 && !(go = arrived(kn))) break;
          make_s(t, kn);  // over P_t, which the product before it reads first
          if (t == w.tiles - 1) mma_commit(&kv_empty[kn % C::kSlots], one);
        }
      }
      at += 2 * w.n;
      ++done[0];
      steps[0] += w.n;
      if (w.tiles == 2) ++done[1], steps[1] += w.n;
    }
  } else if (warp < kTmaWarp) {
    // ---- softmax: a thread half a row, keys [64 half, 64 half + 64) of each tile
    const int t = warp / 8, half = warp / 4 & 1, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t s_at = tmem + lanes + t * kTile + half * 64, o_at = tmem + lanes + C::kO + t * DP + half * (DP / 2);
    const float scale2 = a.scale * kLog2e;
    bool ok = true;
    uint32_t done = 0, steps = 0;  // of this tile
    int at = 0;
#pragma unroll 1
    for (int round = 0; piece(round, w); at += 2 * w.n, ++round) {
      if (t >= w.tiles) continue;
      const int keys = w.keys, first = w.first, n = w.n;
      const int row0 = a.by_group(w.u + t) * kTile, i = row0 + row;  // the query
      const int h = w.c * a.group + a.by_group.mod(w.u + t);
      float* lse = a.lse + (w.b * (int64_t)a.q_heads + h) * a.q_len + i;
      if (n == 0) {
        if (i < a.q_len) {
          T* o = static_cast<T*>(a.o) + w.b * a.os[0] + (int64_t)i * a.os[1] + h * a.os[2];
          for (int d = half * (DP / 2); d < min(a.head_dim, (half + 1) * (DP / 2)); d += 8)
            *reinterpret_cast<uint4*>(o + d) = make_uint4(0, 0, 0, 0);
          if (half == 0) *lse = -INFINITY;
        }
        continue;
      }
      float top, total = 0.0f;
      int lo, hi;
      key_range(a, keys, i, lo, hi);
      {  // nothing to go by yet: the first tile's maximum
        ok = wait(&s_full[t], steps & 1) && ok;
        tc_fence_after();
        const int from = lo - first * kTile - half * 64, to = hi - first * kTile - half * 64;
        float m = -INFINITY;
#pragma unroll 1
        for (int q = 0; q < 64; q += 32) {
          uint32_t r[32];
          tmem_ld32(s_at + q, r);
          tmem_wait_ld();
          mask_row(r, seen_bits(from - q, to - q), kMinusInf);
#pragma unroll
          for (int k = 0; k < 32; k += 2) m = max3(m, __uint_as_float(r[k]), __uint_as_float(r[k + 1]));
        }
        tops[1][t][half][row] = m;
        named_sync(3 + warp / 8 * 4 + (warp & 3), 64);
        top = lo < hi ? fmaxf(m, tops[1][t][half ^ 1][row]) : 0.0f;
      }
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        // a wait that gives up goes on to the barriers with what is there: the
        // other half may be waiting in them
        ok = wait(&s_full[t], (steps + j) & 1) && ok;
        tc_fence_after();
        const int key0 = (first + j) * kTile, from = lo - key0 - half * 64, to = hi - key0 - half * 64;
        // columns [from, to) are seen; most tiles need no mask
        const bool mask = __any_sync(0xFFFFFFFFu, from > 0 || to < 64);
        uint32_t w[2][16];
        float sums;
#pragma unroll 1
        for (int turn = 0;; turn ^= 1) {
          float minus = top == -INFINITY ? 0.0f : -top * scale2;
          if constexpr (kNarrow<T>) minus = __fadd_rn(minus, kLift<T>);  // fused it took a register more, and spilled
          const uint64_t scale_pair = pair(scale2, scale2), minus_pair = pair(minus, minus);
          uint64_t sum[2] = {0, 0};
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t r[32];
            tmem_ld32(s_at + q * 32, r);
            tmem_wait_ld();
            if (mask) mask_row(r, seen_bits(from - q * 32, to - q * 32), kMinusInf);
#pragma unroll
            for (int k = 0; k < 32; k += 8)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                m4[e] = max3(m4[e], __uint_as_float(r[k + e]), __uint_as_float(r[k + 4 + e]));
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float x, y;
              unpair(fma2(pair(__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1])), scale_pair, minus_pair), x, y);
              x = exp2_fast(x);
              y = exp2_fast(y);
              sum[k & 1] = add2(sum[k & 1], pair(x, y));
              w[q][k] = round2<T>(x, y);
            }
          }
          float x, y;
          unpair(add2(sum[0], sum[1]), x, y);
          sums = x + y;
          float m = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]);
          // the other half's maximum, from the warp with the same rows
          tops[turn][t][half][row] = m;
          named_sync(3 + warp / 8 * 4 + (warp & 3), 64);
          m = fmaxf(m, tops[turn][t][half ^ 1][row]);
          // the first maximum, or one that has grown too far: rescale, and again
          const bool raise = m > top && (top == -INFINITY || (m - top) * scale2 > kStale);
          if (!__any_sync(0xFFFFFFFFu, raise)) break;
          const float f = raise ? exp2_fast((top - m) * scale2) : 1.0f;
          if (raise) top = m;
          total *= f;
          // O is complete up to the tile before: its product was issued before this S
#pragma unroll 1
          for (int k = 0; k < DP / 2; k += 16) {
            uint32_t o[16];
            tmem_ld16(o_at + k, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st16(o_at + k, o);
          }
        }
        total += sums;
        tmem_st16(s_at, w[0]);
        tmem_st16(s_at + 16, w[1]);
        if (t == 0 && half == 0 && key0 + kTile > keys && keys < a.k_len) {
          // rows of V past the length: zeros. Tile 0's product is the first to
          // read them, and waits for this thread.
          const int v = at + 2 * j + 1;
          ok = wait(&kv_full[v % C::kSlots], (v / C::kSlots) & 1) && ok;
          if (key0 + row >= keys) zero_row<DP>(smem + (2 + v % C::kSlots) * C::kTileBytes, row);
          fence_async_smem();
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t]);
      }
      ok = wait(&o_full[t], done & 1) && ok;
      tc_fence_after();
      // both halves' sums, in the order of the keys
      tops[0][t][half][row] = total;
      named_sync(3 + warp / 8 * 4 + (warp & 3), 64);
      total = tops[0][t][0][row] + tops[0][t][1][row];
      // No key seen: the sum is 0 and top still is. (Products that are all -inf have
      // a sum of 0 too, but no softmax: NaN, in o by 0 times 1 / 0.)
      const bool none = total == 0.0f && top == 0.0f;
      // The tile leaves from the place of its queries, which are done with.
      stage_row<T, DP / 2>(smem + t * C::kTileBytes, row, half * (DP / 2), o_at, 1.0f / total, !none);
      fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_free[t]);
      if (half == 0 && i < a.q_len && ok) {
        const float l = (top * scale2 + (log2f(total) - kLift<T>)) * kLn2;
        *lse = none ? -INFINITY : total == 0.0f ? __uint_as_float(0x7FC00000u) : l;
      }
      named_sync(1 + t, 256);
      if ((warp & 7) == 0) {
        if (elect_one()) {
          if (!wait.gave_up()) store_tile<DP>(&map_o, base + t * C::kTileBytes, a.head_dim, row0, h, w.b);
          mbar_arrive(&q_free[t]);
        }
        __syncwarp();
      }
      ++done;
      steps += n;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

template <typename T, int DP>
cudaError_t run(const AttnArgs& a, int sms, cudaStream_t s) {
  using C = Fwd<DP>;
  CUtensorMap q, k, v, o;
  // without keys nothing is loaded, but the maps still have to be valid
  const int64_t k_len = a.k_len > 0 ? a.k_len : 1;
  if (!attn_map(&q, a.q, a.dtype, a.qs, a.batch, a.q_len, a.q_heads, a.head_dim) ||
      !attn_map(&o, a.o, a.dtype, a.os, a.batch, a.q_len, a.q_heads, a.head_dim) ||
      !attn_map(&k, a.k_len > 0 ? a.k : a.q, a.dtype, a.ks, a.batch, k_len, a.kv_heads, a.head_dim) ||
      !attn_map(&v, a.k_len > 0 ? a.v : a.q, a.dtype, a.vs, a.batch, k_len, a.kv_heads, a.head_dim))
    return cudaErrorInvalidValue;
  const int64_t q_tiles = (a.q_len + kTile - 1) / kTile, pairs = (q_tiles * a.group + 1) / 2;
  const int64_t blocks = pairs * a.batch * a.kv_heads;
  if (blocks > 0x70000000ll) return cudaErrorInvalidConfiguration;
  static std::atomic<uint64_t> asked{0};
  cudaError_t e = allow_smem(k_attn_fwd<T, DP>, C::kSmem, asked);
  if (e != cudaSuccess) return e;
  k_attn_fwd<T, DP><<<attn_grid(a, blocks, sms), kFwdThreads, C::kSmem, s>>>(
      q, k, v, o, a, (int)(q_tiles * a.group), (int)pairs, (int)blocks);
  return cudaGetLastError();
}

template <typename T>
cudaError_t forward_t(const AttnArgs& a, int sms, cudaStream_t s) {
  return a.head_dim <= 64 ? run<T, 64>(a, sms, s) : run<T, 128>(a, sms, s);
}

}  // namespace

ZG_ERROR_WORD(attn_fwd_error, g_attn_fwd_error)

cudaError_t launch_attention_forward(const AttnArgs& a, int sms, cudaStream_t s) {
  return a.dtype == kF16 ? forward_t<__half>(a, sms, s) : forward_t<__nv_bfloat16>(a, sms, s);
}

}  // namespace zg
