// The experts' products and the products of scaled e4m3 matrices, on the tensor
// cores: out[n][m] = sum over k of a(m, k) b(n, k), a the weights (or the rows
// whose columns are contiguous in out), b the rows.
//
// A pair of blocks (two SMs) makes tiles of 256 along M x up to 256 along N (224
// with scales, which need TMEM too): each block holds half of either operand, so
// an element that comes from L2 meets 256 others. The ragged side is N (rows in
// runs by expert) or K (a weight gradient's rows). How long the runs are is known
// on the device only: every block reads the offsets and takes each pairs-th tile
// of the list that they make. Tiles of a run are equally wide, so its rows fill
// them to within 32; rows of the next run that a tile also reads end in columns
// that nobody stores. Along K a run's last rows are loaded behind rows of zeros: TMA
// counts rows from the step's first (Form), and from a negative start it fills zeros.
//
// Twelve warps: one loads by TMA, one issues MMAs, one brings scales (words of four
// exponents, which the tensor core applies itself), eight take the sums. These leave TMEM
// after a run of steps and are added up in registers, rounded: the tensor core truncates
// where it adds, which over thousands of steps would cost an fp32 result its last bits.
// TMEM holds two tiles' sums, so the MMAs go on meanwhile.
//
// An SM's stores leave at 32 bytes a cycle at most, whatever way they take (measured
// alone and on all SMs at once: by TMA, from registers, by 64 to 512 bytes of a row).
// fp32 sums go straight from registers, a warp 128 bytes of a row. 16-bit ones go
// through shared memory: 8 x 8 matrices are turned on the way in, so that a row of out
// lies there as it does in memory, and TMA stores take 32 rows from there while the
// next are made. From registers, 64 bytes of a row each, they were as fast, but not
// where rows start inside a sector (520 x 1000 weights: 47 us, so 27). Rows behind the
// last whole 32 of a run, and outs whose rows do not start on 16 bytes, go by ordinary
// stores.
//
// Measured (captured, one behind the other): 16384 x 2048 x 2048 in bf16 by 16 even
// experts 78 us forward (1770 TFLOP/s), 98 for the weights' gradient in fp32; 8192 x 8192 x
// 8192 570 us (1930, 0.98 of the library's burst rate); 8192 x 8192 x 4096 in e4m3 150 us
// (3660 TFLOP/s); 74 rows x 2048 x 1024 by 16 experts 9.5 us (6.2 TB/s of weights). Large
// ones are bound by the tensor cores (74 to 84 % of the cycles; the rest is a pair's last
// tile, which others do not have, and each kernel's start and end), long under load by the
// power limit: the clock falls from 1.9 to 1.5 GHz, and the forward products take 91 us, the
// library's batched product 86. fp32 weight gradients: 268 MB of sums beside them (added to
// what is there 479 us: reads that wait for each other). Many small experts: a tile's way
// out (4500 cycles for 128 x 192 sums of a block) is longer than its products.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "block.h"
#include "experts.h"
#include "tc.cuh"
#include "vec.cuh"

namespace zg {
namespace {

__device__ unsigned g_product_error;

constexpr int kTileM = 256;                 // of a pair
constexpr int kStepBytes = 128;             // along the contraction: 64 elements, of e4m3 128
constexpr int kABytes = 128 * kStepBytes;   // of one block
constexpr int kMnRows = 64;                 // rows of a step whose operands are contiguous along M and N
constexpr int kMnChunk = kMnRows * 128;     // bytes of 64 columns of them
// Steps whose sums stay in the tensor core (powers of two). Each of four truncated
// additions a step may cost 2^-23 of the sum: 4e-6 after 8 steps, 8e-6 after 16, of a
// 16-bit result's rounding (4e-4 and up). On the inputs of a layer fp32 results are off
// by 4e-7 with 8 (9e-7 with 16) in norm. 16-bit results of 16384 x 2048 x 2048 in bf16
// differ from rounded fp32 sums by 1.1e-4 in norm with 64, 7e-5 with 16 in the same 82 us,
// 6e-5 with 8 in 84; of 8192 x 8192 x 8192 16 costs 0.8 %. e4m3's steps are of twice as
// many products for each addition: 5e-5 with 64; 16 would take 8 % of a product of 128 x
// 4096 x 4096.
constexpr int kRunF32 = 8, kRunHalf = 16, kRunScaledHalf = 64;
constexpr int kMaxStages = 12;
constexpr int kMostSmem = 232448 - 1024;    // dynamic shared memory; the rest is for the barriers
constexpr int kScaleSteps = 4;              // steps that a word of scales lasts
constexpr int kScaleSlots = 4;
constexpr int kScaleSlot = 3 * 512;         // of 128 rows of a, 256 of b
constexpr int kEpilogue = 8;                // warps
constexpr int kThreadsHere = (4 + kEpilogue) * 32;
struct ProductPlan {
  int tile_n;    // widest tile, a multiple of 32
  int stages;
  int run;       // steps whose sums stay in the tensor core, a power of two
  int b_bytes;   // of a stage and block
  int pairs;
  int store_at, scales_at, runs_at;  // in shared memory, behind the stages
  Divide by_expert, by_band;         // ragged K: by an expert's tiles, by those of 8 along M
  int tiles_out;                     // out is of 16 bits and can be written by TMA
};

template <bool A_MN, bool B_MN, bool SCALED>
struct Form {
  static constexpr bool kRaggedK = B_MN;
  static constexpr int kStepK = SCALED ? 128 : 64;  // elements
  static constexpr int kMaxN = SCALED ? 224 : 256;
  static constexpr int kScaleCols = 2 * kMaxN;      // where the scales' TMEM starts
  // The operands' tensor maps: contiguous side, the other, groups; with a ragged K
  // (both contiguous along M and N): columns, a step's rows, the step's first row, so
  // that rows in front of the first are outside of the tensor.
};

// The runs of rows, in shared memory, with those of no expert at the end.
struct Runs {
  int *first, *rows;  // a run's first row, how many; [groups + 2]
  int* start;         // tiles along N of the runs before; [groups + 3]
  int* reach;         // the lowest and the highest row that runs reach
  __host__ __device__ static constexpr int bytes(int groups) { return (3 * (groups + 3) + 2) * 4; }
  __device__ __forceinline__ Runs(void* at, int groups)
      : first(static_cast<int*>(at)), rows(first + groups + 3), start(rows + groups + 3), reach(start + groups + 3) {}
};

struct Tile {
  int g;
  int m0;             // of the pair
  int n0;             // first row of b and out (ragged K: of an expert's matrix)
  int width, padded;  // rows of it; up to 32
  int k0, rows_k;     // the first row along K, how many (ragged K)
  int steps;
};

// A block's way through the tiles: 32-bit numbers, which the host has checked. (A run
// along K may have 2^31 - 1 rows: its last step's end is not an int.)
template <typename F>
struct Walk {
  const ProductArgs& a;
  const ProductPlan& p;
  const Runs& runs;
  uint32_t m_tiles, n_tiles, i, total;
  int g = 0;

  __device__ __forceinline__ Walk(const ProductArgs& a_, const ProductPlan& p_, const Runs& r_, int pair)
      : a(a_), p(p_), runs(r_), m_tiles((static_cast<uint32_t>(a_.m) + kTileM - 1) / kTileM), i(pair) {
    n_tiles = F::kRaggedK ? (static_cast<uint32_t>(a.n) + p.tile_n - 1) / p.tile_n : 0;
    total = (F::kRaggedK ? a.groups * n_tiles : runs.start[a.groups + 2]) * m_tiles;
  }
  __device__ __forceinline__ bool next(Tile& t) {
    if (i >= total) return false;
    uint32_t local, rows, across;
    if (F::kRaggedK) {
      const uint32_t each = m_tiles * n_tiles;
      g = static_cast<int>(p.by_expert(i));
      local = i - g * each;
      rows = static_cast<uint32_t>(a.n);
      across = n_tiles;
      t.k0 = runs.first[g];
      t.rows_k = runs.rows[g];
      t.steps = static_cast<int>((static_cast<uint32_t>(t.rows_k) + kMnRows - 1) / kMnRows);
    } else {
      while (runs.start[g + 1] * m_tiles <= i) ++g;
      local = i - runs.start[g] * m_tiles;
      rows = runs.rows[g];
      across = runs.start[g + 1] - runs.start[g];
      t.k0 = 0;
      t.steps = g < a.groups ? (static_cast<int>(a.k) + F::kStepK - 1) / F::kStepK : 0;  // else rows of no expert
    }
    // bands of 8 tiles along M: the rows' tiles come round while a band's weights stay in L2
    const uint32_t band = F::kRaggedK ? p.by_band(local) : local / (8 * across), in = local - band * 8 * across;
    const uint32_t wide = min(8u, m_tiles - band * 8), n = wide == 8 ? in / 8 : in / wide;
    t.m0 = static_cast<int>((band * 8 + in - n * wide) * kTileM);
    const uint32_t each = F::kRaggedK ? p.tile_n : ((rows + across - 1) / across + 31) / 32 * 32, at = n * each;
    t.g = g;
    t.n0 = static_cast<int>((F::kRaggedK ? 0 : runs.first[g]) + at);
    t.width = static_cast<int>(min(each, rows - at));
    t.padded = (t.width + 31) / 32 * 32;
    i += p.pairs;
    return true;
  }
  static __device__ __forceinline__ int bound(const ProductArgs& a, int g) {
    const int rows = static_cast<int>(F::kRaggedK ? a.k : a.n);
    if (a.offsets == nullptr) return g == 0 ? 0 : rows;
    return max(0, min(a.offsets[g], rows));
  }
};

// The runs of offsets that decrease, by one thread. Out of line: in the way of every call
// its code cost a kernel whose instructions are in no cache yet 3000 cycles.
template <typename F>
__device__ __noinline__ void join_runs(const ProductArgs& a, Runs runs) {
  const int start = Walk<F>::bound(a, 0);
  int end = start;
  for (int g = 0; g < a.groups; ++g) {
    const int to = max(end, Walk<F>::bound(a, g + 1));
    runs.first[g] = end;
    runs.rows[g] = to - end;
    end = to;
  }
  runs.reach[0] = end > start ? start : static_cast<int>(a.n);
  runs.reach[1] = end > start ? end : 0;
}

// Fill `runs` (all threads of the block).
template <typename F>
__device__ void read_runs(const ProductArgs& a, const ProductPlan& p, const Runs& runs) {
  if (threadIdx.x == 0) {
    runs.reach[0] = static_cast<int>(a.n);
    runs.reach[1] = 0;
  }
  __syncthreads();
  bool falls = false;
  for (int g = threadIdx.x; g < a.groups; g += kThreadsHere) {
    const int from = Walk<F>::bound(a, g), to = Walk<F>::bound(a, g + 1);
    falls = falls || to < from;
    runs.first[g] = from;
    runs.rows[g] = max(0, to - from);
    if (!F::kRaggedK && to > from) {
      atomicMin(&runs.reach[0], from);
      atomicMax(&runs.reach[1], to);
    }
  }
  // An offset that decreases, which no routing makes, counts as the largest before it: runs
  // stay apart, so a row has one writer and there are no more tiles than the host has counted.
  if (__syncthreads_or(falls)) {
    if (threadIdx.x == 0) join_runs<F>(a, runs);
    __syncthreads();
  }
  if (!F::kRaggedK && threadIdx.x < 32) {
    if (threadIdx.x == 0) {
      // rows before the first run and behind the last belong to nobody (all, when there is no run)
      runs.first[a.groups] = runs.reach[1];
      runs.rows[a.groups] = static_cast<int>(a.n) - runs.reach[1];
      runs.first[a.groups + 1] = 0;
      runs.rows[a.groups + 1] = min(runs.reach[0], runs.reach[1]);
    }
    __syncwarp();
    int sum = 0;
    for (int at = 0; at < a.groups + 2; at += 32) {
      const int g = at + threadIdx.x;
      const int own = g < a.groups + 2 ? static_cast<int>((static_cast<uint32_t>(runs.rows[g]) + p.tile_n - 1) / p.tile_n) : 0;
      int v = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (static_cast<int>(threadIdx.x) >= o) v += u;
      }
      if (g < a.groups + 2) runs.start[g] = sum + v - own;
      sum += __shfl_sync(0xFFFFFFFFu, v, 31);
    }
    if (threadIdx.x == 0) runs.start[a.groups + 2] = sum;
  }
  __syncthreads();
}

// A place in a ring of n.
struct Ring {
  int n, at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ explicit Ring(int n_) : n(n_) {}
  __device__ __forceinline__ void step() {
    if (++at == n) {
      at = 0;
      phase ^= 1;
    }
  }
};

template <typename T>
__device__ __forceinline__ uint32_t pair_of(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pair_of<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pair_of<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A buffer of 16-bit results: [64 columns][row][16-byte piece ^ row], as TMA takes
// it; 128 columns of kStoreRows rows.
constexpr int kStoreRows = 32, kStoreBytes = kStoreRows * 128 * 2;
constexpr int kStoreSpace = 4 * kStoreBytes;  // two for each half of the epilogue's warps

// Its first `rows` rows to `out` (its first element) by ordinary stores; four warps.
__device__ __noinline__ void store_rows(const ProductArgs& a, const uint8_t* buf, uint16_t* out, int64_t m, int rows,
                                        int warp, int lane, bool aligned) {
  const int piece = lane % 16;
  const int columns = static_cast<int>(min((int64_t)8, a.m - m - piece * 8));
  for (int r = warp * 2 + lane / 16; r < rows; r += 8) {
    uint16_t e[8];
    *reinterpret_cast<uint4*>(e) =
        *reinterpret_cast<const uint4*>(buf + piece / 8 * (kStoreRows * 128) + r * 128 + (piece % 8 ^ (r & 7)) * 16);
    uint16_t* to = out + r * a.out_row + piece * 8;
    if (aligned && columns == 8) {
      *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(e);
      continue;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j >= columns) break;
      to[j] = e[j];
    }
  }
}

// A tile's sums out, as T (16 bits), from TMEM at `from` (zeros). Four warps (`quarter`:
// 32 columns of out each) have columns [m, m + 128) of `rows` rows from row n of matrix
// g; they share two buffers at `space`, which they take in turn, and barrier `id`. The
// loop is not unrolled: unrolled it is more code than the instruction caches hold, and
// took twice the time.
template <typename T, bool CLIPS>
__device__ __forceinline__ void store_tile(const ProductArgs& a, const CUtensorMap* map, bool tiles, uint32_t from,
                                           bool zero, int64_t m, int64_t n, int g, int rows, int quarter, int lane,
                                           uint8_t* space, uint32_t& turn, int id) {
  const bool issues = quarter == 0 && elect_one() != 0;
  const int boxes = m >= a.m ? 0 : a.m - m > 64 ? 2 : 1;
#pragma unroll 1
  for (int row0 = 0; row0 < rows; row0 += kStoreRows) {
    uint8_t* buf = space + (turn++ & 1) * kStoreBytes;
    uint32_t v[2][16];  // [half of the columns][8 rows, as fragments]
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (zero) {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[h][j] = 0;
      } else {
        tmem_ld_16x32(from + ((uint32_t)h << 20) + row0, v[h]);
      }
    }
    if (issues) tma_store_read<1>();  // the store before last has been read
    some_sync(id, 128);
    tmem_wait_ld();
    tmem_loaded(v[0]);
    tmem_loaded(v[1]);
    auto pair = [&](int h, int j) { return pair_of<T>(__uint_as_float(v[h][j]), __uint_as_float(v[h][j + 1])); };
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = k * 8 + lane % 8;
      store_turned4(smem_u32(buf) + quarter / 2 * (kStoreRows * 128) + r * 128 + (((quarter & 1) * 4 + lane / 8) ^ (r & 7)) * 16,
                    pair(0, k * 4), pair(0, k * 4 + 2), pair(1, k * 4), pair(1, k * 4 + 2));
    }
    fence_async_smem();
    some_sync(id, 128);
    const int left = rows - row0;
    if (tiles && (CLIPS || left >= kStoreRows)) {  // (CLIPS: rows behind these are behind the matrix's end, and dropped)
      if (issues)
        for (int c = 0; c < boxes; ++c)
          tma_store3(map, smem_u32(buf) + c * (kStoreRows * 128), (int)m + c * 64, (int)n + row0, g);
    } else {
      store_rows(a, buf, static_cast<uint16_t*>(a.out) + g * a.out_group + (n + row0) * a.out_row + m, m,
                 min(left, kStoreRows), quarter, lane, tiles);
    }
    if (issues) tma_store_commit();
  }
}

// fp32 sums go out from registers: the thread's column of `rows` rows from `out` on, a
// warp 128 bytes of a row.
__device__ __forceinline__ void store_sums(const ProductArgs& a, uint32_t (&acc)[8][16], float* out, int rows) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i * 16 >= rows) return;
    const int left = rows - i * 16;
    if (a.accumulate) {
      const float* old = out;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        if (j < left) acc[i][j] = __float_as_uint(__uint_as_float(acc[i][j]) + *old);
        old += a.out_row;
        asm volatile("" : "+l"(old));  // one address that moves on, not all at once
      }
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      if (j < left) *out = __uint_as_float(acc[i][j]);
      out += a.out_row;
      asm volatile("" : "+l"(out));
    }
  }
}

template <bool A_MN, bool B_MN, bool SCALED>
__global__ void __launch_bounds__(kThreadsHere, 1) __cluster_dims__(2, 1, 1)
    k_product(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
              const __grid_constant__ CUtensorMap map_out, const __grid_constant__ ProductArgs a, const __grid_constant__ ProductPlan p) {
  using F = Form<A_MN, B_MN, SCALED>;
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], sums_full[2], sums_empty[2],
      scales_full[kScaleSlots], scales_empty[kScaleSlots];
  __shared__ uint32_t tmem_slot, abort_word;
  // the swizzle is a function of address bits: tiles start on 1024 bytes, the same in both blocks
  uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  const uint32_t base = smem_u32(smem), stage_bytes = kABytes + p.b_bytes;
  uint8_t* scales = smem + p.scales_at;
  const Runs runs(smem + p.runs_at, a.groups);
  const int warp = warp_number(), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 2);   // both blocks' loads; rank 0's barrier counts
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sums_full[s], 1);
      mbar_init(&sums_empty[s], 2 * kEpilogue);
    }
    for (int s = 0; s < kScaleSlots; ++s) {
      mbar_init(&scales_full[s], 2);  // both blocks' scales; rank 0's barrier counts
      mbar_init(&scales_empty[s], 1);
    }
    abort_word = 0;
    mbar_init_fence();
    tma_prefetch(&map_a);
    tma_prefetch(&map_b);
    if (p.tiles_out) tma_prefetch(&map_out);
  }
  if (warp == 3) tmem_alloc_pair(&tmem_slot, 512);
  tc_fence_before();
  cluster_sync();  // while the kernel ahead ends: 0.2 us of every product
  tc_fence_after();
  griddep_wait();
  griddep_trigger();
  read_runs<F>(a, p, runs);
  const uint32_t tmem = tmem_slot;
  const PairWaiter wait{&abort_word, cluster_map(smem_u32(&abort_word), rank ^ 1), &g_product_error};
  Walk<F> walk(a, p, runs, static_cast<int>(blockIdx.x / 2));
  Tile t;

  if (warp == 0) {
    // ---- loads: each block its half of both operands
    const uint32_t one = elect_one();
    const uint32_t full0 = cluster_map(smem_u32(&full[0]), 0);
    Ring ring(p.stages);
    bool go = true;
    while (go && walk.next(t)) {
      const int half = t.padded / 2, m = t.m0 + rank * 128, n = t.n0 + rank * half;
      const int b_chunks = B_MN ? (half + 63) / 64 : 1;
      const uint32_t bytes = kABytes + (B_MN ? b_chunks * kMnChunk : p.b_bytes);
#pragma unroll 1
      for (int step = 0; step < t.steps; ++step) {
        const int s = ring.at;
        if (!(go = wait(&empty[s], ring.phase ^ 1))) break;
        const int k = t.k0 + step * F::kStepK;
        const uint32_t to = base + s * stage_bytes;
        if (one) {
          const uint32_t bar = full0 + s * 8;
          mbar_arrive_expect_tx_mapped(bar, bytes);
          // ragged K: `from` rows before the step's first, which read as zeros, so that
          // the stage ends with the run's last row
          const int from = F::kRaggedK ? min(0, t.rows_k - step * kMnRows - kMnRows) : 0;
          if (F::kRaggedK) {
            tma_load3_pair(to, &map_a, m, from, k, bar);
            tma_load3_pair(to + kMnChunk, &map_a, m + 64, from, k, bar);
          } else if (A_MN) {
            tma_load3_pair(to, &map_a, m, k, t.g, bar);
            tma_load3_pair(to + kMnChunk, &map_a, m + 64, k, t.g, bar);
          } else {
            tma_load3_pair(to, &map_a, k, m, t.g, bar);
          }
          if (B_MN) {
            for (int c = 0; c < b_chunks; ++c)
              tma_load3_pair(to + kABytes + c * kMnChunk, &map_b, n + c * 64, from, k, bar);
          } else {
            tma_load3_pair(to + kABytes, &map_b, k, n, 0, bar);
          }
        }
        __syncwarp();
        ring.step();
      }
    }
    if (go) {  // every stage has been read
      for (int s = 0; s < p.stages && go; ++s) {
        go = wait(&empty[ring.at], ring.phase ^ 1);
        ring.step();
      }
    }
    if (!go)  // leave the copies in flight time to land
      for (int i = 0; i < 64; ++i) __nanosleep(1000);
  } else if (warp == 1 && rank == 0) {
    // ---- the tensor cores of both blocks
    const uint32_t one = elect_one();
    const uint64_t a_desc = smem_desc(base, A_MN ? kMnChunk : 0, 1024);
    const uint64_t b_desc = smem_desc(base + kABytes, B_MN ? kMnChunk : 0, 1024);
    Ring ring(p.stages), slots(kScaleSlots), sums(2);
    uint32_t sa = 0;
    bool go = true;
    while (go && walk.next(t)) {
      const uint32_t idesc = SCALED ? 0 : mma_desc(a.dtype == kBF16, kTileM, t.padded, A_MN, B_MN);
      uint32_t d = 0;
#pragma unroll 1
      for (int step = 0; step < t.steps; ++step) {
        if ((step & (p.run - 1)) == 0) {
          if (!(go = wait(&sums_empty[sums.at], sums.phase ^ 1))) break;
          tc_fence_after();
          d = tmem + sums.at * F::kMaxN;
        }
        if (SCALED && step % kScaleSteps == 0) {
          if (!(go = wait.written(&scales_full[slots.at], slots.phase))) break;
          tc_fence_after();
          const uint32_t from = smem_u32(scales) + slots.at * kScaleSlot;
          sa = tmem + F::kScaleCols + (slots.at & 1) * 16;
          tmem_copy_scales_pair(sa, from, one);
          tmem_copy_scales_pair(sa + 4, from + 512, one);
          tmem_copy_scales_pair(sa + 8, from + 1024, one);
          mma_commit_pair(&scales_empty[slots.at], one);
          slots.step();
        }
        const int s = ring.at;
        if (!(go = wait(&full[s], ring.phase))) break;
        tc_fence_after();
        const uint32_t at = s * (stage_bytes / 16);  // in the descriptors' units of 16 bytes
        const bool more = (step & (p.run - 1)) != 0;
        if constexpr (SCALED) {
          const uint32_t scaled = mma_desc_scaled(kTileM, t.padded, step % kScaleSteps);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_scaled_pair(d, a_desc + at + k * 2, b_desc + at + k * 2, scaled, sa, sa + 4, more || k > 0, one);
        } else if constexpr (F::kRaggedK) {
          const int first = (kMnRows - min(kMnRows, t.rows_k - step * kMnRows)) / 16;  // 16s of zeros are left out
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k >= first) mma_ss_pair(d, a_desc + at + k * 128, b_desc + at + k * 128, idesc, more || k > first, one);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ss_pair(d, a_desc + at + k * (A_MN ? 128 : 2), b_desc + at + k * 2, idesc, more || k > 0, one);
        }
        mma_commit_pair(&empty[s], one);
        ring.step();
        if (((step + 1) & (p.run - 1)) == 0 || step + 1 == t.steps) {
          mma_commit_pair(&sums_full[sums.at], one);
          sums.step();
        }
      }
    }
    if (!go)  // leave the MMAs in flight time to end
      for (int i = 0; i < 64; ++i) __nanosleep(1000);
  } else if (SCALED && warp == 2) {
    // ---- scales: a word (four blocks of 128) of every row of the tile. Rank 0's MMAs learn
    // of either block's by fences of shared memory, which cost nothing that shows (8192 x
    // 2048 x 1024: 16.7 us; fences of all memory, in warps of their own, took 17.7).
    const uint32_t full0 = cluster_map(smem_u32(&scales_full[0]), 0);
    Ring slots(kScaleSlots);
    bool go = true;
    while (go && walk.next(t)) {
      const uint8_t* pa[4];
      const uint8_t* pb[8];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        pa[i] = a.a_scales + (t.g * a.m + min(t.m0 + (int64_t)rank * 128 + lane + i * 32, a.m - 1)) * a.scale_pitch;
#pragma unroll
      for (int i = 0; i < 8; ++i) pb[i] = a.b_scales + min((int64_t)t.n0 + lane + i * 32, a.n - 1) * a.scale_pitch;
      const int words = (t.steps + kScaleSteps - 1) / kScaleSteps;
      struct Words {
        uint4 a, b, c;
      } even, odd;  // two words are under way
      auto fetch = [&](int w, Words& v) {
        if (w >= words) return;
        auto word = [&](const uint8_t* q) { return *reinterpret_cast<const uint32_t*>(q + w * 4); };
        v.a = make_uint4(word(pa[0]), word(pa[1]), word(pa[2]), word(pa[3]));
        v.b = make_uint4(word(pb[0]), word(pb[1]), word(pb[2]), word(pb[3]));
        v.c = make_uint4(word(pb[4]), word(pb[5]), word(pb[6]), word(pb[7]));
      };
      auto put = [&](const Words& v) {
        if (!(go = wait(&scales_empty[slots.at], slots.phase ^ 1))) return;
        uint8_t* to = scales + slots.at * kScaleSlot + lane * 16;
        *reinterpret_cast<uint4*>(to) = v.a;
        *reinterpret_cast<uint4*>(to + 512) = v.b;
        *reinterpret_cast<uint4*>(to + 1024) = v.c;
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          fence_release_shared();
          mbar_arrive_mapped(full0 + slots.at * 8);
        }
        slots.step();
      };
      fetch(0, even);
      fetch(1, odd);
#pragma unroll 1
      for (int w = 0; w < words && go; w += 2) {
        put(even);
        fetch(w + 2, even);
        if (!go || w + 1 >= words) break;
        put(odd);
        fetch(w + 3, odd);
      }
    }
    if (go)
      for (int s = 0; s < kScaleSlots && go; ++s) {
        go = wait(&scales_empty[slots.at], slots.phase ^ 1);
        slots.step();
      }
  } else if (warp >= 4) {
    // ---- sums: four warps have the tile's columns of out (lanes of TMEM), each 32, in half of its rows
    const uint32_t empty0 = cluster_map(smem_u32(&sums_empty[0]), 0);
    const int part = (warp - 4) / 4, quarter = warp & 3;
    const uint32_t mine = tmem + ((uint32_t)quarter << 21);  // the warp's lanes
    const bool f32 = a.out_dtype == kF32;
    uint32_t turn = 0;
    Ring sums(2);
    bool go = true;
    while (walk.next(t)) {
      // the first four warps have the first half of the rows, in whole 32s
      const int first = part == 0 ? 0 : (t.padded / 2 + 31) / 32 * 32;
      const int half = part == 0 ? min((t.padded / 2 + 31) / 32 * 32, t.padded) : t.padded - first;
      uint32_t from = 0;
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_mapped(empty0 + sums.at * 8);
        sums.step();
      };
      // fp32 sums go to registers, and their TMEM is free at once; 16-bit results' only
      // where there are several runs, and back after the last. (Of 128 rows, whatever the tile's width.)
      uint32_t acc[8][16];
#pragma unroll 1
      for (int step = 0; step < t.steps; step += p.run) {
        if (!(go = wait(&sums_full[sums.at], sums.phase))) break;
        tc_fence_after();
        from = mine + sums.at * F::kMaxN + first;
        const bool end = step + p.run >= t.steps;
        if (step == 0 && end && !f32) break;
        if (step == 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) tmem_ld16(from + i * 16, acc[i]);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i) tmem_loaded(acc[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            uint32_t r[8];
            tmem_ld8(from + i * 8, r);
            tmem_wait_ld();
            tmem_loaded(r);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              uint32_t& to = acc[i / 2][i % 2 * 8 + j];
              to = __float_as_uint(__uint_as_float(to) + __uint_as_float(r[j]));
            }
          }
        }
        if (end && !f32) break;
        release();
      }
      // the four go on together or not at all
      if (!(go = some_sync_and(1 + part, 128, go))) break;
      if (!f32 && t.steps > p.run) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i * 16 < half) tmem_st16(from + i * 16, acc[i]);
        tmem_wait_st();
      }
      if (f32 && t.steps == 0) {
#pragma unroll
        for (int j = 0; j < 128; ++j) acc[j / 16][j % 16] = 0;
      }
      if (!(a.accumulate && t.steps == 0)) {
        const int64_t m = t.m0 + (int64_t)rank * 128, n = t.n0 + (int64_t)first;
        const int g = F::kRaggedK ? t.g : 0, rows = min(half, t.width - first);
        uint8_t* space = smem + p.store_at + part * (2 * kStoreBytes);
        const int64_t column = m + quarter * 32 + lane;
        if (f32) {
          if (column < a.m)
            store_sums(a, acc, static_cast<float*>(a.out) + g * a.out_group + n * a.out_row + column, rows);
        } else if (a.out_dtype == kF16)
          store_tile<__half, F::kRaggedK>(a, &map_out, p.tiles_out != 0, from, t.steps == 0, m, n, g, rows, quarter, lane,
                                          space, turn, 1 + part);
        else
          store_tile<__nv_bfloat16, F::kRaggedK>(a, &map_out, p.tiles_out != 0, from, t.steps == 0, m, n, g, rows, quarter,
                                                 lane, space, turn, 1 + part);
      }
      if (!f32 && t.steps > 0) release();
    }
    tma_store_written();
  }
  // No block leaves while the other may still reach its memory or arrive at its barriers.
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == 3) {
    tc_fence_after();
    tmem_free_pair(tmem, 512);
  }
}

// A pair whose block `giver` waits `limit` times on a barrier that nothing arrives at,
// the other block until it is told. ends[block]: 1 where the wait ran out, 2 where the
// other block's did (0: neither). Four warps go on together, as the sums' do.
__global__ void __launch_bounds__(128) __cluster_dims__(2, 1, 1) k_pair_that_gives_up(int giver, uint32_t limit, int32_t* ends) {
  __shared__ __align__(8) uint64_t bar;
  __shared__ uint32_t abort_word;
  __shared__ unsigned late;
  const int rank = static_cast<int>(cluster_rank());
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    mbar_init_fence();
    abort_word = 0;
    late = 0;
  }
  __syncthreads();
  cluster_sync();
  const PairWaiter wait{&abort_word, cluster_map(smem_u32(&abort_word), rank ^ 1), &late, rank == giver ? limit : kSpinLimit};
  bool go = true;
  if (threadIdx.x < 32) go = wait(&bar, 0);
  __syncwarp();
  go = some_sync_and(1, 128, go);
  if (threadIdx.x == 0) {
    ends[rank] = go ? 0 : late != 0 ? 1 : 2;
    if (late != 0) atomicAdd(&g_product_error, 1u);
  }
  __syncwarp();
  cluster_sync();
}

// out of no rows along K: zero.
__global__ void __launch_bounds__(256) k_product_zero(const ProductArgs a) {
  griddep_wait();
  griddep_trigger();
  const int64_t rows = a.n * a.groups;
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const int64_t at = r / a.n * a.out_group + r % a.n * a.out_row;
    for (int64_t m = threadIdx.x; m < a.m; m += 256) {
      if (a.out_dtype == kF32)
        static_cast<float*>(a.out)[at + m] = 0.0f;
      else
        static_cast<uint16_t*>(a.out)[at + m] = 0;
    }
  }
}

// The width of tiles with the least estimated time, in cycles: a step of 64 (e4m3: 128)
// along K takes 2 for each row of the tile, 200 at least and what its bytes need at 96
// a cycle; a tile's sums leave at 16 a row (fp32 30), and 3000 more lie around it. Wide
// tiles win but where they leave most of a round empty. 2048 x 2048 x 4096 in e4m3
// takes 25 us with tiles of 128, 27 with 224; 8192 x 2048 x 1024 27 and 23; 16384 x
// 2048 x 2048 in bf16 by 16 experts 99 us with tiles of 128, 83 with 256.
int choose_width(const ProductArgs& a, bool ragged_k, int step_k, int most, int pairs) {
  const double m_tiles = std::ceil(a.m / (double)kTileM), mean = (ragged_k ? a.k : a.n) / (double)a.groups;
  const double steps = std::ceil((ragged_k ? mean : (double)a.k) / step_k);
  const bool known = ragged_k || a.offsets == nullptr;  // how many tiles there are
  int best = most;
  double least = 1e300;
  for (int w = a.n <= 32 ? 32 : 64; w <= most; w += 32) {
    const double across = known ? std::ceil(a.n / (double)w) : std::max(1.0, mean / w + 0.5);
    const double tiles = m_tiles * across * (ragged_k || !known ? a.groups : 1);
    const double rounds = known ? std::ceil(tiles / pairs) : std::max(1.0, tiles / pairs + 0.5);
    const double width = std::min((double)w, std::ceil((known ? a.n / across : mean) / 32) * 32);
    const double step = std::max({2 * width, 200.0, (kABytes + 64.0 * w) / 96});
    const double time = rounds * (std::max(steps * step, (a.out_dtype == kF32 ? 30 : 16) * width) + 3000);
    if (time <= least) {
      least = time;
      best = w;
    }
    if (w >= a.n) break;
  }
  return best;
}

template <bool A_MN, bool B_MN, bool SCALED>
cudaError_t run(const ProductArgs& a, cudaStream_t s) {
  using F = Form<A_MN, B_MN, SCALED>;
  constexpr uint64_t elem = SCALED ? 1 : 2;
  auto kernel = k_product<A_MN, B_MN, SCALED>;
  static std::atomic<uint64_t> asked{0};
  cudaError_t e = allow_smem(kernel, kMostSmem, asked);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kThreadsHere);
  cfg.dynamicSmemBytes = kMostSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // As many pairs as run at once; asked once per kernel and device.
  constexpr int kDevices = 64;
  static std::atomic<int> found[kDevices];
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  int pairs = dev < kDevices ? found[dev].load(std::memory_order_relaxed) : 0;
  if (pairs == 0) {
    cfg.gridDim = dim3(2);
    if ((e = cudaOccupancyMaxActiveClusters(&pairs, kernel, &cfg)) != cudaSuccess) return e;
    if (pairs < 1) return cudaErrorLaunchOutOfResources;
    if (dev < kDevices) found[dev].store(pairs, std::memory_order_relaxed);
  }

  ProductPlan p{};
  p.run = a.out_dtype == kF32 ? kRunF32 : SCALED ? kRunScaledHalf : kRunHalf;
  const int width = choose_width(a, F::kRaggedK, F::kStepK, F::kMaxN, pairs);
  const int64_t across = (a.n + width - 1) / width;
  if (F::kRaggedK) {  // every expert's tiles are the same: as narrow as they can be
    p.tile_n = static_cast<int>((a.n + across - 1) / across + 31) / 32 * 32;
    p.b_bytes = (p.tile_n / 2 + 63) / 64 * kMnChunk;
  } else {
    p.tile_n = width;
    p.b_bytes = p.tile_n / 2 * kStepBytes;
  }
  const int stage = kABytes + p.b_bytes, behind = kStoreSpace + (SCALED ? kScaleSlots * kScaleSlot : 0) + Runs::bytes(a.groups);
  p.stages = min((kMostSmem - 1024 - behind) / stage, kMaxStages);
  p.store_at = p.stages * stage;
  p.scales_at = p.store_at + kStoreSpace;
  p.runs_at = p.scales_at + (SCALED ? kScaleSlots * kScaleSlot : 0);

  // a: along M and K (in either order) by group; b: its rows, all groups' together
  const uint64_t groups = F::kRaggedK ? 1 : a.groups, rows = a.k;
  const uint64_t a_extent[3] = {(uint64_t)(A_MN ? a.m : a.k), F::kRaggedK ? kMnRows : (uint64_t)(A_MN ? a.k : a.m),
                                F::kRaggedK ? rows : groups};
  const uint64_t a_strides[2] = {(uint64_t)a.a_row * elem, (uint64_t)(groups > 1 ? a.a_group : a.a_row) * elem};
  const uint64_t b_extent[3] = {(uint64_t)(B_MN ? a.n : a.k), F::kRaggedK ? kMnRows : (uint64_t)a.n, F::kRaggedK ? rows : 1};
  const uint64_t b_strides[2] = {(uint64_t)a.b_row * elem, (uint64_t)a.b_row * elem};
  const uint64_t out_groups = F::kRaggedK ? a.groups : 1;
  const uint64_t out_extent[3] = {(uint64_t)a.m, (uint64_t)a.n, out_groups};
  const uint64_t out_strides[2] = {(uint64_t)a.out_row * 2, (uint64_t)(out_groups > 1 ? a.out_group : a.out_row) * 2};
  p.tiles_out = a.out_dtype != kF32 && reinterpret_cast<uintptr_t>(a.out) % 16 == 0 && out_strides[0] % 16 == 0 &&
                out_strides[1] % 16 == 0;
  CUtensorMap map_a, map_b, map_out{};
  if (!make_tensor_map(&map_a, a.a, a.dtype, 3, a_extent, a_strides, A_MN ? kMnRows : 128) ||
      !make_tensor_map(&map_b, a.b, a.dtype, 3, b_extent, b_strides, B_MN ? kMnRows : p.tile_n / 2) ||
      (p.tiles_out && !make_tensor_map(&map_out, a.out, a.out_dtype, 3, out_extent, out_strides, kStoreRows)))
    return cudaErrorInvalidValue;

  const int64_t m_tiles = (a.m + kTileM - 1) / kTileM, n_tiles = (a.n + p.tile_n - 1) / p.tile_n;
  const int64_t most = m_tiles * (F::kRaggedK ? n_tiles * a.groups : n_tiles + a.groups + 2);
  if (most > (int64_t)0x7FFFFFFF || a.n > 0x7FFFFFFF || a.k > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  if (F::kRaggedK) {
    p.by_expert = Divide(static_cast<uint32_t>(m_tiles * n_tiles));
    p.by_band = Divide(static_cast<uint32_t>(8 * n_tiles));
  }
  p.pairs = static_cast<int>(most < pairs ? most : pairs);
  cfg.gridDim = dim3(2 * p.pairs);
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, map_a, map_b, map_out, a, p);
}

}  // namespace

ZG_ERROR_WORD(product_error, g_product_error)

cudaError_t launch_pair_that_gives_up(int giver, uint32_t limit, int32_t* ends, cudaStream_t s) {
  k_pair_that_gives_up<<<2, 128, 0, s>>>(giver, limit, ends);
  return cudaGetLastError();
}

cudaError_t launch_product(const ProductArgs& a, cudaStream_t s) {
  if (a.dtype == kE4M3) return run<false, false, true>(a, s);
  if (a.ragged_k && a.k == 0) {
    if (a.accumulate) return cudaSuccess;
    return launch_next(k_product_zero, dim3((unsigned)std::min<int64_t>(a.n * a.groups, 4096)), 256, 0, s, a);
  }
  if (a.ragged_k) return run<true, true, false>(a, s);
  return a.a_mn ? run<true, false, false>(a, s) : run<false, false, false>(a, s);
}

}  // namespace zg
