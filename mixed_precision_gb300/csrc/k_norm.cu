// RMSNorm with the residual's addition, forward and backward.
//
// forward:  s = RNE(x + residual); rstd = (mean(s^2) + eps)^(-1/2);
//           y = RNE(s * rstd * w); optionally y packed to 8 bits.
// backward: xhat = s * rstd, g = dy * w;
//           dx = RNE(dsum + rstd * (g - xhat * mean(g * xhat)));
//           dw[c] = sum over rows of dy * xhat.
//
// Both are bound by HBM: every tensor is read once and written once, a row
// stays in registers between its reduction and its output, in the tensors'
// own type (the stored sum is what is normalised, so nothing is lost). A row
// belongs to a team of threads (a power of two; lanes of one warp, or whole
// warps), each holding CH chunks of 8 neighbouring columns, so every access of
// a warp covers whole 128-byte lines, and all of a row's loads are issued
// before the first is used. dw: a thread keeps the same columns for all
// the rows of its block and sums them in registers; the blocks' sums go to
// the workspace and a second kernel adds them in a fixed order (no atomics).
//
// Measured at 16384 x 2048 in bf16: forward with a residual 44.6 us (6.0 TB/s),
// 55.0 us with the packed output (5.5 TB/s; the codes' instructions share the
// issue slots); backward with dsum 48.7 us (5.5 TB/s; the weight gradient's
// second kernel is 5 us of it). At 64 x 1024 forward takes 2.3 us, backward 5.0:
// two kernels' start and end.
#include <atomic>

#include "act.cuh"
#include "block.h"
#include "tc.cuh"
#include "vec.cuh"

namespace zg {
namespace {

__device__ unsigned g_norm_error;

constexpr int kNormThreads = 256;

constexpr int kMaxVecCols = 8192;  // 256 threads x 4 chunks x 8 columns
constexpr int64_t kStreamRows = 1024;  // backward: rows from which they go through shared memory

__device__ __forceinline__ float load_any(const void* p, int dtype, int64_t i) {
  if (dtype == kF32) return static_cast<const float*>(p)[i];
  if (dtype == kF16) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void store_any(void* p, int dtype, int64_t i, float v) {
  if (dtype == kF32)
    static_cast<float*>(p)[i] = v;
  else if (dtype == kF16)
    static_cast<__half*>(p)[i] = __float2half_rn(v);
  else
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// 8 weights from column c (c % 8 == 0, the buffer 16-byte aligned); read again
// for every row, so cached as ordinary loads.
__device__ __forceinline__ void load8_weight(const NormArgs& a, int c, float (&w)[8]) {
  if (a.weight_dtype == kF32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.weight) + c);
    const float4 u = p[0], v = p[1];
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    w[4] = v.x; w[5] = v.y; w[6] = v.z; w[7] = v.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.weight) + c);
    const bool half = a.weight_dtype == kF16;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t b = (j < 2 ? u.x : j < 4 ? u.y : j < 6 ? u.z : u.w) >> 16 * (j & 1) & 0xFFFFu;
      w[j] = half ? __half2float(__ushort_as_half(static_cast<unsigned short>(b)))
                  : __uint_as_float(b << 16);
    }
  }
}

// Sum over a team of `team` threads (a power of two). Teams wider than a warp
// are whole blocks; `smem` holds one float per warp and is reused after the
// second barrier.
__device__ __forceinline__ float team_sum(float v, int team, float* smem) {
  const int width = team < 32 ? team : 32;
  for (int o = width / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (team > 32) {
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) smem[warp] = v;
    __syncthreads();
    v = 0.0f;
    for (int w = 0; w < team / 32; ++w) v += smem[w];
    __syncthreads();
  }
  return v;
}

// RNE(x + r) of 8 elements.
template <typename T>
__device__ __forceinline__ Pack8<T> add8(const Pack8<T>& x, const Pack8<T>& r) {
  float u[8], v[8];
  widen8(x, u);
  widen8(r, v);
#pragma unroll
  for (int j = 0; j < 8; ++j) u[j] += v[j];
  return round8<T>(u);
}
template <typename T>
__device__ __forceinline__ float squares8(const Pack8<T>& x, float ss) {
  float u[8];
  widen8(x, u);
#pragma unroll
  for (int j = 0; j < 8; ++j) ss = fmaf(u[j], u[j], ss);
  return ss;
}

// The outputs of 8 columns of a row, from the stored sum. Whole warps call it:
// four lanes share a group of the packed row.
template <typename T>
__device__ __forceinline__ void write8(const NormArgs& a, int64_t row, int c, bool live, const Pack8<T>& s,
                                       float rstd) {
  Pack8<T> y{};
  if (c < a.cols) {
    float w[8], f[8];
    load8_weight(a, c, w);
    widen8(s, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = f[j] * rstd * w[j];
    y = round8<T>(f);
    if (live && a.y != nullptr) store8_raw(static_cast<T*>(a.y) + row * a.cols + c, y);
  }
  if (a.q != nullptr) {
    float f[8];
    widen8(y, f);
    const uint32_t byte = act_group_byte(f);
    if (live && c < a.pitch) {
      *reinterpret_cast<uint2*>(a.q + row * a.pitch + c) = act_codes8(f, act_inv_scale(byte));
      if ((threadIdx.x & 3) == 0) a.scales[row * (a.pitch / kActGroup) + c / kActGroup] = byte;
    }
  }
}

// The block's sum of its slots' dw, in slot order, to the workspace.
template <int CH>
__device__ __forceinline__ void sum_slots(const NormArgs& a, float* acc, const float (&dw)[CH][8], int slot, int slots,
                                          int lane, int team) {
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = (lane + k * team) * 8;
    if (c < a.cols) {
      float4* p = reinterpret_cast<float4*>(acc + (size_t)slot * a.cols + c);
      p[0] = make_float4(dw[k][0], dw[k][1], dw[k][2], dw[k][3]);
      p[1] = make_float4(dw[k][4], dw[k][5], dw[k][6], dw[k][7]);
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
    float t = 0.0f;
    for (int s = 0; s < slots; ++s) t += acc[(size_t)s * a.cols + c];
    a.part[(int64_t)blockIdx.x * a.cols + c] = t;
  }
}

// Whether any thread of a team of 32 n threads says yes; a barrier of the team.
__device__ __forceinline__ bool team_any(bool v, int team, int id) {
  if (team == 32) return __any_sync(0xFFFFFFFFu, v);
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "barrier.cta.red.or.pred p, %2, %3, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v)), "r"(id + 1), "r"(team)
      : "memory");
  return r != 0;
}

// Many rows. A team (whole warps of a block) walks over rows, three deep: bulk
// copies bring the rows ahead into shared memory while one is worked on, so
// the bytes in flight do not depend on registers. At most N tensors a row.
template <typename T, int N>
struct RowStream {
  static constexpr int kStages = 3;
  uint8_t* stages;   // this team's
  uint64_t* full;    // this team's kStages barriers
  float* red;        // this team's sums, one a warp
  const void* src[N];
  int64_t stride[N];
  uint32_t bytes;    // of a row
  int team, id, lane, n;
  int64_t row, rows, step;
  int s = 0;
  uint32_t parity = 0;

  __device__ __forceinline__ int stage_bytes() const { return static_cast<int>(bytes) * n; }
  // 8 elements of tensor i's row from column c, as one 16-byte load.
  __device__ __forceinline__ Pack8<T> at(int i, int c) const {
    const uint4 u = *reinterpret_cast<const uint4*>(stages + s * stage_bytes() + i * bytes + c * sizeof(T));
    Pack8<T> v;
    *reinterpret_cast<uint4*>(v.e) = u;
    return v;
  }
  __device__ __forceinline__ void fetch(int64_t r, int st) const {  // one thread
    mbar_arrive_expect_tx(&full[st], bytes * n);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n)
        bulk_g2s(stages + st * stage_bytes() + i * bytes, static_cast<const T*>(src[i]) + r * stride[i], bytes,
                 &full[st]);
  }
  // Called by all threads; the block synchronises after it.
  __device__ __forceinline__ void start() const {
    if (lane != 0) return;
    for (int i = 0; i < kStages; ++i) mbar_init(&full[i], 1);
    mbar_init_fence();
    for (int i = 0; i < kStages; ++i)
      if (row + i * step < rows) fetch(row + i * step, i);
  }
  // The next row is in its stage; false after the last, or when a wait gave up
  // (then the copies in flight are given time to land).
  __device__ __forceinline__ bool next() {
    if (row >= rows) return false;
    const bool late = !mbar_wait(&full[s], parity);
    if (!team_any(late, team, id)) return true;
    if (late) atomicAdd(&g_norm_error, 1u);
    for (int i = 0; i < kStages && row + i * step < rows; ++i)
      mbar_wait(&full[(s + i) % kStages], parity ^ (s + i >= kStages), kSpinLimit >> 10);
    return false;
  }
  // The team's sum; every thread has then done its reads before it.
  __device__ __forceinline__ float sum(float v) const {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (team > 32) {
      if ((lane & 31) == 0) red[lane / 32] = v;
      team_any(false, team, id);
      v = 0.0f;
      for (int w = 0; w < team / 32; ++w) v += red[w];
    }
    return v;
  }
  __device__ __forceinline__ void advance() {
    row += step;
    if (++s == kStages) s = 0, parity ^= 1;
  }
};

template <typename T, int CH>
__global__ void __launch_bounds__(256) k_norm_backward_rows(const NormArgs a, int team) {
  extern __shared__ __align__(16) uint8_t stages[];  // afterwards [teams][cols] floats
  constexpr int kStages = RowStream<T, 3>::kStages;
  __shared__ __align__(8) uint64_t full[4 * kStages];
  __shared__ float red[8];
  const int id = threadIdx.x / team, teams = blockDim.x / team, n = a.res != nullptr ? 3 : 2;
  const uint32_t bytes = a.cols * sizeof(T);
  RowStream<T, 3> in{stages + (size_t)id * kStages * n * bytes, full + id * kStages, red + id * (team / 32),
                     {a.x, a.dy, a.res}, {a.x_stride, a.dy_stride, a.r_stride}, bytes, team, id,
                     (int)threadIdx.x % team, n, (int64_t)blockIdx.x * teams + id, a.rows, (int64_t)gridDim.x * teams};
  in.start();
  float w[CH][8], dw[CH][8];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = (in.lane + k * team) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[k][j] = dw[k][j] = 0.0f;
    if (c < a.cols) load8_weight(a, c, w[k]);
  }
  const float inv_cols = 1.0f / static_cast<float>(a.cols);
  float rstd = in.row < a.rows ? a.rstd_in[in.row] : 0.0f;
  __syncthreads();
  for (; in.next(); in.advance()) {
    const float ahead = in.row + in.step < a.rows ? a.rstd_in[in.row + in.step] : 0.0f;
    float dot = 0.0f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (in.lane + k * team) * 8;
      if (c < a.cols) {
        float x[8], g[8];
        widen8(in.at(0, c), x);
        widen8(in.at(1, c), g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float xh = x[j] * rstd;
          dw[k][j] = fmaf(g[j], xh, dw[k][j]);
          dot = fmaf(g[j] * w[k][j], xh, dot);
        }
      }
    }
    dot = in.sum(dot) * inv_cols;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (in.lane + k * team) * 8;
      if (c < a.cols) {
        float x[8], g[8], d[8] = {};
        widen8(in.at(0, c), x);
        widen8(in.at(1, c), g);
        if (n == 3) widen8(in.at(2, c), d);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = fmaf(rstd, fmaf(-dot, x[j] * rstd, g[j] * w[k][j]), d[j]);
        store8(static_cast<T*>(a.dx) + in.row * a.cols + c, d);
      }
    }
    team_any(false, team, id);  // the stage has been read
    if (in.lane == 0 && in.row + kStages * in.step < a.rows) in.fetch(in.row + kStages * in.step, in.s);
    rstd = ahead;
  }
  griddep_trigger();
  __syncthreads();  // every team's copies have landed and been read
  sum_slots<CH>(a, reinterpret_cast<float*>(stages), dw, id, teams, in.lane, team);
}

// Rows as vectors. blockDim.x is a multiple of `team`, or equal to it when a
// team is wider than a warp.
template <typename T, int CH>
__global__ void __launch_bounds__(256) k_norm_forward(const NormArgs a, int team) {
  __shared__ float red[32];
  const int lane = threadIdx.x % team, slot = threadIdx.x / team, slots = blockDim.x / team;
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.res);
  // every team of a block makes the same number of rounds (shuffles and barriers)
  for (int64_t base = (int64_t)blockIdx.x * slots; base < a.rows; base += (int64_t)gridDim.x * slots) {
    const int64_t row = base + slot;
    const bool live = row < a.rows;
    Pack8<T> v[CH];
    float ss = 0.0f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (lane + k * team) * 8;
      v[k] = Pack8<T>{};
      if (live && c < a.cols) v[k] = load8_raw(x + row * a.x_stride + c);
    }
    if (res != nullptr) {
      Pack8<T> r[CH];
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int c = (lane + k * team) * 8;
        r[k] = Pack8<T>{};
        if (live && c < a.cols) r[k] = load8_raw(res + row * a.r_stride + c);
      }
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int c = (lane + k * team) * 8;
        v[k] = add8(v[k], r[k]);
        if (live && c < a.cols) store8_raw(static_cast<T*>(a.sum) + row * a.cols + c, v[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < CH; ++k) ss = squares8(v[k], ss);
    ss = team_sum(ss, team, red);
    const float rstd = 1.0f / sqrtf(ss / static_cast<float>(a.cols) + a.eps);
    if (live && lane == 0 && a.rstd != nullptr) a.rstd[row] = rstd;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (lane + k * team) * 8;
      write8(a, row, c, live, v[k], rstd);
    }
  }
}

// Any cols and strides: a block per row, element by element, the row read
// again for its output. Rows that are not whole vectors, or too wide for a
// team's registers, come here.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) k_norm_forward_any(const NormArgs a) {
  __shared__ float red[32];
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.res);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* src = x + row * a.x_stride;
    float ss = 0.0f;
    if (res != nullptr) {
      T* sum = static_cast<T*>(a.sum) + row * a.cols;
      for (int c = threadIdx.x; c < a.cols; c += kNormThreads) {
        const T s = DT<T>::from_f32(DT<T>::to_f32(src[c]) + DT<T>::to_f32(res[row * a.r_stride + c]));
        sum[c] = s;
        ss = fmaf(DT<T>::to_f32(s), DT<T>::to_f32(s), ss);
      }
      src = sum;
    } else {
      for (int c = threadIdx.x; c < a.cols; c += kNormThreads)
        ss = fmaf(DT<T>::to_f32(src[c]), DT<T>::to_f32(src[c]), ss);
    }
    ss = team_sum(ss, kNormThreads, red);  // its barriers also order the sum's writes and reads
    const float rstd = 1.0f / sqrtf(ss / static_cast<float>(a.cols) + a.eps);
    if (threadIdx.x == 0 && a.rstd != nullptr) a.rstd[row] = rstd;
    // whole rounds of 32 columns, so that a warp holds one group of the packed row
    const int end = a.q != nullptr ? a.pitch : (a.cols + 31) / 32 * 32;
    for (int c = threadIdx.x; c < end; c += kNormThreads) {
      T y = DT<T>::from_f32(0.0f);
      if (c < a.cols) {
        y = DT<T>::from_f32(DT<T>::to_f32(src[c]) * rstd * load_any(a.weight, a.weight_dtype, c));
        if (a.y != nullptr) static_cast<T*>(a.y)[row * a.cols + c] = y;
      }
      if (a.q != nullptr) {
        const uint32_t byte = act_scale_byte(
            __reduce_max_sync(0xFFFFFFFFu, abs_bits(DT<T>::to_f32(y))));
        const float one[8] = {DT<T>::to_f32(y)};
        a.q[row * a.pitch + c] = static_cast<int8_t>(act_codes8(one, act_inv_scale(byte)).x & 0xFFu);
        if ((threadIdx.x & 31) == 0) a.scales[row * (a.pitch / kActGroup) + c / kActGroup] = byte;
      }
    }
    __syncthreads();  // y may be x's or the residual's buffer: the next row's reads come after
  }
}

template <typename T, int CH>
__global__ void __launch_bounds__(256) k_norm_backward(const NormArgs a, int team) {
  extern __shared__ float acc_smem[];  // [slots][cols], after the rows
  __shared__ float red[32];
  const int lane = threadIdx.x % team, slot = threadIdx.x / team, slots = blockDim.x / team;
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  const T* dsum = static_cast<const T*>(a.res);
  float w[CH][8], dw[CH][8];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = (lane + k * team) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[k][j] = dw[k][j] = 0.0f;
    if (c < a.cols) load8_weight(a, c, w[k]);
  }
  const float inv_cols = 1.0f / static_cast<float>(a.cols);
  struct Row {
    Pack8<T> x[CH], g[CH], d[CH];
    float rstd;
  };
  auto load = [&](int64_t row, Row& r) {
    r.rstd = row < a.rows ? a.rstd_in[row] : 0.0f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (lane + k * team) * 8;
      r.x[k] = r.g[k] = r.d[k] = Pack8<T>{};
      if (row < a.rows && c < a.cols) {
        r.x[k] = load8_raw(x + row * a.x_stride + c);
        r.g[k] = load8_raw(dy + row * a.dy_stride + c);
        if (dsum != nullptr) r.d[k] = load8_raw(dsum + row * a.r_stride + c);
      }
    }
  };
  // With a chunk a thread the next row's loads are issued before this row's
  // sums; with more they would not fit beside them.
  constexpr bool kAhead = CH == 1;
  const int64_t step = (int64_t)gridDim.x * slots;
  Row now, ahead;
  if (kAhead) load((int64_t)blockIdx.x * slots + slot, ahead);
  for (int64_t base = (int64_t)blockIdx.x * slots; base < a.rows; base += step) {
    const int64_t row = base + slot;
    const bool live = row < a.rows;
    if (kAhead) {
      now = ahead;
      load(row + step, ahead);
    } else {
      load(row, now);
    }
    const float rstd = now.rstd;
    float dot = 0.0f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      float xf[8], g[8];
      widen8(now.x[k], xf);
      widen8(now.g[k], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xh = xf[j] * rstd;
        dw[k][j] = fmaf(g[j], xh, dw[k][j]);
        dot = fmaf(g[j] * w[k][j], xh, dot);
      }
    }
    dot = team_sum(dot, team, red) * inv_cols;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (lane + k * team) * 8;
      if (live && c < a.cols) {
        float xf[8], g[8], d[8];
        widen8(now.x[k], xf);
        widen8(now.g[k], g);
        widen8(now.d[k], d);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = fmaf(rstd, fmaf(-dot, xf[j] * rstd, g[j] * w[k][j]), d[j]);
        store8(static_cast<T*>(a.dx) + row * a.cols + c, d);
      }
    }
  }
  griddep_trigger();
  sum_slots<CH>(a, acc_smem, dw, slot, slots, lane, team);
}

// dx of any cols and strides.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) k_norm_backward_any(const NormArgs a) {
  __shared__ float red[32];
  const T* dsum = static_cast<const T*>(a.res);
  const float inv_cols = 1.0f / static_cast<float>(a.cols);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* dy = static_cast<const T*>(a.dy) + row * a.dy_stride;
    const float rstd = a.rstd_in[row];
    float dot = 0.0f;
    for (int c = threadIdx.x; c < a.cols; c += kNormThreads)
      dot = fmaf(DT<T>::to_f32(dy[c]) * load_any(a.weight, a.weight_dtype, c),
                 DT<T>::to_f32(x[c]) * rstd, dot);
    dot = team_sum(dot, kNormThreads, red) * inv_cols;
    for (int c = threadIdx.x; c < a.cols; c += kNormThreads) {
      const float g = DT<T>::to_f32(dy[c]) * load_any(a.weight, a.weight_dtype, c);
      const float d = dsum != nullptr ? DT<T>::to_f32(dsum[row * a.r_stride + c]) : 0.0f;
      static_cast<T*>(a.dx)[row * a.cols + c] =
          DT<T>::from_f32(fmaf(rstd, fmaf(-dot, DT<T>::to_f32(x[c]) * rstd, g), d));
    }
  }
}

// dw partials of any cols and strides: a block takes 32 columns and every
// gridDim.y-th run of 8 rows. Runs before k_norm_backward_any, which may
// overwrite dy.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) k_norm_dweight_any(const NormArgs a) {
  __shared__ float acc[8][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), r0 = threadIdx.x >> 5;
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  float t = 0.0f;
  if (c < a.cols)
    for (int64_t row = blockIdx.y * 8ll + r0; row < a.rows; row += gridDim.y * 8ll)
      t = fmaf(DT<T>::to_f32(dy[row * a.dy_stride + c]),
               DT<T>::to_f32(x[row * a.x_stride + c]) * a.rstd_in[row], t);
  acc[r0][threadIdx.x & 31] = t;
  __syncthreads();
  if (r0 == 0 && c < a.cols) {
    for (int s = 1; s < 8; ++s) t += acc[s][threadIdx.x & 31];
    a.part[(int64_t)blockIdx.y * a.cols + c] = t;
  }
}

// dw[c] = the parts' sums in a fixed order: 32 columns x 32 runs of parts.
__global__ void __launch_bounds__(1024) k_norm_dweight_sum(const NormArgs a, int parts) {
  __shared__ float acc[32][33];
  griddep_wait();
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float t = 0.0f;
  if (c < a.cols) {
    // eight loads in flight: the parts come from L2, one at a time they would
    // cost its latency each
    int p = run;
    for (; p + 7 * 32 < parts; p += 8 * 32) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = a.part[(int64_t)(p + j * 32) * a.cols + c];
#pragma unroll
      for (int j = 0; j < 8; ++j) t += v[j];
    }
    float v[7];
#pragma unroll
    for (int j = 0; j < 7; ++j) v[j] = p + j * 32 < parts ? a.part[(int64_t)(p + j * 32) * a.cols + c] : 0.0f;
#pragma unroll
    for (int j = 0; j < 7; ++j) t += v[j];
  }
  acc[run][lane] = t;
  __syncthreads();
  if (run == 0 && c < a.cols) {
    for (int s = 1; s < 32; ++s) t += acc[s][lane];
    store_any(a.dweight, a.dweight_dtype, c, t);
  }
}

int pow2_at_least(int n) {
  int p = 1;
  while (p < n) p *= 2;
  return p;
}

// How a call's rows are worked on. stream: through shared memory (k_norm_*_rows);
// else straight from global memory.
struct Shape {
  bool stream;
  int team, threads, chunks, grid, smem;
};

// Rows of n chunks of 8 columns. A team's threads take up to 4 chunks each, so
// that few rows' sums go between warps and many loads are in flight. Where the
// rows are too few to fill the machine (152 SMs of 512 threads) a row is spread
// over more threads instead: at 64 rows of 1024 a chunk a thread takes 2.2 us,
// 4 chunks 4.2 us.
Shape direct_shape(int64_t rows, int n) {
  Shape s{};
  s.chunks = 1;
  while (s.chunks < 4 && n > 32 * s.chunks) s.chunks *= 2;
  while (s.chunks > 1 && rows * (pow2_at_least(n) / s.chunks) < 152 * 512 && pow2_at_least(n) / s.chunks < 256)
    s.chunks /= 2;  // a team is 256 threads at most
  const int team = pow2_at_least((n + s.chunks - 1) / s.chunks);
  s.team = team < 4 ? 4 : team;  // the packed output's groups are 4 neighbouring lanes
  s.threads = s.team > 32 ? s.team : 128;
  return s;
}

constexpr int kSmemPerSm = 220 * 1024;

// All of a block's shapes depend on sizes alone (152 SMs, a constant), so the
// backward's workspace and the order of its sums are the same everywhere.
// `tensors`: that a row reads.
//
// Backward keeps the weights and dw in registers, which leaves too few for the
// loads in flight: many rows of 16-bit types go through shared memory. us,
// direct against through shared memory, bf16 with dsum:
//   16384 x 1024   33.1, 28.7     4096 x 8192   74.6, 56.8    1024 x 1024   7.7, 6.9
//   16384 x 2048   69.0, 49.1     1024 x 4096   19.7, 15.2     512 x 4096   9.6, 13.0
// Short rows do better directly than with a bulk copy a row and tensor (65536 x
// 256: 27.6, 31.8; x 128: 16.4, 31.0; several rows a copy were not tried),
// and so does fp32, whose loads are twice as long (16384 x 1024: 47 us,
// 5.7 TB/s). Forward has the registers: through shared memory it took 48 us
// where it takes 23 (16384 x 1024).
Shape norm_shape(int64_t rows, int n, int elem_bytes, int tensors, bool backward) {
  Shape s = direct_shape(rows, n);
  const int stage = n * 8 * elem_bytes * tensors;
  // what the registers allow
  const int fit_threads = !backward ? 2048 : s.chunks > 1 ? 512 : elem_bytes == 2 ? 1024 : 768;
  // Backward with short rows that fill the machine: larger blocks leave fewer
  // parts of dw to add up. 128 threads against 256, bf16 with dsum: 65536 x 256
  // 28.6, 27.6 us; 65536 x 64 9.8, 8.8.
  if (backward && s.team <= 32 && rows >= 152ll * fit_threads / s.team) s.threads = 256;
  int per_sm = fit_threads / s.threads;
  if (backward) s.smem = s.threads / s.team * n * 32;
  if (backward && n > 32 && rows >= kStreamRows && elem_bytes == 2) {
    s.stream = true;
    s.chunks = n <= 64 ? 2 : 4;
    s.team = n <= 128 ? 32 : pow2_at_least(n) / 4;
    s.threads = s.team > 128 ? s.team : 128;
    const int ring = s.threads / s.team * RowStream<__half, 3>::kStages * stage, sums = s.threads / s.team * n * 32;
    s.smem = ring > sums ? ring : sums;
    const int fit = kSmemPerSm / s.smem, most = 512 / s.threads;
    per_sm = fit < most ? fit : most;
  }
  const int slots = s.threads / s.team;
  const int64_t want = (rows + slots - 1) / slots, most = 152ll * per_sm;
  s.grid = static_cast<int>(want < most ? want : most);
  return s;
}

bool vec_cols(int cols) { return cols % 8 == 0 && cols <= kMaxVecCols; }
bool norm_vec(const NormArgs& a) {
  return vec_cols(a.cols) && a.x_stride % 8 == 0 && a.r_stride % 8 == 0 && a.dy_stride % 8 == 0;
}

template <typename T, int CH>
cudaError_t forward_launch(const NormArgs& a, const Shape& sh, cudaStream_t s) {
  k_norm_forward<T, CH><<<sh.grid, sh.threads, 0, s>>>(a, sh.team);
  return cudaGetLastError();
}

template <typename T>
cudaError_t forward_t(const NormArgs& a, int sms, cudaStream_t s) {
  if (!norm_vec(a)) {
    const int64_t most = sms * 8ll;
    k_norm_forward_any<T><<<(int)(a.rows < most ? a.rows : most), kNormThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  const Shape sh = norm_shape(a.rows, (a.q != nullptr ? a.pitch : a.cols) / 8, (int)sizeof(T),
                              a.res != nullptr ? 2 : 1, false);
  switch (sh.chunks) {
    case 1: return forward_launch<T, 1>(a, sh, s);
    case 2: return forward_launch<T, 2>(a, sh, s);
    default: return forward_launch<T, 4>(a, sh, s);
  }
}

template <typename T, int CH>
cudaError_t backward_launch(const NormArgs& a, const Shape& sh, cudaStream_t s) {
  static std::atomic<uint64_t> asked{0}, asked_rows{0};
  if (!sh.stream) {
    cudaError_t e = allow_smem(k_norm_backward<T, CH>, kSmemPerSm, asked);
    if (e != cudaSuccess) return e;
    k_norm_backward<T, CH><<<sh.grid, sh.threads, sh.smem, s>>>(a, sh.team);
    return cudaGetLastError();
  }
  if constexpr (CH > 1 && sizeof(T) == 2) {
    cudaError_t e = allow_smem(k_norm_backward_rows<T, CH>, kSmemPerSm, asked_rows);
    if (e != cudaSuccess) return e;
    k_norm_backward_rows<T, CH><<<sh.grid, sh.threads, sh.smem, s>>>(a, sh.team);
  }
  return cudaGetLastError();
}

constexpr int kAnyParts = 64;

template <typename T>
cudaError_t backward_t(const NormArgs& a, int sms, cudaStream_t s) {
  int parts;
  cudaError_t e;
  if (norm_vec(a)) {
    const Shape sh = norm_shape(a.rows, a.cols / 8, (int)sizeof(T), a.res != nullptr ? 3 : 2, true);
    parts = sh.grid;
    switch (sh.chunks) {
      case 1: e = backward_launch<T, 1>(a, sh, s); break;
      case 2: e = backward_launch<T, 2>(a, sh, s); break;
      default: e = backward_launch<T, 4>(a, sh, s); break;
    }
  } else {
    parts = (int)((a.rows + 7) / 8 < kAnyParts ? (a.rows + 7) / 8 : kAnyParts);
    k_norm_dweight_any<T><<<dim3((a.cols + 31) / 32, parts), kNormThreads, 0, s>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t most = sms * 8ll;
    k_norm_backward_any<T><<<(int)(a.rows < most ? a.rows : most), kNormThreads, 0, s>>>(a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  // launched while the rows' kernel ends; it waits for it before its first read
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((a.cols + 31) / 32);
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_norm_dweight_sum, a, parts);
}

}  // namespace

ZG_ERROR_WORD(norm_error, g_norm_error)

int norm_backward_parts(int64_t rows, int cols) {
  int parts = (int)((rows + 7) / 8 < kAnyParts ? (rows + 7) / 8 : kAnyParts);
  if (!vec_cols(cols)) return parts;
  // whichever type, strides and tensors the call has
  for (int size : {2, 4})
    for (int tensors : {2, 3}) {
      const int grid = norm_shape(rows, cols / 8, size, tensors, true).grid;
      parts = grid > parts ? grid : parts;
    }
  return parts;
}

cudaError_t launch_norm_forward(const NormArgs& a, int sms, cudaStream_t s) {
  switch (a.dtype) {
    case kF32: return forward_t<float>(a, sms, s);
    case kF16: return forward_t<__half>(a, sms, s);
    default: return forward_t<__nv_bfloat16>(a, sms, s);
  }
}

cudaError_t launch_norm_backward(const NormArgs& a, int sms, cudaStream_t s) {
  if (a.rows == 0) {
    return cudaMemsetAsync(a.dweight, 0, (size_t)a.cols * (a.dweight_dtype == kF32 ? 4 : 2), s);
  }
  switch (a.dtype) {
    case kF32: return backward_t<float>(a, sms, s);
    case kF16: return backward_t<__half>(a, sms, s);
    default: return backward_t<__nv_bfloat16>(a, sms, s);
  }
}

}  // namespace zg
