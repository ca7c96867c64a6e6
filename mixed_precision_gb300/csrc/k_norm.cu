// RMSNorm with the residual's addition, forward and backward.
//
// forward:  s = RNE(x + residual); rstd = (mean(s^2) + eps)^(-1/2);
//           y = RNE(s * rstd * w); optionally y packed to 8 bits.
// backward: xhat = s * rstd, g = dy * w;
//           dx = RNE(dsum + rstd * (g - xhat * mean(g * xhat)));
//           dw[c] = sum over rows of dy * xhat.
//
// Both are bound by HBM: every tensor is read once and written once, a row
// stays in registers between its reduction and its output. A row belongs to
// a team of threads (a power of two; lanes of one warp, or whole warps), each
// holding CH chunks of 8 neighbouring columns, so every access of a warp
// covers whole 128-byte lines. dw: a thread keeps the same columns for all
// the rows of its block and sums them in registers; the blocks' sums go to
// the workspace and a second kernel adds them in a fixed order (no atomics).
#include "act.cuh"
#include "block.h"
#include "vec.cuh"

namespace zg {
namespace {

constexpr int kNormThreads = 256;
constexpr int kMaxVecCols = 16384;  // 512 threads x 4 chunks x 8 columns

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

// Rows as vectors. blockDim.x is a multiple of `team`, or equal to it when a
// team is wider than a warp.
template <typename T, int CH>
__global__ void __launch_bounds__(512) k_norm_forward(const NormArgs a, int team) {
  __shared__ float red[32];
  const int lane = threadIdx.x % team, slot = threadIdx.x / team, slots = blockDim.x / team;
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.res);
  // every team of a block makes the same number of rounds (shuffles and barriers)
  for (int64_t base = (int64_t)blockIdx.x * slots; base < a.rows; base += (int64_t)gridDim.x * slots) {
    const int64_t row = base + slot;
    const bool live = row < a.rows;
    float v[CH][8];
    float ss = 0.0f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (lane + k * team) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] = 0.0f;
      if (live && c < a.cols) load8(x + row * a.x_stride + c, v[k]);
    }
    if (res != nullptr) {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int c = (lane + k * team) * 8;
        if (live && c < a.cols) {
          float r[8];
          load8(res + row * a.r_stride + c, r);
          Pack8<T> s;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            s.e[j] = DT<T>::from_f32(v[k][j] + r[j]);
            v[k][j] = DT<T>::to_f32(s.e[j]);
          }
          store8_raw(static_cast<T*>(a.sum) + row * a.cols + c, s);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(v[k][j], v[k][j], ss);
    ss = team_sum(ss, team, red);
    const float rstd = 1.0f / sqrtf(ss / static_cast<float>(a.cols) + a.eps);
    if (live && lane == 0 && a.rstd != nullptr) a.rstd[row] = rstd;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (lane + k * team) * 8;
      const bool in = live && c < a.cols;
      Pack8<T> y;
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = 0.0f;
      if (in) {
        float w[8];
        load8_weight(a, c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          y.e[j] = DT<T>::from_f32(v[k][j] * rstd * w[j]);
          f[j] = DT<T>::to_f32(y.e[j]);
        }
        if (a.y != nullptr) store8_raw(static_cast<T*>(a.y) + row * a.cols + c, y);
      }
      if (a.q != nullptr) {
        const uint32_t byte = act_group_byte(f);
        if (live && c < a.pitch) {
          *reinterpret_cast<uint2*>(a.q + row * a.pitch + c) = act_codes8(f, act_inv_scale(byte));
          if ((threadIdx.x & 3) == 0)
            a.scales[row * (a.pitch / kActGroup) + c / kActGroup] = byte;
        }
      }
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
        a.q[row * a.pitch + c] = static_cast<int8_t>(act_code(DT<T>::to_f32(y), act_inv_scale(byte)));
        if ((threadIdx.x & 31) == 0) a.scales[row * (a.pitch / kActGroup) + c / kActGroup] = byte;
      }
    }
    __syncthreads();  // y may be x's or the residual's buffer: the next row's reads come after
  }
}

template <typename T, int CH>
__global__ void __launch_bounds__(512) k_norm_backward(const NormArgs a, int team) {
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
  for (int64_t base = (int64_t)blockIdx.x * slots; base < a.rows; base += (int64_t)gridDim.x * slots) {
    const int64_t row = base + slot;
    const bool live = row < a.rows;
    const float rstd = live ? a.rstd_in[row] : 0.0f;
    float xh[CH][8], g[CH][8];
    float dot = 0.0f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (lane + k * team) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) xh[k][j] = g[k][j] = 0.0f;
      if (live && c < a.cols) {
        load8(x + row * a.x_stride + c, xh[k]);
        load8(dy + row * a.dy_stride + c, g[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xh[k][j] *= rstd;
        dw[k][j] = fmaf(g[k][j], xh[k][j], dw[k][j]);
        g[k][j] *= w[k][j];
        dot = fmaf(g[k][j], xh[k][j], dot);
      }
    dot = team_sum(dot, team, red) * inv_cols;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (lane + k * team) * 8;
      if (live && c < a.cols) {
        float d[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = 0.0f;
        if (dsum != nullptr) load8(dsum + row * a.r_stride + c, d);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = fmaf(rstd, fmaf(-dot, xh[k][j], g[k][j]), d[j]);
        store8(static_cast<T*>(a.dx) + row * a.cols + c, d);
      }
    }
  }
  // the block's sum over its slots, in slot order
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = (lane + k * team) * 8;
    if (c < a.cols)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc_smem[slot * a.cols + c + j] = dw[k][j];
  }
  __syncthreads();
  for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
    float t = 0.0f;
    for (int s = 0; s < slots; ++s) t += acc_smem[s * a.cols + c];
    a.part[(int64_t)blockIdx.x * a.cols + c] = t;
  }
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
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float t = 0.0f;
  if (c < a.cols)
    for (int p = run; p < parts; p += 32) t += a.part[(int64_t)p * a.cols + c];
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

struct Shape {
  int team, threads, chunks;
};

// The team for a row of n chunks of 8 columns: up to 4 chunks a thread, at
// least 4 threads (the packed output's groups are 4 neighbouring lanes).
Shape norm_shape(int n) {
  Shape s;
  s.chunks = n <= 32 ? 1 : n <= 64 ? 2 : 4;
  const int team = pow2_at_least((n + s.chunks - 1) / s.chunks);
  s.team = team < 4 ? 4 : team;
  s.threads = s.team > kNormThreads ? s.team : kNormThreads;
  if (s.team > 32) s.threads = s.team;  // wider than a warp: one team a block
  return s;
}

bool norm_vec(const NormArgs& a) {
  return a.cols % 8 == 0 && a.cols <= kMaxVecCols - kActPitch && a.x_stride % 8 == 0 &&
         a.r_stride % 8 == 0 && a.dy_stride % 8 == 0;
}

// Blocks of a row kernel. 152 SMs' worth, a constant: the backward's workspace
// and the order of its sums are the same wherever they are asked for.
int norm_grid(int64_t rows, const Shape& s) {
  const int slots = s.threads / s.team;
  const int64_t want = (rows + slots - 1) / slots;
  const int64_t most = 152ll * (2048 / s.threads);
  return static_cast<int>(want < most ? want : most);
}

template <typename T>
cudaError_t forward_t(const NormArgs& a, int sms, cudaStream_t s) {
  if (!norm_vec(a)) {
    const int64_t most = sms * 8ll;
    k_norm_forward_any<T><<<(int)(a.rows < most ? a.rows : most), kNormThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  const Shape sh = norm_shape((a.q != nullptr ? a.pitch : a.cols) / 8);
  const int grid = norm_grid(a.rows, sh);
  switch (sh.chunks) {
    case 1: k_norm_forward<T, 1><<<grid, sh.threads, 0, s>>>(a, sh.team); break;
    case 2: k_norm_forward<T, 2><<<grid, sh.threads, 0, s>>>(a, sh.team); break;
    default: k_norm_forward<T, 4><<<grid, sh.threads, 0, s>>>(a, sh.team); break;
  }
  return cudaGetLastError();
}

template <typename T, int CH>
cudaError_t backward_launch(const NormArgs& a, const Shape& sh, int grid, cudaStream_t s) {
  const int smem = sh.threads / sh.team * a.cols * 4;
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(k_norm_backward<T, CH>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  k_norm_backward<T, CH><<<grid, sh.threads, smem, s>>>(a, sh.team);
  return cudaGetLastError();
}

constexpr int kAnyParts = 64;

template <typename T>
cudaError_t backward_t(const NormArgs& a, int sms, cudaStream_t s) {
  int parts;
  cudaError_t e;
  if (norm_vec(a)) {
    const Shape sh = norm_shape(a.cols / 8);
    const int grid = parts = norm_grid(a.rows, sh);
    switch (sh.chunks) {
      case 1: e = backward_launch<T, 1>(a, sh, grid, s); break;
      case 2: e = backward_launch<T, 2>(a, sh, grid, s); break;
      default: e = backward_launch<T, 4>(a, sh, grid, s); break;
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
  k_norm_dweight_sum<<<(a.cols + 31) / 32, 1024, 0, s>>>(a, parts);
  return cudaGetLastError();
}

}  // namespace

int norm_backward_parts(int64_t rows, int cols) {
  int parts = (int)((rows + 7) / 8 < kAnyParts ? (rows + 7) / 8 : kAnyParts);
  if (cols % 8 == 0 && cols <= kMaxVecCols - kActPitch) {
    const int grid = norm_grid(rows, norm_shape(cols / 8));
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
