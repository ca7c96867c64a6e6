// Weight gradient from a packed activation: dw = dy^T X, X restored in dy's
// type. Plain tiled form: 64 x 64 outputs a block, fp32 sums over the tokens.
#include "act.cuh"
#include "block.h"
#include "vec.cuh"

namespace zg {
namespace {

constexpr int kTile = 64, kDepth = 16;

template <typename T>
__global__ void __launch_bounds__(256) k_wgrad(const WgradArgs a) {
  __shared__ float sa[kDepth][kTile + 4], sb[kDepth][kTile + 4];
  const int64_t m0 = (int64_t)blockIdx.y * kTile;
  const int n0 = blockIdx.x * kTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const T* dy = static_cast<const T*>(a.dy);
  float acc[4][4] = {};
  for (int64_t t0 = 0; t0 < a.tokens; t0 += kDepth) {
    for (int i = threadIdx.x; i < kDepth * kTile; i += 256) {
      const int r = i / kTile, c = i % kTile;
      const int64_t t = t0 + r;
      const bool live = t < a.tokens;
      sa[r][c] = live && m0 + c < a.n_out ? DT<T>::to_f32(dy[t * a.dy_stride + m0 + c]) : 0.0f;
      float x = 0.0f;
      if (live && n0 + c < a.n_in)
        x = static_cast<float>(a.q[t * a.pitch + n0 + c]) *
            act_scale(a.scales[t * (a.pitch / kActGroup) + (n0 + c) / kActGroup]);
      sb[r][c] = DT<T>::to_f32(DT<T>::from_f32(x));
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kDepth; ++r) {
      float u[4], v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = sa[r][ty * 4 + i], v[i] = sb[r][tx * 4 + i];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(u[i], v[j], acc[i][j]);
    }
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty * 4 + i;
      const int n = n0 + tx * 4 + j;
      if (m >= a.n_out || n >= a.n_in) continue;
      const int64_t at = m * a.n_in + n;
      if (a.dw_dtype == kF32) {
        float* dw = static_cast<float*>(a.dw);
        dw[at] = a.accumulate ? dw[at] + acc[i][j] : acc[i][j];
      } else {
        static_cast<T*>(a.dw)[at] = DT<T>::from_f32(acc[i][j]);
      }
    }
}

}  // namespace

// No kernel of the block operators waits on anything yet.
cudaError_t block_error_read_clear(unsigned* value, cudaStream_t s) {
  *value = 0;
  return cudaStreamSynchronize(s);
}

cudaError_t launch_wgrad(const WgradArgs& a, int sms, cudaStream_t s) {
  (void)sms;
  const dim3 grid((a.n_in + kTile - 1) / kTile, (unsigned)((a.n_out + kTile - 1) / kTile));
  if (a.dtype == kF16)
    k_wgrad<__half><<<grid, 256, 0, s>>>(a);
  else
    k_wgrad<__nv_bfloat16><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace zg
