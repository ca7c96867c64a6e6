// The experts' products and the products of scaled e4m3 matrices: one thread an
// output element, fp32 sums.
#include <cuda_fp8.h>

#include "block.h"
#include "experts.h"
#include "vec.cuh"

namespace zg {
namespace {

__device__ unsigned g_product_error;

struct E4M3 {
  uint8_t bits;
};

template <typename T>
__device__ __forceinline__ float value(const ProductArgs&, const void* p, const uint8_t*, int64_t, int64_t, int64_t at) {
  return DT<T>::to_f32(static_cast<const T*>(p)[at]);
}
template <>
__device__ __forceinline__ float value<E4M3>(const ProductArgs& a, const void* p, const uint8_t* scales, int64_t row,
                                             int64_t k, int64_t at) {
  const uint32_t byte = scales[row * a.scale_pitch + k / kScaledBlock];
  const float s = __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7FC00000u : byte << 23);
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(p)[at], __NV_E4M3))) * s;
}

__device__ __forceinline__ int64_t bound(const ProductArgs& a, int g, int64_t rows) {
  if (a.offsets == nullptr) return g == 0 ? 0 : rows;
  const int64_t o = a.offsets[g];
  return o < 0 ? 0 : o < rows ? o : rows;
}

template <typename T, typename Out>
__global__ void __launch_bounds__(256) k_product_plain(const ProductArgs a) {
  const int64_t m = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
  const int64_t rows = a.ragged_k ? a.n * a.groups : a.n;
  if (m >= a.m) return;
  for (int64_t r = (int64_t)blockIdx.y * 8 + threadIdx.x / 32; r < rows; r += (int64_t)gridDim.y * 8) {
    int g;
    int64_t n = r, k0 = 0, k1 = a.k;
    if (a.ragged_k) {
      g = (int)(r / a.n);
      n = r - g * a.n;
      k0 = bound(a, g, a.k);
      k1 = bound(a, g + 1, a.k);
    } else {
      for (g = 0; g < a.groups; ++g)
        if (bound(a, g, a.n) <= r && r < bound(a, g + 1, a.n)) break;
    }
    float sum = 0.0f;
    if (g < a.groups)
      for (int64_t k = k0; k < k1; ++k) {
        const int64_t at_a = a.a_mn ? k * a.a_row + m : m * a.a_row + k;
        const int64_t at_b = a.b_mn ? k * a.b_row + n : n * a.b_row + k;
        const int64_t group = a.ragged_k ? 0 : g;
        sum += value<T>(a, a.a, a.a_scales, group * a.m + m, k, group * a.a_group + at_a) *
               value<T>(a, a.b, a.b_scales, n, k, at_b);
      }
    Out* out = static_cast<Out*>(a.out) + (a.ragged_k ? g * a.out_group : 0) + n * a.out_row + m;
    if (sizeof(Out) == 4 && a.accumulate)
      *out = DT<Out>::from_f32(DT<Out>::to_f32(*out) + sum);
    else
      *out = DT<Out>::from_f32(sum);
  }
}

template <typename T>
cudaError_t run(const ProductArgs& a, cudaStream_t s) {
  const int64_t rows = a.ragged_k ? a.n * a.groups : a.n;
  const int64_t down = (rows + 7) / 8;
  const dim3 grid((unsigned)((a.m + 31) / 32), (unsigned)(down < 65535 ? down : 65535));
  if (a.out_dtype == kF32)
    k_product_plain<T, float><<<grid, 256, 0, s>>>(a);
  else if (a.out_dtype == kF16)
    k_product_plain<T, __half><<<grid, 256, 0, s>>>(a);
  else
    k_product_plain<T, __nv_bfloat16><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t product_error(unsigned** at) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(at), g_product_error);
}

cudaError_t launch_product(const ProductArgs& a, int sms, cudaStream_t s) {
  (void)sms;
  if (a.dtype == kE4M3) return run<E4M3>(a, s);
  return a.dtype == kF16 ? run<__half>(a, s) : run<__nv_bfloat16>(a, s);
}

}  // namespace zg
