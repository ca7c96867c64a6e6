// Internal interface between the host side of the expert layer's operators and
// the 8-bit floating-point products (experts_api.cpp) and their kernels
// (k_route.cu, k_rows.cu, k_scaled.cu, k_products.cu). Not part of the public ABI.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "internal.h"

namespace zg {

constexpr int kMaxExperts = 1024;
constexpr int kMaxChoices = 32;
constexpr int kScaledBlock = 128;  // elements along the contraction that share a scale
constexpr int kE4M3 = 3;           // a dtype of its own, beside kF32, kF16 and kBF16

struct RouteArgs {
  const void* logits;
  int64_t stride;
  int64_t tokens;
  int experts, k;
  int dtype, normalize;
  float* weights;
  int32_t *chosen, *offsets, *source, *place;
  int32_t* counts;  // workspace: [blocks][experts]
  // backward
  const float *dweights, *weights_in;
  const int32_t* chosen_in;
  void* dlogits;
};
int64_t route_workspace_bytes(int64_t tokens, int experts, int k);
cudaError_t launch_route(const RouteArgs& a, cudaStream_t s);
cudaError_t launch_route_backward(const RouteArgs& a, cudaStream_t s);

struct RowsArgs {
  int64_t tokens, hidden;
  int k, dtype;
  const void *x, *y;  // x: gather's input or combine_backward's dout
  int64_t x_stride, y_stride;
  const int32_t *place, *source;
  const float* weights;
  void* out;  // rows, out or dy
  float* dweights;
};
cudaError_t launch_gather(const RowsArgs& a, cudaStream_t s);
cudaError_t launch_combine(const RowsArgs& a, cudaStream_t s);
cudaError_t launch_combine_backward(const RowsArgs& a, cudaStream_t s);

struct ScaledArgs {
  const void* x;
  int64_t batch_stride, stride;
  int64_t batch, rows, cols;
  int dtype;
  int64_t pitch, scale_pitch;      // of q
  int64_t pitch_t, scale_pitch_t;  // of qt
  uint8_t *q, *scales, *qt, *scales_t;
  const uint8_t *q_in, *scales_in;
  void* out;
};
cudaError_t launch_scaled_pack(const ScaledArgs& a, cudaStream_t s);
cudaError_t launch_scaled_unpack(const ScaledArgs& a, cudaStream_t s);

// out[g][n][m] = sum over k of a(g, m, k) * b(n, k), for the products by expert.
// M is the weights' or the output's contiguous side. The ragged side is N (rows
// of b and out, split into groups by offsets) or K (a and b in groups along k,
// one output matrix a group). Strides in elements.
struct ProductArgs {
  const void *a, *b;
  void* out;
  int64_t m, n, k;         // of a ragged side: all groups' rows together
  int64_t a_group, a_row;  // a_group: between the groups' matrices (ragged N)
  int64_t b_row;
  int64_t out_group, out_row;  // out_group: ragged K
  bool a_mn, b_mn;             // contiguous along M or N (else along K)
  bool ragged_k;
  int groups;
  const int32_t* offsets;  // NULL: one group of all rows
  int dtype, out_dtype, accumulate;
  const uint8_t *a_scales, *b_scales;  // kE4M3
  int64_t scale_pitch;
};
cudaError_t launch_product(const ProductArgs& a, cudaStream_t s);
cudaError_t product_error(unsigned** at);
cudaError_t launch_pair_that_gives_up(int giver, uint32_t limit, int32_t* ends, cudaStream_t s);

#ifdef __CUDACC__
// A launch that may begin while the kernel ahead of it in the stream still runs: the
// kernel calls griddep_wait() before its first access to memory.
template <typename... P, typename... A>
cudaError_t launch_next(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
#endif

}  // namespace zg
