// Internal interface between the host side of the block operators
// (block_api.cpp) and their kernels (k_norm.cu, k_act.cu, k_wgrad.cu,
// k_attn_fwd.cu, k_attn_bwd.cu). Not part of the public ABI (include/zero.h is).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "internal.h"

namespace zg {

constexpr int kActGroup = 32;   // elements of a packed row that share one scale
constexpr int kActPitch = 128;  // a packed row is padded to a multiple of this

// Division of numbers below 2^31 by a fixed one: n / d = n * mul >> shift, with
// mul = floor(2^shift / d) + 1 and shift = 31 + ceil(log2 d).
struct Divide {
  uint64_t mul;
  uint32_t d, shift;
  Divide() = default;
  explicit Divide(uint32_t by) : d(by) {
    uint32_t l = 0;
    while ((1ull << l) < by) ++l;
    shift = 31 + l;
    mul = (1ull << shift) / by + 1;
  }
#ifdef __CUDACC__
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return static_cast<uint32_t>(n * mul >> shift); }
  __device__ __forceinline__ uint32_t mod(uint32_t n) const { return n - (*this)(n) * d; }
#endif
};

struct NormArgs {
  int64_t rows;
  int cols, pitch;  // pitch: of the packed output
  int64_t x_stride, r_stride, dy_stride;
  int dtype, weight_dtype, dweight_dtype;
  float eps;
  const void *x, *res, *weight, *dy;  // res: residual (forward) or dsum (backward)
  const float* rstd_in;
  void *sum, *y, *dx, *dweight;
  int8_t* q;
  uint8_t* scales;
  float* rstd;
  float* part;  // backward: [parts][cols] partial sums of dweight
};
cudaError_t launch_norm_forward(const NormArgs& a, int sms, cudaStream_t s);
// Rows of partial sums that the backward writes (its workspace is parts x cols floats).
int norm_backward_parts(int64_t rows, int cols);
cudaError_t launch_norm_backward(const NormArgs& a, int sms, cudaStream_t s);

struct ActArgs {
  int64_t rows;
  int cols, pitch;
  int64_t stride;  // of x or out
  int dtype;
  const void* x;
  void* out;
  const int8_t* q_in;
  const uint8_t* scales_in;
  int8_t* q;
  uint8_t* scales;
};
cudaError_t launch_act_pack(const ActArgs& a, cudaStream_t s);
cudaError_t launch_act_unpack(const ActArgs& a, cudaStream_t s);

struct WgradArgs {
  const void* dy;
  int64_t dy_stride;
  int dtype;
  const int8_t* q;
  const uint8_t* scales;
  int64_t tokens, n_out;
  int n_in, pitch;
  void* dw;
  int dw_dtype, accumulate;
};
cudaError_t launch_wgrad(const WgradArgs& a, int sms, cudaStream_t s);

struct AttnArgs {
  int64_t batch, q_len, k_len;
  int q_heads, kv_heads, head_dim, group;  // group = q_heads / kv_heads
  int dtype, causal;
  int64_t window;  // 0: none
  float scale;
  int64_t qs[3], ks[3], vs[3], os[3], dos[3], dqs[3], dks[3], dvs[3];  // {batch, token, head}
  const void *q, *k, *v, *dout;
  const void* o_in;
  void *o, *dq, *dk, *dv;
  const int32_t* lengths;
  float* lse;
  const float* lse_in;
  // backward, from the workspace (k_attn_bwd.cu): the rows' statistics; in fp16
  // the key heads' largest |v| in v_parts parts and bounds of |dp - delta|
  float* stats;
  uint32_t *v_top, *ds_top;
  int v_parts;
  Divide by_group, by_kv_heads, by_q_heads, by_batch_kv, by_batch_q;  // batch x heads
};
cudaError_t launch_attention_forward(const AttnArgs& a, int sms, cudaStream_t s);
int64_t attention_backward_bytes(const AttnArgs& a);
cudaError_t launch_attention_backward(const AttnArgs& a, int sms, cudaStream_t s);

// Where the kernels' error words are on the current device: each counts the waits
// that gave up, and is never cleared.
cudaError_t norm_error(unsigned** at);
cudaError_t wgrad_error(unsigned** at);
cudaError_t attn_fwd_error(unsigned** at);
cudaError_t attn_bwd_error(unsigned** at);

// A kernel whose one wait gives up after `limit` tries (k_misc.cu).
cudaError_t launch_wait_that_gives_up(unsigned* error, uint32_t limit, cudaStream_t s);

}  // namespace zg
