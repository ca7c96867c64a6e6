// Attention's backward pass, plain form: a warp per row, each lane holding
// four neighbouring elements of the head, one dot product (five shuffles) per
// query-key pair.
#include "block.h"
#include "vec.cuh"

namespace zg {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

template <typename T>
__device__ __forceinline__ void load4(const T* p, int d, int dim, float (&x)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = d + j < dim ? DT<T>::to_f32(p[d + j]) : 0.0f;
}
template <typename T>
__device__ __forceinline__ void save4(T* p, int d, int dim, const float (&x)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (d + j < dim) p[d + j] = DT<T>::from_f32(x[j]);
}
__device__ __forceinline__ float dot4(const float (&x)[4], const float (&y)[4]) {
  return fmaf(x[0], y[0], fmaf(x[1], y[1], fmaf(x[2], y[2], x[3] * y[3])));
}

__device__ __forceinline__ int64_t valid_keys(const AttnArgs& a, int64_t b) {
  return a.lengths == nullptr ? a.k_len : min((int64_t)max(a.lengths[b], 0), a.k_len);
}

// Keys [lo, hi) that query i of batch entry b sees.
__device__ __forceinline__ void key_range(const AttnArgs& a, int64_t b, int64_t i, int64_t& lo,
                                          int64_t& hi) {
  const int64_t d = i + a.k_len - a.q_len;
  hi = valid_keys(a, b);
  if (a.causal) hi = min(hi, d + 1);
  lo = a.window > 0 ? max((int64_t)0, d - a.window + 1) : 0;
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) k_attn_dq(const AttnArgs a) {
  const int64_t row = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
  if (row >= a.batch * a.q_heads * a.q_len) return;
  const int d = (threadIdx.x & 31) * 4;
  const int64_t i = row % a.q_len, h = row / a.q_len % a.q_heads, b = row / a.q_len / a.q_heads;
  const int64_t c = h / a.group;
  float q[4], o[4], g[4], dq[4] = {};
  load4(static_cast<const T*>(a.q) + b * a.qs[0] + i * a.qs[1] + h * a.qs[2], d, a.head_dim, q);
  load4(static_cast<const T*>(a.o_in) + b * a.os[0] + i * a.os[1] + h * a.os[2], d, a.head_dim, o);
  load4(static_cast<const T*>(a.dout) + b * a.dos[0] + i * a.dos[1] + h * a.dos[2], d, a.head_dim, g);
  int64_t lo, hi;
  key_range(a, b, i, lo, hi);
  const float delta = warp_sum(dot4(o, g));
  if ((threadIdx.x & 31) == 0) a.delta[row] = delta;
  const float lse = a.lse_in[row];
  for (int64_t j = lo; j < hi; ++j) {
    float k[4], v[4];
    load4(static_cast<const T*>(a.k) + b * a.ks[0] + j * a.ks[1] + c * a.ks[2], d, a.head_dim, k);
    load4(static_cast<const T*>(a.v) + b * a.vs[0] + j * a.vs[1] + c * a.vs[2], d, a.head_dim, v);
    const float p = expf(warp_sum(dot4(q, k)) * a.scale - lse);
    const float ds = p * (warp_sum(dot4(g, v)) - delta) * a.scale;
#pragma unroll
    for (int e = 0; e < 4; ++e) dq[e] = fmaf(ds, k[e], dq[e]);
  }
  save4(static_cast<T*>(a.dq) + b * a.dqs[0] + i * a.dqs[1] + h * a.dqs[2], d, a.head_dim, dq);
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) k_attn_dkv(const AttnArgs a) {
  const int64_t row = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
  if (row >= a.batch * a.kv_heads * a.k_len) return;
  const int d = (threadIdx.x & 31) * 4;
  const int64_t j = row % a.k_len, c = row / a.k_len % a.kv_heads, b = row / a.k_len / a.kv_heads;
  float k[4], v[4], dk[4] = {}, dv[4] = {};
  load4(static_cast<const T*>(a.k) + b * a.ks[0] + j * a.ks[1] + c * a.ks[2], d, a.head_dim, k);
  load4(static_cast<const T*>(a.v) + b * a.vs[0] + j * a.vs[1] + c * a.vs[2], d, a.head_dim, v);
  const int64_t off = a.k_len - a.q_len;
  const int64_t lo = a.causal ? max((int64_t)0, j - off) : 0;
  int64_t hi = a.window > 0 ? min(a.q_len, j - off + a.window) : a.q_len;
  if (j >= valid_keys(a, b)) hi = lo;
  for (int g = 0; g < a.group; ++g) {
    const int64_t h = c * a.group + g;
    for (int64_t i = lo; i < hi; ++i) {
      const int64_t at = (b * a.q_heads + h) * a.q_len + i;
      float q[4], go[4];
      load4(static_cast<const T*>(a.q) + b * a.qs[0] + i * a.qs[1] + h * a.qs[2], d, a.head_dim, q);
      load4(static_cast<const T*>(a.dout) + b * a.dos[0] + i * a.dos[1] + h * a.dos[2], d, a.head_dim, go);
      const float p = expf(warp_sum(dot4(q, k)) * a.scale - a.lse_in[at]);
      const float ds = p * (warp_sum(dot4(go, v)) - a.delta[at]) * a.scale;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        dk[e] = fmaf(ds, q[e], dk[e]);
        dv[e] = fmaf(p, go[e], dv[e]);
      }
    }
  }
  save4(static_cast<T*>(a.dk) + b * a.dks[0] + j * a.dks[1] + c * a.dks[2], d, a.head_dim, dk);
  save4(static_cast<T*>(a.dv) + b * a.dvs[0] + j * a.dvs[1] + c * a.dvs[2], d, a.head_dim, dv);
}

unsigned blocks(int64_t rows) { return (unsigned)((rows + kWarps - 1) / kWarps); }

template <typename T>
cudaError_t backward_t(const AttnArgs& a, cudaStream_t s) {
  const int64_t rq = a.batch * a.q_heads * a.q_len, rk = a.batch * a.kv_heads * a.k_len;
  if (rq > 0) k_attn_dq<T><<<blocks(rq), kWarps * 32, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (rk > 0) k_attn_dkv<T><<<blocks(rk), kWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_backward(const AttnArgs& a, int sms, cudaStream_t s) {
  (void)sms;
  return a.dtype == kF16 ? backward_t<__half>(a, s) : backward_t<__nv_bfloat16>(a, s);
}

}  // namespace zg
