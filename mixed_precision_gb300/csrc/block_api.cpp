// Host side of the block operators declared in include/zero.h: argument
// checks and launches. No compute happens here.
#include "zero.h"

#include <cmath>

#include <cuda_runtime.h>

#include "block.h"
#include "checks.h"
#include "experts.h"

using namespace zg;

namespace {

constexpr int kMaxNormCols = 65536;
constexpr int64_t kMaxLen = int64_t(1) << 28;

int check_norm(const zero_rmsnorm_desc* d) {
  if (d == nullptr) return fail(ZERO_ERR_INVALID, "desc is NULL");
  if (int rc = check_rows(d->rows, d->cols, kMaxNormCols)) return rc;
  if (!valid_dtype(d->dtype) || !valid_dtype(d->weight_dtype))
    return fail(ZERO_ERR_INVALID, "bad dtype %d or weight_dtype %d", d->dtype, d->weight_dtype);
  if (!(d->eps >= 0.0) || !std::isfinite(d->eps))
    return fail(ZERO_ERR_INVALID, "eps %g is not a finite number >= 0", d->eps);
  if (int rc = check_stride(d->x_stride, d->cols, "x_stride")) return rc;
  if (int rc = check_stride(d->residual_stride, d->cols, "residual_stride")) return rc;
  return check_stride(d->dy_stride, d->cols, "dy_stride");
}

int64_t act_pitch(int64_t cols) { return (cols + kActPitch - 1) / kActPitch * kActPitch; }

NormArgs norm_args(const zero_rmsnorm_desc* d) {
  NormArgs a{};
  a.rows = d->rows;
  a.cols = (int)d->cols;
  a.pitch = (int)act_pitch(d->cols);
  a.x_stride = d->x_stride;
  a.r_stride = d->residual_stride;
  a.dy_stride = d->dy_stride;
  a.dtype = d->dtype;
  a.weight_dtype = d->weight_dtype;
  a.eps = (float)d->eps;
  return a;
}

constexpr int64_t kMaxActCols = int64_t(1) << 30;

int check_strides(const int64_t s[3], const int64_t n[3], int64_t dim, const char* name,
                  int64_t out[3]) {
  for (int i = 0; i < 3; ++i) {
    out[i] = n[i] > 1 ? s[i] : 8 * ((dim + 7) / 8);  // a dimension of size 1 is never stepped over
    if (out[i] < dim || out[i] > kMaxStride || out[i] % 8 != 0)
      return fail(ZERO_ERR_INVALID, "%s stride %d is %lld: a multiple of 8, at least head_dim %lld",
                  name, i, (long long)s[i], (long long)dim);
  }
  return ZERO_OK;
}

// The {batch, token, head} strides of an output: no two elements may share an
// address. Sorted by stride, each dimension must step over all of the last.
int check_disjoint(const int64_t s[3], const int64_t n[3], int64_t dim, const char* name) {
  int order[3] = {0, 1, 2};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (s[order[j]] > s[order[j + 1]]) {
        const int t = order[j];
        order[j] = order[j + 1];
        order[j + 1] = t;
      }
  int64_t span = dim;
  for (int i = 0; i < 3; ++i) {
    const int d = order[i];
    if (n[d] <= 1) continue;
    if (s[d] < span) return fail(ZERO_ERR_INVALID, "%s: its elements overlap", name);
    span += (n[d] - 1) * s[d];
  }
  return ZERO_OK;
}

// A [batch, token, head, dim] tensor of 16-bit elements.
struct View {
  const void* base;
  const int64_t *s, *n;
  int64_t dim;
  const char* name;

  int64_t span() const {  // elements from the first to behind the last
    int64_t e = dim;
    for (int i = 0; i < 3; ++i) e += (n[i] - 1) * s[i];
    return e;
  }
  // Where steps of the period are left out: the elements' extent in it; 0 if it
  // is none (a stride above it that is no multiple).
  int64_t extent(int64_t period) const {
    int64_t e = dim;
    for (int i = 0; i < 3; ++i) {
      if (n[i] == 1 || s[i] % period == 0) continue;
      if (s[i] > period) return 0;
      e += (n[i] - 1) * s[i];
    }
    return e <= period ? e : 0;
  }
};

bool same_place(const View& x, const View& y) {
  bool same = x.base == y.base;
  for (int i = 0; i < 3; ++i) same = same && x.n[i] == y.n[i] && (x.n[i] == 1 || x.s[i] == y.s[i]);
  return same;
}

// Whether no element of x is one of y's: their ranges are apart, or they lie side
// by side in the steps of one of their strides (heads of one projection, halves
// of one row). Interleaved in any other way they count as overlapping.
bool apart(const View& x, const View& y) {
  for (int i = 0; i < 3; ++i)
    if (x.n[i] == 0 || y.n[i] == 0) return true;
  const int64_t d = (static_cast<const char*>(y.base) - static_cast<const char*>(x.base)) / 2;
  if (d >= x.span() || -d >= y.span()) return true;
  for (const View* v : {&x, &y})
    for (int i = 0; i < 3; ++i) {
      const int64_t period = v->s[i], ex = x.extent(period), ey = y.extent(period);
      if (v->n[i] == 1 || ex == 0 || ey == 0) continue;
      const int64_t r = (d % period + period) % period;
      if (r >= ex && r + ey <= period) return true;
    }
  return false;
}

// An output may not overlap an input that is read after it has been written.
// in_place: but be exactly it, where each element is read by whom it is written.
int check_output(const View& out, const View& in, bool in_place) {
  if ((in_place && same_place(out, in)) || apart(out, in)) return ZERO_OK;
  return fail(ZERO_ERR_INVALID, "%s overlaps %s", out.name, in.name);
}

int attention_args(const zero_attention_desc* d, bool backward, AttnArgs& a) {
  if (d == nullptr) return fail(ZERO_ERR_INVALID, "desc is NULL");
  if (d->batch < 0 || d->batch > kMaxLen || d->q_len < 0 || d->q_len > kMaxLen || d->k_len < 0 ||
      d->k_len > kMaxLen)
    return fail(ZERO_ERR_INVALID, "batch %lld, q_len %lld or k_len %lld out of range",
                (long long)d->batch, (long long)d->q_len, (long long)d->k_len);
  if (d->q_heads < 1 || d->kv_heads < 1 || d->q_heads % d->kv_heads != 0 || d->q_heads > 65536)
    return fail(ZERO_ERR_INVALID, "%d query heads over %d key heads", d->q_heads, d->kv_heads);
  if (d->head_dim < 8 || d->head_dim > 128 || d->head_dim % 8 != 0)
    return fail(ZERO_ERR_INVALID, "head_dim %d: multiples of 8 up to 128", d->head_dim);
  if (!half_dtype(d->dtype)) return fail(ZERO_ERR_INVALID, "dtype %d: fp16 or bf16", d->dtype);
  if (d->window < 0) return fail(ZERO_ERR_INVALID, "window %lld < 0", (long long)d->window);
  if (!(d->scale > 0.0) || !(d->scale < 1e37))  // in powers of two, times log2 e, still an fp32 number
    return fail(ZERO_ERR_INVALID, "scale %g is not between 0 and 1e37", d->scale);
  // row counts and tile counts stay inside the kernels' index types
  if ((double)d->batch * d->q_heads * ((double)d->q_len + 128) > 2e11 ||
      (double)d->batch * d->kv_heads * ((double)d->k_len + 128) > 2e11)
    return fail(ZERO_ERR_INVALID, "too many rows");
  a = AttnArgs{};
  a.batch = d->batch;
  a.q_len = d->q_len;
  a.k_len = d->k_len;
  a.q_heads = d->q_heads;
  a.kv_heads = d->kv_heads;
  a.group = d->q_heads / d->kv_heads;
  a.head_dim = d->head_dim;
  a.dtype = d->dtype;
  if (d->batch * d->q_heads > 0x7FFFFFFF) return fail(ZERO_ERR_INVALID, "too many heads");
  if (d->batch > 0) {
    a.by_group = Divide(a.group);
    a.by_kv_heads = Divide(a.kv_heads);
    a.by_q_heads = Divide(a.q_heads);
    a.by_batch_kv = Divide((uint32_t)(d->batch * d->kv_heads));
    a.by_batch_q = Divide((uint32_t)(d->batch * d->q_heads));
  }
  a.causal = d->causal != 0;
  // a window wider than any distance is none
  a.window = d->window < d->q_len + d->k_len ? d->window : 0;
  a.scale = (float)d->scale;
  const int64_t nq[3] = {d->batch, d->q_len, d->q_heads}, nk[3] = {d->batch, d->k_len, d->kv_heads};
  const struct {
    const int64_t *s, *n;
    int64_t* out;
    const char* name;
    bool used, written;
  } all[] = {
      {d->q_strides, nq, a.qs, "q", true, false},
      {d->k_strides, nk, a.ks, "k", true, false},
      {d->v_strides, nk, a.vs, "v", true, false},
      {d->o_strides, nq, a.os, "o", true, !backward},
      {d->do_strides, nq, a.dos, "dout", backward, false},
      {d->dq_strides, nq, a.dqs, "dq", backward, true},
      {d->dk_strides, nk, a.dks, "dk", backward, true},
      {d->dv_strides, nk, a.dvs, "dv", backward, true},
  };
  for (const auto& t : all) {
    if (!t.used) continue;
    if (int rc = check_strides(t.s, t.n, d->head_dim, t.name, t.out)) return rc;
    if (t.written)
      if (int rc = check_disjoint(t.out, t.n, d->head_dim, t.name)) return rc;
  }
  return ZERO_OK;
}

constexpr int kErrorWords = 5, kBlockErrorWords = 4;  // of the block operators and of the experts' products
cudaError_t (*const kErrorWord[kErrorWords])(unsigned**) = {norm_error, wgrad_error, attn_fwd_error, attn_bwd_error,
                                                           product_error};

}  // namespace

extern "C" {

int zero_rmsnorm_forward(const zero_rmsnorm_desc* desc, const void* x, const void* residual,
                         const void* weight, void* sum_out, void* y, int8_t* q, uint8_t* scales,
                         float* rstd, void* stream) {
  Range r("zero_rmsnorm_forward");
  if (int rc = check_norm(desc)) return rc;
  if (desc->rows == 0) return ZERO_OK;
  NEED(x);
  NEED(weight);
  ALIGNED(y);
  ALIGNED(rstd);
  if (residual != nullptr) {
    ALIGNED(residual);
    NEED(sum_out);
    if ((sum_out == x && desc->x_stride != desc->cols) ||
        (sum_out == residual && desc->residual_stride != desc->cols))
      return fail(ZERO_ERR_INVALID, "sum_out may be an input itself only when its stride is cols");
  } else if (sum_out != nullptr) {
    return fail(ZERO_ERR_INVALID, "sum_out without a residual");
  }
  if (y != nullptr) {
    if (y == sum_out) return fail(ZERO_ERR_INVALID, "y may not be sum_out itself");
    if ((y == x && desc->x_stride != desc->cols) || (y == residual && desc->residual_stride != desc->cols))
      return fail(ZERO_ERR_INVALID, "y may be an input itself only when its stride is cols");
  }
  if ((q == nullptr) != (scales == nullptr))
    return fail(ZERO_ERR_INVALID, "q and scales come together");
  if (q != nullptr) {
    NEED(q);
    NEED(scales);
  } else if (y == nullptr) {
    return fail(ZERO_ERR_INVALID, "neither y nor a packed output");
  }
  NormArgs a = norm_args(desc);
  a.x = x;
  a.res = residual;
  if (residual == nullptr) a.r_stride = a.x_stride;
  a.dy_stride = a.x_stride;
  a.weight = weight;
  a.sum = sum_out;
  a.y = y;
  a.q = q;
  a.scales = scales;
  a.rstd = rstd;
  int sms;
  if (int rc = device_sms(&sms)) return rc;
  cudaError_t e = launch_norm_forward(a, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "RMSNorm forward launch");
}

int zero_rmsnorm_backward_workspace(const zero_rmsnorm_desc* desc, int64_t* bytes) {
  if (bytes == nullptr) return fail(ZERO_ERR_INVALID, "bytes is NULL");
  if (int rc = check_norm(desc)) return rc;
  *bytes = (int64_t)norm_backward_parts(desc->rows, (int)desc->cols) * desc->cols * 4;
  return ZERO_OK;
}

int zero_rmsnorm_backward(const zero_rmsnorm_desc* desc, const void* dy, const void* x,
                          const void* weight, const float* rstd, const void* dsum, void* dx,
                          void* dweight, int dweight_dtype, void* workspace,
                          int64_t workspace_bytes, void* stream) {
  Range r("zero_rmsnorm_backward");
  if (int rc = check_norm(desc)) return rc;
  if (!valid_dtype(dweight_dtype)) return fail(ZERO_ERR_INVALID, "bad dweight_dtype %d", dweight_dtype);
  NEED(dweight);
  NormArgs a = norm_args(desc);
  if (desc->rows > 0) {
    NEED(dy);
    NEED(x);
    NEED(weight);
    NEED(rstd);
    NEED(dx);
    ALIGNED(dsum);
    if (dx == x) return fail(ZERO_ERR_INVALID, "dx may not be x itself");
    if ((dx == dy && desc->dy_stride != desc->cols) ||
        (dx == dsum && desc->residual_stride != desc->cols))
      return fail(ZERO_ERR_INVALID, "dx may be an input itself only when its stride is cols");
    NEED(workspace);
    const int64_t want = (int64_t)norm_backward_parts(a.rows, a.cols) * a.cols * 4;
    if (workspace_bytes < want)
      return fail(ZERO_ERR_INVALID, "workspace of %lld bytes, %lld needed",
                  (long long)workspace_bytes, (long long)want);
  }
  a.dy = dy;
  a.x = x;
  a.weight = weight;
  a.rstd_in = rstd;
  a.res = dsum;
  if (dsum == nullptr) a.r_stride = a.x_stride;
  a.dx = dx;
  a.dweight = dweight;
  a.dweight_dtype = dweight_dtype;
  a.part = static_cast<float*>(workspace);
  int sms;
  if (int rc = device_sms(&sms)) return rc;
  cudaError_t e = launch_norm_backward(a, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "RMSNorm backward launch");
}

int zero_act_layout(int64_t rows, int64_t cols, int64_t* pitch, int64_t* q_bytes,
                    int64_t* scale_bytes) {
  if (int rc = check_rows(rows, cols, kMaxActCols)) return rc;
  if (pitch == nullptr || q_bytes == nullptr || scale_bytes == nullptr)
    return fail(ZERO_ERR_INVALID, "an output pointer is NULL");
  const int64_t p = act_pitch(cols);
  if ((double)rows * (double)p > 4e18) return fail(ZERO_ERR_INVALID, "too many elements");
  *pitch = p;
  *q_bytes = rows * p;
  *scale_bytes = rows * (p / kActGroup);
  return ZERO_OK;
}

int zero_act_pack(const void* x, int64_t x_stride, int64_t rows, int64_t cols, int dtype, int8_t* q,
                  uint8_t* scales, void* stream) {
  Range r("zero_act_pack");
  if (int rc = check_rows(rows, cols, kMaxActCols)) return rc;
  if (!valid_dtype(dtype)) return fail(ZERO_ERR_INVALID, "bad dtype %d", dtype);
  if (int rc = check_stride(x_stride, cols, "x_stride")) return rc;
  if (rows == 0) return ZERO_OK;
  NEED(x);
  NEED(q);
  NEED(scales);
  ActArgs a{};
  a.rows = rows;
  a.cols = (int)cols;
  a.pitch = (int)act_pitch(cols);
  a.stride = x_stride;
  a.dtype = dtype;
  a.x = x;
  a.q = q;
  a.scales = scales;
  cudaError_t e = launch_act_pack(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "activation pack launch");
}

int zero_act_unpack(const int8_t* q, const uint8_t* scales, int64_t rows, int64_t cols, void* out,
                    int64_t out_stride, int dtype, void* stream) {
  Range r("zero_act_unpack");
  if (int rc = check_rows(rows, cols, kMaxActCols)) return rc;
  if (!valid_dtype(dtype)) return fail(ZERO_ERR_INVALID, "bad dtype %d", dtype);
  if (int rc = check_stride(out_stride, cols, "out_stride")) return rc;
  if (rows == 0) return ZERO_OK;
  NEED(q);
  NEED(scales);
  NEED(out);
  ActArgs a{};
  a.rows = rows;
  a.cols = (int)cols;
  a.pitch = (int)act_pitch(cols);
  a.stride = out_stride;
  a.dtype = dtype;
  a.q_in = q;
  a.scales_in = scales;
  a.out = out;
  cudaError_t e = launch_act_unpack(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "activation restore launch");
}

int zero_act_weight_grad_workspace(int64_t tokens, int64_t n_out, int64_t n_in, int64_t* bytes) {
  if (bytes == nullptr) return fail(ZERO_ERR_INVALID, "bytes is NULL");
  if (int rc = check_rows(tokens, n_in, kMaxActCols)) return rc;
  if (int rc = check_rows(n_out, n_in, kMaxActCols)) return rc;
  *bytes = 0;
  return ZERO_OK;
}

int zero_act_weight_grad(const void* dy, int64_t dy_stride, int dtype, const int8_t* q,
                         const uint8_t* scales, int64_t tokens, int64_t n_out, int64_t n_in,
                         void* dw, int dw_dtype, int accumulate, void* workspace,
                         int64_t workspace_bytes, void* stream) {
  Range r("zero_act_weight_grad");
  (void)workspace, (void)workspace_bytes;  // no plan needs one
  if (int rc = check_rows(tokens, n_in, kMaxActCols)) return rc;
  if (n_out < 1 || n_out > kMaxActCols)
    return fail(ZERO_ERR_INVALID, "n_out %lld out of range", (long long)n_out);
  if (!half_dtype(dtype)) return fail(ZERO_ERR_INVALID, "dtype %d: fp16 or bf16", dtype);
  if (dw_dtype != ZERO_F32 && dw_dtype != dtype)
    return fail(ZERO_ERR_INVALID, "dw_dtype %d: fp32 or dy's type", dw_dtype);
  if (accumulate && dw_dtype != ZERO_F32)
    return fail(ZERO_ERR_INVALID, "accumulate needs an fp32 dw");
  if (int rc = check_stride(dy_stride, n_out, "dy_stride")) return rc;
  if (dy_stride % 8 != 0)
    return fail(ZERO_ERR_INVALID, "dy_stride %lld is not a multiple of 8", (long long)dy_stride);
  NEED(dw);
  if (tokens > 0) {
    NEED(dy);
    NEED(q);
    NEED(scales);
  }
  WgradArgs a{};
  a.dy = dy;
  a.dy_stride = dy_stride;
  a.dtype = dtype;
  a.q = q;
  a.scales = scales;
  a.tokens = tokens;
  a.n_out = n_out;
  a.n_in = (int)n_in;
  a.pitch = (int)act_pitch(n_in);
  a.dw = dw;
  a.dw_dtype = dw_dtype;
  a.accumulate = accumulate != 0;
  int sms;
  if (int rc = device_sms(&sms)) return rc;
  cudaError_t e = launch_wgrad(a, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "weight gradient launch");
}

int zero_attention_forward(const zero_attention_desc* desc, const void* q, const void* k,
                           const void* v, const int32_t* key_lengths, void* o, float* lse,
                           void* stream) {
  Range r("zero_attention_forward");
  AttnArgs a;
  if (int rc = attention_args(desc, false, a)) return rc;
  if (a.batch == 0 || a.q_len == 0) return ZERO_OK;
  NEED(q);
  if (a.k_len > 0) {
    NEED(k);
    NEED(v);
  }
  NEED(o);
  NEED(lse);
  if ((reinterpret_cast<uintptr_t>(key_lengths) & 3u) != 0)
    return fail(ZERO_ERR_INVALID, "key_lengths is not 4-byte aligned");
  const int64_t nq[3] = {a.batch, a.q_len, a.q_heads}, nk[3] = {a.batch, a.k_len, a.kv_heads}, dim = a.head_dim;
  const View to{o, a.os, nq, dim, "o"};
  if (int rc = check_output(to, {q, a.qs, nq, dim, "q"}, true)) return rc;
  if (int rc = check_output(to, {k, a.ks, nk, dim, "k"}, false)) return rc;
  if (int rc = check_output(to, {v, a.vs, nk, dim, "v"}, false)) return rc;
  a.q = q;
  a.k = k;
  a.v = v;
  a.lengths = key_lengths;
  a.o = o;
  a.lse = lse;
  int sms;
  if (int rc = device_sms(&sms)) return rc;
  cudaError_t e = launch_attention_forward(a, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "attention forward launch");
}

int zero_attention_backward_workspace(const zero_attention_desc* desc, int64_t* bytes) {
  if (bytes == nullptr) return fail(ZERO_ERR_INVALID, "bytes is NULL");
  AttnArgs a;
  if (int rc = attention_args(desc, true, a)) return rc;
  *bytes = attention_backward_bytes(a);
  return ZERO_OK;
}

int zero_attention_backward(const zero_attention_desc* desc, const void* dout, const void* q,
                            const void* k, const void* v, const void* o, const float* lse,
                            const int32_t* key_lengths, void* dq, void* dk, void* dv,
                            void* workspace, int64_t workspace_bytes, void* stream) {
  Range r("zero_attention_backward");
  AttnArgs a;
  if (int rc = attention_args(desc, true, a)) return rc;
  if (a.batch == 0 || (a.q_len == 0 && a.k_len == 0)) return ZERO_OK;
  if (a.q_len > 0) {
    NEED(dout);
    NEED(q);
    NEED(o);
    NEED(lse);
    NEED(dq);
    NEED(workspace);
    if (workspace_bytes < attention_backward_bytes(a))
      return fail(ZERO_ERR_INVALID, "workspace of %lld bytes, %lld needed",
                  (long long)workspace_bytes, (long long)attention_backward_bytes(a));
  }
  if (a.k_len > 0) {
    NEED(k);
    NEED(v);
    NEED(dk);
    NEED(dv);
  }
  if ((reinterpret_cast<uintptr_t>(key_lengths) & 3u) != 0)
    return fail(ZERO_ERR_INVALID, "key_lengths is not 4-byte aligned");
  const int64_t nq[3] = {a.batch, a.q_len, a.q_heads}, nk[3] = {a.batch, a.k_len, a.kv_heads}, dim = a.head_dim;
  const View tq{dq, a.dqs, nq, dim, "dq"}, tk{dk, a.dks, nk, dim, "dk"}, tv{dv, a.dvs, nk, dim, "dv"};
  const View from_q{q, a.qs, nq, dim, "q"}, from_do{dout, a.dos, nq, dim, "dout"}, from_k{k, a.ks, nk, dim, "k"},
      from_v{v, a.vs, nk, dim, "v"}, from_o{o, a.os, nq, dim, "o"};
  const struct {
    const View &out, &in;
    bool in_place;
  } pairs[] = {
      {tq, from_q, false}, {tq, from_do, false}, {tq, from_k, false}, {tq, from_v, false}, {tq, from_o, true},
      {tk, from_q, false}, {tk, from_do, false}, {tk, from_k, true},  {tk, from_v, true},  {tv, from_q, false},
      {tv, from_do, false}, {tv, from_k, true},  {tv, from_v, true},  {tq, tk, false},     {tq, tv, false},
      {tk, tv, false}};
  for (const auto& p : pairs)
    if (int rc = check_output(p.out, p.in, p.in_place)) return rc;
  a.dout = dout;
  a.q = q;
  a.k = k;
  a.v = v;
  a.o_in = o;
  a.lse_in = lse;
  a.lengths = key_lengths;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.stats = static_cast<float*>(workspace);
  int sms;
  if (int rc = device_sms(&sms)) return rc;
  cudaError_t e = launch_attention_backward(a, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "attention backward launch");
}

int zero_operator_status(void* stream) {
  Range r("zero_operator_status");
  constexpr int kDevices = 64;
  // What the thread last saw. Device counts are never cleared, so no thread takes
  // a time-out from another, and none is lost between a read and a write.
  static thread_local unsigned seen[kDevices][kErrorWords];
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int dev = 0;
  unsigned now[kErrorWords];
  cudaError_t e = cudaGetDevice(&dev);
  for (int i = 0; i < kErrorWords && e == cudaSuccess; ++i) {
    unsigned* at = nullptr;
    e = kErrorWord[i](&at);
    if (e == cudaSuccess) e = cudaMemcpyAsync(&now[i], at, sizeof(unsigned), cudaMemcpyDeviceToHost, s);
  }
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail(e, "operator status");
  if (dev >= kDevices) return fail(ZERO_ERR_INVALID, "device %d", dev);
  bool late = false;
  for (int i = 0; i < kErrorWords; ++i) {
    late = late || now[i] != seen[dev][i];
    seen[dev][i] = now[i];
  }
  if (late) return fail(ZERO_ERR_TIMEOUT, "a bounded wait gave up in an operator");
  return ZERO_OK;
}

int zero_selftest_operator_timeout(int kernels, uint32_t spin_limit, void* stream) {
  Range r("zero_selftest_operator_timeout");
  if (kernels < 0 || kernels >= kBlockErrorWords)
    return fail(ZERO_ERR_INVALID, "kernels %d outside 0..%d", kernels, kBlockErrorWords - 1);
  if (spin_limit < 1 || spin_limit > kSpinLimit) return fail(ZERO_ERR_INVALID, "spin_limit outside 1..2^22");
  unsigned* at = nullptr;
  cudaError_t e = kErrorWord[kernels](&at);
  if (e == cudaSuccess) e = launch_wait_that_gives_up(at, spin_limit, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "operator self-test");
}

int zero_selftest_pair_timeout(int block, uint32_t spin_limit, int32_t* ends, void* stream) {
  Range r("zero_selftest_pair_timeout");
  if (block < 0 || block > 1) return fail(ZERO_ERR_INVALID, "block %d: 0 or 1", block);
  if (spin_limit < 1 || spin_limit > kSpinLimit) return fail(ZERO_ERR_INVALID, "spin_limit outside 1..2^22");
  if (ends == nullptr || reinterpret_cast<uintptr_t>(ends) % 4 != 0)
    return fail(ZERO_ERR_INVALID, "ends is NULL or not 4-byte aligned");
  cudaError_t e = launch_pair_that_gives_up(block, spin_limit, ends, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "pair self-test");
}

}  // extern "C"
