// Host side of the expert layer's operators and of the 8-bit floating-point
// products declared in include/zero.h: argument checks and launches.
#include "zero.h"

#include <cuda_runtime.h>

#include "checks.h"
#include "experts.h"

using namespace zg;

namespace {

constexpr int64_t kMaxIndex = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxDim = int64_t(1) << 24;
constexpr int64_t kMaxHidden = int64_t(1) << 30;
constexpr int64_t kMaxPackCols = 65535 * 128;

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }
int64_t dtype_bytes(int d) { return d == ZERO_F32 ? 4 : 2; }

// A buffer of a call: its bytes from first to behind the last.
struct Buffer {
  const void* p;
  int64_t bytes;
  const char* name;
};

// From the first to behind the last of rows x cols elements, `stride` between
// rows; at most 2^60 (further apart than any two addresses).
int64_t span(int64_t rows, int64_t cols, int64_t stride) {
  if (rows <= 0 || cols <= 0) return 0;
  const __int128 n = (__int128)(rows - 1) * stride + cols;
  return n < ((int64_t)1 << 60) ? (int64_t)n : (int64_t)1 << 60;
}

Buffer buffer(const void* p, int64_t rows, int64_t cols, int64_t stride, int64_t bytes, const char* name) {
  return {p, span(rows, cols, stride) * bytes, name};
}

bool overlap(const Buffer& a, const Buffer& b) {
  if (a.p == nullptr || b.p == nullptr || a.bytes == 0 || b.bytes == 0) return false;
  const auto x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + (uint64_t)b.bytes && y < x + (uint64_t)a.bytes;
}

// The first `outputs` buffers overlap nothing.
template <int N>
int check_apart(const Buffer (&all)[N], int outputs) {
  for (int i = 0; i < outputs; ++i)
    for (int j = i + 1; j < N; ++j)
      if (overlap(all[i], all[j])) return fail(ZERO_ERR_INVALID, "%s overlaps %s", all[i].name, all[j].name);
  return ZERO_OK;
}

int check_input_stride(int64_t stride, const char* name) {
  if (stride % 8 != 0)
    return fail(ZERO_ERR_INVALID, "%s %lld is not a multiple of 8", name, (long long)stride);
  return ZERO_OK;
}

// A required buffer whose elements are moved one by one: aligned to them.
int need_elements(const void* p, int dtype, const char* name) {
  if (p == nullptr) return fail(ZERO_ERR_INVALID, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) % dtype_bytes(dtype) != 0)
    return fail(ZERO_ERR_INVALID, "%s is not aligned to its elements", name);
  return ZERO_OK;
}
#define NEED_ELEMENTS(p, dtype)                              \
  do {                                                       \
    if (int rc_ = need_elements(p, dtype, #p)) return rc_;   \
  } while (0)

int check_choice(int64_t tokens, int experts, int k) {
  if (experts < 1 || experts > kMaxExperts)
    return fail(ZERO_ERR_INVALID, "%d experts: 1 to %d", experts, kMaxExperts);
  if (k < 1 || k > experts || k > kMaxChoices)
    return fail(ZERO_ERR_INVALID, "k %d of %d experts: 1 to %d", k, experts, kMaxChoices);
  if (tokens < 0 || tokens > kMaxIndex / k)
    return fail(ZERO_ERR_INVALID, "%lld tokens out of range", (long long)tokens);
  return ZERO_OK;
}

int check_rows_call(int64_t tokens, int k, int64_t hidden, int dtype) {
  if (k < 1 || k > kMaxChoices) return fail(ZERO_ERR_INVALID, "k %d: 1 to %d", k, kMaxChoices);
  if (tokens < 0 || tokens > kMaxIndex / k)
    return fail(ZERO_ERR_INVALID, "%lld tokens out of range", (long long)tokens);
  if (hidden < 1 || hidden > kMaxHidden)
    return fail(ZERO_ERR_INVALID, "hidden %lld out of range", (long long)hidden);
  if (!valid_dtype(dtype)) return fail(ZERO_ERR_INVALID, "bad dtype %d", dtype);
  return ZERO_OK;
}

int check_experts(const zero_experts_desc* d) {
  if (d == nullptr) return fail(ZERO_ERR_INVALID, "desc is NULL");
  if (d->rows < 0 || d->rows > kMaxIndex)
    return fail(ZERO_ERR_INVALID, "%lld rows out of range", (long long)d->rows);
  if (d->n_out < 1 || d->n_out > kMaxDim || d->n_in < 1 || d->n_in > kMaxDim)
    return fail(ZERO_ERR_INVALID, "n_out %lld or n_in %lld out of range", (long long)d->n_out, (long long)d->n_in);
  if (d->experts < 1 || d->experts > kMaxExperts)
    return fail(ZERO_ERR_INVALID, "%d experts: 1 to %d", d->experts, kMaxExperts);
  if (!half_dtype(d->dtype)) return fail(ZERO_ERR_INVALID, "dtype %d: fp16 or bf16", d->dtype);
  if (int rc = check_stride(d->x_stride, d->n_in, "x_stride")) return rc;
  if (int rc = check_stride(d->y_stride, d->n_out, "y_stride")) return rc;
  if (int rc = check_stride(d->w_row_stride, d->n_in, "w_row_stride")) return rc;
  if (d->experts == 1) return ZERO_OK;  // w_stride is not stepped over
  return check_stride(d->w_stride, span(d->n_out, d->n_in, d->w_row_stride), "w_stride");
}

// The step between experts' matrices; of a lone one some multiple of 8.
int64_t expert_step(const zero_experts_desc* d) {
  return d->experts > 1 ? d->w_stride : up(span(d->n_out, d->n_in, d->w_row_stride), 8);
}

Buffer expert_matrices(const void* p, const zero_experts_desc* d, int64_t bytes, const char* name) {
  return buffer(p, d->experts, span(d->n_out, d->n_in, d->w_row_stride), expert_step(d), bytes, name);
}

int launch(const ProductArgs& a, const char* what, void* stream) {
  cudaError_t e = launch_product(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZERO_OK : cuda_fail(e, what);
}

ScaledArgs scaled_args(int64_t batch, int64_t rows, int64_t cols) {
  ScaledArgs a{};
  a.batch = batch;
  a.rows = rows;
  a.cols = cols;
  a.pitch = up(cols, kScaledBlock);
  a.scale_pitch = up(a.pitch / kScaledBlock, 4);
  a.pitch_t = up(rows, kScaledBlock);
  a.scale_pitch_t = up(a.pitch_t / kScaledBlock, 4);
  return a;
}

}  // namespace

extern "C" {

int zero_route_workspace(int64_t tokens, int experts, int k, int64_t* bytes) {
  if (bytes == nullptr) return fail(ZERO_ERR_INVALID, "bytes is NULL");
  if (int rc = check_choice(tokens, experts, k)) return rc;
  *bytes = route_workspace_bytes(tokens, experts, k);
  return ZERO_OK;
}

int zero_route(const void* logits, int64_t logits_stride, int64_t tokens, int experts, int k, int dtype, int normalize,
               float* weights, int32_t* chosen, int32_t* offsets, int32_t* source, int32_t* place, void* workspace,
               int64_t workspace_bytes, void* stream) {
  Range r("zero_route");
  if (int rc = check_choice(tokens, experts, k)) return rc;
  if (!valid_dtype(dtype)) return fail(ZERO_ERR_INVALID, "bad dtype %d", dtype);
  if (int rc = check_stride(logits_stride, experts, "logits_stride")) return rc;
  NEED(offsets);
  const int64_t slots = tokens * k, want = route_workspace_bytes(tokens, experts, k);
  if (tokens > 0) {
    NEED_ELEMENTS(logits, dtype);
    NEED(weights);
    NEED(chosen);
    NEED(source);
    NEED(place);
    NEED(workspace);
    if (workspace_bytes < want)
      return fail(ZERO_ERR_INVALID, "workspace of %lld bytes, %lld needed", (long long)workspace_bytes,
                  (long long)want);
  }
  const Buffer all[] = {{weights, slots * 4, "weights"},
                        {chosen, slots * 4, "chosen"},
                        {offsets, (experts + 1) * 4ll, "offsets"},
                        {source, slots * 4, "source"},
                        {place, slots * 4, "place"},
                        {workspace, tokens > 0 ? want : 0, "workspace"},
                        buffer(logits, tokens, experts, logits_stride, dtype_bytes(dtype), "logits")};
  if (int rc = check_apart(all, 6)) return rc;
  RouteArgs a{};
  a.logits = logits;
  a.stride = logits_stride;
  a.tokens = tokens;
  a.experts = experts;
  a.k = k;
  a.dtype = dtype;
  a.normalize = normalize != 0;
  a.weights = weights;
  a.chosen = chosen;
  a.offsets = offsets;
  a.source = source;
  a.place = place;
  a.counts = static_cast<int32_t*>(workspace);
  cudaError_t e = launch_route(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "routing launch");
}

int zero_route_backward(const float* dweights, const float* weights, const int32_t* chosen, const void* logits,
                        int64_t logits_stride, int64_t tokens, int experts, int k, int dtype, int normalize,
                        void* dlogits, void* stream) {
  Range r("zero_route_backward");
  if (int rc = check_choice(tokens, experts, k)) return rc;
  if (!valid_dtype(dtype)) return fail(ZERO_ERR_INVALID, "bad dtype %d", dtype);
  if (int rc = check_stride(logits_stride, experts, "logits_stride")) return rc;
  if (tokens == 0) return ZERO_OK;
  NEED(dweights);
  NEED(weights);
  NEED(chosen);
  NEED(dlogits);
  if (!normalize) NEED_ELEMENTS(logits, dtype);
  const int64_t slots = tokens * k, b = dtype_bytes(dtype);
  const Buffer all[] = {{dlogits, tokens * experts * b, "dlogits"},
                        {dweights, slots * 4, "dweights"},
                        {weights, slots * 4, "weights"},
                        {chosen, slots * 4, "chosen"},
                        buffer(normalize ? nullptr : logits, tokens, experts, logits_stride, b, "logits")};
  if (int rc = check_apart(all, 1)) return rc;
  RouteArgs a{};
  a.logits = logits;
  a.stride = logits_stride;
  a.tokens = tokens;
  a.experts = experts;
  a.k = k;
  a.dtype = dtype;
  a.normalize = normalize != 0;
  a.dweights = dweights;
  a.weights_in = weights;
  a.chosen_in = chosen;
  a.dlogits = dlogits;
  cudaError_t e = launch_route_backward(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "routing backward launch");
}

int zero_experts_gather(const void* x, int64_t x_stride, int64_t tokens, int k, int64_t hidden, int dtype,
                        const int32_t* place, const int32_t* source, void* rows, void* stream) {
  Range r("zero_experts_gather");
  if (int rc = check_rows_call(tokens, k, hidden, dtype)) return rc;
  if (int rc = check_stride(x_stride, hidden, "x_stride")) return rc;
  if (tokens == 0) return ZERO_OK;
  NEED(x);
  NEED(place);
  NEED(source);
  NEED(rows);
  const int64_t slots = tokens * k, b = dtype_bytes(dtype);
  const Buffer all[] = {{rows, slots * hidden * b, "rows"},
                        buffer(x, tokens, hidden, x_stride, b, "x"),
                        {place, slots * 4, "place"},
                        {source, slots * 4, "source"}};
  if (int rc = check_apart(all, 1)) return rc;
  RowsArgs a{};
  a.tokens = tokens;
  a.hidden = hidden;
  a.k = k;
  a.dtype = dtype;
  a.x = x;
  a.x_stride = x_stride;
  a.place = place;
  a.source = source;
  a.out = rows;
  cudaError_t e = launch_gather(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "gather launch");
}

int zero_experts_combine(const void* y, int64_t y_stride, int64_t tokens, int k, int64_t hidden, int dtype,
                         const int32_t* place, const float* weights, void* out, void* stream) {
  Range r("zero_experts_combine");
  if (int rc = check_rows_call(tokens, k, hidden, dtype)) return rc;
  if (int rc = check_stride(y_stride, hidden, "y_stride")) return rc;
  if (tokens == 0) return ZERO_OK;
  NEED(y);
  NEED(place);
  ALIGNED(weights);
  NEED(out);
  const int64_t slots = tokens * k, b = dtype_bytes(dtype);
  const Buffer all[] = {{out, tokens * hidden * b, "out"},
                        buffer(y, slots, hidden, y_stride, b, "y"),
                        {place, slots * 4, "place"},
                        {weights, slots * 4, "weights"}};
  if (int rc = check_apart(all, 1)) return rc;
  RowsArgs a{};
  a.tokens = tokens;
  a.hidden = hidden;
  a.k = k;
  a.dtype = dtype;
  a.y = y;
  a.y_stride = y_stride;
  a.place = place;
  a.weights = weights;
  a.out = out;
  cudaError_t e = launch_combine(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "combine launch");
}

int zero_experts_combine_backward(const void* dout, int64_t dout_stride, const void* y, int64_t y_stride,
                                  int64_t tokens, int k, int64_t hidden, int dtype, const int32_t* place,
                                  const int32_t* source, const float* weights, void* dy, float* dweights,
                                  void* stream) {
  Range r("zero_experts_combine_backward");
  if (int rc = check_rows_call(tokens, k, hidden, dtype)) return rc;
  if (int rc = check_stride(dout_stride, hidden, "dout_stride")) return rc;
  if (int rc = check_stride(y_stride, hidden, "y_stride")) return rc;
  if (tokens == 0) return ZERO_OK;
  NEED(dout);
  NEED(y);
  NEED(place);
  NEED(source);
  NEED(weights);
  NEED(dy);
  NEED(dweights);
  const int64_t slots = tokens * k, b = dtype_bytes(dtype);
  const Buffer all[] = {{dy, slots * hidden * b, "dy"},
                        {dweights, slots * 4, "dweights"},
                        buffer(dout, tokens, hidden, dout_stride, b, "dout"),
                        buffer(y, slots, hidden, y_stride, b, "y"),
                        {place, slots * 4, "place"},
                        {source, slots * 4, "source"},
                        {weights, slots * 4, "weights"}};
  if (int rc = check_apart(all, 2)) return rc;
  RowsArgs a{};
  a.tokens = tokens;
  a.hidden = hidden;
  a.k = k;
  a.dtype = dtype;
  a.x = dout;
  a.x_stride = dout_stride;
  a.y = y;
  a.y_stride = y_stride;
  a.place = place;
  a.source = source;
  a.weights = weights;
  a.out = dy;
  a.dweights = dweights;
  cudaError_t e = launch_combine_backward(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "combine backward launch");
}

int zero_experts_forward(const zero_experts_desc* d, const void* x, const void* weights, const int32_t* offsets,
                         void* y, void* stream) {
  Range r("zero_experts_forward");
  if (int rc = check_experts(d)) return rc;
  if (int rc = check_input_stride(d->x_stride, "x_stride")) return rc;
  if (int rc = check_input_stride(expert_step(d), "w_stride")) return rc;
  if (int rc = check_input_stride(d->w_row_stride, "w_row_stride")) return rc;
  if (d->rows == 0) return ZERO_OK;
  NEED(x);
  NEED(weights);
  NEED(offsets);
  NEED_ELEMENTS(y, d->dtype);
  const Buffer all[] = {buffer(y, d->rows, d->n_out, d->y_stride, 2, "y"),
                        buffer(x, d->rows, d->n_in, d->x_stride, 2, "x"),
                        expert_matrices(weights, d, 2, "weights"),
                        {offsets, (d->experts + 1) * 4ll, "offsets"}};
  if (int rc = check_apart(all, 1)) return rc;
  ProductArgs a{};
  a.a = weights;
  a.b = x;
  a.out = y;
  a.m = d->n_out;
  a.n = d->rows;
  a.k = d->n_in;
  a.a_group = expert_step(d);
  a.a_row = d->w_row_stride;
  a.b_row = d->x_stride;
  a.out_row = d->y_stride;
  a.groups = d->experts;
  a.offsets = offsets;
  a.dtype = a.out_dtype = d->dtype;
  return launch(a, "experts' forward launch", stream);
}

int zero_experts_input_grad(const zero_experts_desc* d, const void* dy, const void* weights, const int32_t* offsets,
                            void* dx, void* stream) {
  Range r("zero_experts_input_grad");
  if (int rc = check_experts(d)) return rc;
  if (int rc = check_input_stride(d->y_stride, "y_stride")) return rc;
  if (int rc = check_input_stride(expert_step(d), "w_stride")) return rc;
  if (int rc = check_input_stride(d->w_row_stride, "w_row_stride")) return rc;
  if (d->rows == 0) return ZERO_OK;
  NEED(dy);
  NEED(weights);
  NEED(offsets);
  NEED_ELEMENTS(dx, d->dtype);
  const Buffer all[] = {buffer(dx, d->rows, d->n_in, d->x_stride, 2, "dx"),
                        buffer(dy, d->rows, d->n_out, d->y_stride, 2, "dy"),
                        expert_matrices(weights, d, 2, "weights"),
                        {offsets, (d->experts + 1) * 4ll, "offsets"}};
  if (int rc = check_apart(all, 1)) return rc;
  ProductArgs a{};
  a.a = weights;
  a.a_mn = true;
  a.b = dy;
  a.out = dx;
  a.m = d->n_in;
  a.n = d->rows;
  a.k = d->n_out;
  a.a_group = expert_step(d);
  a.a_row = d->w_row_stride;
  a.b_row = d->y_stride;
  a.out_row = d->x_stride;
  a.groups = d->experts;
  a.offsets = offsets;
  a.dtype = a.out_dtype = d->dtype;
  return launch(a, "experts' input gradient launch", stream);
}

int zero_experts_weight_grad(const zero_experts_desc* d, const void* dy, const void* x, const int32_t* offsets,
                             void* dw, int dw_dtype, int accumulate, void* stream) {
  Range r("zero_experts_weight_grad");
  if (int rc = check_experts(d)) return rc;
  if (dw_dtype != ZERO_F32 && dw_dtype != d->dtype)
    return fail(ZERO_ERR_INVALID, "dw_dtype %d: fp32 or the inputs' type", dw_dtype);
  if (accumulate && dw_dtype != ZERO_F32) return fail(ZERO_ERR_INVALID, "accumulate needs an fp32 dw");
  if (int rc = check_input_stride(d->x_stride, "x_stride")) return rc;
  if (int rc = check_input_stride(d->y_stride, "y_stride")) return rc;
  NEED_ELEMENTS(dw, dw_dtype);
  NEED(offsets);
  if (d->rows > 0) {
    NEED(dy);
    NEED(x);
  }
  const Buffer all[] = {expert_matrices(dw, d, dtype_bytes(dw_dtype), "dw"),
                        buffer(dy, d->rows, d->n_out, d->y_stride, 2, "dy"),
                        buffer(x, d->rows, d->n_in, d->x_stride, 2, "x"),
                        {offsets, (d->experts + 1) * 4ll, "offsets"}};
  if (int rc = check_apart(all, 1)) return rc;
  ProductArgs a{};
  a.a = x;
  a.a_mn = true;
  a.b = dy;
  a.b_mn = true;
  a.out = dw;
  a.m = d->n_in;
  a.n = d->n_out;
  a.k = d->rows;
  a.a_row = d->x_stride;
  a.b_row = d->y_stride;
  a.out_group = expert_step(d);
  a.out_row = d->w_row_stride;
  a.ragged_k = true;
  a.groups = d->experts;
  a.offsets = offsets;
  a.dtype = d->dtype;
  a.out_dtype = dw_dtype;
  a.accumulate = accumulate != 0;
  return launch(a, "experts' weight gradient launch", stream);
}

int zero_scaled_layout(int64_t rows, int64_t cols, int64_t* pitch, int64_t* scale_pitch) {
  if (int rc = check_rows(rows, cols, kMaxIndex)) return rc;
  if (pitch == nullptr || scale_pitch == nullptr) return fail(ZERO_ERR_INVALID, "an output pointer is NULL");
  const ScaledArgs a = scaled_args(1, rows, cols);
  *pitch = a.pitch;
  *scale_pitch = a.scale_pitch;
  return ZERO_OK;
}

int zero_scaled_pack(const void* x, int64_t batch_stride, int64_t x_stride, int64_t batch, int64_t rows, int64_t cols,
                     int dtype, void* q, uint8_t* scales, void* qt, uint8_t* scales_t, void* stream) {
  Range r("zero_scaled_pack");
  if (int rc = check_rows(rows, cols, kMaxPackCols)) return rc;
  if (batch < 0 || batch > 65535 || (double)batch * (double)up(rows, 128) > (double)kMaxIndex ||
      (double)batch * (double)up(cols, 128) > (double)kMaxIndex)
    return fail(ZERO_ERR_INVALID, "batch %lld of %lld x %lld out of range", (long long)batch, (long long)rows,
                (long long)cols);
  if (!valid_dtype(dtype)) return fail(ZERO_ERR_INVALID, "bad dtype %d", dtype);
  if (int rc = check_stride(x_stride, cols, "x_stride")) return rc;
  if (batch > 1)
    if (int rc = check_stride(batch_stride, span(rows, cols, x_stride), "batch_stride")) return rc;
  if ((q == nullptr) != (scales == nullptr)) return fail(ZERO_ERR_INVALID, "q and scales come together");
  if ((qt == nullptr) != (scales_t == nullptr)) return fail(ZERO_ERR_INVALID, "qt and scales_t come together");
  if (batch == 0 || rows == 0) return ZERO_OK;
  if (q == nullptr && qt == nullptr) return fail(ZERO_ERR_INVALID, "neither form is wanted");
  NEED(x);
  ALIGNED(q);
  ALIGNED(scales);
  ALIGNED(qt);
  ALIGNED(scales_t);
  ScaledArgs a = scaled_args(batch, rows, cols);
  const int64_t each = span(rows, cols, x_stride);
  const Buffer all[] = {{q, batch * rows * a.pitch, "q"},
                        {scales, batch * rows * a.scale_pitch, "scales"},
                        {qt, batch * cols * a.pitch_t, "qt"},
                        {scales_t, batch * cols * a.scale_pitch_t, "scales_t"},
                        buffer(x, batch, each, batch > 1 ? batch_stride : each, dtype_bytes(dtype), "x")};
  if (int rc = check_apart(all, 4)) return rc;
  a.x = x;
  a.batch_stride = batch > 1 ? batch_stride : 0;
  a.stride = x_stride;
  a.dtype = dtype;
  a.q = static_cast<uint8_t*>(q);
  a.scales = scales;
  a.qt = static_cast<uint8_t*>(qt);
  a.scales_t = scales_t;
  cudaError_t e = launch_scaled_pack(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "scaled pack launch");
}

int zero_scaled_unpack(const void* q, const uint8_t* scales, int64_t rows, int64_t cols, void* out, int64_t out_stride,
                       int dtype, void* stream) {
  Range r("zero_scaled_unpack");
  if (int rc = check_rows(rows, cols, kMaxIndex)) return rc;
  if (!valid_dtype(dtype)) return fail(ZERO_ERR_INVALID, "bad dtype %d", dtype);
  if (int rc = check_stride(out_stride, cols, "out_stride")) return rc;
  if (rows == 0) return ZERO_OK;
  NEED(q);
  NEED(scales);
  NEED(out);
  ScaledArgs a = scaled_args(1, rows, cols);
  const Buffer all[] = {buffer(out, rows, cols, out_stride, dtype_bytes(dtype), "out"),
                        {q, rows * a.pitch, "q"},
                        {scales, rows * a.scale_pitch, "scales"}};
  if (int rc = check_apart(all, 1)) return rc;
  a.q_in = static_cast<const uint8_t*>(q);
  a.scales_in = scales;
  a.out = out;
  a.stride = out_stride;
  a.dtype = dtype;
  cudaError_t e = launch_scaled_unpack(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "scaled restore launch");
}

int zero_scaled_matmul(const zero_scaled_desc* d, const void* a, const uint8_t* a_scales, const void* b,
                       const uint8_t* b_scales, const int32_t* offsets, void* out, void* stream) {
  Range r("zero_scaled_matmul");
  if (d == nullptr) return fail(ZERO_ERR_INVALID, "desc is NULL");
  if (d->rows < 0 || d->rows > kMaxIndex)
    return fail(ZERO_ERR_INVALID, "%lld rows out of range", (long long)d->rows);
  if (d->n < 1 || d->n > kMaxDim || d->k < 1 || d->k > kMaxDim)
    return fail(ZERO_ERR_INVALID, "n %lld or k %lld out of range", (long long)d->n, (long long)d->k);
  if (d->experts < 0 || d->experts > kMaxExperts)
    return fail(ZERO_ERR_INVALID, "%d experts: 0 to %d", d->experts, kMaxExperts);
  if (!valid_dtype(d->out_dtype)) return fail(ZERO_ERR_INVALID, "bad out_dtype %d", d->out_dtype);
  if (d->accumulate && d->out_dtype != ZERO_F32) return fail(ZERO_ERR_INVALID, "accumulate needs an fp32 out");
  if (int rc = check_stride(d->out_stride, d->n, "out_stride")) return rc;
  if (d->experts == 0 && offsets != nullptr) return fail(ZERO_ERR_INVALID, "offsets without experts");
  if (d->rows == 0) return ZERO_OK;
  NEED(a);
  NEED(a_scales);
  NEED(b);
  NEED(b_scales);
  NEED_ELEMENTS(out, d->out_dtype);
  if (d->experts > 0) NEED(offsets);
  const int groups = d->experts > 0 ? d->experts : 1;
  const ScaledArgs s = scaled_args(1, d->rows, d->k);
  const Buffer all[] = {buffer(out, d->rows, d->n, d->out_stride, dtype_bytes(d->out_dtype), "out"),
                        {a, d->rows * s.pitch, "a"},
                        {a_scales, d->rows * s.scale_pitch, "a_scales"},
                        {b, groups * d->n * s.pitch, "b"},
                        {b_scales, groups * d->n * s.scale_pitch, "b_scales"},
                        {offsets, (d->experts + 1) * 4ll, "offsets"}};
  if (int rc = check_apart(all, 1)) return rc;
  ProductArgs p{};
  p.a = b;
  p.b = a;
  p.a_scales = b_scales;
  p.b_scales = a_scales;
  p.out = out;
  p.m = d->n;
  p.n = d->rows;
  p.k = d->k;
  p.a_group = d->n * s.pitch;
  p.a_row = p.b_row = s.pitch;
  p.scale_pitch = s.scale_pitch;
  p.out_row = d->out_stride;
  p.groups = groups;
  p.offsets = offsets;
  p.dtype = kE4M3;
  p.out_dtype = d->out_dtype;
  p.accumulate = d->accumulate != 0;
  return launch(p, "scaled product launch", stream);
}

}  // extern "C"
