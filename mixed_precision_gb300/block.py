"""Operators of a transformer block's forward and backward, on torch tensors.

Each function checks its tensors, allocates what the caller did not pass, and
makes one call of the C ABI (mixed_precision_gb300._abi); every computation is
in the library's CUDA kernels. Work is enqueued on `stream` (default: torch's
current stream) and nothing waits. With a `stream` that is not the current
one, outputs and scratch are allocated on it and the inputs are marked as used
on it, so the caching allocator reuses none of them too early; ordering the
streams' work stays the caller's job, as with any torch operation.

Wrong shapes, types, devices or layouts raise ValueError here, or ZeroError
(ZERO_ERR_INVALID) from the library; nothing is enqueued then.
"""
from __future__ import annotations

import torch

from . import _abi as abi

DTYPE_CODE = {torch.float32: abi.ZERO_F32, torch.float16: abi.ZERO_F16,
              torch.bfloat16: abi.ZERO_BF16}


def _need(ok, message: str) -> None:
    if not ok:
        raise ValueError(message)


class _On:
    """The stream of one call: its handle, and allocations that belong to it."""

    __slots__ = ("stream", "handle", "other")

    def __init__(self, stream, tensors):
        device = tensors[0].device
        if device.type != "cuda" or device.index != torch.cuda.current_device():
            raise ValueError(f"tensors must be on the current CUDA device, got {device}")
        for t in tensors:
            if t is not None and t.device != device:
                raise ValueError(f"tensors on {device} and {t.device}")
        current = torch.cuda.current_stream()
        self.stream = current if stream is None else stream
        self.handle = self.stream.cuda_stream
        self.other = self.handle != current.cuda_stream
        if self.other:
            for t in tensors:
                if t is not None:
                    t.record_stream(self.stream)

    def empty(self, shape, dtype, device):
        if not self.other:
            return torch.empty(shape, dtype=dtype, device=device)
        with torch.cuda.stream(self.stream):
            return torch.empty(shape, dtype=dtype, device=device)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _rows(t, name, shape, dtype):
    """The row stride of a [rows, cols] tensor whose rows are contiguous."""
    _need(t.shape == shape and t.dtype == dtype,
          f"{name}: expected {tuple(shape)} of {dtype}, got {tuple(t.shape)} of {t.dtype}")
    step, inner = t.stride()
    _need(inner == 1 or shape[1] <= 1, f"{name}: the elements of a row must be contiguous")
    return step if shape[0] > 1 else shape[1]


def _out(t, on, name, shape, dtype, device):
    if t is None:
        return on.empty(shape, dtype, device)
    _need(tuple(t.shape) == tuple(shape) and t.dtype == dtype and t.is_contiguous(),
          f"{name}: expected a contiguous {tuple(shape)} of {dtype}, got {tuple(t.shape)} of {t.dtype}")
    return t


# ---------------------------------------------------------------------------
# Packed activations
# ---------------------------------------------------------------------------

class PackedActivation:
    """A [rows, cols] activation held in 8 bits: int8 codes ``q`` [rows, pitch]
    and one power-of-two scale for each 32 elements, ``scales`` [rows, pitch / 32]
    (1.03 bytes per element). ``save`` fills it in the forward pass (or
    rmsnorm_forward does, with its output); ``restore`` and ``weight_grad`` use
    it in the backward pass."""

    __slots__ = ("rows", "cols", "q", "scales")

    def __init__(self, rows: int, cols: int, q=None, scales=None, device="cuda", stream=None):
        _need(rows >= 0 and cols >= 1, f"a packed activation of {rows} x {cols}")
        pitch = (cols + 127) // 128 * 128
        self.rows, self.cols = rows, cols
        if q is None:
            on = torch.cuda.stream(stream) if stream is not None else None
            if on is not None:
                on.__enter__()
            try:
                q = torch.empty((rows, pitch), dtype=torch.int8, device=device)
                scales = torch.empty((rows, pitch // 32), dtype=torch.uint8, device=device)
            finally:
                if on is not None:
                    on.__exit__(None, None, None)
        _need(q.dtype == torch.int8 and q.shape == (rows, pitch) and q.is_contiguous(),
              f"q: expected a contiguous int8 [{rows}, {pitch}]")
        _need(scales is not None and scales.dtype == torch.uint8 and scales.is_contiguous()
              and scales.shape == (rows, pitch // 32),
              f"scales: expected a contiguous uint8 [{rows}, {pitch // 32}]")
        self.q, self.scales = q, scales

    def save(self, x: torch.Tensor, stream=None) -> "PackedActivation":
        """Pack x [rows, cols] (fp32, fp16 or bf16; its row stride is free)."""
        _need(x.dtype in DTYPE_CODE, f"x: unsupported type {x.dtype}")
        step = _rows(x, "x", (self.rows, self.cols), x.dtype)
        on = _On(stream, (x, self.q, self.scales))
        abi.zero_act_pack(x.data_ptr(), step, self.rows, self.cols, DTYPE_CODE[x.dtype],
                          self.q.data_ptr(), self.scales.data_ptr(), on.handle)
        return self

    def restore(self, dtype: torch.dtype | None = None, out=None, stream=None) -> torch.Tensor:
        """The activation's values in `dtype` (default: out's, or bf16)."""
        if dtype is None:
            dtype = out.dtype if out is not None else torch.bfloat16
        _need(dtype in DTYPE_CODE, f"unsupported type {dtype}")
        on = _On(stream, (self.q, self.scales, out))
        if out is None:
            out = on.empty((self.rows, self.cols), dtype, self.q.device)
        step = _rows(out, "out", (self.rows, self.cols), dtype)
        abi.zero_act_unpack(self.q.data_ptr(), self.scales.data_ptr(), self.rows, self.cols,
                            out.data_ptr(), step, DTYPE_CODE[dtype], on.handle)
        return out


def weight_grad(dy: torch.Tensor, packed: PackedActivation, out=None, dtype=None,
                accumulate: bool = False, stream=None) -> torch.Tensor:
    """dw [n_out, n_in] = dy^T X of a linear layer y = x W^T, X the packed
    input restored in dy's type (fp16 or bf16).

    dy [tokens, n_out]: its row stride is a multiple of 8 elements. dw is fp32
    or dy's type (`dtype`; default out's, or dy's). `accumulate` adds to an
    fp32 `out` (main gradients over micro-batches)."""
    _need(dy.dim() == 2 and dy.shape[0] == packed.rows,
          f"dy: expected [{packed.rows}, n_out], got {tuple(dy.shape)}")
    _need(dy.dtype in (torch.float16, torch.bfloat16), f"dy: unsupported type {dy.dtype}")
    _need(not accumulate or out is not None, "accumulate needs out")
    tokens, n_out = dy.shape
    step = dy.stride(0) if tokens > 1 else (n_out + 7) // 8 * 8
    _need(dy.stride(1) == 1 or n_out <= 1, "dy: the elements of a row must be contiguous")
    if dtype is None:
        dtype = out.dtype if out is not None else dy.dtype
    _need(dtype in DTYPE_CODE, f"unsupported type {dtype}")
    on = _On(stream, (dy, packed.q, packed.scales, out))
    out = _out(out, on, "out", (n_out, packed.cols), dtype, dy.device)
    nbytes = abi.zero_act_weight_grad_workspace(tokens, n_out, packed.cols)
    space = on.empty(nbytes, torch.uint8, dy.device) if nbytes else None
    abi.zero_act_weight_grad(dy.data_ptr(), step, DTYPE_CODE[dy.dtype], packed.q.data_ptr(),
                             packed.scales.data_ptr(), tokens, n_out, packed.cols, out.data_ptr(),
                             DTYPE_CODE[dtype], accumulate, _ptr(space), nbytes, on.handle)
    return out


# ---------------------------------------------------------------------------
# RMSNorm with the residual's addition
# ---------------------------------------------------------------------------

def rmsnorm_forward(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual=None, out=None,
                    sum_out=None, rstd=None, packed: PackedActivation | None = None,
                    want_out: bool = True, stream=None):
    """(y, s, rstd) of x [rows, cols]: s = x + residual (x itself without one),
    y = s * rstd * weight, rstd = (mean(s^2) + eps)^(-1/2) in fp32.

    `packed` also receives y in 8 bits, from the same pass; with want_out=False
    y is not written (returned as None). sum_out may be x or residual itself."""
    _need(x.dim() == 2 and x.dtype in DTYPE_CODE, f"x: expected [rows, cols], got {tuple(x.shape)} of {x.dtype}")
    rows, cols = x.shape
    x_step = _rows(x, "x", x.shape, x.dtype)
    r_step = cols if residual is None else _rows(residual, "residual", x.shape, x.dtype)
    _need(weight.dtype in DTYPE_CODE and weight.shape == (cols,) and weight.is_contiguous(),
          f"weight: expected a contiguous [{cols}]")
    _need(want_out or packed is not None, "want_out=False needs packed")
    q = scales = None
    if packed is not None:
        _need(packed.rows == rows and packed.cols == cols,
              f"packed: {packed.rows} x {packed.cols} for x of {rows} x {cols}")
        q, scales = packed.q, packed.scales
    on = _On(stream, (x, weight, residual, out, sum_out, rstd, q, scales))
    if want_out:
        out = _out(out, on, "out", x.shape, x.dtype, x.device)
    else:
        _need(out is None, "out with want_out=False")
    if residual is not None:
        sum_out = _out(sum_out, on, "sum_out", x.shape, x.dtype, x.device)
    else:
        _need(sum_out is None, "sum_out without a residual")
    rstd = _out(rstd, on, "rstd", (rows,), torch.float32, x.device)
    desc = abi.zero_rmsnorm_desc(rows, cols, x_step, r_step, cols, DTYPE_CODE[x.dtype],
                                 DTYPE_CODE[weight.dtype], eps)
    abi.zero_rmsnorm_forward(desc, x.data_ptr(), _ptr(residual), weight.data_ptr(), _ptr(sum_out),
                             _ptr(out), _ptr(q), _ptr(scales), rstd.data_ptr(), on.handle)
    return out, (x if residual is None else sum_out), rstd


def rmsnorm_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                     dsum=None, dx=None, dweight=None, dweight_dtype=None, stream=None):
    """(dx, dweight) from dy [rows, cols], the forward's s as `x`, and rstd. dx
    is the gradient of x and of the residual; dsum, the gradient that reaches
    s by its other use, is added to it. dweight: fp32 sums stored as
    dweight_dtype (default: dweight's type, or weight's)."""
    _need(x.dim() == 2 and x.dtype in DTYPE_CODE, f"x: expected [rows, cols], got {tuple(x.shape)} of {x.dtype}")
    rows, cols = x.shape
    x_step = _rows(x, "x", x.shape, x.dtype)
    dy_step = _rows(dy, "dy", x.shape, x.dtype)
    r_step = cols if dsum is None else _rows(dsum, "dsum", x.shape, x.dtype)
    _need(weight.dtype in DTYPE_CODE and weight.shape == (cols,) and weight.is_contiguous(),
          f"weight: expected a contiguous [{cols}]")
    _need(rstd.dtype == torch.float32 and rstd.shape == (rows,) and rstd.is_contiguous(),
          f"rstd: expected a contiguous fp32 [{rows}]")
    if dweight_dtype is None:
        dweight_dtype = dweight.dtype if dweight is not None else weight.dtype
    _need(dweight_dtype in DTYPE_CODE, f"unsupported type {dweight_dtype}")
    on = _On(stream, (x, dy, weight, rstd, dsum, dx, dweight))
    dx = _out(dx, on, "dx", x.shape, x.dtype, x.device)
    dweight = _out(dweight, on, "dweight", (cols,), dweight_dtype, x.device)
    desc = abi.zero_rmsnorm_desc(rows, cols, x_step, r_step, dy_step, DTYPE_CODE[x.dtype],
                                 DTYPE_CODE[weight.dtype], 0.0)
    nbytes = abi.zero_rmsnorm_backward_workspace(desc)
    space = on.empty(nbytes, torch.uint8, x.device) if nbytes else None
    abi.zero_rmsnorm_backward(desc, dy.data_ptr(), x.data_ptr(), weight.data_ptr(), rstd.data_ptr(),
                              _ptr(dsum), dx.data_ptr(), dweight.data_ptr(),
                              DTYPE_CODE[dweight_dtype], _ptr(space), nbytes, on.handle)
    return dx, dweight


# ---------------------------------------------------------------------------
# Attention's training pair
# ---------------------------------------------------------------------------

def _steps(t, name, shape, dtype):
    """{batch, token, head} strides of a [batch, length, heads, head_dim] tensor."""
    _need(t.shape == shape and t.dtype == dtype,
          f"{name}: expected {tuple(shape)} of {dtype}, got {tuple(t.shape)} of {t.dtype}")
    b, s, h, inner = t.stride()
    _need(inner == 1, f"{name}: the elements of a head must be contiguous")
    return b, s, h


def _attention_desc(q, k, v, causal, window, key_lengths, scale):
    _need(q.dim() == 4 and k.dim() == 4, "q, k, v: expected [batch, length, heads, head_dim]")
    batch, q_len, q_heads, dim = q.shape
    k_len, kv_heads = k.shape[1], k.shape[2]
    _need(q.dtype in (torch.float16, torch.bfloat16), f"q: unsupported type {q.dtype}")
    if key_lengths is not None:
        _need(key_lengths.dtype == torch.int32 and key_lengths.shape == (batch,)
              and key_lengths.is_contiguous(), f"key_lengths: expected a contiguous int32 [{batch}]")
    shape = (batch, k_len, kv_heads, dim)
    d = abi.zero_attention_desc(batch, q_len, k_len, q_heads, kv_heads, dim, DTYPE_CODE[q.dtype],
                                causal, 0, window, dim ** -0.5 if scale is None else scale)
    d.q_strides = _steps(q, "q", q.shape, q.dtype)
    d.k_strides = _steps(k, "k", shape, q.dtype)
    d.v_strides = _steps(v, "v", shape, q.dtype)
    return d


def _like(t, on, ref, name):
    """The given output, or a new contiguous one of ref's shape; its strides."""
    if t is None:
        t = on.empty(ref.shape, ref.dtype, ref.device)
    return t, _steps(t, name, ref.shape, ref.dtype)


def attention_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False,
                      window: int = 0, key_lengths=None, scale: float | None = None, out=None, lse=None,
                      stream=None):
    """(o, lse) of q [batch, q_len, q_heads, head_dim] and k, v [batch, k_len,
    kv_heads, head_dim] (fp16 or bf16; strides are free multiples of 8).

    Query i sees key j when j < key_lengths[b], j <= i + k_len - q_len
    (`causal`) and j > i + k_len - q_len - window (`window` > 0). A query that
    sees no key has o = 0 and lse = -inf. scale: default head_dim^-1/2. lse is
    fp32 [batch, q_heads, q_len]."""
    d = _attention_desc(q, k, v, causal, window, key_lengths, scale)
    on = _On(stream, (q, k, v, key_lengths, out, lse))
    out, d.o_strides = _like(out, on, q, "out")
    lse = _out(lse, on, "lse", (q.shape[0], q.shape[2], q.shape[1]), torch.float32, q.device)
    abi.zero_attention_forward(d, q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(key_lengths),
                               out.data_ptr(), lse.data_ptr(), on.handle)
    return out, lse


def attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                       o: torch.Tensor, lse: torch.Tensor, causal: bool = False, window: int = 0,
                       key_lengths=None, scale: float | None = None, dq=None, dk=None, dv=None,
                       stream=None):
    """(dq, dk, dv) from dout, the forward's tensors and the same mask; the
    probabilities are recomputed from lse. dk and dv are summed over the query
    heads that share a key head."""
    d = _attention_desc(q, k, v, causal, window, key_lengths, scale)
    d.o_strides = _steps(o, "o", q.shape, q.dtype)
    d.do_strides = _steps(dout, "dout", q.shape, q.dtype)
    _need(lse.dtype == torch.float32 and lse.is_contiguous()
          and lse.shape == (q.shape[0], q.shape[2], q.shape[1]), "lse: expected the forward's")
    on = _On(stream, (q, k, v, o, dout, lse, key_lengths, dq, dk, dv))
    dq, d.dq_strides = _like(dq, on, q, "dq")
    dk, d.dk_strides = _like(dk, on, k, "dk")
    dv, d.dv_strides = _like(dv, on, v, "dv")
    nbytes = abi.zero_attention_backward_workspace(d)
    space = on.empty(nbytes, torch.uint8, q.device) if nbytes else None
    abi.zero_attention_backward(d, dout.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                o.data_ptr(), lse.data_ptr(), _ptr(key_lengths), dq.data_ptr(),
                                dk.data_ptr(), dv.data_ptr(), _ptr(space), nbytes, on.handle)
    return dq, dk, dv


def check(stream=None) -> None:
    """Raise ZeroError(ZERO_ERR_TIMEOUT) if a kernel of this module gave up a
    bounded wait since the last check. Synchronises the stream."""
    abi.zero_operator_status((stream or torch.cuda.current_stream()).cuda_stream)
