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
HALF = (torch.float16, torch.bfloat16)
_F32 = torch.float32
_raw_stream = torch._C._cuda_getCurrentRawStream  # without building a Stream object


def _stream(stream, *tensors):
    """(the handle to launch on, `stream` if it is not torch's current one, else
    None). All tensors (None: absent) must be on the current device."""
    index = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors on {tensors[0].device} and {t.device}")
    if index < 0 or index != torch.cuda.current_device():
        raise ValueError(f"tensors must be on the current CUDA device, got {tensors[0].device}")
    handle = _raw_stream(index)
    if stream is None or stream.cuda_stream == handle:
        return handle, None
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return stream.cuda_stream, stream


def _empty(side, shape, dtype, device):
    if side is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(side):
        return torch.empty(shape, dtype=dtype, device=device)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _rows(t, name, shape, dtype) -> int:
    """The row stride of a [rows, cols] tensor whose rows are contiguous."""
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name}: expected {tuple(shape)} of {dtype}, got {tuple(t.shape)} of {t.dtype}")
    step, inner = t.stride()
    if inner != 1 and shape[1] > 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    return step if shape[0] > 1 else shape[1]


def _given(t, name, shape, dtype) -> None:
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {tuple(shape)} of {dtype}, got "
                         f"{tuple(t.shape)} of {t.dtype}")


def _matrix(x, name) -> None:
    if x.dim() != 2 or x.dtype not in DTYPE_CODE:
        raise ValueError(f"{name}: expected [rows, cols] of fp32, fp16 or bf16, got {tuple(x.shape)} of {x.dtype}")


def _weight(weight, cols) -> None:
    if weight.dtype not in DTYPE_CODE or weight.shape != (cols,) or not weight.is_contiguous():
        raise ValueError(f"weight: expected a contiguous [{cols}]")


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
        if rows < 0 or cols < 1:
            raise ValueError(f"a packed activation of {rows} x {cols}")
        pitch = (cols + 127) // 128 * 128
        self.rows, self.cols = rows, cols
        if q is None:
            q = _empty(stream, (rows, pitch), torch.int8, device)
            scales = _empty(stream, (rows, pitch // 32), torch.uint8, device)
        else:
            _given(q, "q", (rows, pitch), torch.int8)
            if scales is None:
                raise ValueError("q without scales")
            _given(scales, "scales", (rows, pitch // 32), torch.uint8)
        self.q, self.scales = q, scales

    def save(self, x: torch.Tensor, stream=None) -> "PackedActivation":
        """Pack x [rows, cols] (fp32, fp16 or bf16; its row stride is free)."""
        _matrix(x, "x")
        step = _rows(x, "x", (self.rows, self.cols), x.dtype)
        handle, _ = _stream(stream, x, self.q, self.scales)
        abi.zero_act_pack(x.data_ptr(), step, self.rows, self.cols, DTYPE_CODE[x.dtype],
                          self.q.data_ptr(), self.scales.data_ptr(), handle)
        return self

    def restore(self, dtype: torch.dtype | None = None, out=None, stream=None) -> torch.Tensor:
        """The activation's values in `dtype` (default: out's, or bf16)."""
        if dtype is None:
            dtype = out.dtype if out is not None else torch.bfloat16
        if dtype not in DTYPE_CODE:
            raise ValueError(f"unsupported type {dtype}")
        handle, side = _stream(stream, self.q, self.scales, out)
        step = self.cols
        if out is None:
            out = _empty(side, (self.rows, self.cols), dtype, self.q.device)
        else:
            step = _rows(out, "out", (self.rows, self.cols), dtype)
        abi.zero_act_unpack(self.q.data_ptr(), self.scales.data_ptr(), self.rows, self.cols,
                            out.data_ptr(), step, DTYPE_CODE[dtype], handle)
        return out


def weight_grad(dy: torch.Tensor, packed: PackedActivation, out=None, dtype=None,
                accumulate: bool = False, stream=None) -> torch.Tensor:
    """dw [n_out, n_in] = dy^T X of a linear layer y = x W^T, X the packed
    input restored in dy's type (fp16 or bf16).

    dy [tokens, n_out]: its row stride is a multiple of 8 elements. dw is fp32
    or dy's type (`dtype`; default out's, or dy's). `accumulate` adds to an
    fp32 `out` (main gradients over micro-batches)."""
    if dy.dim() != 2 or dy.shape[0] != packed.rows or dy.dtype not in HALF:
        raise ValueError(f"dy: expected [{packed.rows}, n_out] of fp16 or bf16, got {tuple(dy.shape)} of {dy.dtype}")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    tokens, n_out = dy.shape
    step, inner = dy.stride()
    if inner != 1 and n_out > 1:
        raise ValueError("dy: the elements of a row must be contiguous")
    if tokens <= 1:
        step = (n_out + 7) // 8 * 8
    if dtype is None:
        dtype = out.dtype if out is not None else dy.dtype
    if dtype not in DTYPE_CODE:
        raise ValueError(f"unsupported type {dtype}")
    handle, side = _stream(stream, dy, packed.q, packed.scales, out)
    if out is None:
        out = _empty(side, (n_out, packed.cols), dtype, dy.device)
    else:
        _given(out, "out", (n_out, packed.cols), dtype)
    abi.zero_act_weight_grad(dy.data_ptr(), step, DTYPE_CODE[dy.dtype], packed.q.data_ptr(),
                             packed.scales.data_ptr(), tokens, n_out, packed.cols, out.data_ptr(),
                             DTYPE_CODE[dtype], accumulate, None, 0, handle)
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
    _matrix(x, "x")
    shape, dtype = x.shape, x.dtype
    rows, cols = shape
    x_step = _rows(x, "x", shape, dtype)
    r_step = cols if residual is None else _rows(residual, "residual", shape, dtype)
    _weight(weight, cols)
    q = scales = None
    if packed is not None:
        if packed.rows != rows or packed.cols != cols:
            raise ValueError(f"packed: {packed.rows} x {packed.cols} for x of {rows} x {cols}")
        q, scales = packed.q, packed.scales
    handle, side = _stream(stream, x, weight, residual, out, sum_out, rstd, q, scales)
    if not want_out:
        if out is not None or packed is None:
            raise ValueError("want_out=False goes with packed and without out")
    elif out is None:
        out = _empty(side, shape, dtype, x.device)
    else:
        _given(out, "out", shape, dtype)
    if residual is None:
        if sum_out is not None:
            raise ValueError("sum_out without a residual")
    elif sum_out is None:
        sum_out = _empty(side, shape, dtype, x.device)
    else:
        _given(sum_out, "sum_out", shape, dtype)
    if rstd is None:
        rstd = _empty(side, (rows,), _F32, x.device)
    else:
        _given(rstd, "rstd", (rows,), _F32)
    desc = abi.zero_rmsnorm_desc(rows, cols, x_step, r_step, cols, DTYPE_CODE[dtype],
                                 DTYPE_CODE[weight.dtype], eps)
    abi.zero_rmsnorm_forward(desc, x.data_ptr(), _ptr(residual), weight.data_ptr(), _ptr(sum_out),
                             _ptr(out), _ptr(q), _ptr(scales), rstd.data_ptr(), handle)
    return out, (x if residual is None else sum_out), rstd


def rmsnorm_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                     dsum=None, dx=None, dweight=None, dweight_dtype=None, stream=None):
    """(dx, dweight) from dy [rows, cols], the forward's s as `x`, and rstd. dx
    is the gradient of x and of the residual; dsum, the gradient that reaches
    s by its other use, is added to it. dweight: fp32 sums stored as
    dweight_dtype (default: dweight's type, or weight's)."""
    _matrix(x, "x")
    shape, dtype = x.shape, x.dtype
    rows, cols = shape
    x_step = _rows(x, "x", shape, dtype)
    dy_step = _rows(dy, "dy", shape, dtype)
    r_step = cols if dsum is None else _rows(dsum, "dsum", shape, dtype)
    _weight(weight, cols)
    _given(rstd, "rstd", (rows,), _F32)
    if dweight_dtype is None:
        dweight_dtype = dweight.dtype if dweight is not None else weight.dtype
    if dweight_dtype not in DTYPE_CODE:
        raise ValueError(f"unsupported type {dweight_dtype}")
    handle, side = _stream(stream, x, dy, weight, rstd, dsum, dx, dweight)
    if dx is None:
        dx = _empty(side, shape, dtype, x.device)
    else:
        _given(dx, "dx", shape, dtype)
    if dweight is None:
        dweight = _empty(side, (cols,), dweight_dtype, x.device)
    else:
        _given(dweight, "dweight", (cols,), dweight_dtype)
    desc = abi.zero_rmsnorm_desc(rows, cols, x_step, r_step, dy_step, DTYPE_CODE[dtype],
                                 DTYPE_CODE[weight.dtype], 0.0)
    nbytes = abi.zero_rmsnorm_backward_workspace(desc)
    space = _empty(side, nbytes, torch.uint8, x.device) if nbytes else None
    abi.zero_rmsnorm_backward(desc, dy.data_ptr(), x.data_ptr(), weight.data_ptr(), rstd.data_ptr(),
                              _ptr(dsum), dx.data_ptr(), dweight.data_ptr(),
                              DTYPE_CODE[dweight_dtype], _ptr(space), nbytes, handle)
    return dx, dweight


# ---------------------------------------------------------------------------
# Attention's training pair
# ---------------------------------------------------------------------------


def _steps(t, name, shape, dtype):
    """{batch, token, head} strides of a [batch, length, heads, head_dim] tensor."""
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name}: expected {tuple(shape)} of {dtype}, got {tuple(t.shape)} of {t.dtype}")
    steps = t.stride()
    if steps[3] != 1:
        raise ValueError(f"{name}: the elements of a head must be contiguous")
    return steps[:3]


def _attention_sizes(q, k, causal, window, key_lengths, scale):
    """The leading fields of the call's descriptor, and the shape of k and v."""
    if q.dim() != 4 or k.dim() != 4 or q.dtype not in HALF:
        raise ValueError("q, k, v: expected [batch, length, heads, head_dim] of fp16 or bf16, got "
                         f"{tuple(q.shape)} and {tuple(k.shape)} of {q.dtype}")
    batch, q_len, q_heads, dim = q.shape
    _, k_len, kv_heads, _ = k.shape
    if key_lengths is not None:
        _given(key_lengths, "key_lengths", (batch,), torch.int32)
    sizes = (batch, q_len, k_len, q_heads, kv_heads, dim, DTYPE_CODE[q.dtype], causal, 0, window,
             dim ** -0.5 if scale is None else scale)
    return sizes, (batch, k_len, kv_heads, dim)


def _like(t, side, ref, name):
    """The given output, or a new contiguous one of ref's shape; its strides."""
    if t is None:
        t = _empty(side, ref.shape, ref.dtype, ref.device)
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
    sizes, shape = _attention_sizes(q, k, causal, window, key_lengths, scale)
    dtype = q.dtype
    q_steps, k_steps, v_steps = _steps(q, "q", q.shape, dtype), _steps(k, "k", shape, dtype), _steps(v, "v", shape, dtype)
    handle, side = _stream(stream, q, k, v, key_lengths, out, lse)
    out, o_steps = _like(out, side, q, "out")
    rows = (sizes[0], sizes[3], sizes[1])
    if lse is None:
        lse = _empty(side, rows, _F32, q.device)
    else:
        _given(lse, "lse", rows, _F32)
    desc = abi.attention_desc_flat(*sizes, *q_steps, *k_steps, *v_steps, *o_steps)
    abi.zero_attention_forward(desc, q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(key_lengths),
                               out.data_ptr(), lse.data_ptr(), handle)
    return out, lse


def attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                       o: torch.Tensor, lse: torch.Tensor, causal: bool = False, window: int = 0,
                       key_lengths=None, scale: float | None = None, dq=None, dk=None, dv=None,
                       stream=None):
    """(dq, dk, dv) from dout, the forward's tensors and the same mask; the
    probabilities are recomputed from lse. dk and dv are summed over the query
    heads that share a key head."""
    sizes, shape = _attention_sizes(q, k, causal, window, key_lengths, scale)
    dtype, q_shape = q.dtype, q.shape
    steps = (*_steps(q, "q", q_shape, dtype), *_steps(k, "k", shape, dtype), *_steps(v, "v", shape, dtype),
             *_steps(o, "o", q_shape, dtype), *_steps(dout, "dout", q_shape, dtype))
    _given(lse, "lse", (sizes[0], sizes[3], sizes[1]), _F32)
    handle, side = _stream(stream, q, k, v, o, dout, lse, key_lengths, dq, dk, dv)
    dq, dq_steps = _like(dq, side, q, "dq")
    dk, dk_steps = _like(dk, side, k, "dk")
    dv, dv_steps = _like(dv, side, v, "dv")
    desc = abi.attention_desc_flat(*sizes, *steps, *dq_steps, *dk_steps, *dv_steps)
    nbytes = abi.zero_attention_backward_workspace(desc)
    space = _empty(side, nbytes, torch.uint8, q.device) if nbytes else None
    abi.zero_attention_backward(desc, dout.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                o.data_ptr(), lse.data_ptr(), _ptr(key_lengths), dq.data_ptr(),
                                dk.data_ptr(), dv.data_ptr(), _ptr(space), nbytes, handle)
    return dq, dk, dv


def check(stream=None) -> None:
    """Raise ZeroError(ZERO_ERR_TIMEOUT) if a kernel of this module gave up a
    bounded wait since the last check. Synchronises the stream."""
    abi.zero_operator_status((stream or torch.cuda.current_stream()).cuda_stream)
