"""Operators of a transformer block's forward and backward, on torch tensors.

Each function checks its tensors, allocates what the caller did not pass, and
makes one call of the C ABI (mixed_precision_gb300._abi); every computation is
in the library's CUDA kernels. Work is enqueued on `stream` (default: torch's
current stream) and nothing waits. With a `stream` that is not the current
one, outputs and scratch are allocated on it and the inputs are marked as used
on it, so the caching allocator reuses none of them too early; ordering the
streams' work stays the caller's job, as with any torch operation.

Nothing is recorded for autograd: the results carry no graph, also where an
input requires a gradient, and the gradients come from the backward functions
(called by hand, or in a torch.autograd.Function of the caller's).

Wrong shapes, types, devices or layouts raise ValueError here, or ZeroError
(ZERO_ERR_INVALID) from the library; nothing is enqueued then.

The checks are written out in each function and the library's entry points
called directly: at a few microseconds a kernel, helper calls would be a good
part of a short call's time.
"""
from __future__ import annotations

import functools

import torch

from . import _abi as abi

DTYPE_CODE = {torch.float32: abi.ZERO_F32, torch.float16: abi.ZERO_F16,
              torch.bfloat16: abi.ZERO_BF16}
HALF_CODE = {torch.float16: abi.ZERO_F16, torch.bfloat16: abi.ZERO_BF16}
_F32 = torch.float32
_empty = torch.empty
_current_device = torch._C._cuda_getDevice
_norm_desc, _attention_desc = abi.RMSNORM_DESC.pack, abi.ATTENTION_DESC.pack
_raw_stream = torch._C._cuda_getCurrentRawStream  # without building a Stream object


def _stream(stream, tensors):
    """(the handle to launch on, `stream` if it is not torch's current one, else
    None). All tensors (None: absent) must be on the current device."""
    index = _current_device()
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors must be on the current CUDA device {index}, got {t.device}")
    handle = _raw_stream(index)
    if stream is None or stream.cuda_stream == handle:
        return handle, None
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return stream.cuda_stream, stream


def _new(side, shape, dtype, device):
    """A new tensor, of the side stream if the call has one."""
    if side is None:
        return _empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(side):
        return _empty(shape, dtype=dtype, device=device)


def _library():
    """The loaded library (abi.lib(), without the call once it is loaded)."""
    return abi._lib or abi.lib()


def _got(name, t, want):
    return ValueError(f"{name}: expected {want}, got {tuple(t.shape)} of {t.dtype}, strides {t.stride()}")


def _row_step(t, name, shape, dtype) -> int:
    """The row stride of a [rows, cols] tensor whose rows are contiguous."""
    step, inner = t.stride() if t.dim() == 2 else (0, 0)
    if t.shape != shape or t.dtype is not dtype or (inner != 1 and shape[1] > 1):
        raise _got(name, t, f"{tuple(shape)} of {dtype} with contiguous rows")
    return step if shape[0] > 1 else shape[1]


def _given(t, name, shape, dtype) -> None:
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous():
        raise _got(name, t, f"a contiguous {tuple(shape)} of {dtype}")


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
            q = _new(stream, (rows, pitch), torch.int8, device)
            scales = _new(stream, (rows, pitch // 32), torch.uint8, device)
        else:
            _given(q, "q", (rows, pitch), torch.int8)
            if scales is None:
                raise ValueError("q without scales")
            _given(scales, "scales", (rows, pitch // 32), torch.uint8)
        self.q, self.scales = q, scales

    def save(self, x: torch.Tensor, stream=None) -> "PackedActivation":
        """Pack x [rows, cols] (fp32, fp16 or bf16; its row stride is free)."""
        dtype, q, scales = x.dtype, self.q, self.scales
        code = DTYPE_CODE.get(dtype)
        if code is None:
            raise _got("x", x, "fp32, fp16 or bf16")
        step = _row_step(x, "x", (self.rows, self.cols), dtype)
        handle, _ = _stream(stream, (x, q, scales))
        rc = _library().zero_act_pack(x.data_ptr(), step, self.rows, self.cols, code, q.data_ptr(), scales.data_ptr(),
                                      handle)
        if rc:
            abi._check(rc)
        return self

    def restore(self, dtype: torch.dtype | None = None, out=None, stream=None) -> torch.Tensor:
        """The activation's values in `dtype` (default: out's, or bf16)."""
        if dtype is None:
            dtype = out.dtype if out is not None else torch.bfloat16
        code, q, scales, rows, cols = DTYPE_CODE.get(dtype), self.q, self.scales, self.rows, self.cols
        if code is None:
            raise ValueError(f"unsupported type {dtype}")
        step = cols if out is None else _row_step(out, "out", (rows, cols), dtype)
        handle, side = _stream(stream, (q, scales, out))
        if out is None:
            out = _new(side, (rows, cols), dtype, q.device)
        rc = _library().zero_act_unpack(q.data_ptr(), scales.data_ptr(), rows, cols, out.data_ptr(), step, code, handle)
        if rc:
            abi._check(rc)
        return out


def weight_grad(dy: torch.Tensor, packed: PackedActivation, out=None, dtype=None,
                accumulate: bool = False, stream=None) -> torch.Tensor:
    """dw [n_out, n_in] = dy^T X of a linear layer y = x W^T, X the packed
    input restored in dy's type (fp16 or bf16).

    dy [tokens, n_out]: its row stride is a multiple of 8 elements. dw is fp32
    or dy's type (`dtype`; default out's, or dy's). `accumulate` adds to an
    fp32 `out` (main gradients over micro-batches)."""
    code, q, scales, cols = HALF_CODE.get(dy.dtype), packed.q, packed.scales, packed.cols
    if code is None or dy.dim() != 2 or dy.shape[0] != packed.rows:
        raise _got("dy", dy, f"[{packed.rows}, n_out] of fp16 or bf16")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    tokens, n_out = dy.shape
    step, inner = dy.stride()
    if inner != 1 and n_out > 1:
        raise _got("dy", dy, "contiguous rows")
    if tokens <= 1:
        step = (n_out + 7) // 8 * 8
    if dtype is None:
        dtype = out.dtype if out is not None else dy.dtype
    if dtype not in DTYPE_CODE:
        raise ValueError(f"unsupported type {dtype}")
    handle, side = _stream(stream, (dy, q, scales, out))
    if out is None:
        out = _new(side, (n_out, cols), dtype, q.device)
    else:
        _given(out, "out", (n_out, cols), dtype)
    rc = _library().zero_act_weight_grad(dy.data_ptr(), step, code, q.data_ptr(), scales.data_ptr(), tokens, n_out,
                                         cols, out.data_ptr(), DTYPE_CODE[dtype], accumulate, None, 0, handle)
    if rc:
        abi._check(rc)
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
    y is not written (returned as None). sum_out may be x or residual itself, out
    too if it is not sum_out."""
    shape, dtype, device = x.shape, x.dtype, x.device
    code, wcode = DTYPE_CODE.get(dtype), DTYPE_CODE.get(weight.dtype)
    if code is None or len(shape) != 2:
        raise _got("x", x, "[rows, cols] of fp32, fp16 or bf16")
    rows, cols = shape
    x_step, inner = x.stride()
    if inner != 1 and cols > 1:
        raise _got("x", x, "contiguous rows")
    if rows <= 1:
        x_step = cols
    if wcode is None or weight.shape != (cols,) or not weight.is_contiguous():
        raise _got("weight", weight, f"a contiguous [{cols}] of fp32, fp16 or bf16")
    q = scales = q_ptr = scales_ptr = None
    if packed is not None:
        if packed.rows != rows or packed.cols != cols:
            raise ValueError(f"packed: {packed.rows} x {packed.cols} for x of {rows} x {cols}")
        q, scales = packed.q, packed.scales
        q_ptr, scales_ptr = q.data_ptr(), scales.data_ptr()
    handle, side = _stream(stream, (x, weight, residual, out, sum_out, rstd, q, scales))
    r_step, r_ptr, sum_ptr, total = cols, None, None, x
    if residual is not None:
        r_step, r_ptr = _row_step(residual, "residual", shape, dtype), residual.data_ptr()
        if sum_out is None:
            sum_out = _new(side, shape, dtype, device)
        else:
            _given(sum_out, "sum_out", shape, dtype)
        total, sum_ptr = sum_out, sum_out.data_ptr()
    elif sum_out is not None:
        raise ValueError("sum_out without a residual")
    out_ptr = None
    if want_out:
        if out is None:
            out = _new(side, shape, dtype, device)
        else:
            _given(out, "out", shape, dtype)
        out_ptr = out.data_ptr()
    elif out is not None or packed is None:
        raise ValueError("want_out=False goes with packed and without out")
    if rstd is None:
        rstd = _new(side, rows, _F32, device)
    else:
        _given(rstd, "rstd", (rows,), _F32)
    rc = _library().zero_rmsnorm_forward(_norm_desc(rows, cols, x_step, r_step, cols, code, wcode, eps), x.data_ptr(),
                                         r_ptr, weight.data_ptr(), sum_ptr, out_ptr, q_ptr, scales_ptr,
                                         rstd.data_ptr(), handle)
    if rc:
        abi._check(rc)
    return out, total, rstd


@functools.lru_cache(maxsize=256)
def _norm_scratch(rows, cols) -> int:
    """Scratch bytes of a norm's backward: a function of its sizes."""
    return abi.zero_rmsnorm_backward_workspace(
        _norm_desc(rows, cols, cols, cols, cols, abi.ZERO_F32, abi.ZERO_F32, 0.0))


def rmsnorm_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                     dsum=None, dx=None, dweight=None, dweight_dtype=None, stream=None):
    """(dx, dweight) from dy [rows, cols], the forward's s as `x`, and rstd. dx
    is the gradient of x and of the residual; dsum, the gradient that reaches
    s by its other use, is added to it. dweight: fp32 sums stored as
    dweight_dtype (default: dweight's type, or weight's)."""
    shape, dtype, device = x.shape, x.dtype, x.device
    code, wcode = DTYPE_CODE.get(dtype), DTYPE_CODE.get(weight.dtype)
    if code is None or len(shape) != 2:
        raise _got("x", x, "[rows, cols] of fp32, fp16 or bf16")
    rows, cols = shape
    x_step, dy_step = _row_step(x, "x", shape, dtype), _row_step(dy, "dy", shape, dtype)
    r_step, r_ptr = cols, None
    if dsum is not None:
        r_step, r_ptr = _row_step(dsum, "dsum", shape, dtype), dsum.data_ptr()
    if wcode is None or weight.shape != (cols,) or not weight.is_contiguous():
        raise _got("weight", weight, f"a contiguous [{cols}] of fp32, fp16 or bf16")
    _given(rstd, "rstd", (rows,), _F32)
    if dweight_dtype is None:
        dweight_dtype = dweight.dtype if dweight is not None else weight.dtype
    dcode = DTYPE_CODE.get(dweight_dtype)
    if dcode is None:
        raise ValueError(f"unsupported type {dweight_dtype}")
    handle, side = _stream(stream, (x, dy, weight, rstd, dsum, dx, dweight))
    if dx is None:
        dx = _new(side, shape, dtype, device)
    else:
        _given(dx, "dx", shape, dtype)
    if dweight is None:
        dweight = _new(side, cols, dweight_dtype, device)
    else:
        _given(dweight, "dweight", (cols,), dweight_dtype)
    nbytes = _norm_scratch(rows, cols)
    space = _new(side, nbytes, torch.uint8, device)
    rc = _library().zero_rmsnorm_backward(_norm_desc(rows, cols, x_step, r_step, dy_step, code, wcode, 0.0),
                                          dy.data_ptr(), x.data_ptr(), weight.data_ptr(), rstd.data_ptr(), r_ptr,
                                          dx.data_ptr(), dweight.data_ptr(), dcode, space.data_ptr(), nbytes, handle)
    if rc:
        abi._check(rc)
    return dx, dweight


# ---------------------------------------------------------------------------
# Attention's training pair
# ---------------------------------------------------------------------------

def _steps(t, name, shape, dtype):
    """Strides of a [batch, length, heads, head_dim] tensor, head elements contiguous."""
    steps = t.stride()
    if t.shape != shape or t.dtype is not dtype or steps[3] != 1:
        raise _got(name, t, f"{tuple(shape)} of {dtype} with contiguous heads")
    return steps


def _attention_sizes(q, k, causal, window, key_lengths, scale):
    """The leading fields of the call's descriptor, and the shape of k and v."""
    q_shape, k_shape = q.shape, k.shape
    code = HALF_CODE.get(q.dtype)
    if code is None or len(q_shape) != 4 or len(k_shape) != 4:
        raise _got("q", q, "[batch, length, heads, head_dim] of fp16 or bf16, as k and v")
    batch, q_len, q_heads, dim = q_shape
    _, k_len, kv_heads, _ = k_shape
    if key_lengths is not None:
        _given(key_lengths, "key_lengths", (batch,), torch.int32)
    return (batch, q_len, k_len, q_heads, kv_heads, dim, code, causal, 0, window,
            dim ** -0.5 if scale is None else scale), (batch, k_len, kv_heads, dim)


def attention_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False,
                      window: int = 0, key_lengths=None, scale: float | None = None, out=None, lse=None,
                      stream=None):
    """(o, lse) of q [batch, q_len, q_heads, head_dim] and k, v [batch, k_len,
    kv_heads, head_dim] (fp16 or bf16; strides are free multiples of 8).

    Query i sees key j when j < key_lengths[b], j <= i + k_len - q_len
    (`causal`) and j > i + k_len - q_len - window (`window` > 0). A query that
    sees no key has o = 0 and lse = -inf. scale: default head_dim^-1/2. lse is
    fp32 [batch, q_heads, q_len]. out may be q itself."""
    sizes, kv_shape = _attention_sizes(q, k, causal, window, key_lengths, scale)
    dtype, shape, device = q.dtype, q.shape, q.device
    qb, qt, qh, _ = _steps(q, "q", shape, dtype)
    kb, kt, kh, _ = _steps(k, "k", kv_shape, dtype)
    vb, vt, vh, _ = _steps(v, "v", kv_shape, dtype)
    handle, side = _stream(stream, (q, k, v, key_lengths, out, lse))
    if out is None:
        out = _new(side, shape, dtype, device)
        ob, ot, oh, _ = out.stride()
    else:
        ob, ot, oh, _ = _steps(out, "out", shape, dtype)
    rows = (sizes[0], sizes[3], sizes[1])
    if lse is None:
        lse = _new(side, rows, _F32, device)
    else:
        _given(lse, "lse", rows, _F32)
    rc = _library().zero_attention_forward(
        _attention_desc(*sizes, qb, qt, qh, kb, kt, kh, vb, vt, vh, ob, ot, oh, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0),
        q.data_ptr(), k.data_ptr(), v.data_ptr(), None if key_lengths is None else key_lengths.data_ptr(),
        out.data_ptr(), lse.data_ptr(), handle)
    if rc:
        abi._check(rc)
    return out, lse


@functools.lru_cache(maxsize=256)
def _attention_scratch(batch, q_len, q_heads) -> int:
    """Scratch bytes of attention's backward, enough for both types and any sharing of keys."""
    steps = (max(q_len, 1) * q_heads * 8, q_heads * 8, 8)
    return abi.zero_attention_backward_workspace(
        _attention_desc(batch, q_len, q_len, q_heads, q_heads, 8, abi.ZERO_F16, 0, 0, 0, 1.0, *steps * 8))


def attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                       o: torch.Tensor, lse: torch.Tensor, causal: bool = False, window: int = 0,
                       key_lengths=None, scale: float | None = None, dq=None, dk=None, dv=None,
                       stream=None):
    """(dq, dk, dv) from dout, the forward's tensors and the same mask; the
    probabilities are recomputed from lse. dk and dv are summed over the query
    heads that share a key head. dq may be o itself, dk and dv k or v; they may
    overlap no other input."""
    sizes, kv_shape = _attention_sizes(q, k, causal, window, key_lengths, scale)
    dtype, shape, device = q.dtype, q.shape, q.device
    qb, qt, qh, _ = _steps(q, "q", shape, dtype)
    kb, kt, kh, _ = _steps(k, "k", kv_shape, dtype)
    vb, vt, vh, _ = _steps(v, "v", kv_shape, dtype)
    ob, ot, oh, _ = _steps(o, "o", shape, dtype)
    gb, gt, gh, _ = _steps(dout, "dout", shape, dtype)
    batch, q_heads, q_len = sizes[0], sizes[3], sizes[1]
    _given(lse, "lse", (batch, q_heads, q_len), _F32)
    handle, side = _stream(stream, (q, k, v, o, dout, lse, key_lengths, dq, dk, dv))
    if dq is None:
        dq = _new(side, shape, dtype, device)
        dqb, dqt, dqh, _ = dq.stride()
    else:
        dqb, dqt, dqh, _ = _steps(dq, "dq", shape, dtype)
    if dk is None:
        dk = _new(side, kv_shape, dtype, device)
        dkb, dkt, dkh, _ = dk.stride()
    else:
        dkb, dkt, dkh, _ = _steps(dk, "dk", kv_shape, dtype)
    if dv is None:
        dv = _new(side, kv_shape, dtype, device)
        dvb, dvt, dvh, _ = dv.stride()
    else:
        dvb, dvt, dvh, _ = _steps(dv, "dv", kv_shape, dtype)
    nbytes = _attention_scratch(batch, q_len, q_heads)
    space = _new(side, nbytes, torch.uint8, device)
    rc = _library().zero_attention_backward(
        _attention_desc(*sizes, qb, qt, qh, kb, kt, kh, vb, vt, vh, ob, ot, oh, gb, gt, gh, dqb, dqt, dqh,
                        dkb, dkt, dkh, dvb, dvt, dvh),
        dout.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
        None if key_lengths is None else key_lengths.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
        space.data_ptr(), nbytes, handle)
    if rc:
        abi._check(rc)
    return dq, dk, dv


def check(stream=None) -> None:
    """Raise ZeroError(ZERO_ERR_TIMEOUT) if a kernel of this module gave up a
    bounded wait, on any stream of the device, since this thread's last check.
    Synchronises the stream."""
    abi.zero_operator_status((stream or torch.cuda.current_stream()).cuda_stream)
