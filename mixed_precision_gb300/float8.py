"""Products of 8-bit floating-point matrices with block scales, on torch tensors.

A Float8Matrix holds e4m3 codes and one power-of-two scale for each 128
elements along its rows, which are the contraction of a product. For a linear
layer y = x W^T all three products of a training step are ``matmul``s of packed
forms, each made by ``pack`` from one read of a tensor:

    x8, x8t = pack(x, transposed=True)      # forward; backward's weight gradient
    w8, w8t = pack(w, transposed=True)
    y = matmul(x8, w8)
    g8, g8t = pack(dy, transposed=True)
    dx = matmul(g8, w8t)
    dw = matmul(g8t, x8t, dtype=torch.float32)

Streams, errors and checks are those of mixed_precision_gb300.block.
"""
from __future__ import annotations

import torch

from . import _abi as abi
from .block import _given, _got, _library, _new, _row_step, _stream, DTYPE_CODE, check

__all__ = ["Float8Matrix", "pack", "matmul", "check"]

_E4M3, _U8 = torch.float8_e4m3fn, torch.uint8
_scaled_desc = abi.SCALED_DESC.pack


class Float8Matrix:
    """rows x cols elements, or one such matrix for each of `experts`: codes ``q``
    [(experts,) rows, pitch], e4m3 with cols rounded up to 128, and ``scales``
    [(experts,) rows, scale_pitch], uint8: b stands for 2^(b - 127) (1.01 bytes
    per element). An inf or a NaN becomes NaN."""

    __slots__ = ("rows", "cols", "experts", "q", "scales")

    def __init__(self, rows: int, cols: int, experts: int | None = None, q=None, scales=None, device="cuda",
                 stream=None):
        if rows < 0 or cols < 1 or (experts is not None and experts < 1):
            raise ValueError(f"a float8 matrix of {rows} x {cols}, experts {experts}")
        blocks = (cols + 127) // 128
        lead = (rows,) if experts is None else (experts, rows)
        q_shape, s_shape = lead + (blocks * 128,), lead + ((blocks + 3) // 4 * 4,)
        self.rows, self.cols, self.experts = rows, cols, experts
        if q is None:
            q = _new(stream, q_shape, _E4M3, device)
            scales = _new(stream, s_shape, _U8, device)
        else:
            _given(q, "q", q_shape, _E4M3)
            if scales is None:
                raise ValueError("q without scales")
            _given(scales, "scales", s_shape, _U8)
        self.q, self.scales = q, scales

    def restore(self, dtype: torch.dtype | None = None, out=None, stream=None) -> torch.Tensor:
        """The values [(experts,) rows, cols] in `dtype` (default: out's, or bf16)."""
        if dtype is None:
            dtype = out.dtype if out is not None else torch.bfloat16
        code, q, scales, rows, cols = DTYPE_CODE.get(dtype), self.q, self.scales, self.rows, self.cols
        if code is None:
            raise ValueError(f"unsupported type {dtype}")
        shape, step = (rows, cols), cols
        if self.experts is not None:
            shape = (self.experts, rows, cols)
            if out is not None:
                _given(out, "out", shape, dtype)
        elif out is not None:
            step = _row_step(out, "out", shape, dtype)
        handle, side = _stream(stream, (q, scales, out))
        if out is None:
            out = _new(side, shape, dtype, q.device)
        rc = _library().zero_scaled_unpack(q.data_ptr(), scales.data_ptr(), rows * (self.experts or 1), cols,
                                           out.data_ptr(), step, code, handle)
        if rc:
            abi._check(rc)
        return out


def _form(want, name, rows, cols, experts, side, device):
    """The Float8Matrix to fill: a new one for True, a given one, None for False."""
    if want is False or want is None:
        return None
    if want is True:
        return Float8Matrix(rows, cols, experts, device=device, stream=side)
    if (want.rows, want.cols, want.experts) != (rows, cols, experts):
        raise ValueError(f"{name}: {want.rows} x {want.cols}, experts {want.experts}, for {rows} x {cols}, {experts}")
    return want


def pack(x: torch.Tensor, direct=True, transposed=False, stream=None):
    """(packed x, packed x^T) of x [rows, cols] or [experts, rows, cols] (fp32,
    fp16 or bf16; row and expert strides are free) from one read of it. Each of
    `direct` and `transposed` is True (a new Float8Matrix), a Float8Matrix to
    fill, or False (None is returned in its place)."""
    dtype, shape = x.dtype, x.shape
    code = DTYPE_CODE.get(dtype)
    if code is None or len(shape) not in (2, 3):
        raise _got("x", x, "[rows, cols] or [experts, rows, cols] of fp32, fp16 or bf16")
    experts = shape[0] if len(shape) == 3 else None
    rows, cols = shape[-2:]
    if cols < 1 or experts == 0 or (transposed is not False and transposed is not None and rows < 1):
        raise _got("x", x, "no empty dimension")
    step, inner = x.stride()[-2:]
    if inner != 1 and cols > 1:
        raise _got("x", x, "contiguous rows")
    if rows <= 1:
        step = cols
    each = x.stride()[0] if experts is not None else 0
    tensors = [x]
    for m in (direct, transposed):
        if isinstance(m, Float8Matrix):
            tensors += [m.q, m.scales]
    handle, side = _stream(stream, tensors)
    a = _form(direct, "direct", rows, cols, experts, side, x.device)
    b = _form(transposed, "transposed", cols, rows, experts, side, x.device)
    rc = _library().zero_scaled_pack(x.data_ptr(), each, step, experts or 1, rows, cols, code,
                                     a and a.q.data_ptr(), a and a.scales.data_ptr(),
                                     b and b.q.data_ptr(), b and b.scales.data_ptr(), handle)
    if rc:
        abi._check(rc)
    return a, b


def matmul(a: Float8Matrix, b: Float8Matrix, offsets=None, out=None, dtype=None, accumulate: bool = False,
           stream=None) -> torch.Tensor:
    """out [a.rows, b.rows]: the products of a's rows with b's, summed in fp32.

    With offsets (int32 [experts + 1]) b has a matrix for each expert, which the
    rows offsets[e] <= r < offsets[e + 1] of a meet; rows of no expert are zero.
    dtype: fp32, fp16 or bf16 (default: out's, or bf16). `accumulate` adds to an
    fp32 `out`."""
    rows, n, k = a.rows, b.rows, a.cols
    experts = b.experts or 0
    if a.experts is not None or b.cols != k:
        raise ValueError(f"a of {rows} x {k}, experts {a.experts}; b of {n} x {b.cols}, experts {b.experts}")
    if (offsets is None) != (b.experts is None):
        raise ValueError("offsets go with a matrix for each expert")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    if dtype is None:
        dtype = out.dtype if out is not None else torch.bfloat16
    code = DTYPE_CODE.get(dtype)
    if code is None:
        raise ValueError(f"unsupported type {dtype}")
    if offsets is not None:
        _given(offsets, "offsets", (experts + 1,), torch.int32)
    aq, a_scales, bq, b_scales = a.q, a.scales, b.q, b.scales
    handle, side = _stream(stream, (aq, a_scales, bq, b_scales, offsets, out))
    if out is None:
        out, step = _new(side, (rows, n), dtype, aq.device), n
    else:
        step = _row_step(out, "out", (rows, n), dtype)
    rc = _library().zero_scaled_matmul(_scaled_desc(rows, n, k, step, experts, code, accumulate, 0), aq.data_ptr(),
                                       a_scales.data_ptr(), bq.data_ptr(), b_scales.data_ptr(),
                                       None if offsets is None else offsets.data_ptr(), out.data_ptr(), handle)
    if rc:
        abi._check(rc)
    return out
