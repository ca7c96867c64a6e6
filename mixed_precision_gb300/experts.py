"""Operators of an expert layer (mixture of experts), on torch tensors.

A layer's forward pass: ``route`` chooses k experts for each token, ``gather``
copies the tokens' rows in the experts' order, ``forward`` multiplies each
expert's run of rows with its weights, ``combine`` sums the weighted rows back.
The backward pass: ``combine_backward``, ``input_grad`` and ``weight_grad``,
``combine`` without weights (the gradient of ``gather``), ``route_backward``.

The conventions are those of mixed_precision_gb300.block: each function checks
its tensors, allocates what the caller did not pass and makes one call of the C
ABI; work is enqueued on `stream` (default: torch's current stream) and nothing
waits, so calls can be captured into a CUDA graph; nothing is recorded for
autograd; wrong shapes, types, devices or layouts raise ValueError here or
ZeroError from the library, and nothing is enqueued then. How many rows each
expert has stays on the device.
"""
from __future__ import annotations

import functools

import torch

from . import _abi as abi
from .block import (_F32, _given, _got, _library, _new, _row_step, _stream, DTYPE_CODE, HALF_CODE, check)

__all__ = ["Routing", "route", "route_backward", "gather", "combine", "combine_backward", "forward", "input_grad",
           "weight_grad", "check"]

_I32 = torch.int32
_new_routing = object.__new__
_experts_desc = abi.EXPERTS_DESC.pack


class Routing:
    """The choice of k of num_experts experts for each token, and the chosen
    slots (token, position) in the experts' order:

    weights [tokens, k] fp32; experts [tokens, k] (-1: none taken); offsets
    [num_experts + 1], where each expert's rows start; source [tokens * k], the
    slot token * k + position of each row (-1 behind the last); place [tokens,
    k], the row of each slot (-1: none). All but weights are int32."""

    __slots__ = ("num_experts", "normalize", "tokens", "k", "weights", "experts", "offsets", "source", "place")

    def __init__(self, num_experts: int, normalize: bool, weights, experts, offsets, source, place):
        if weights.dim() != 2:
            raise _got("weights", weights, "[tokens, k] of fp32")
        tokens, k = shape = weights.shape
        _given(weights, "weights", shape, _F32)
        _given(experts, "experts", shape, _I32)
        _given(offsets, "offsets", (num_experts + 1,), _I32)
        _given(source, "source", (tokens * k,), _I32)
        _given(place, "place", shape, _I32)
        self.num_experts, self.normalize, self.tokens, self.k = num_experts, bool(normalize), tokens, k
        self.weights, self.experts, self.offsets, self.source, self.place = weights, experts, offsets, source, place


@functools.lru_cache(maxsize=256)
def _route_scratch(tokens, num_experts, k) -> int:
    return abi.zero_route_workspace(tokens, num_experts, k)


def _logits(logits):
    code = DTYPE_CODE.get(logits.dtype)
    if code is None or logits.dim() != 2:
        raise _got("logits", logits, "[tokens, experts] of fp32, fp16 or bf16")
    return code, _row_step(logits, "logits", logits.shape, logits.dtype)


def route(logits: torch.Tensor, k: int, normalize: bool = True, stream=None) -> Routing:
    """Choose the k largest of logits [tokens, num_experts] for each token, the
    lower expert where they are equal. A logit of -inf is never taken: a row of
    nothing else (a padding token) goes to no expert and has weights 0.

    The weights are the softmax over the taken logits (normalize) or over all of
    the row. Up to 1024 experts and 32 choices; the row stride is free."""
    code, step = _logits(logits)
    tokens, num_experts = logits.shape
    handle, side = _stream(stream, (logits,))
    device = logits.device
    # one allocation: four arrays of tokens * k, the offsets, the scratch, each from a 16-byte boundary
    nbytes = _route_scratch(tokens, num_experts, k)
    slots = tokens * k
    each, ends = (slots + 3) // 4 * 4, (num_experts + 4) // 4 * 4
    space = _new(side, 4 * each + ends + nbytes // 4, _I32, logits.device)
    at = space.data_ptr()
    rc = _library().zero_route(logits.data_ptr(), step, tokens, num_experts, k, code, normalize, at, at + 4 * each,
                               at + 16 * each, at + 8 * each, at + 12 * each, at + 16 * each + 4 * ends, nbytes, handle)
    if rc:
        abi._check(rc)
    r = _new_routing(Routing)
    r.num_experts, r.normalize, r.tokens, r.k = num_experts, bool(normalize), tokens, k
    shape, steps = (tokens, k), (k, 1)
    r.weights = space.view(_F32).as_strided(shape, steps)
    r.experts = space.as_strided(shape, steps, each)
    r.source = space.as_strided((slots,), (1,), 2 * each)
    r.place = space.as_strided(shape, steps, 3 * each)
    r.offsets = space.as_strided((num_experts + 1,), (1,), 4 * each)
    return r


def route_backward(dweights: torch.Tensor, logits: torch.Tensor, routing: Routing, out=None,
                   stream=None) -> torch.Tensor:
    """dlogits [tokens, num_experts], in the logits' type, of dweights [tokens, k] fp32."""
    code, step = _logits(logits)
    tokens, k, num_experts = routing.tokens, routing.k, routing.num_experts
    if logits.shape != (tokens, num_experts):
        raise _got("logits", logits, f"{(tokens, num_experts)}, the routing's")
    _given(dweights, "dweights", (tokens, k), _F32)
    weights, experts = routing.weights, routing.experts
    handle, side = _stream(stream, (logits, dweights, weights, experts, out))
    if out is None:
        out = _new(side, (tokens, num_experts), logits.dtype, logits.device)
    else:
        _given(out, "out", (tokens, num_experts), logits.dtype)
    rc = _library().zero_route_backward(dweights.data_ptr(), weights.data_ptr(), experts.data_ptr(), logits.data_ptr(),
                                        step, tokens, num_experts, k, code, routing.normalize, out.data_ptr(), handle)
    if rc:
        abi._check(rc)
    return out


def _hidden(t, name, rows):
    """Code, row step and elements a row of a [rows, hidden] tensor."""
    code = DTYPE_CODE.get(t.dtype)
    if code is None or t.dim() != 2 or t.shape[0] != rows:
        raise _got(name, t, f"[{rows}, hidden] of fp32, fp16 or bf16")
    return code, _row_step(t, name, t.shape, t.dtype), t.shape[1]


def gather(x: torch.Tensor, routing: Routing, out=None, stream=None) -> torch.Tensor:
    """The rows of x [tokens, hidden] in the experts' order, [tokens * k,
    hidden]; rows behind the last expert's are zero."""
    tokens, k = routing.tokens, routing.k
    code, step, hidden = _hidden(x, "x", tokens)
    place, source = routing.place, routing.source
    handle, side = _stream(stream, (x, place, source, out))
    if out is None:
        out = _new(side, (tokens * k, hidden), x.dtype, x.device)
    else:
        _given(out, "out", (tokens * k, hidden), x.dtype)
    rc = _library().zero_experts_gather(x.data_ptr(), step, tokens, k, hidden, code, place.data_ptr(),
                                        source.data_ptr(), out.data_ptr(), handle)
    if rc:
        abi._check(rc)
    return out


def combine(y: torch.Tensor, routing: Routing, weighted: bool = True, out=None, stream=None) -> torch.Tensor:
    """out [tokens, hidden]: each token's sum over its k rows of y [tokens * k,
    hidden], times the routing's weights; in fp32, rounded once. weighted=False:
    the plain sum, which is the gradient of ``gather``."""
    tokens, k = routing.tokens, routing.k
    code, step, hidden = _hidden(y, "y", tokens * k)
    place, weights = routing.place, routing.weights if weighted else None
    handle, side = _stream(stream, (y, place, weights, out))
    if out is None:
        out = _new(side, (tokens, hidden), y.dtype, y.device)
    else:
        _given(out, "out", (tokens, hidden), y.dtype)
    rc = _library().zero_experts_combine(y.data_ptr(), step, tokens, k, hidden, code, place.data_ptr(),
                                         weights.data_ptr() if weighted else None, out.data_ptr(), handle)
    if rc:
        abi._check(rc)
    return out


def combine_backward(dout: torch.Tensor, y: torch.Tensor, routing: Routing, dy=None, dweights=None, stream=None):
    """(dy [tokens * k, hidden], dweights [tokens, k] fp32) of the weighted
    ``combine``; dy is zero in rows behind the last expert's, dweights where no
    expert was taken."""
    tokens, k = routing.tokens, routing.k
    code, step, hidden = _hidden(dout, "dout", tokens)
    y_step = _row_step(y, "y", (tokens * k, hidden), dout.dtype)
    place, source, weights = routing.place, routing.source, routing.weights
    handle, side = _stream(stream, (dout, y, place, source, weights, dy, dweights))
    if dy is None:
        dy = _new(side, (tokens * k, hidden), y.dtype, y.device)
    else:
        _given(dy, "dy", (tokens * k, hidden), y.dtype)
    if dweights is None:
        dweights = _new(side, (tokens, k), _F32, y.device)
    else:
        _given(dweights, "dweights", (tokens, k), _F32)
    rc = _library().zero_experts_combine_backward(dout.data_ptr(), step, y.data_ptr(), y_step, tokens, k, hidden, code,
                                                  place.data_ptr(), source.data_ptr(), weights.data_ptr(),
                                                  dy.data_ptr(), dweights.data_ptr(), handle)
    if rc:
        abi._check(rc)
    return dy, dweights


# ---------------------------------------------------------------------------
# The experts' products
# ---------------------------------------------------------------------------

def _eights(n):
    return (n + 7) // 8 * 8


def _rows(t, name, cols, dtype=None):
    """(rows, row stride) of a [rows, cols] tensor of fp16 or bf16."""
    shape = t.shape
    if t.dtype not in HALF_CODE or len(shape) != 2 or (cols is not None and shape[1] != cols) or \
            (dtype is not None and t.dtype is not dtype):
        raise _got(name, t, f"[rows, {'cols' if cols is None else cols}] of {dtype or 'fp16 or bf16'}")
    step, inner = t.stride()
    if inner != 1 and shape[1] > 1:
        raise _got(name, t, "contiguous rows")
    return shape[0], step if shape[0] > 1 else _eights(shape[1])


def _matrices(t, name, shape=None, dtype=None):
    """Strides (between experts' matrices, between rows) of a [experts, n_out, n_in] tensor."""
    if t.dim() != 3 or (shape is not None and t.shape != shape) or (dtype is not None and t.dtype is not dtype):
        raise _got(name, t, "[experts, n_out, n_in] of fp16 or bf16" if shape is None else f"{shape} of {dtype}")
    experts, n_out, n_in = t.shape
    each, step, inner = t.stride()
    if inner != 1 and n_in > 1:
        raise _got(name, t, "contiguous rows")
    step = step if n_out > 1 else _eights(n_in)
    return each if experts > 1 else _eights(n_out * step), step


def _output(out, name, shape, dtype, side, device):
    """The output tensor and its row stride."""
    if out is None:
        return _new(side, shape, dtype, device), shape[1]
    return out, _row_step(out, name, shape, dtype)


def forward(x: torch.Tensor, weight: torch.Tensor, offsets: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    """y [rows, n_out]: y[r] = x[r] W_e^T for the rows offsets[e] <= r <
    offsets[e + 1] of expert e; rows of no expert are zero.

    x [rows, n_in] and weight [experts, n_out, n_in] are fp16 or bf16, their
    strides free multiples of 8 (of one projection, or of all experts' in a flat
    parameter buffer). offsets: int32 [experts + 1], as ``route`` gives.

    A new result has rows without gaps: with an n_out that is no multiple of 8 it
    (and a dy of its shape) is no input of another product. `out` may be columns of
    a wider buffer, ``buffer[:, :n_out]``, whose row stride is a multiple of 8."""
    each, w_step = _matrices(weight, "weight")
    experts, n_out, n_in = weight.shape
    dtype = weight.dtype
    rows, x_step = _rows(x, "x", n_in, dtype)
    _given(offsets, "offsets", (experts + 1,), _I32)
    handle, side = _stream(stream, (x, weight, offsets, out))
    out, y_step = _output(out, "out", (rows, n_out), dtype, side, x.device)
    rc = _library().zero_experts_forward(
        _experts_desc(rows, n_out, n_in, x_step, y_step, each, w_step, experts, HALF_CODE[dtype]), x.data_ptr(),
        weight.data_ptr(), offsets.data_ptr(), out.data_ptr(), handle)
    if rc:
        abi._check(rc)
    return out


def input_grad(dy: torch.Tensor, weight: torch.Tensor, offsets: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    """dx [rows, n_in]: dx[r] = dy[r] W_e for each expert's rows; rows of no
    expert are zero. dy's and weight's strides are multiples of 8 (``forward``
    says how an odd n_out meets that)."""
    each, w_step = _matrices(weight, "weight")
    experts, n_out, n_in = weight.shape
    dtype = weight.dtype
    rows, y_step = _rows(dy, "dy", n_out, dtype)
    _given(offsets, "offsets", (experts + 1,), _I32)
    handle, side = _stream(stream, (dy, weight, offsets, out))
    out, x_step = _output(out, "out", (rows, n_in), dtype, side, dy.device)
    rc = _library().zero_experts_input_grad(
        _experts_desc(rows, n_out, n_in, x_step, y_step, each, w_step, experts, HALF_CODE[dtype]), dy.data_ptr(),
        weight.data_ptr(), offsets.data_ptr(), out.data_ptr(), handle)
    if rc:
        abi._check(rc)
    return out


def weight_grad(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor, out=None, dtype=None,
                accumulate: bool = False, stream=None) -> torch.Tensor:
    """dw [experts, n_out, n_in]: the sum over each expert's rows of dy[r]^T
    x[r]; zero for an expert without rows.

    dy's and x's row strides are multiples of 8. dw is fp32 or the inputs' type
    (`dtype`; default out's, or theirs), its strides free: `out` may be all experts' gradients in a flat buffer.
    `accumulate` adds to an fp32 `out` (main gradients over micro-batches)."""
    rows, y_step = _rows(dy, "dy", None)
    x_rows, x_step = _rows(x, "x", None, dy.dtype)
    if x_rows != rows:
        raise _got("x", x, f"{rows} rows, as dy")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    if dtype is None:
        dtype = out.dtype if out is not None else dy.dtype
    if dtype not in DTYPE_CODE:
        raise ValueError(f"unsupported type {dtype}")
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise _got("offsets", offsets, "int32 [experts + 1]")
    experts, n_out, n_in = shape = (offsets.shape[0] - 1, dy.shape[1], x.shape[1])
    _given(offsets, "offsets", (experts + 1,), _I32)
    handle, side = _stream(stream, (dy, x, offsets, out))
    if out is None:
        out = _new(side, shape, dtype, dy.device)
        each, w_step = n_out * n_in, n_in
    else:
        each, w_step = _matrices(out, "out", shape, dtype)
    rc = _library().zero_experts_weight_grad(
        _experts_desc(rows, n_out, n_in, x_step, y_step, each, w_step, experts, HALF_CODE[dy.dtype]), dy.data_ptr(),
        x.data_ptr(), offsets.data_ptr(), out.data_ptr(), DTYPE_CODE[dtype], accumulate, handle)
    if rc:
        abi._check(rc)
    return out
