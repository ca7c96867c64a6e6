"""The block operators' host side, without a GPU: outputs in the place of inputs.
The pointers are made-up addresses that are never read."""
import itertools

import pytest
import torch

from test_block_host import P, attention, norm, refused, z  # noqa: F401

# batch 2, 10 queries of 4 heads, 12 keys of 2 heads, head_dim 64, in bytes
NQ, NK = 2 * 10 * 256 * 2, 2 * 12 * 128 * 2


def addresses(names, **at):
    """Buffers far from one another, except those given."""
    a = {n: (i + 1) << 24 for i, n in enumerate(names)}
    a.update(at)
    return a


def forward(z, desc=None, **at):
    a = addresses(("q", "k", "v", "o", "lse"), **at)
    return (z.zero_attention_forward, desc or attention(z), a["q"], a["k"], a["v"], 0, a["o"], a["lse"], 0)


def backward(z, desc=None, **at):
    a = addresses(("do", "q", "k", "v", "o", "lse", "dq", "dk", "dv", "ws"), **at)
    return (z.zero_attention_backward, desc or attention(z), a["do"], a["q"], a["k"], a["v"], a["o"], a["lse"], 0, a["dq"],
            a["dk"], a["dv"], a["ws"], 1 << 30, 0)


def accepted(z, call, *args):
    """Past every check: without a device the call fails with another code, or it would run."""
    if torch.cuda.is_available():
        pytest.skip("made-up addresses")
    with pytest.raises(z.ZeroError) as e:
        call(*args)
    assert e.value.code == 2, e.value  # ZERO_ERR_CUDA


def test_attention_outputs_over_inputs(z):  # noqa: F811
    for step in (0, 16, NQ - 16):
        refused(z, *forward(z, o=(1 << 24) + step, q=1 << 24) if step else forward(z, o=2 << 24))
        refused(z, *forward(z, o=(3 << 24) + min(step, NK - 16)))
        for out, other in itertools.product(("dq",), ("q", "do", "k", "v")):
            size = NQ if other in ("q", "do") else NK
            at = addresses(("do", "q", "k", "v", "o", "lse", "dq", "dk", "dv", "ws"))[other]
            refused(z, *backward(z, **{out: at + min(step, size - 16)}))
        for out, other in itertools.product(("dk", "dv"), ("q", "do")):
            at = addresses(("do", "q", "k", "v", "o", "lse", "dq", "dk", "dv", "ws"))[other]
            refused(z, *backward(z, **{out: at + step}))
        refused(z, *backward(z, dk=9 << 24, dv=(9 << 24) + min(step, NK - 16)))
        refused(z, *backward(z, dq=9 << 24, dk=(9 << 24) + step))
    # shifted, or with other strides, an input is not the output itself
    refused(z, *backward(z, dk=(3 << 24) + 16))
    refused(z, *backward(z, attention(z, dk_strides=(12 * 256, 256, 64)), dk=3 << 24))
    refused(z, *backward(z, dq=(5 << 24) + 512))


def test_attention_outputs_in_place(z):  # noqa: F811
    accepted(z, *forward(z))
    accepted(z, *forward(z, q=4 << 24, o=4 << 24))
    accepted(z, *backward(z))
    at = dict(do=1 << 24, q=2 << 24, k=3 << 24, v=4 << 24, o=5 << 24)
    accepted(z, *backward(z, **at, dq=5 << 24, dk=3 << 24, dv=4 << 24))
    accepted(z, *backward(z, **at, dq=5 << 24, dk=4 << 24, dv=3 << 24))


def test_attention_outputs_side_by_side(z):  # noqa: F811
    """dq, dk and dv as parts of one buffer, beside q, k and v in another or in the same rows."""
    W = 256 + 128 + 128  # heads of q, k and v in a row
    d = {n + "_strides": (10 * W, W, 64) for n in ("q", "k", "v", "dq", "dk", "dv")}
    packed = attention(z, k_len=10, **d)
    part = dict(q=P, k=P + 512, v=P + 768, dq=2 * P, dk=2 * P + 512, dv=2 * P + 768)
    accepted(z, *backward(z, packed, **part))
    refused(z, *backward(z, packed, **{**part, "dk": 2 * P + 496}))
    refused(z, *backward(z, packed, **{**part, "dv": 2 * P + 640}))
    # a row of [heads][q, dq] halves
    two = attention(z, q_strides=(10 * 512, 512, 128), dq_strides=(10 * 512, 512, 128))
    accepted(z, *backward(z, two, q=P, dq=P + 128))
    refused(z, *backward(z, two, q=P, dq=P + 112))
    # the gradients' rows behind the tensors' in each token
    rows = attention(z, k_len=10, **{n: (10 * 2 * W, 2 * W, 64) for n in d})
    part = dict(q=P, k=P + 512, v=P + 768, dq=P + 1024, dk=P + 1536, dv=P + 1792)
    accepted(z, *backward(z, rows, **part))
    refused(z, *backward(z, rows, **{**part, "dv": P + 2048 - 128}))


def test_norm_outputs_in_place(z):  # noqa: F811
    call = z.zero_rmsnorm_forward
    accepted(z, call, norm(z), P, 0, 2 * P, 0, P, 0, 0, 0, 0)
    accepted(z, call, norm(z), P, 3 * P, 2 * P, P, 3 * P, 0, 0, 0, 0)
    refused(z, call, norm(z), P, 3 * P, 2 * P, 4 * P, 4 * P, 0, 0, 0, 0)  # the sum would be lost
    refused(z, call, norm(z), P, 3 * P, 2 * P, P, P, 0, 0, 0, 0)
    refused(z, call, norm(z, x_stride=72), P, 0, 2 * P, 0, P, 0, 0, 0, 0)  # rows not yet read
    refused(z, call, norm(z, residual_stride=72), P, 3 * P, 2 * P, 4 * P, 3 * P, 0, 0, 0, 0)


def test_operator_timeout_arguments(z):  # noqa: F811
    for kernels, limit in ((-1, 100), (4, 100), (0, 0), (0, (1 << 22) + 1)):
        refused(z, z.zero_selftest_operator_timeout, kernels, limit, 0)


@pytest.mark.parametrize("scale", [1e37, 1e39, 1e300, float("inf")])
def test_attention_scale_beyond_fp32(z, scale):  # noqa: F811
    refused(z, *forward(z, attention(z, scale=scale)))
    accepted(z, *forward(z, attention(z, scale=9e36)))
