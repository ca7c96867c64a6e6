"""The block operators at their edges: the largest sizes they take, infinities in
queries, fp16 gradients far from one, non-finite rows beside masked ones, every
way out of the weight gradient, outputs in place of inputs, scratch sizes."""
import math

import pytest
import torch

import _block_ref as ref
from mixed_precision_gb300 import block

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def same_bits(a, b):
    t = torch.int32 if a.dtype == F32 else torch.int16
    return torch.equal(a.contiguous().view(t), b.contiguous().view(t))


def qkv(g, B, Sq, Sk, H, K, D, dtype, dout=0.1):
    return (normal(g, B, Sq, H, D, dtype=dtype), normal(g, B, Sk, K, D, dtype=dtype, scale=1.5),
            normal(g, B, Sk, K, D, dtype=dtype), normal(g, B, Sq, H, D, dtype=dtype, scale=dout))


# ---------------------------------------------------------------------------
# Attention: infinities in q
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_row_of_infinite_products(dtype, D):
    """A row that sees keys, every one of whose products is -inf, has no softmax:
    NaN in o, lse and dq, not the zeros of a row that sees no key."""
    g = gen(D)
    q, k, v, do = qkv(g, 1, 300, 300, 2, 1, D, dtype)
    k[..., 0] = k[..., 0].abs() + 0.5
    clean = block.attention_forward(q, k, v, causal=True)
    for row in (0, 5, 150):  # one key, a few, more than a tile
        q[0, row, 0, 0] = -math.inf
    q[0, 200, 0, 0] = math.inf
    bad = torch.zeros(300, dtype=torch.bool, device="cuda")
    bad[[0, 5, 150, 200]] = True
    o, lse = block.attention_forward(q, k, v, causal=True)
    assert bool(o[0, bad, 0].isnan().all()) and bool(lse[0, 0, bad].isnan().all())
    assert same_bits(o[0, ~bad], clean[0][0, ~bad]) and same_bits(lse[0, :, ~bad], clean[1][0, :, ~bad])
    assert same_bits(o[0, :, 1], clean[0][0, :, 1])
    dq, _, _ = block.attention_backward(do, q, k, v, o, lse, causal=True)
    assert bool(dq[0, bad, 0].isnan().all()) and bool(dq[0, :, 1].isfinite().all())
    assert bool(dq[0, ~bad, 0].isfinite().all())


# ---------------------------------------------------------------------------
# Attention in fp16: weights and gradients over the range of the type
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("Sk", [4096, 65536])
def test_attention_fp16_weak_keys_add_up(Sk):
    """A key takes nearly all of the weight, and its value is zero: what is left is
    the others' (Sk - 1) e^-18. A weight is off by its rounding, or by half a step
    of fp16's smallest numbers, 2^-25, of which 2^7 are taken out again."""
    D = 64
    q = torch.zeros(1, 128, 1, D, dtype=F16, device="cuda")
    k = torch.zeros(1, Sk, 1, D, dtype=F16, device="cuda")
    q[..., 0], k[0, 7, 0, 0] = 12, 12  # a logit of 12 * 12 / 8
    v = torch.ones_like(k)
    v[0, 7] = 0
    o, _ = block.attention_forward(q, k, v)
    p = math.exp(-18.0)
    want = (Sk - 1) * p / (1 + (Sk - 1) * p)
    assert float((o.double() - want).abs().max()) <= (Sk - 1) * 2 ** -32 + want * (2 * ref.U[F16] + 2 ** -16) + 2 ** -25


# ---------------------------------------------------------------------------
# Attention: non-finite rows beside rows and keys that are masked
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_what_nobody_sees_stays_zero(dtype, D):
    """A query that sees no key has o = 0 and dq = 0, a key that no query sees dk =
    dv = 0, whatever the tile's other rows hold."""
    g = gen(D + 1)
    q, k, v, do = qkv(g, 2, 300, 200, 2, 1, D, dtype)  # causal: queries below 100 see nothing
    lengths = torch.tensor([200, 150], dtype=torch.int32, device="cuda")
    k[0, 3], v[0, 4] = math.nan, math.inf
    do[1, 299, 1, 5], q[1, 280, 0, 7] = math.nan, math.inf
    mask = dict(causal=True, key_lengths=lengths)
    o, lse = block.attention_forward(q, k, v, **mask)
    assert bool((o[:, :100] == 0).all()) and bool((lse[:, :, :100] == -math.inf).all())
    assert bool(o[0, 104:].isnan().all())
    dq, dk, dv = block.attention_backward(do, q, k, v, o, lse, **mask)
    assert bool((dq[:, :100] == 0).all())
    assert bool((dk[1, 150:] == 0).all()) and bool((dv[1, 150:] == 0).all())
    assert bool(dv[1, :150].isnan().any())


# ---------------------------------------------------------------------------
# Weight gradient
# ---------------------------------------------------------------------------

def test_weight_grad_of_the_widest_rows():
    """2^30 columns: two rows of codes are further apart than 32 bits reach."""
    tokens, n_in = 64, 1 << 30
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of device memory")
    codes = torch.arange(tokens, device="cuda") % 7 - 3
    q = torch.empty(tokens, n_in, dtype=torch.int8, device="cuda")
    q.copy_(codes.to(torch.int8)[:, None].expand_as(q))
    scales = torch.full((tokens, n_in // 32), 127, dtype=torch.uint8, device="cuda")
    dy = torch.zeros(tokens, 8, dtype=BF16, device="cuda")[:, :1]
    dy[:, 0] = torch.arange(tokens, device="cuda") % 5 - 1
    dw = block.weight_grad(dy, block.PackedActivation(tokens, n_in, q=q, scales=scales))
    want = float((dy[:, 0].double() * codes).sum())  # small whole numbers: exact
    assert bool((dw == want).all())
    block.check()
