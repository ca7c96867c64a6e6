"""The block operators at their edges: the largest sizes they take, infinities in
queries, fp16 gradients far from one, non-finite rows beside masked ones, every
way out of the weight gradient, outputs in place of inputs, scratch sizes."""
import ctypes
import math
import threading

import pytest
import torch

import _block_ref as ref
from mixed_precision_gb300 import _abi as abi
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


class Guarded:
    """A tensor of the given shape between two guard regions of a pattern."""

    def __init__(self, shape, dtype):
        n = math.prod(shape) * torch.empty(0, dtype=dtype).element_size()
        self.raw = torch.full((8192 + (n + 15) // 16 * 16,), 0xA5, dtype=torch.uint8, device="cuda")
        self.n = n
        self.t = self.raw[4096:4096 + n].view(dtype).view(shape)

    def intact(self):
        return bool((self.raw[:4096] == 0xA5).all()) and bool((self.raw[4096 + self.n:] == 0xA5).all())


# ---------------------------------------------------------------------------
# RMSNorm: outputs in the place of inputs
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("rows,cols", [(50, 1024), (7, 33), (3000, 520), (300, 4100)])
def test_norm_in_place(rows, cols):
    g = gen(cols)
    x, res, w = normal(g, rows, cols, dtype=BF16), normal(g, rows, cols, dtype=BF16), normal(g, cols, dtype=BF16)
    y, s, rstd = block.rmsnorm_forward(x, w, residual=res)
    a, b = x.clone(), res.clone()
    got = block.rmsnorm_forward(a, w, residual=b, out=b, sum_out=a)
    assert all(same_bits(p, q) for p, q in zip(got, (y, s, rstd)))
    a = s.clone()
    assert same_bits(block.rmsnorm_forward(a, w, out=a)[0], y)
    with pytest.raises(abi.ZeroError):
        block.rmsnorm_forward(x, w, residual=res, out=a, sum_out=a)


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


def gradients(do, q, k, v, o, lse, causal, lengths, scale):
    """{name: (gradient in 64 bits, tolerance)}, and the largest |p (dp - delta)|.

    p and ds are operands of the type with a power of two taken out that keeps
    the largest possible one below 2^15: each is off by U of itself, and by
    half the type's smallest step, which that power makes 2^-39 of the bound
    |dp - delta| <= |do|_1 max|v| + |delta| of the key head's rows (for p, whose
    bound is 1, 2^-39). The rest as in _block_ref.attention_backward."""
    U, E = ref.U[q.dtype], ref.E
    B, Sq, H, D = q.shape
    Sk, K = k.shape[1], k.shape[2]
    z = lambda t: torch.zeros(t.shape, dtype=torch.float64, device=t.device)  # noqa: E731
    g, top = {n: z(t) for n, t in (("dq", q), ("dk", k), ("dv", v))}, 0.0
    tol = {n: torch.zeros_like(t) for n, t in g.items()}
    for b in range(B):
        n = Sk if lengths is None else int(lengths[b])
        ok = ref.seen(Sq, Sk, causal, 0, n).to(q.device)[:, :n]
        rows = ok.any(1)
        if n == 0:
            continue
        ok = ok[rows]
        for c in range(K):
            kk, vv = k[b, :n, c].double(), v[b, :n, c].double()
            heads = []
            for h in range(c * H // K, (c + 1) * H // K):
                qq, gg, oo = (t[b, rows, h].double() for t in (q, do, o))
                delta = (gg * oo).sum(1, keepdim=True)
                heads.append((h, qq, gg, oo, delta, gg.abs().sum(1, keepdim=True) * vv.abs().max() + delta.abs()))
            bound = max(float(x[-1].max()) for x in heads)
            for h, qq, gg, oo, delta, own in heads:
                ll = lse[b, h, rows].double()[:, None]
                d = 2 * D * E * (qq.abs() @ kk.abs().t() * scale).amax(1, keepdim=True) + 2 ** -17 + 4 * E * ll.abs()
                p = (qq @ kk.t() * scale - ll).masked_fill(~ok, -math.inf).exp()
                x = gg @ vv.t() - delta
                ds = p * x
                top = max(top, float(ds.abs().max()))
                dots = 2 * D * E * (gg.abs() @ vv.abs().t() + (gg * oo).abs().sum(1, keepdim=True))
                off = p * (d * x.abs() + 2 * dots) + U * ds.abs()
                # a row's own bound for dq, the head's for dk
                off_q, off_k = off + 2 ** -39 * own * ok, off + 2 ** -39 * bound * ok
                off_p = p * (d + U) + 2 ** -39 * ok
                g["dq"][b, rows, h] = scale * (ds @ kk)
                tol["dq"][b, rows, h] = scale * (off_q @ kk.abs() + Sk * E * (ds.abs() @ kk.abs()))
                g["dk"][b, :n, c] += scale * (ds.t() @ qq)
                tol["dk"][b, :n, c] += scale * (off_k.t() @ qq.abs() + Sq * E * (ds.abs().t() @ qq.abs()))
                g["dv"][b, :n, c] += p.t() @ gg
                tol["dv"][b, :n, c] += off_p.t() @ gg.abs() + Sq * E * (p.t() @ gg.abs())
    return {n: (g[n], tol[n] + U * g[n].abs() + ref.TINY[q.dtype] / 2) for n in g}, top


def check_range(q, k, v, do, causal=True, lengths=None):
    scale = q.shape[-1] ** -0.5
    o, lse = block.attention_forward(q, k, v, causal=causal, key_lengths=lengths)
    got = block.attention_backward(do, q, k, v, o, lse, causal=causal, key_lengths=lengths)
    want, top = gradients(do, q, k, v, o, lse, causal, lengths, scale)
    for t, name in zip(got, ("dq", "dk", "dv")):
        assert float(want[name][0].abs().max()) < 65504  # the result itself fits the type
        ref.close(t, *want[name], name)
    block.check()
    return top


@pytest.mark.parametrize("D,dout", [(64, 7e3), (128, 6e3)])
def test_attention_fp16_large_gradients(D, dout):
    """p (dp - delta) leaves fp16, dq, dk and dv do not."""
    g = torch.Generator()
    g.manual_seed(1)
    q, k, v, do = ((torch.randn(1, 512, heads, D, generator=g) * scale).to(F16).cuda()
                   for heads, scale in ((2, 1), (1, 1.5), (1, 2), (2, dout)))
    assert check_range(q, k, v, do) > 65504


@pytest.mark.parametrize("Sq,D,dout", [(2048, 64, 1e-4), (1000, 128, 1e-4), (1500, 80, 1e-5)])
def test_attention_fp16_small_gradients(Sq, D, dout):
    """p (dp - delta) is below fp16's normal numbers."""
    q, k, v, do = qkv(gen(Sq), 1, Sq, Sq, 2, 1, D, F16, dout=dout)
    assert check_range(q, k, v, do) < 2 ** -10


def test_attention_fp16_rows_of_unlike_size():
    g = gen(6)
    q, k, v, do = qkv(g, 2, 700, 700, 4, 2, 64, F16, dout=1.0)
    do = (do.float() * torch.exp2(torch.randint(-13, 9, (2, 700, 4, 1), generator=g, device="cuda").float())).half()
    do[0, 100:300] = 0
    lengths = torch.tensor([700, 391], dtype=torch.int32, device="cuda")
    k[1, 391:] = math.nan
    v[1, 391:] = math.inf
    check_range(q, k, v, do, lengths=lengths)
    check_range(q, k, v.mul_(100), (do.float() / 256).half(), causal=False, lengths=lengths)


def test_attention_fp16_weak_weights_in_dv():
    """128 x 100 e^-18, of weights below fp16's smallest normal number."""
    Sk, D = 4096, 64
    q = torch.zeros(1, 128, 1, D, dtype=F16, device="cuda")
    k = torch.zeros(1, Sk, 1, D, dtype=F16, device="cuda")
    q[..., 0], k[0, 7, 0, 0] = 12, 12  # a logit of 12 * 12 / 8
    v = torch.ones_like(k)
    o, lse = block.attention_forward(q, k, v)
    _, _, dv = block.attention_backward(torch.full_like(q, 100), q, k, v, o, lse)
    want = 128 * 100 * math.exp(-18.0) / (1 + (Sk - 1) * math.exp(-18.0))
    weak = torch.cat([dv[0, :7], dv[0, 8:]]).double()
    # the weight's rounding and the result's, the exponent's; half a step of the smallest numbers
    assert float((weak - want).abs().max()) <= want * (2 * ref.U[F16] + 2 ** -14) + 2 ** -25


@pytest.mark.parametrize("D", [64, 128])
def test_attention_fp16_repeats_and_replays(D):
    """The bounds are collected by maxima, the same in any order; captured, the three
    kernels are ordered as in a stream."""
    q, k, v, do = qkv(gen(D), 2, 700, 900, 8, 2, D, F16)
    lengths = torch.tensor([900, 611], dtype=torch.int32, device="cuda")
    mask = dict(causal=True, key_lengths=lengths)
    o, lse = block.attention_forward(q, k, v, **mask)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = block.attention_backward(do, q, k, v, o, lse, **mask)
    for scale in (1.0, 2.0 ** -9, 300.0):
        do.copy_(normal(gen(D + 1), *do.shape, scale=scale))
        v.copy_(normal(gen(D + 2), *v.shape, scale=1 / scale))
        a = block.attention_forward(q, k, v, **mask)
        o.copy_(a[0])
        lse.copy_(a[1])
        want = block.attention_backward(do, q, k, v, o, lse, **mask)
        for _ in range(3):
            graph.replay()
            again = block.attention_backward(do, q, k, v, o, lse, **mask)
            assert all(same_bits(x, y) and same_bits(x, z) for x, y, z in zip(want, held, again))
        assert all(bool(x.isfinite().all()) for x in want)


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
# Attention: outputs in the place of inputs
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,D", [(F16, 64), (BF16, 128), (BF16, 72)])
def test_attention_in_place(dtype, D):
    q, k, v, do = qkv(gen(D), 3, 700, 500, 4, 2, D, dtype)
    lengths = torch.tensor([500, 0, 333], dtype=torch.int32, device="cuda")
    mask = dict(causal=True, key_lengths=lengths)
    o, lse = block.attention_forward(q, k, v, **mask)
    want = block.attention_backward(do, q, k, v, o, lse, **mask)
    held = q.clone()
    o2, lse2 = block.attention_forward(held, k, v, out=held, **mask)
    assert o2 is held and same_bits(o, o2) and same_bits(lse, lse2)
    for first in (0, 1):  # dk over k and dv over v, and the other way round
        a, b, c = o.clone(), k.clone(), v.clone()
        places = (b, c) if first == 0 else (c, b)
        got = block.attention_backward(do, q, b, c, a, lse, dq=a, dk=places[0], dv=places[1], **mask)
        assert all(same_bits(x, y) for x, y in zip(got, want))


def test_attention_gradients_in_one_buffer():
    """q, k and v as parts of a projection's rows, dq, dk and dv as parts of its gradient."""
    g = gen(4)
    B, S, H, K, D = 2, 300, 4, 2, 64
    rows = normal(g, B, S, H + 2 * K, D, dtype=BF16)
    grad = torch.full_like(rows, math.nan)
    parts = lambda t: (t[:, :, :H], t[:, :, H:H + K], t[:, :, H + K:])  # noqa: E731
    q, k, v = parts(rows)
    do = normal(g, B, S, H, D, dtype=BF16)
    o, lse = block.attention_forward(q, k, v, causal=True)
    dq, dk, dv = parts(grad)
    block.attention_backward(do, q, k, v, o, lse, causal=True, dq=dq, dk=dk, dv=dv)
    want = block.attention_backward(do, *(t.contiguous() for t in (q, k, v)), o, lse, causal=True)
    assert same_bits(grad, torch.cat(want, 2))


def test_attention_refuses_outputs_over_inputs():
    q, k, v, do = qkv(gen(5), 1, 64, 64, 2, 2, 64, BF16)
    o, lse = block.attention_forward(q, k, v)
    for call in (lambda: block.attention_forward(q, k, v, out=k), lambda: block.attention_forward(q, k, v, out=v),
                 lambda: block.attention_backward(do, q, k, v, o, lse, dq=q),
                 lambda: block.attention_backward(do, q, k, v, o, lse, dq=do),
                 lambda: block.attention_backward(do, q, k, v, o, lse, dk=q),
                 lambda: block.attention_backward(do, q, k, v, o, lse, dv=do),
                 lambda: block.attention_backward(do, q, k, v, o, lse, dk=k, dv=k)):
        with pytest.raises(abi.ZeroError) as e:
            call()
        assert e.value.code == abi.ZERO_ERR_INVALID


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


# few and many tokens; outputs that fill the machine (a tile's sums leave by bulk
# stores or additions) or do not (clusters); rows that are whole vectors or not;
# above 1024 tokens fp32 sums are moved in rounded runs
@pytest.mark.parametrize("tokens,n_out,n_in", [
    (130, 5000, 4104), (1000, 4104, 5000), (1024, 8200, 2056), (1030, 3000, 4100), (1100, 4104, 5000), (2500, 5001, 4100),
    (1100, 4100, 4105), (200, 3001, 4110), (3000, 300, 520), (700, 136, 521), (65, 40, 72), (1500, 20, 33)])
def test_weight_grad_accumulates_every_way_out(tokens, n_out, n_in):
    g = gen(tokens + n_out)
    pad = (-n_out) % 8
    def micro(seed):
        dy = normal(gen(seed), tokens, n_out + pad, dtype=BF16)[:, :n_out]
        return dy, block.PackedActivation(tokens, n_in).save(normal(gen(seed + 1), tokens, n_in, dtype=BF16, scale=2))
    main = normal(g, n_out, n_in)
    out = Guarded((n_out, n_in), F32)
    out.t.copy_(main)
    want, size = main.double(), main.double().abs()
    total = main.clone()
    for seed in (11, 21):  # two micro-batches in a row
        dy, p = micro(seed)
        one = block.weight_grad(dy, p, dtype=F32)
        block.weight_grad(dy, p, out=out.t, accumulate=True)
        total += one  # the addition to what is there is one fp32 rounding
        assert same_bits(out.t, total) and out.intact()
        x = p.restore(BF16).double()
        want = want + dy.double().t() @ x
        size = size + dy.double().abs().t() @ x.abs()
    ref.close(out.t, want, (tokens / 8 + 32) * 2 * ref.E * size + 4 * ref.E * want.abs(), "dw")
    plain = Guarded((n_out, n_in), F32)
    block.weight_grad(dy, p, out=plain.t)
    assert same_bits(plain.t, one) and plain.intact()
    block.check()


@pytest.mark.parametrize("tokens,n_out,n_in", [(8192, 264, 328), (8192, 4096, 4096), (40000, 64, 96)])
def test_weight_grad_fp32_sums_are_rounded(tokens, n_out, n_in):
    """Sums of one sign, where truncated additions would all err the same way. A run
    of 64 additions is off by 64 truncations of at most 2^-24 of it (2^-18), the runs'
    rounded sums by one rounding each in random directions (2^-24 sqrt(runs) in the
    mean, six times that at the worst of all outputs)."""
    g = gen(tokens)
    dy = (torch.rand(tokens, n_out, generator=g, device="cuda") + 0.5).to(BF16)
    x = (torch.rand(tokens, n_in, generator=g, device="cuda") + 0.5).to(BF16)
    p = block.PackedActivation(tokens, n_in).save(x)
    dw = block.weight_grad(dy, p, dtype=F32)
    n = min(n_out, 256)  # columns are enough
    want = dy[:, :n].double().t() @ p.restore(BF16).double()
    rel = (dw[:n].double() - want) / want
    assert float(rel.mean().abs()) < 1e-6 and float(rel.abs().max()) < 1e-6 + 6 * ref.E * math.sqrt(tokens / 1024)


@pytest.mark.parametrize("dtype,tokens", [(F16, 1 << 20), (F16, 1 << 18), (BF16, 1 << 20)])
def test_weight_grad_of_many_tokens(dtype, tokens):
    """16-bit results of very long sums of one sign, which are made in rounded runs:
    the sums' own error stays below a sixteenth of the type's rounding. The mean
    over the outputs, spread over a binade, averages the rounding away (as it does
    for the exact sums)."""
    g = gen(3)
    n_out, n_in = 128, 128
    spread = torch.exp2(torch.rand(n_out, generator=g, device="cuda")) * (256 / tokens)
    dy = ((torch.rand(tokens, n_out, generator=g, device="cuda") + 0.5) * spread).to(dtype)
    x = ((torch.rand(tokens, n_in, generator=g, device="cuda") + 0.5) *
         torch.exp2(torch.rand(n_in, generator=g, device="cuda"))).to(dtype)
    p = block.PackedActivation(tokens, n_in).save(x)
    dw = block.weight_grad(dy, p)
    want = dy.double().t() @ p.restore(dtype).double()
    u, n = ref.U[dtype], want.numel()
    rounded = (want.to(dtype).double() - want) / want
    assert float(rounded.mean().abs()) < 6 * u / math.sqrt(3 * n)
    rel = (dw.double() - want) / want
    assert float(rel.mean().abs()) < u / 16 + 6 * u / math.sqrt(3 * n)
    assert float(rel.abs().max()) < u + u / 16


# ---------------------------------------------------------------------------
# Scratch of exactly the reported size
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("rows,cols,pad", [(1, 8, 0), (33, 1024, 0), (700, 3000, 0), (2500, 2048, 0), (5000, 512, 8),
                                           (65536, 128, 0), (40000, 256, 0), (777, 33, 0), (50, 72, 3), (3, 20000, 0)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_norm_backward_scratch_is_enough(rows, cols, pad, dtype):
    g = gen(rows)
    x, dy, dsum = (normal(g, rows, cols + pad, dtype=dtype)[:, :cols] for _ in range(3))
    w = normal(g, cols, dtype=dtype)
    rstd = x.float().square().mean(1).rsqrt()
    code = block.DTYPE_CODE[dtype]
    desc = abi.RMSNORM_DESC.pack(rows, cols, *[cols + pad if rows > 1 else cols] * 3, code, code, 0.0)
    space = Guarded((abi.zero_rmsnorm_backward_workspace(desc),), torch.uint8)
    for extra in (None, dsum):
        dx, dw = torch.empty(rows, cols, dtype=dtype, device="cuda"), torch.empty(cols, device="cuda")
        abi.zero_rmsnorm_backward(desc, dy.data_ptr(), x.data_ptr(), w.data_ptr(), rstd.data_ptr(),
                                  None if extra is None else extra.data_ptr(), dx.data_ptr(), dw.data_ptr(), abi.ZERO_F32,
                                  space.t.data_ptr(), space.n, torch.cuda.current_stream().cuda_stream)
        want = block.rmsnorm_backward(dy, x, w, rstd, dsum=extra, dweight_dtype=F32)
        assert same_bits(dx, want[0]) and same_bits(dw, want[1]) and space.intact()


@pytest.mark.parametrize("B,Sq,Sk,H,K,D", [(1, 1, 1, 1, 1, 8), (2, 300, 200, 4, 2, 64), (3, 129, 700, 6, 1, 128),
                                           (5, 100, 1000, 5, 5, 72), (40, 100, 130, 1, 1, 64)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_backward_scratch_is_enough(B, Sq, Sk, H, K, D, dtype):
    q, k, v, do = qkv(gen(B), B, Sq, Sk, H, K, D, dtype)
    o, lse = block.attention_forward(q, k, v, causal=True)
    tensors = (q, k, v, o, do, q, k, v)
    desc = abi.zero_attention_desc(B, Sq, Sk, H, K, D, block.DTYPE_CODE[dtype], 1, 0, 0, D ** -0.5,
                                   *[(ctypes.c_int64 * 3)(*t.stride()[:3]) for t in tensors])
    space = Guarded((abi.zero_attention_backward_workspace(desc),), torch.uint8)
    out = [torch.empty_like(t) for t in (q, k, v)]
    abi.zero_attention_backward(desc, do.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                None, *[t.data_ptr() for t in out], space.t.data_ptr(), space.n,
                                torch.cuda.current_stream().cuda_stream)
    want = block.attention_backward(do, q, k, v, o, lse, causal=True)
    assert all(same_bits(a, b) for a, b in zip(out, want)) and space.intact()


# ---------------------------------------------------------------------------
# Waits that give up
# ---------------------------------------------------------------------------

def timed_out():
    try:
        block.check()
    except abi.ZeroError as e:
        assert e.code == abi.ZERO_ERR_TIMEOUT
        return True
    return False


@pytest.mark.parametrize("kernels", range(4))
def test_a_wait_that_gives_up_is_reported(kernels):
    """Once, to every thread, from whichever stream; the operators run on."""
    timed_out()  # what other tests may have left to this thread
    assert not timed_out()
    side = torch.cuda.Stream()
    told = []

    def other():
        told.append(timed_out())  # a thread's first call tells it of all since the start
        told.append(timed_out())
        abi.zero_selftest_operator_timeout(kernels, 1000, side.cuda_stream)
        side.synchronize()
        told.append(timed_out())
        told.append(timed_out())

    t = threading.Thread(target=other)
    t.start()
    t.join()
    assert told[1:] == [False, True, False]
    assert timed_out() and not timed_out()
    x, w = normal(gen(1), 4, 64), torch.ones(64, device="cuda")
    y, _, _ = block.rmsnorm_forward(x, w)
    assert bool(y.isfinite().all()) and not timed_out()
