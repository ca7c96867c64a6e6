"""The expert layer's operators on the GPU against their definitions in 64 bits:
routing, rows to the experts and back, the experts' products. Sizes, types,
strides and masks where they can go wrong, with the tolerances of _experts_ref."""
import math
import os
import subprocess
import sys

import pytest
import torch

import _experts_ref as ref
from _block_ref import E, TINY, U, close
from mixed_precision_gb300 import block, experts

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
I32 = torch.int32


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


# ---------------------------------------------------------------------------
# Routing
# ---------------------------------------------------------------------------

def check_route(logits, k, normalize, r=None):
    if r is None:
        r = experts.route(logits, k, normalize=normalize)
    want = ref.route(logits, k, normalize)
    for n in ("experts", "offsets", "source", "place"):
        assert torch.equal(getattr(r, n).cpu(), want[n]), n
    close(r.weights.cpu(), want["weights"], ref.weights_tol(logits, want["weights"]), "weights")
    return r, want


@pytest.mark.parametrize("tokens,n,k", [(1, 1, 1), (1, 16, 2), (33, 16, 2), (7, 3, 3), (100, 33, 5), (65, 64, 8),
                                        (257, 128, 8), (31, 200, 4), (40, 256, 32), (50, 1024, 32), (3, 1000, 1),
                                        (5000, 8, 2), (4865, 17, 3)])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("normalize", [True, False])
def test_route(tokens, n, k, dtype, normalize):
    g = gen(tokens * 31 + n)
    logits = normal(g, tokens, n, dtype=dtype, scale=2)  # 16-bit ones tie
    check_route(logits, k, normalize)
    check_route((logits.float().round() + 0.0).to(dtype), k, normalize)


def test_route_special_logits():
    inf, nan = math.inf, math.nan
    rows = [[0.0, -0.0, 0.0, -0.0], [-inf] * 4, [-inf, 1.0, -inf, -inf], [-inf, 3.0, 1.0, -inf], [3e38, -3e38, 1.0, 2.0],
            [1e-45, 0.0, -1e-45, 2e-45], [-3.4e38, -3.3e38, -inf, -3.4e38]]
    for normalize in (True, False):
        check_route(torch.tensor(rows, device="cuda"), 3, normalize)
        check_route(torch.tensor(rows, device="cuda").to(BF16), 2, normalize)
    # infinities and NaN: the choice is defined, the weights are NaN
    r = experts.route(torch.tensor([[1.0, inf, 0.0, inf], [nan, 2.0, inf, 3.0], [0.0, 5.0, nan, nan]], device="cuda"), 2)
    assert r.experts.tolist() == [[1, 3], [0, 2], [2, 3]]
    assert bool(r.weights.isnan().all()) and r.offsets.tolist() == [0, 1, 2, 4, 6]


@pytest.mark.parametrize("normalize", [True, False])
def test_route_padding(normalize):
    g = gen(5)
    logits = normal(g, 700, 24)
    logits[torch.rand(700, generator=g, device="cuda") < 0.4] = -math.inf
    logits[:, 5] = -math.inf
    r, _ = check_route(logits, 4, normalize)
    assert int(r.offsets[-1]) < 700 * 4
    all_padding = torch.full((70, 24), -math.inf, device="cuda")
    r, _ = check_route(all_padding, 4, normalize)
    assert int(r.offsets[-1]) == 0


def test_route_strides_and_no_tokens():
    g = gen(6)
    wide = normal(g, 300, 61)
    check_route(wide[:, 3:40], 3, True)
    r = experts.route(torch.empty(0, 16, device="cuda"), 2)
    assert r.offsets.tolist() == [0] * 17 and r.weights.shape == (0, 2)
    x = experts.gather(torch.empty(0, 64, device="cuda"), r)
    assert x.shape == (0, 64)
    assert experts.forward(torch.empty(0, 64, device="cuda", dtype=BF16), torch.ones(16, 8, 64, device="cuda", dtype=BF16),
                           r.offsets).shape == (0, 8)


@pytest.mark.parametrize("tokens,n,k", [(1, 2, 2), (33, 16, 2), (100, 33, 5), (257, 128, 8), (50, 1024, 32), (9, 300, 7)])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("normalize", [True, False])
def test_route_backward(tokens, n, k, dtype, normalize):
    g = gen(tokens + n)
    logits = normal(g, tokens, n + 3, dtype=dtype)[:, :n]
    logits[::5] = -math.inf
    logits[::3, 0] = -math.inf
    r = experts.route(logits, k, normalize=normalize)
    dw = normal(g, tokens, k)
    dw[r.experts < 0] = math.nan  # nothing was taken there
    got = experts.route_backward(dw, logits, r)
    # by the formula in 64 bits, from the kernel's weights
    w, taken = r.weights.double(), r.experts >= 0
    d = torch.where(taken, dw.double(), 0.0)
    s = (w * d).sum(1, keepdim=True)
    size_s = (w * d).abs().sum(1, keepdim=True)
    at = torch.where(taken, r.experts, n).long()
    wide = torch.zeros(tokens, n + 1, dtype=torch.float64, device="cuda")
    if normalize:
        want = wide.scatter(1, at, w * (d - s))[:, :n]
        size = wide.scatter(1, at, w * (d.abs() + size_s))[:, :n]
    else:
        p = torch.nan_to_num(torch.softmax(logits.double(), 1), nan=0.0)
        want = wide.scatter(1, at, w * d)[:, :n] - p * s
        size = wide.scatter(1, at, (w * d).abs())[:, :n] + p * size_s
    # a sum of 5 shuffles; p as the weights; the last additions
    spread = 12.0  # of the logits: normal ones lie within 6 of zero
    rel = 8 * E + 2 * (spread * E + 4 * E) + (n / 32 + 8) * E
    close(got, want, rel * size + U[dtype] * want.abs() + TINY[dtype], "dlogits")


def test_route_gradient_by_differences():
    """d(sum of c * weights) / dlogits against central differences of the definition."""
    g = gen(9)
    logits, c = normal(g, 20, 12), normal(g, 20, 3)
    for normalize in (True, False):
        r = experts.route(logits, 3, normalize=normalize)
        got = experts.route_backward(c, logits, r).double()
        at = r.experts.long()

        def weights(v):
            t = v.gather(1, at)
            return (t - torch.logsumexp(t if normalize else v, 1, keepdim=True)).exp()

        h = 1e-5
        for e in range(12):
            step = torch.zeros(12, dtype=torch.float64, device="cuda")
            step[e] = h
            want = ((weights(logits.double() + step) - weights(logits.double() - step)) * c.double()).sum(1) / (2 * h)
            # differences: h^2 of the third derivative and 1e-16 / h; the kernel: fp32
            assert float((got[:, e] - want).abs().max()) < 1e-5


# ---------------------------------------------------------------------------
# Rows to the experts and back
# ---------------------------------------------------------------------------

ROWS = [(1, 8, 2, 64), (33, 16, 2, 2048), (100, 33, 5, 72), (65, 8, 8, 1000), (50, 40, 32, 264), (9, 4, 1, 1), (70, 6, 3, 33),
        (600, 16, 4, 520)]


def routed(g, tokens, n, k, padded):
    logits = normal(g, tokens, n)
    if padded:
        logits[torch.rand(tokens, generator=g, device="cuda") < 0.3] = -math.inf
        if n > k:
            logits[:, 1] = -math.inf
    return experts.route(logits, k)


@pytest.mark.parametrize("tokens,n,k,hidden", ROWS)
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("padded", [False, True])
def test_gather_and_combine(tokens, n, k, hidden, dtype, padded):
    g = gen(tokens + hidden)
    r = routed(g, tokens, n, k, padded)
    last = int(r.offsets[-1])
    x = normal(g, tokens, hidden + 8, dtype=dtype)[:, :hidden]
    rows = experts.gather(x, r)
    slot = r.source[:last].long()
    assert torch.equal(rows[:last], x[slot // k]) and not bool(rows[last:].any())

    y = normal(g, tokens * k, hidden + 16, dtype=dtype)[:, 8:hidden + 8]
    y[last:] = math.nan  # rows of nobody
    w = r.weights.view(-1)[slot].double()
    for weighted in (True, False):
        part = y[:last].double() * (w[:, None] if weighted else 1.0)
        want = torch.zeros(tokens, hidden, dtype=torch.float64, device="cuda").index_add_(0, slot // k, part)
        size = torch.zeros_like(want).index_add_(0, slot // k, part.abs())
        got = experts.combine(y, r, weighted=weighted)
        close(got, want, 2 * k * E * size + U[dtype] * want.abs() + TINY[dtype], "combined")

    dout = normal(g, tokens, hidden + 24, dtype=dtype)[:, :hidden]
    dy, dw = experts.combine_backward(dout, y, r)
    want = w[:, None] * dout.double()[slot // k]
    close(dy[:last], want, (U[dtype] + E) * want.abs() + TINY[dtype], "dy")
    assert not bool(dy[last:].any())
    d = dout.double()[slot // k]
    full, size = torch.zeros(tokens * k, dtype=torch.float64, device="cuda"), torch.zeros(tokens * k, device="cuda").double()
    full[slot], size[slot] = (d * y[:last].double()).sum(1), (d * y[:last].double()).abs().sum(1)
    # a lane's chain is hidden / 32 long (element by element too), then 5 shuffles
    close(dw, full.view(tokens, k), ((hidden / 32 + 16) * E * size).view(tokens, k) + 2.0 ** -149, "dweights")


def test_the_same_token_to_every_expert_and_far_rows():
    """All rows of one token; rows whose offsets pass 32 bits of bytes."""
    r = experts.route(torch.zeros(1, 32, device="cuda"), 32)
    x = normal(gen(1), 1, 128, dtype=BF16)
    assert torch.equal(experts.gather(x, r), x.expand(32, 128))
    g = gen(2)
    r = experts.route(normal(g, 3, 4), 2)
    base = torch.empty(3 * 2 ** 30 + 256, dtype=BF16, device="cuda")
    x = base.as_strided((3, 128), (2 ** 30 + 64, 1))
    x.copy_(normal(g, 3, 128))
    assert torch.equal(experts.gather(x, r), x[r.source.long() // 2])


def test_places_out_of_range_reach_nothing():
    """What a routing's device arrays say is not trusted: a place outside the order is passed by."""
    g = gen(3)
    r = experts.route(normal(g, 10, 4), 2)
    bad = experts.Routing(4, True, r.weights, r.experts, r.offsets, r.source, r.place + 2 ** 20)
    x = normal(g, 10, 64)
    held = torch.full((20, 64), 7.0, device="cuda")
    experts.gather(x, bad, out=held)
    assert bool((held == 7).all())
    assert not bool(experts.combine(normal(g, 20, 64), bad).any())


# ---------------------------------------------------------------------------
# The experts' products
# ---------------------------------------------------------------------------

def offsets_of(counts, before=0):
    return torch.tensor([before] + [before + sum(counts[:i + 1]) for i in range(len(counts))], dtype=I32, device="cuda")


COUNTS = [([1],), ([5, 0, 3],), ([0, 0, 0],), ([64, 64],), ([256, 0, 1, 255],), ([300, 17, 513, 2, 31, 33],),
          ([1] * 40,), ([0, 1030],), ([15, 16, 17, 47, 48, 49, 63, 64, 65, 127, 128, 129],), ([3] * 130 + [0] * 20,)]
SIZES = [(64, 64), (8, 8), (200, 136), (256, 512), (520, 264), (33, 72), (130, 1000), (16, 2048)]


def padded_rows(g, rows, cols, dtype, scale=1.0):
    """Rows that start on 16 bytes, their padding NaN."""
    t = torch.full((rows, (cols + 7) // 8 * 8 + 8), math.nan, dtype=dtype, device="cuda")
    t[:, :cols] = normal(g, rows, cols, scale=scale)
    return t[:, :cols]


def check_products(counts, n_out, n_in, dtype):
    g = gen(n_out + n_in + sum(counts))
    rows, extra = sum(counts), 5  # rows of no expert behind the last
    off = offsets_of(counts)
    o = off.tolist()
    x = padded_rows(g, rows + extra, n_in, dtype)
    dy = padded_rows(g, rows + extra, n_out, dtype)
    x[rows:], dy[rows:] = math.nan, math.inf
    w = normal(g, len(counts), n_out, (n_in + 7) // 8 * 8, dtype=dtype)[:, :, :n_in]
    y = experts.forward(x, w, off)
    want, size = ref.forward(x[:rows], w, o)
    close(y[:rows], want, ref.product_tol(n_in, size, want, dtype, dtype), "y")
    dx = experts.input_grad(dy, w, off)
    want, size = ref.input_grad(dy[:rows], w, o)
    close(dx[:rows], want, ref.product_tol(n_out, size, want, dtype, dtype), "dx")
    assert not bool(y[rows:].any()) and not bool(dx[rows:].any())
    want, size = ref.weight_grad(dy[:rows], x[:rows], o)
    for out in (dtype, F32):
        dw = experts.weight_grad(dy, x, off, dtype=out)
        close(dw, want, ref.product_tol(max(counts), size, want, dtype, out, run=1024), f"dw {out}")
    start = normal(g, *want.shape)
    dw = start.clone()
    experts.weight_grad(dy, x, off, out=dw, accumulate=True)
    tol = ref.product_tol(max(counts), size, want, dtype, F32, run=1024)
    close(dw, want + start.double(), tol + E * (want + start.double()).abs(), "dw added")
    experts.check()


@pytest.mark.parametrize("counts", [c[0] for c in COUNTS], ids=lambda c: f"{len(c)}x{sum(c)}")
@pytest.mark.parametrize("n_out,n_in", SIZES)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_products(counts, n_out, n_in, dtype):
    check_products(counts, n_out, n_in, dtype)


@pytest.mark.parametrize("counts,n_out,n_in", [([2000, 1, 2096, 0], 512, 768), ([700] * 9, 1024, 512), ([4100], 768, 520),
                                               ([1, 2, 3, 4], 2048, 4096), ([9000, 90], 264, 256)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_products_of_many_tiles(counts, n_out, n_in, dtype):
    check_products(counts, n_out, n_in, dtype)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_weight_grad_of_one_sign(dtype):
    """Long sums of terms of one sign, where cut additions would add up: fp32 results by rounded runs."""
    g = gen(3)
    off = offsets_of([20000, 1500])
    x, dy = normal(g, 21500, 136, dtype=dtype).abs(), normal(g, 21500, 72, dtype=dtype).abs()
    want, size = ref.weight_grad(dy, x, off.tolist())
    dw = experts.weight_grad(dy, x, off, dtype=F32)
    close(dw, want, ref.product_tol(20000, size, want, dtype, F32, run=1024), "dw")
    dw = experts.weight_grad(dy, x, off)
    close(dw, want, ref.product_tol(20000, size, want, dtype, dtype), "dw")


def test_products_over_flat_buffers():
    """All experts' matrices as a view of a flat parameter buffer (gate, up and down of each in turn), and
    their gradients written into the flat gradient; nothing else there changes."""
    g = gen(4)
    n, hidden, ffn, rows = 5, 264, 136, 400
    each = 3 * ffn * hidden
    flat, grad = normal(g, n * each + 64, dtype=BF16), normal(g, n * each + 64, dtype=BF16)
    both = lambda t: t.as_strided((n, 2 * ffn, hidden), (each, hidden, 1), 0)  # noqa: E731
    down = lambda t: t.as_strided((n, hidden, ffn), (each, ffn, 1), 2 * ffn * hidden)  # noqa: E731
    off = offsets_of([100, 0, 7, 200, 93])
    x, act = normal(g, rows, hidden, dtype=BF16), normal(g, rows, ffn, dtype=BF16)
    want, size = ref.forward(x, both(flat), off.tolist())
    close(experts.forward(x, both(flat), off), want, ref.product_tol(hidden, size, want, BF16, BF16))
    want, size = ref.input_grad(x, down(flat), off.tolist())
    close(experts.input_grad(x, down(flat), off), want, ref.product_tol(hidden, size, want, BF16, BF16))
    before = grad.clone()
    experts.weight_grad(x, act, off, out=down(grad))
    want, size = ref.weight_grad(x, act, off.tolist())
    close(down(grad), want, ref.product_tol(200, size, want, BF16, BF16))
    assert torch.equal(both(grad), both(before)) and torch.equal(grad[n * each:], before[n * each:])


def test_outputs_with_free_strides():
    g = gen(5)
    off = offsets_of([70, 30])
    x, w, dy = normal(g, 100, 72, dtype=F16), normal(g, 2, 40, 72, dtype=F16), normal(g, 100, 40, dtype=F16)
    wide = torch.full((100, 91), 5.0, dtype=F16, device="cuda")
    y = experts.forward(x, w, off, out=wide[:, 11:51])
    assert torch.equal(y, experts.forward(x, w, off)) and bool((wide[:, :11] == 5).all()) and bool((wide[:, 51:] == 5).all())
    wide.fill_(5.0)
    dx = experts.input_grad(dy, w, off, out=wide[:, 3:75])
    assert torch.equal(dx, experts.input_grad(dy, w, off)) and bool((wide[:, :3] == 5).all())
    big = torch.full((2, 45, 77), 5.0, device="cuda")
    dw = experts.weight_grad(dy, x, off, out=big[:, 2:42, 3:75])
    assert torch.equal(dw, experts.weight_grad(dy, x, off, dtype=F32))
    assert float(big.sum() - dw.sum()) == pytest.approx(5.0 * (2 * 45 * 77 - 2 * 40 * 72), rel=1e-4)


def test_offsets_out_of_range_stay_inside():
    """Offsets are clamped to the rows; the results of sound experts do not change."""
    g = gen(6)
    x, w = normal(g, 50, 64, dtype=BF16), normal(g, 3, 64, 64, dtype=BF16)
    off = torch.tensor([0, 20, 50, 2 ** 30], dtype=I32, device="cuda")
    want = experts.forward(x, w, torch.tensor([0, 20, 50, 50], dtype=I32, device="cuda"))
    assert torch.equal(experts.forward(x, w, off), want)
    off = torch.tensor([-7, 20, 50, 10], dtype=I32, device="cuda")
    assert torch.equal(experts.forward(x, w, off)[:50], want)
    dw = experts.weight_grad(x, x, off)
    assert torch.equal(dw[0], experts.weight_grad(x, x, torch.tensor([0, 20], dtype=I32, device="cuda"))[0])
    assert not bool(dw[2].any())


def test_another_experts_rows_reach_nothing():
    """NaN and inf in one expert's rows and weights, beside others' in the same tiles."""
    g = gen(7)
    counts = [33, 5, 90, 40]
    off = offsets_of(counts)
    x, dy, w = normal(g, 168, 72, dtype=F16), normal(g, 168, 136, dtype=F16), normal(g, 4, 136, 72, dtype=F16)
    clean = [experts.forward(x, w, off), experts.input_grad(dy, w, off), experts.weight_grad(dy, x, off, dtype=F32)]
    x2, dy2, w2 = x.clone(), dy.clone(), w.clone()
    x2[33:38], dy2[33:38], w2[1] = math.nan, math.inf, math.nan
    for a, b in zip(clean[:2], (experts.forward(x2, w2, off), experts.input_grad(dy2, w2, off))):
        assert torch.equal(a[:33], b[:33]) and torch.equal(a[38:], b[38:]) and not bool(b[33:38].isfinite().any())
    dw = experts.weight_grad(dy2, x2, off, dtype=F32)
    assert bool(dw[1].isnan().all())
    for e in (0, 2, 3):
        assert torch.equal(dw[e], clean[2][e])


# ---------------------------------------------------------------------------
# As a user's program runs them
# ---------------------------------------------------------------------------

def layer(logits, x, w_up, w_down, dout, k):
    """Forward and backward of an expert layer with a ReLU between: (out, dx, dw_up, dw_down, dlogits)."""
    r = experts.route(logits, k)
    rows = experts.gather(x, r)
    h = experts.forward(rows, w_up, r.offsets)
    act = h.relu()
    y = experts.forward(act, w_down, r.offsets)
    out = experts.combine(y, r)
    dy, dweights = experts.combine_backward(dout, y, r)
    d_act = experts.input_grad(dy, w_down, r.offsets)
    dw_down = experts.weight_grad(dy, act, r.offsets, dtype=F32)
    dh = d_act * (h > 0)
    dw_up = experts.weight_grad(dh, rows, r.offsets, dtype=F32)
    dx = experts.combine(experts.input_grad(dh, w_up, r.offsets), r, weighted=False)
    return out, dx, dw_up, dw_down, experts.route_backward(dweights, logits, r)


def layer_inputs(seed, tokens=300, n=8, hidden=136, ffn=264, dtype=BF16):
    g = gen(seed)
    logits = normal(g, tokens, n)
    logits[torch.rand(tokens, generator=g, device="cuda") < 0.1] = -math.inf
    logits[:, 3] = -math.inf  # an idle expert
    return (logits, normal(g, tokens, hidden, dtype=dtype), normal(g, n, ffn, hidden, dtype=dtype, scale=hidden ** -0.5),
            normal(g, n, hidden, ffn, dtype=dtype, scale=ffn ** -0.5), normal(g, tokens, hidden, dtype=dtype))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_layer_matches_autograd(dtype):
    """The whole layer against autograd in 64 bits of the same choice. On the longest path (dx) lie seven
    roundings to dtype, each of relative size U at most and independent: their rms is below sqrt(7) U of
    the result's size; 4 U is allowed in norm."""
    logits, x, w_up, w_down, dout = inputs = layer_inputs(1, dtype=dtype)
    got = layer(*inputs, 2)
    real = [t.double().requires_grad_() for t in (logits, x, w_up, w_down)]
    r = experts.route(logits, 2)
    at, taken = r.experts.clamp(min=0).long(), r.experts >= 0
    picked = real[0].gather(1, at)
    w = torch.where(taken, torch.softmax(torch.where(taken, picked, -1e30), 1), 0.0)
    h = torch.einsum("th,tkfh->tkf", real[1], real[2][at]).relu()
    y = torch.einsum("tkf,tkhf->tkh", h, real[3][at])
    out = (y * w[..., None]).sum(1)
    out.backward(dout.double())
    want = [out.detach(), real[1].grad, real[2].grad, real[3].grad, torch.nan_to_num(real[0].grad)]
    for name, a, b in zip(("out", "dx", "dw_up", "dw_down", "dlogits"), got, want):
        err = float((a.double() - b).norm() / b.norm())
        assert err < 4 * U[dtype], (name, err)
    assert not bool(got[2][3].any()) and not bool(got[3][3].any())


def test_layer_captured_and_replayed():
    """Two captured layers that share nothing but the code, replayed in turn with new inputs: bit for bit the
    eager results."""
    held = [list(layer_inputs(s)) for s in (2, 3)]
    stream = torch.cuda.Stream()
    graphs, outs = [], []
    with torch.cuda.stream(stream):
        for inputs in held:
            layer(*inputs, 2)
            stream.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                outs.append(layer(*inputs, 2))
            graphs.append(graph)
    torch.cuda.synchronize()
    for seed in (4, 5):
        for i, inputs in enumerate(held):
            for t, new in zip(inputs, layer_inputs(seed + 10 * i)):
                t.copy_(new)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for inputs, out in zip(held, outs):
            for a, b in zip(out, layer(*inputs, 2)):
                assert torch.equal(a, b)
    experts.check()


def test_repeated_and_concurrent_calls_agree():
    inputs = layer_inputs(6, tokens=900)
    want = layer(*inputs, 2)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    results = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                results.append(layer(*inputs, 2))
    torch.cuda.synchronize()
    for got in results:
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_side_stream():
    """`stream` other than the current one: outputs belong to it, inputs are kept for it."""
    g = gen(8)
    logits, x, w, _, _ = layer_inputs(9)
    want = experts.forward(experts.gather(x, experts.route(logits, 2)), w, experts.route(logits, 2).offsets)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = experts.route(logits, 2, stream=side)
    y = experts.forward(experts.gather(x, r, stream=side), w, r.offsets, stream=side)
    side.synchronize()
    assert torch.equal(y, want)


def test_python_refusals():
    g = gen(10)
    x, w = normal(g, 20, 64, dtype=BF16), normal(g, 4, 32, 64, dtype=BF16)
    off = offsets_of([5, 5, 5, 5])
    for bad in (lambda: experts.forward(x.float(), w, off), lambda: experts.forward(x, w.half(), off),
                lambda: experts.forward(x[:, :56], w, off), lambda: experts.forward(x.t(), w, off),
                lambda: experts.forward(x, w, off[:4]), lambda: experts.forward(x, w, off.long()),
                lambda: experts.forward(x, w[0], off), lambda: experts.forward(x, w, off.cpu()),
                lambda: experts.forward(x, w.transpose(1, 2), off),
                lambda: experts.forward(x, w, off, out=torch.empty(20, 31, dtype=BF16, device="cuda")),
                lambda: experts.input_grad(x, w, off), lambda: experts.weight_grad(x, x[:19], off),
                lambda: experts.weight_grad(x, x.half(), off), lambda: experts.weight_grad(x, x, off, dtype=F16),
                lambda: experts.weight_grad(x, x, off, accumulate=True),
                lambda: experts.weight_grad(x, x, off, out=torch.empty(4, 64, 64, device="cuda", dtype=BF16),
                                            accumulate=True),
                lambda: experts.route(x.long(), 2), lambda: experts.route(x[0], 2), lambda: experts.route(x, 0),
                lambda: experts.route(x, 33), lambda: experts.route(x, 65),
                lambda: experts.gather(x, experts.route(x[:7], 2)),
                lambda: experts.combine(x, experts.route(x, 2)),
                lambda: experts.combine_backward(x, x.repeat(2, 1).float(), experts.route(x, 2)),
                lambda: experts.Routing(64, True, *[getattr(experts.route(x, 2), n) for n in (
                    "weights", "place", "offsets", "source", "source")])):
        with pytest.raises((ValueError, RuntimeError)):
            bad()
    assert block.check is experts.check


# ---------------------------------------------------------------------------
# What the tensor-core products add: tiles, runs, ways out, kernels that overlap
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("tokens", [63, 64, 65, 127, 128, 129, 256])
@pytest.mark.parametrize("n,k", [(8, 3), (1000, 32)])
def test_route_at_one_blocks_border(tokens, n, k):
    g = gen(tokens + n)
    logits = normal(g, tokens, n, scale=2)
    logits[::9] = -math.inf
    check_route(logits, k, True)
    check_route(logits.round() + 0.0, k, False)


def test_routing_arrays_start_on_16_bytes_and_are_apart():
    """The arrays of a routing are parts of one allocation: each passes the checks that a user's own would."""
    for tokens, n, k in ((1, 1, 1), (3, 5, 3), (129, 7, 5)):
        r = experts.route(normal(gen(tokens), tokens, n), k)
        again = experts.Routing(n, True, r.weights, r.experts, r.offsets, r.source, r.place)
        x = normal(gen(1), tokens, 40, dtype=BF16)
        assert torch.equal(experts.gather(x, r), experts.gather(x, again))
        before = [t.clone() for t in (r.weights, r.experts, r.offsets, r.source, r.place)]
        r.weights.fill_(7.0), r.offsets.fill_(3)
        assert torch.equal(r.experts, before[1]) and torch.equal(r.source, before[3]) and torch.equal(r.place, before[4])


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_weight_grad_of_no_rows(dtype):
    off = torch.zeros(4, dtype=I32, device="cuda")
    x, dy = torch.empty(0, 72, dtype=dtype, device="cuda"), torch.empty(0, 33, dtype=dtype, device="cuda")
    for out in (dtype, F32):
        dw = torch.full((3, 33, 80), 5.0, dtype=out, device="cuda")
        experts.weight_grad(dy, x, off, out=dw[:, :, :72])
        assert not bool(dw[:, :, :72].any()) and bool((dw[:, :, 72:] == 5).all())
    dw = torch.full((3, 33, 72), 5.0, device="cuda")
    experts.weight_grad(dy, x, off, out=dw, accumulate=True)
    assert bool((dw == 5).all())


@pytest.mark.parametrize("counts", [[1] * 1024, [0] * 1023 + [5], [3, 0] * 512])
def test_products_of_a_thousand_experts(counts):
    check_products(counts, 40, 72, BF16)


# run lengths around the tiles' widths (32 to 256) and the steps' rows (64), outs that leave by
# whole tiles, by ragged ends and element by element
@pytest.mark.parametrize("counts", [[255, 257, 223, 225], [31, 32, 33, 511, 513], [2049]])
@pytest.mark.parametrize("n_out,n_in", [(128, 136), (257, 264), (255, 520), (1, 8), (2, 1), (511, 72)])
def test_products_around_the_tiles(counts, n_out, n_in):
    check_products(counts, n_out, n_in, BF16)


@pytest.mark.parametrize("shift", [0, 1, 2, 4, 8])
@pytest.mark.parametrize("pad", [0, 1, 2, 8])
def test_outputs_at_any_alignment(shift, pad):
    """y, dx and dw that start on any element, rows any elements apart: the same bits, and nothing beside them."""
    g = gen(11)
    off = offsets_of([90, 40, 0, 133])
    x, w, dy = normal(g, 263, 136, dtype=F16), normal(g, 4, 264, 136, dtype=F16), normal(g, 263, 264, dtype=F16)

    def placed(want, call):
        shape = want.shape
        row = shape[-1] + pad
        each = shape[-2] * row
        count = each * (shape[0] if want.dim() == 3 else 1)
        flat = torch.full((count + 32,), 5.0, dtype=want.dtype, device="cuda")
        out = flat.as_strided(shape, (each, row, 1) if want.dim() == 3 else (row, 1), shift)
        call(out)
        assert torch.equal(out, want)
        out.fill_(5.0)
        assert bool((flat == 5).all())

    placed(experts.forward(x, w, off), lambda o: experts.forward(x, w, off, out=o))
    placed(experts.input_grad(dy, w, off), lambda o: experts.input_grad(dy, w, off, out=o))
    for out in (F16, F32):
        placed(experts.weight_grad(dy, x, off, dtype=out), lambda o: experts.weight_grad(dy, x, off, out=o))


def test_sums_of_many_runs():
    """K beyond the steps that stay in the tensor core: 8 of 64 for fp32 results, 64 for 16-bit ones."""
    for k in (511, 512, 513, 4095, 4097, 9000):
        g = gen(k)
        off = offsets_of([70, 0, 190])
        x, w = normal(g, 260, (k + 7) // 8 * 8, dtype=BF16)[:, :k], normal(g, 3, 72, (k + 7) // 8 * 8, dtype=BF16)[:, :, :k]
        want, size = ref.forward(x, w, off.tolist())
        close(experts.forward(x, w, off), want, ref.product_tol(k, size, want, BF16, BF16, run=4096), f"y {k}")
        off = offsets_of([k, 3])
        x, dy = normal(g, k + 3, 136, dtype=F16).abs(), normal(g, k + 3, 264, dtype=F16).abs()
        want, size = ref.weight_grad(dy, x, off.tolist())
        close(experts.weight_grad(dy, x, off, dtype=F32), want, ref.product_tol(k, size, want, F16, F32, run=512), f"dw {k}")


def test_calls_one_behind_the_other():
    """Kernels of neighbouring calls overlap: buffers that are read by one call and overwritten by the next,
    in every order, hold what they hold when each call is waited for."""
    logits, x, w_up, w_down, dout = layer_inputs(5, tokens=700)

    def passes(wait):
        g, kept = gen(77), []
        rows = h = y = None
        for i in range(12):
            r = experts.route(logits + 0.1 * i, 2)
            wait()
            rows = experts.gather(x, r, out=rows)
            wait()
            h = experts.forward(rows, w_up, r.offsets, out=h)
            wait()
            y = experts.forward(h, w_down, r.offsets, out=y)
            wait()
            out = experts.combine(y, r)
            wait()
            dw = experts.weight_grad(y, h, r.offsets, dtype=F32)
            wait()
            experts.input_grad(y, w_down, r.offsets, out=h)
            wait()
            experts.weight_grad(y, h, r.offsets, out=dw, accumulate=True)
            wait()
            kept.append((r.place, out, dw, h.clone()))
        return kept

    want = passes(torch.cuda.synchronize)
    for _ in range(3):
        got = passes(lambda: None)
        assert all(torch.equal(a, b) for p, q in zip(got, want) for a, b in zip(p, q))
    experts.check()


def test_products_on_two_streams_at_once():
    g = gen(8)
    off = offsets_of([500, 0, 900, 600])
    x, w = normal(g, 2000, 520, dtype=BF16), normal(g, 4, 776, 520, dtype=BF16)
    want = experts.forward(x, w, off)
    dw = experts.weight_grad(want, x, off, dtype=F32)
    sides = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for i in range(6):
        outs.append((experts.forward(x, w, off, stream=sides[0]), experts.weight_grad(want, x, off, dtype=F32, stream=sides[1])))
    torch.cuda.synchronize()
    assert all(torch.equal(a, want) and torch.equal(b, dw) for a, b in outs)


def test_products_of_two_graphs():
    """Captured calls hold no workspace: two graphs of the same products replayed at once."""
    g = gen(9)
    off = offsets_of([300, 10, 90])
    x, w = normal(g, 400, 264, dtype=F16), normal(g, 3, 136, 264, dtype=F16)
    want = experts.forward(x, w, off)
    sides, graphs, outs = [torch.cuda.Stream() for _ in range(2)], [], []
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs.append(experts.forward(x, w, off))
        graphs.append(graph)
    torch.cuda.synchronize()
    for _ in range(5):
        for s, graph in zip(sides, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_first_calls_captured():
    """A process whose first calls of all are recorded into a graph."""
    code = """
import torch
from mixed_precision_gb300 import experts, float8
x = torch.randn(300, 136, device='cuda').bfloat16()
w = torch.randn(4, 264, 136, device='cuda').bfloat16()
off = torch.tensor([0, 100, 100, 250, 300], dtype=torch.int32, device='cuda')
logits = torch.randn(300, 4, device='cuda')
torch.cuda.synchronize()
def calls():
    y = experts.forward(x, w, off)
    r = experts.route(logits, 2)
    return (y, experts.input_grad(y, w, off), experts.weight_grad(y, x, off, dtype=torch.float32), experts.gather(x, r),
            float8.matmul(float8.pack(x)[0], float8.pack(x)[0], dtype=torch.float32))
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = calls()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, calls()))
experts.check()
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]
