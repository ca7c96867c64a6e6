"""Scaled e4m3 matrices and their products on the GPU against the definition in 64 bits."""
import math

import pytest
import torch

import _experts_ref as ref
from _block_ref import E, close
from mixed_precision_gb300 import float8
from test_gpu_experts import offsets_of

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def check_packed(m, x):
    """Codes, scale bytes and padding of a Float8Matrix made from x [rows, cols]."""
    value, byte = ref.scaled(x)
    assert (m.scales.cpu().numpy() == byte).all()
    got = m.restore(F32).cpu().double()
    value = value.float().double()  # exact but for 2^128 and above, which is beyond fp32
    close(got, value, torch.zeros_like(value), "restored")
    codes = m.q.view(torch.uint8).cpu()
    assert not bool(codes[:, x.shape[1]:].any())
    return got


SIZES = [(1, 1), (1, 128), (3, 129), (128, 128), (130, 520), (257, 1000), (64, 2048), (5, 33), (1000, 72), (300, 700)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_pack(rows, cols, dtype):
    g = gen(rows + cols)
    x = normal(g, rows, cols + 8, dtype=dtype)[:, :cols]
    x *= torch.exp2(torch.randint(-8, 8, (rows, 1), generator=g, device="cuda").float()).to(dtype)
    a, b = float8.pack(x, transposed=True)
    check_packed(a, x)
    check_packed(b, x.t())
    # each form alone, into matrices that hold something else: the same bytes
    for direct in (True, False):
        m = float8.Float8Matrix(*((rows, cols) if direct else (cols, rows)))
        m.q.view(torch.uint8).fill_(77), m.scales.fill_(99)
        got = float8.pack(x, direct=m if direct else False, transposed=False if direct else m)
        assert got[1 if direct else 0] is None
        same = a if direct else b
        assert torch.equal(m.q.view(torch.uint8), same.q.view(torch.uint8)) and torch.equal(m.scales, same.scales)
    for out in (F32, F16, BF16):
        assert torch.equal(a.restore(out), a.restore(F32).to(out))


def test_pack_borders():
    """Largest magnitudes around 448 times a power of two, ties between codes, the smallest and largest numbers."""
    top = torch.tensor([448.0, 448.0 + 2 ** -15, 447.9, 224.0, 1.0, 1.75, 1.7500001, 2.0 ** -126, 1e-45, 0.0, 3.4e38,
                        2.0 ** -118, 1.75 * 2 ** -118], device="cuda")
    x = torch.zeros(len(top), 128, device="cuda")
    x[:, 0] = top
    frac = torch.linspace(-1, 1, 127, device="cuda")
    x[:, 1:] = top[:, None] * frac
    a, _ = float8.pack(x)
    check_packed(a, x)
    ties = torch.arange(-64, 64, device="cuda", dtype=F32)[None] * 2.0 ** -10
    ties = torch.cat([ties, ties * 17, ties * 1.125])
    ties[:, 0] = 256.0
    a, _ = float8.pack(ties)
    check_packed(a, ties)


def test_pack_not_finite():
    g = gen(1)
    for dtype in (F32, F16, BF16):
        x = normal(g, 40, 300, dtype=dtype)
        x[3, 5], x[4, 130], x[5, 200], x[39, 299] = math.inf, -math.inf, math.nan, math.inf
        x[6] = math.nan
        a, b = float8.pack(x, transposed=True)
        check_packed(a, x)
        check_packed(b, x.t())


def test_pack_experts():
    g = gen(2)
    base = normal(g, 3, 140, 300, dtype=BF16)
    x = base[:, :131, :264]
    a, b = float8.pack(x, transposed=True)
    assert a.q.shape == (3, 131, 384) and b.q.shape == (3, 264, 256)
    r, rt = a.restore(), b.restore()
    for e in range(3):
        one, one_t = float8.pack(x[e], transposed=True)
        assert torch.equal(a.q[e].view(torch.uint8), one.q.view(torch.uint8)) and torch.equal(a.scales[e], one.scales)
        assert torch.equal(b.q[e].view(torch.uint8), one_t.q.view(torch.uint8)) and torch.equal(b.scales[e], one_t.scales)
        assert torch.equal(r[e], one.restore()) and torch.equal(rt[e], one_t.restore())


def check_matmul(m, n, k, out, g, scale=1.0, sign=False):
    x, w = normal(g, m, k, scale=scale), normal(g, n, k)
    if sign:
        x, w = x.abs(), w.abs()
    a, b = float8.pack(x)[0], float8.pack(w)[0]
    ra, rb = a.restore(F32).double(), b.restore(F32).double()
    want, size = ra @ rb.t(), ra.abs() @ rb.abs().t()
    got = float8.matmul(a, b, dtype=out)
    tol = ref.product_tol(k, size, want, None, out, per_mma=32, run=2048 if out == F32 else None)
    close(got, want, tol, "product")
    return a, b, got, want, tol


@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 64, 128), (5, 33, 129), (32, 256, 256), (128, 128, 512), (130, 520, 640),
                                   (257, 300, 1000), (600, 16, 2048), (17, 1100, 72), (300, 260, 4000), (1025, 2049, 264)])
@pytest.mark.parametrize("out", [F32, F16, BF16])
def test_matmul(m, n, k, out):
    check_matmul(m, n, k, out, gen(m + n + k))


@pytest.mark.parametrize("out", [F32, BF16])
def test_matmul_of_many_tiles(out):
    check_matmul(5000, 3300, 1100, out, gen(3))
    check_matmul(300, 9000, 700, out, gen(4))


def test_matmul_scales():
    """Every row and block with a scale of its own, over a wide range."""
    g = gen(5)
    x, w = normal(g, 200, 1300), normal(g, 330, 1300)
    for t in (x, w):
        blocks = torch.exp2(torch.randint(-20, 20, (t.shape[0], 11), generator=g, device="cuda").float())
        t *= blocks.repeat_interleave(128, 1)[:, :1300]
    a, b = float8.pack(x)[0], float8.pack(w)[0]
    ra, rb = a.restore(F32).double(), b.restore(F32).double()
    want, size = ra @ rb.t(), ra.abs() @ rb.abs().t()
    close(float8.matmul(a, b, dtype=F32), want, ref.product_tol(1300, size, want, None, F32, per_mma=32), "product")


def test_matmul_of_one_sign():
    """Long sums of terms of one sign, where cut additions would add up."""
    check_matmul(70, 40, 20000, F32, gen(6), sign=True)
    check_matmul(70, 40, 20000, BF16, gen(6), sign=True)


def test_matmul_accumulates():
    g = gen(7)
    a, b, got, want, tol = check_matmul(150, 270, 900, F32, g)
    start = normal(g, 150, 270)
    out = start.clone()
    assert float8.matmul(a, b, out=out, accumulate=True) is out
    close(out, want + start.double(), tol + E * (want + start.double()).abs(), "added")
    wide = torch.full((150, 301), 3.0, device="cuda")
    float8.matmul(a, b, out=wide[:, 7:277])
    assert torch.equal(wide[:, 7:277], got) and bool((wide[:, :7] == 3).all()) and bool((wide[:, 277:] == 3).all())


@pytest.mark.parametrize("counts", [[5], [0, 40, 0], [33, 300, 0, 1, 257, 64], [1] * 20, [0] * 4, [3] * 130])
@pytest.mark.parametrize("n,k", [(64, 128), (300, 520), (257, 1100)])
def test_matmul_by_expert(counts, n, k):
    g = gen(sum(counts) + n)
    rows = sum(counts)
    off = offsets_of(counts)
    x, w = normal(g, rows + 3, k, dtype=BF16), normal(g, len(counts), n, k, dtype=BF16)
    x[rows:] = math.nan
    a, b = float8.pack(x)[0], float8.pack(w)[0]
    want, size = ref.forward(a.restore(F32)[:rows], b.restore(F32), off.tolist())
    got = float8.matmul(a, b, off)
    close(got[:rows], want, ref.product_tol(k, size, want, None, BF16, per_mma=32), "product")
    assert not bool(got[rows:].any())


def test_not_finite_reaches_what_depends_on_it():
    g = gen(8)
    x, w = normal(g, 100, 300), normal(g, 80, 300)
    clean = float8.matmul(float8.pack(x)[0], float8.pack(w)[0])
    x[7, 200], w[60, 10] = math.inf, math.nan
    got = float8.matmul(float8.pack(x)[0], float8.pack(w)[0])
    hit = torch.zeros(100, 80, dtype=torch.bool, device="cuda")
    hit[7], hit[:, 60] = True, True
    assert torch.equal(got.isnan(), hit)
    # the block of the inf has another scale without it; all other rows are the same
    assert torch.equal(got[~hit], clean[~hit])


def linear(x, w, dy):
    x8, x8t = float8.pack(x, transposed=True)
    w8, w8t = float8.pack(w, transposed=True)
    g8, g8t = float8.pack(dy, transposed=True)
    return float8.matmul(x8, w8), float8.matmul(g8, w8t), float8.matmul(g8t, x8t, dtype=F32)


def test_linear_layer():
    """A linear layer's three products. A code is off by 2^-4 of its element at most (half a step of 2^-3 at
    the low end of a power of two), uniformly: 2^-4 / sqrt(3) / 1.4 rms = 2.6 % of the element; two operands
    3.7 %; 5 % is allowed in norm."""
    g = gen(9)
    x, w, dy = normal(g, 777, 520, dtype=BF16), normal(g, 264, 520, dtype=BF16), normal(g, 777, 264, dtype=BF16)
    y, dx, dw = linear(x, w, dy)
    for got, want in ((y, x.double() @ w.double().t()), (dx, dy.double() @ w.double()), (dw, dy.double().t() @ x.double())):
        assert float((got.double() - want).norm() / want.norm()) < 0.05
    for _ in range(3):
        for a, b in zip(linear(x, w, dy), (y, dx, dw)):
            assert torch.equal(a, b)


def test_linear_layer_captured():
    g = gen(10)
    held = [normal(g, 300, 264, dtype=BF16), normal(g, 136, 264, dtype=BF16), normal(g, 300, 136, dtype=BF16)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        linear(*held)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = linear(*held)
    for seed in (1, 2):
        for t in held:
            t.copy_(normal(gen(seed), *t.shape))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, linear(*held)):
            assert torch.equal(a, b)
    float8.check()


def test_side_stream():
    g = gen(11)
    x, w = normal(g, 200, 300, dtype=BF16), normal(g, 100, 300, dtype=BF16)
    want = float8.matmul(float8.pack(x)[0], float8.pack(w)[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = float8.pack(x, stream=side)[0], float8.pack(w, stream=side)[0]
    got = float8.matmul(a, b, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


def test_refusals():
    g = gen(12)
    x = normal(g, 20, 64)
    a, at = float8.pack(x, transposed=True)
    e, _ = float8.pack(normal(g, 3, 20, 64))
    off = offsets_of([5, 5, 10])
    for bad in (lambda: float8.matmul(a, at), lambda: float8.matmul(e, a), lambda: float8.matmul(a, e),
                lambda: float8.matmul(a, a, off), lambda: float8.matmul(a, e, off[:3]),
                lambda: float8.matmul(a, e, off.long()), lambda: float8.matmul(a, a, accumulate=True),
                lambda: float8.matmul(a, a, out=torch.empty(20, 20, dtype=BF16, device="cuda"), accumulate=True),
                lambda: float8.matmul(a, a, dtype=torch.int8),
                lambda: float8.matmul(a, a, out=torch.empty(20, 21, dtype=BF16, device="cuda")),
                lambda: float8.pack(x.long()), lambda: float8.pack(x[0]), lambda: float8.pack(x.t()),
                lambda: float8.pack(x, direct=at), lambda: float8.pack(x, transposed=a),
                lambda: float8.pack(x, direct=False), lambda: float8.pack(x[:0], transposed=True),
                lambda: float8.Float8Matrix(4, 0), lambda: float8.Float8Matrix(4, 8, q=a.q, scales=a.scales),
                lambda: float8.Float8Matrix(20, 64, q=a.q), lambda: a.restore(torch.int8),
                lambda: a.restore(out=torch.empty(20, 63, device="cuda"))):
        with pytest.raises((ValueError, RuntimeError)):
            bad()
    assert float8.pack(x[:0])[0].restore().shape == (0, 64)


@pytest.mark.parametrize("rows", [1, 31, 33, 113, 223, 225, 449])
@pytest.mark.parametrize("n", [1, 127, 129, 255, 257])
def test_matmul_around_the_tiles(rows, n):
    check_matmul(rows, n, 520, F32, gen(rows + n))
    check_matmul(rows, n, 520, F16, gen(rows + n))


@pytest.mark.parametrize("k", [1, 511, 512, 513, 1023, 1025, 2047, 4097, 9000])
def test_matmul_of_many_steps(k):
    """Words of four scales, runs of 8 steps of 128 (fp32) and of 64."""
    g = gen(k)
    x, w = normal(g, 70, k).abs(), normal(g, 300, k).abs()
    a, b = float8.pack(x)[0], float8.pack(w)[0]
    ra, rb = a.restore(F32).double(), b.restore(F32).double()
    want, size = ra @ rb.t(), ra.abs() @ rb.abs().t()
    for out, run in ((F32, 1024), (BF16, 8192)):
        close(float8.matmul(a, b, dtype=out), want, ref.product_tol(k, size, want, None, out, per_mma=32, run=run), f"{out}")


def test_matmul_reads_nothing_behind_the_columns():
    """The codes and scales of the padding belong to the caller: what they hold does not matter."""
    g = gen(4)
    a, b = float8.pack(normal(g, 40, 300))[0], float8.pack(normal(g, 50, 300))[0]
    want = float8.matmul(a, b, dtype=F32)
    for m in (a, b):
        m.q.view(torch.uint8)[:, 300:] = 0x7F  # NaN
        m.scales[:, 3:] = 255
    assert torch.equal(float8.matmul(a, b, dtype=F32), want)


def test_experts_matmul_of_a_thousand():
    g = gen(6)
    counts = [1, 0] * 512
    x, w = normal(g, 512, 264), normal(g, 1024, 33, 264)
    a, b = float8.pack(x)[0], float8.pack(w)[0]
    y = float8.matmul(a, b, offsets_of(counts), dtype=F32)
    ra, rb = a.restore(F32).double(), b.restore(F32).double()[::2]
    want, size = torch.einsum("rk,rnk->rn", ra, rb), torch.einsum("rk,rnk->rn", ra.abs(), rb.abs())
    close(y, want, ref.product_tol(264, size, want, None, F32, per_mma=32, run=1024), "y")
