"""The expert layer's operators and the scaled products at their edges: sums that
would be lost in truncated additions, the largest sizes, offsets that no routing
makes, the smallest choices."""
import math

import pytest
import torch

import _experts_ref as ref
from _block_ref import E, TINY, U, close
from mixed_precision_gb300 import _abi as abi
from mixed_precision_gb300 import experts, float8
from test_gpu_experts import check_route, gen, normal, offsets_of

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


# ---------------------------------------------------------------------------
# Truncated additions
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("product", ["forward", "input_grad", "weight_grad"])
def test_small_terms_behind_a_large_one(product, dtype):
    """1 + U + 4094 terms of 1.5 * 2^-28: 16 of them are 0.75 steps of an fp32 number next to 1, which a
    truncated addition drops. All together lift the sum 2.3e-5 above the border between two 16-bit results;
    runs of 1024 terms may lose (64 + 4 + 16) * 2^-23 = 1.0e-5."""
    k, n, m = 4096, 40, 72
    left = torch.full((n, k), 2.0 ** -14, dtype=dtype, device="cuda")
    right = torch.full((m, k), 1.5 * 2.0 ** -14, dtype=dtype, device="cuda")
    left[:, :2], right[:, 0], right[:, 1] = 1.0, 1.0, U[dtype]
    want, size = left.double() @ right.double().t(), left.double() @ right.double().t()
    tol = ref.product_tol(k, size, want, dtype, dtype, run=1024)
    if product == "forward":
        got = experts.forward(left, right[None], offsets_of([n]))
    elif product == "input_grad":
        got = experts.input_grad(left, right.t().contiguous()[None], offsets_of([n]))
    else:
        got = experts.weight_grad(left.t().contiguous(), right.t().contiguous(), offsets_of([k]))[0]
    close(got, want, tol, product)


# ---------------------------------------------------------------------------
# Sizes
# ---------------------------------------------------------------------------

def test_products_of_the_most_rows():
    """Runs of 2^31 - 6 and 5 rows, whose steps of 64 end behind the largest int. A few rows are not zero."""
    rows = 2 ** 31 - 1
    x = torch.zeros(rows, 8, dtype=BF16, device="cuda")
    at = torch.tensor([0, 63, 64, 2 ** 30 + 7, rows - 70, rows - 65, rows - 64, rows - 6, rows - 5, rows - 1], device="cuda")
    some = torch.randint(-8, 9, (len(at), 8), device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(BF16)
    x[at] = some
    dw = experts.weight_grad(x, x, offsets_of([rows - 5, 5]), dtype=F32)
    some = some.float()
    assert torch.equal(dw[0], some[:-2].t() @ some[:-2])
    assert torch.equal(dw[1], some[-2:].t() @ some[-2:])
    # forward: the last tile's other half starts behind the largest int
    w = torch.randint(-8, 9, (2, 8, 8), device="cuda", generator=torch.Generator("cuda").manual_seed(2)).to(BF16)
    y = experts.forward(x, w, offsets_of([rows - 5, 5]))
    assert torch.equal(y[at[:-2]].float(), (some[:-2] @ w[0].float().t()).to(BF16).float())
    assert torch.equal(y[at[-2:]].float(), (some[-2:] @ w[1].float().t()).to(BF16).float())
    assert int(y[:2 ** 30].count_nonzero()) + int(y[2 ** 30:].count_nonzero()) == int(y[at].count_nonzero())
    experts.check()
    del x, y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("n_out,n_in", [(8, 264), (300, 72), (33, 520)])
def test_weight_grad_of_every_last_step(dtype, n_out, n_in):
    """Runs of 0 to 66 rows and of 190 to 200, between runs of NaN and inf: each run's last step holds its rows
    and nothing of its neighbours'."""
    g = gen(n_out)
    counts = [c for n in list(range(67)) + list(range(190, 201)) for c in (n, 1 + n % 3)] + [2]
    off = offsets_of([3] + counts)
    rows = sum(counts) + 3 + 5  # and rows of no expert at both ends
    wide = [torch.zeros(rows, (n + 7) // 8 * 8, dtype=dtype, device="cuda") for n in (n_out, n_in)]
    dy, x = wide[0][:, :n_out], wide[1][:, :n_in]
    dy.copy_(normal(g, rows, n_out)), x.copy_(normal(g, rows, n_in))
    o = off.tolist()
    dy[:3], x[rows - 5:] = float("nan"), float("inf")
    for e in range(2, len(o) - 1, 2):
        x[o[e]:o[e + 1]], dy[o[e]:o[e + 1]] = float("nan"), float("inf")
    want, size = ref.weight_grad(dy, x, o)
    for out in (dtype, F32):
        dw = experts.weight_grad(dy, x, off, dtype=out)
        assert bool(dw[2::2].isnan().all())
        close(dw[1::2], want[1::2], ref.product_tol(200, size[1::2], want[1::2], dtype, out), f"{out}")
    experts.check()


# ---------------------------------------------------------------------------
# Offsets that no routing makes
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("offsets,as_if", [([0, 300, 100, 400], [0, 300, 300, 400]), ([500, 100, 200, 300], [500] * 4),
                                           ([20, 10, 400, 390], [20, 20, 400, 400]), ([0, 450, 0, 450], [0, 450, 450, 450]),
                                           ([70, 900, -5, 460], [70, 500, 500, 500])])
def test_offsets_that_decrease(offsets, as_if):
    """Each counts as the largest before it: no row belongs to two experts, and none is left unwritten."""
    g = gen(21)
    rows, n_out, n_in = 500, 136, 264
    x, dy, w = normal(g, rows, n_in, dtype=BF16), normal(g, rows, n_out, dtype=BF16), normal(g, 3, n_out, n_in, dtype=BF16)
    x8, w8 = float8.pack(x)[0], float8.pack(w)[0]

    def calls(off):
        off = torch.tensor(off, dtype=torch.int32, device="cuda")
        y, dx = (torch.full((rows, n), 5.0, dtype=BF16, device="cuda") for n in (n_out, n_in))
        y8 = torch.full((rows, n_out), 5.0, device="cuda")
        return (experts.forward(x, w, off, out=y), experts.input_grad(dy, w, off, out=dx),
                experts.weight_grad(dy, x, off, dtype=F32), float8.matmul(x8, w8, off, out=y8))

    for a, b in zip(calls(offsets), calls(as_if)):
        assert torch.equal(a, b)
    experts.check()


# ---------------------------------------------------------------------------
# Scales on their way to the tensor cores
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("m,n,k", [(70, 300, 700), (300, 260, 4000), (600, 2049, 264)])
def test_products_whose_scales_change(m, n, k):
    """Products with other scales in every row and block, one behind the other beside another stream's traffic:
    none takes a scale of the one before, in either half of a tile."""
    g = gen(m)

    def packed(rows):
        scale = torch.exp2(torch.randint(-12, 12, (rows, (k + 127) // 128), generator=g, device="cuda").float())
        return float8.pack(normal(g, rows, k) * scale.repeat_interleave(128, 1)[:, :k])[0]

    sets = []
    for _ in range(3):
        a, b = packed(m), packed(n)
        ra, rb = a.restore(F32).double(), b.restore(F32).double()
        want, size = ra @ rb.t(), ra.abs() @ rb.abs().t()
        out = float8.matmul(a, b, dtype=F32)
        close(out, want, ref.product_tol(k, size, want, None, F32, per_mma=32, run=1024), "product")
        sets.append((a, b, out))
    side, other = torch.cuda.Stream(), torch.zeros(1 << 24, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(150):
        if i % 10 == 0:
            with torch.cuda.stream(side):
                other.add_(1.0)
        a, b, out = sets[i % 3]
        differ += (float8.matmul(a, b, dtype=F32) != out).any()
    torch.cuda.synchronize()
    assert int(differ) == 0
    float8.check()


# ---------------------------------------------------------------------------
# A wait that gives up
# ---------------------------------------------------------------------------

def timed_out():
    try:
        experts.check()
    except abi.ZeroError as e:
        assert e.code == abi.ZERO_ERR_TIMEOUT
        return True
    return False


@pytest.mark.parametrize("block", [0, 1])
def test_a_pair_that_gives_up_is_reported(block):
    """One block's wait runs out, the other's ends because it is told; both leave, the time-out is reported
    once, and products run on."""
    timed_out()  # what other tests may have left to this thread
    ends = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    abi.zero_selftest_pair_timeout(block, 1000, ends.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert timed_out() and not timed_out()
    assert ends.tolist() == [1 + block, 2 - block]
    g = gen(5)
    x, w = normal(g, 70, 264, dtype=BF16), normal(g, 1, 136, 264, dtype=BF16)
    want, size = ref.forward(x, w, [0, 70])
    close(experts.forward(x, w, offsets_of([70])), want, ref.product_tol(264, size, want, BF16, BF16), "y")
    assert not timed_out()


# ---------------------------------------------------------------------------
# Wide scaled matrices
# ---------------------------------------------------------------------------

def test_restore_of_wide_rows():
    """More columns than one grid takes (65535 x 32 scale blocks of 128): what packing makes of the transpose of
    very many rows."""
    cols = 65535 * 32 * 128 + 1000
    x = torch.zeros(cols, 2, dtype=BF16, device="cuda")
    at = torch.tensor([0, 127, 65535 * 32 * 128 - 1, 65535 * 32 * 128, cols - 500, cols - 1], device="cuda")
    x[at] = torch.tensor([[1.0, -2.0], [3.0, 4.0], [5.0, 6.0], [-7.0, 8.0], [9.0, 10.0], [11.0, 12.0]], device="cuda").to(BF16)
    _, xt = float8.pack(x, direct=False, transposed=True)
    y = xt.restore(BF16)
    assert torch.equal(y, x.t())
    wide = torch.full((2, cols + 3), 5.0, dtype=F16, device="cuda")  # element by element
    xt.restore(out=wide[:, :cols])
    assert torch.equal(wide[:, :cols], x.t().to(F16)) and bool((wide[:, cols:] == 5).all())
    del x, y, xt, wide
    torch.cuda.empty_cache()


# ---------------------------------------------------------------------------
# A lone choice
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("tokens,n", [(1, 1), (70, 1), (33, 16), (200, 2), (65, 128), (40, 300), (9, 1024)])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_top_1(tokens, n, dtype):
    """k = 1: normalised weights are 1 and pass nothing back, the softmax over all gives w dw (delta - p)."""
    g = gen(tokens + n)
    logits = normal(g, tokens, n, dtype=dtype)
    logits[::5] = -math.inf
    dw = normal(g, tokens, 1)
    r, _ = check_route(logits, 1, True)
    taken = r.experts >= 0
    assert torch.equal(r.weights, taken.float())
    assert not bool(experts.route_backward(dw, logits, r).any())

    r, _ = check_route(logits, 1, False)
    w = r.weights.double()
    d = torch.where(taken, dw.double(), 0.0)
    at = torch.where(taken, r.experts, n).long()
    p = torch.nan_to_num(torch.softmax(logits.double(), 1), nan=0.0)
    own = torch.zeros(tokens, n + 1, dtype=torch.float64, device="cuda").scatter(1, at, w * d)[:, :n]
    want, size = own - p * (w * d), own.abs() + p * (w * d).abs()
    # p as the weights (logits within 6 of zero, n / 32 additions and 5 shuffles), the product, one addition
    rel = 8 * E + 2 * (12.0 * E + 4 * E) + (n / 32 + 8) * E
    close(experts.route_backward(dw, logits, r), want, rel * size + U[dtype] * want.abs() + TINY[dtype], "dlogits")

    y = normal(g, tokens, 72, dtype=dtype)
    rows = experts.gather(y, r)
    last = int(r.offsets[-1])
    assert torch.equal(rows[:last], y[r.source[:last].long()]) and not bool(rows[last:].any())
    out = experts.combine(rows, r)
    assert torch.equal(out, torch.where(taken, (r.weights * y.float()).to(dtype), torch.zeros((), dtype=dtype, device="cuda")))
    dy, dweights = experts.combine_backward(y, rows, r)
    assert torch.equal(dy[:last], (r.weights.view(-1)[r.source[:last].long()][:, None] * y.float()[r.source[:last].long()]).to(dtype))
    sq = torch.where(taken, (y.double() ** 2).sum(1, keepdim=True), 0.0)
    close(dweights, sq, (72 / 32 + 16) * E * sq, "dweights")


def test_top_1_gradient_by_differences():
    g = gen(31)
    logits, c = normal(g, 20, 12), normal(g, 20, 1)
    r = experts.route(logits, 1, normalize=False)
    got, at = experts.route_backward(c, logits, r).double(), r.experts.long()
    h = 1e-5
    for e in range(12):
        step = torch.zeros(12, dtype=torch.float64, device="cuda")
        step[e] = h
        up, down = (torch.softmax(logits.double() + s * step, 1).gather(1, at) for s in (1, -1))
        # differences: h^2 of the third derivative and 1e-16 / h; the kernel: fp32
        assert float((got[:, e] - ((up - down) * c.double()).sum(1) / (2 * h)).abs().max()) < 1e-5


# ---------------------------------------------------------------------------
# fp32 sums by their runs: 512 rows of 16 bits, 1024 of 8
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("sign", [False, True])
@pytest.mark.parametrize("counts,n_out,n_in", [([20000, 1500], 136, 72), ([2000, 1, 2096, 0], 512, 768), ([700] * 9, 1024, 512),
                                               ([511, 513, 1025], 33, 264)])
def test_weight_grad_by_runs(counts, n_out, n_in, dtype, sign):
    g = gen(sum(counts) + n_out)
    rows, off = sum(counts), offsets_of(counts)
    dy = torch.zeros(rows, (n_out + 7) // 8 * 8, dtype=dtype, device="cuda")[:, :n_out]
    x = normal(g, rows, n_in, dtype=dtype)
    dy.copy_(normal(g, rows, n_out))
    if sign:
        dy, x = dy.abs_(), x.abs()
    want, size = ref.weight_grad(dy, x, off.tolist())
    tol = ref.product_tol(max(counts), size, want, dtype, F32, run=512)
    close(experts.weight_grad(dy, x, off, dtype=F32), want, tol, "dw")
    start = normal(g, *want.shape)
    dw = start.clone()
    experts.weight_grad(dy, x, off, out=dw, accumulate=True)
    close(dw, want + start.double(), tol + E * (want + start.double()).abs(), "dw added")
    close(experts.weight_grad(dy, x, off), want, ref.product_tol(max(counts), size, want, dtype, dtype, run=1024), "dw rounded")


@pytest.mark.parametrize("sign", [False, True])
@pytest.mark.parametrize("m,n,k", [(70, 40, 20000), (1025, 2049, 1100), (257, 300, 4097)])
def test_scaled_products_by_runs(m, n, k, sign):
    g = gen(m + k)
    x, w = normal(g, m, k), normal(g, n, k)
    if sign:
        x, w = x.abs(), w.abs()
    a, b = float8.pack(x)[0], float8.pack(w)[0]
    ra, rb = a.restore(F32).double(), b.restore(F32).double()
    want, size = ra @ rb.t(), ra.abs() @ rb.abs().t()
    tol = ref.product_tol(k, size, want, None, F32, per_mma=32, run=1024)
    close(float8.matmul(a, b, dtype=F32), want, tol, "product")
    start = normal(g, m, n)
    out = start.clone()
    float8.matmul(a, b, out=out, accumulate=True)
    close(out, want + start.double(), tol + E * (want + start.double()).abs(), "added")


# ---------------------------------------------------------------------------
# Odd widths from product to product
# ---------------------------------------------------------------------------

def test_products_of_an_odd_width_in_padded_rows():
    """n_out = 33: a result without gaps is refused as an input, columns of a wider buffer are taken."""
    g = gen(41)
    off = offsets_of([50, 30])
    x, w = normal(g, 80, 72, dtype=BF16), normal(g, 2, 33, 72, dtype=BF16)
    tight = experts.forward(x, w, off)
    for call in (lambda: experts.input_grad(tight, w, off), lambda: experts.weight_grad(tight, x, off)):
        with pytest.raises(abi.ZeroError):
            call()
    y = experts.forward(x, w, off, out=torch.zeros(80, 40, dtype=BF16, device="cuda")[:, :33])
    assert torch.equal(y, tight)
    want, size = ref.input_grad(y, w, off.tolist())
    close(experts.input_grad(y, w, off), want, ref.product_tol(33, size, want, BF16, BF16), "dx")
    want, size = ref.weight_grad(y, x, off.tolist())
    close(experts.weight_grad(y, x, off, dtype=F32), want, ref.product_tol(50, size, want, BF16, F32), "dw")
