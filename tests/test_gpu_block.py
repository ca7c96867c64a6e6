"""The block operators on the GPU against their definitions in 64 bits.

RMSNorm with the residual's addition, packed activations and the weight
gradient from them, attention's training pair: sizes, types, strides and masks
where they can go wrong, with the tolerances of _block_ref.
"""
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


# ---------------------------------------------------------------------------
# RMSNorm
# ---------------------------------------------------------------------------

ROWS_COLS = [(1, 8), (3, 1), (5, 33), (2, 128), (67, 128), (1, 1000), (33, 1024), (130, 2048), (7, 4100),
             (9, 4096), (4, 8192), (2, 16256), (2, 20000), (1, 65536), (513, 72), (4099, 264)]


# few rows, which are spread over as many threads as a block has
FEW_ROWS = [(1, 2056), (60, 2368), (83, 3256), (3, 4088), (40, 4104), (5, 5000), (300, 6000), (2, 8184), (700, 3000)]


# enough rows to go through shared memory, in teams of one to eight warps
MANY_ROWS = [(2432, 264), (2500, 512), (3001, 520), (2433, 1024), (2432, 1032), (5000, 2048), (2600, 4096), (2440, 5000),
             (2433, 8192)]


def check_forward(x, w, eps, res, y, s, rstd):
    if res is not None:
        assert same_bits(s, (x.float() + res.float()).to(x.dtype))
    want, r64 = ref.norm_forward(s, w, eps)
    rel = ref.row_chain(x.shape[1]) * ref.E
    ref.close(rstd, r64, rel * r64, "rstd")
    if y is not None:
        ref.close(y, want, want.abs() * (ref.U[x.dtype] + rel + 4 * ref.E) + ref.TINY[x.dtype], "y")


@pytest.mark.parametrize("rows,cols", ROWS_COLS + FEW_ROWS + MANY_ROWS)
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("with_res", [False, True])
def test_norm_forward(rows, cols, dtype, with_res):
    g = gen(rows * 7919 + cols)
    x = normal(g, rows, cols, dtype=dtype, scale=3)
    res = normal(g, rows, cols, dtype=dtype) if with_res else None
    w = normal(g, cols, dtype=[F32, F16, BF16][(rows + cols) % 3])
    packed = block.PackedActivation(rows, cols)
    y, s, rstd = block.rmsnorm_forward(x, w, 1e-5, residual=res, packed=packed)
    check_forward(x, w, 1e-5, res, y, s, rstd)
    q, byte, finite = ref.pack(y)
    assert finite.all()
    assert (packed.q.cpu().numpy() == q).all() and (packed.scales.cpu().numpy() == byte).all()
    # without the packed copy, and with the packed copy alone: the same values
    y2, s2, _ = block.rmsnorm_forward(x, w, 1e-5, residual=res)
    assert same_bits(y, y2) and same_bits(s, s2)
    alone = block.PackedActivation(rows, cols)
    y3, _, _ = block.rmsnorm_forward(x, w, 1e-5, residual=res, packed=alone, want_out=False)
    assert y3 is None and torch.equal(alone.q, packed.q) and torch.equal(alone.scales, packed.scales)


@pytest.mark.parametrize("rows,cols,pad", [(50, 128, 8), (50, 1024, 40), (50, 72, 3), (50, 33, 5), (2500, 1024, 40),
                                           (2500, 2056, 8)])
def test_norm_strided_rows_and_in_place_sum(rows, cols, pad):
    g = gen(cols)
    x = normal(g, rows, cols + pad, dtype=BF16)[:, :cols]
    res = normal(g, rows, 2 * cols + 8, dtype=BF16)[:, 8:cols + 8]
    w = normal(g, cols, dtype=BF16)
    y, s, rstd = block.rmsnorm_forward(x, w, 1e-6, residual=res)
    check_forward(x, w, 1e-6, res, y, s, rstd)
    xc, rc = x.contiguous(), res.contiguous()
    a = block.rmsnorm_forward(xc.clone(), w, 1e-6, residual=rc)
    held = rc.clone()
    b = block.rmsnorm_forward(xc, w, 1e-6, residual=held, sum_out=held)
    assert same_bits(a[0], b[0]) and same_bits(a[1], held)
    held = xc.clone()
    b = block.rmsnorm_forward(held, w, 1e-6, residual=rc, sum_out=held)
    assert same_bits(a[0], b[0]) and same_bits(a[1], held)


def test_norm_rows_far_apart():
    """Row offsets beyond 32 bits."""
    base = torch.empty(3 * 2 ** 30 + 256, dtype=BF16, device="cuda")
    x = base.as_strided((3, 128), (2 ** 30 + 64, 1))
    x.copy_(normal(gen(1), 3, 128))
    w = torch.ones(128, device="cuda")
    y, s, rstd = block.rmsnorm_forward(x, w, 1e-6)
    check_forward(x, w, 1e-6, None, y, x, rstd)
    p = block.PackedActivation(3, 128).save(x)
    q, byte, _ = ref.pack(x)
    assert (p.q.cpu().numpy() == q).all() and (p.scales.cpu().numpy() == byte).all()
    dx, dw = block.rmsnorm_backward(x, x, w, rstd, dweight_dtype=F32)
    assert same_bits(dx, block.rmsnorm_backward(x.contiguous(), x.contiguous(), w, rstd)[0])


@pytest.mark.parametrize("rows,cols", ROWS_COLS + FEW_ROWS + MANY_ROWS + [(20000, 128), (3000, 1024)])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("with_dsum", [False, True])
def test_norm_backward(rows, cols, dtype, with_dsum):
    g = gen(rows * 7919 + cols + 1)
    x = normal(g, rows, cols, dtype=dtype, scale=3)
    dy = normal(g, rows, cols, dtype=dtype)
    dsum = normal(g, rows, cols, dtype=dtype) if with_dsum else None
    w = normal(g, cols, dtype=[F32, F16, BF16][(rows + cols) % 3])
    rstd = (x.double().square().mean(1) + 1e-6).rsqrt().float()
    dx, dw = block.rmsnorm_backward(dy, x, w, rstd, dsum=dsum, dweight_dtype=F32)
    rdx, rdw, tol, size = ref.norm_backward(dy, x, w, rstd, dsum)
    ref.close(dx, rdx, tol + ref.U[dtype] * (rdx.abs() + tol) + ref.TINY[dtype], "dx")
    # the longest chain of a column: every eighth row of a 64th of them at most, then 232 partial sums
    ref.close(dw, rdw, (rows / 8 + 240) * ref.E * size + ref.TINY[F32], "dweight")
    dx2, dw2 = block.rmsnorm_backward(dy, x, w, rstd, dsum=dsum, dweight_dtype=BF16)
    assert same_bits(dx, dx2) and same_bits(dw.to(BF16), dw2)
    held = dy.clone()  # in place of dy
    _, dw3 = block.rmsnorm_backward(held, x, w, rstd, dsum=dsum, dx=held, dweight_dtype=F32)
    assert same_bits(dx, held) and same_bits(dw, dw3)


def test_norm_backward_against_differences():
    """<gradient, direction> against central differences of the forward's definition in 64 bits."""
    g = gen(5)
    rows, cols, eps = 6, 96, 1e-3
    x, c = normal(g, rows, cols).double(), normal(g, rows, cols).double()
    w = normal(g, cols).double()
    rstd = (x.square().mean(1) + eps).rsqrt()
    dx, dw = block.rmsnorm_backward(c.float(), x.float(), w.float(), rstd.float(), dweight_dtype=F32)
    loss = lambda a, b: (ref.norm_forward(a, b, eps)[0] * c.float().double()).sum()  # noqa: E731
    x, w = x.float().double(), w.float().double()
    for seed in range(4):
        d, e = normal(gen(seed + 50), rows, cols).double(), normal(gen(seed + 90), cols).double()
        h = 1e-5
        num = (loss(x + h * d, w) - loss(x - h * d, w)) / (2 * h)
        # h^2 / 6 of the third derivative (below 1e3 for unit rows) and fp32 outputs of unit size
        assert abs(float((dx.double() * d).sum() - num)) < 1e-7 + 200 * ref.E * float(d.abs().sum())
        num = (loss(x, w + h * e) - loss(x, w - h * e)) / (2 * h)
        assert abs(float((dw.double() * e).sum() - num)) < 1e-7 + 200 * ref.E * rows * float(e.abs().sum())


def test_norm_special_rows():
    """A zero row, an infinity and a NaN: their own rows alone, and the packed copy marks them."""
    x = normal(gen(9), 4, 256, dtype=BF16)
    x[0] = 0
    x[1, 17] = math.inf
    x[2, 40] = math.nan
    w = torch.ones(256, device="cuda", dtype=BF16)
    packed = block.PackedActivation(4, 256)
    y, _, rstd = block.rmsnorm_forward(x, w, 1e-6, packed=packed)
    assert bool((y[0] == 0).all()) and abs(float(rstd[0]) - 1e3) < 1e-2
    assert bool(y[1, 17].isnan()) and bool((y[1, :17] == 0).all()) and bool(y[2].isnan().all())
    assert bool(y[3].isfinite().all())
    back = packed.restore(BF16)
    assert bool((back[0] == 0).all()) and bool(back[1, :32].isnan().all()) and bool((back[1, 32:] == 0).all())
    assert bool(back[2].isnan().all()) and bool(back[3].isfinite().all())
    dy = torch.ones_like(x)
    dx, dw = block.rmsnorm_backward(dy, x, w, rstd, dweight_dtype=F32)
    assert bool(dx[2].isnan().all()) and bool(dx[3].isfinite().all()) and bool(dw.isnan().any())


def test_norm_no_rows():
    w = torch.ones(64, device="cuda")
    x = torch.empty(0, 64, device="cuda")
    y, _, rstd = block.rmsnorm_forward(x, w)
    assert y.shape == (0, 64) and rstd.shape == (0,)
    dx, dw = block.rmsnorm_backward(x, x, w, rstd, dweight=torch.full((64,), 7.0, device="cuda"))
    assert dx.shape == (0, 64) and bool((dw == 0).all())


# ---------------------------------------------------------------------------
# Packed activations
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (3, 33), (5, 127), (2, 128), (7, 129), (64, 1024), (1001, 72),
                                       (3, 70000)])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_pack_and_restore(rows, cols, dtype):
    g = gen(rows + cols)
    x = normal(g, rows, cols) * torch.exp2(torch.randint(-30, 14, (rows, 1), generator=g, device="cuda").float())
    x = x.to(dtype)
    x[0, 0] = 0
    x[rows // 2, cols // 2] = torch.finfo(dtype).max
    x[rows - 1, cols - 1] = torch.finfo(dtype).smallest_normal / 2  # subnormal
    for view in (x, torch.nn.functional.pad(x, (0, 5))[:, :cols]):
        p = block.PackedActivation(rows, cols).save(view)
        q, byte, _ = ref.pack(x)
        assert (p.q.cpu().numpy() == q).all() and (p.scales.cpu().numpy() == byte).all()
    for out in (F32, F16, BF16):
        got = p.restore(out)
        assert same_bits(got.cpu(), ref.restore(q, byte, cols, out))
    wide = torch.full((rows, cols + 3), 5.0, dtype=dtype, device="cuda")
    p.restore(out=wide[:, :cols])
    assert same_bits(wide[:, :cols], p.restore(dtype)) and bool((wide[:, cols:] == 5).all())
    # an element is off by half a code at most, one where the largest rounds to 128
    step = torch.from_numpy(ref.restore(q * 0 + 1, byte, cols, F32).numpy()).double()
    err = (ref.restore(q, byte, cols, F32).double() - x.cpu().double()).abs()
    assert bool((err <= step * torch.where(torch.from_numpy(abs(q[:, :cols]) == 127), 1.0, 0.5)).all())


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_pack_marks_non_finite_groups(bad):
    x = normal(gen(3), 4, 100, dtype=BF16)
    x[1, 40] = bad
    got = block.PackedActivation(4, 100).save(x).restore(F32)
    assert bool(got[1, 32:64].isnan().all())
    keep = torch.ones(4, 100, dtype=torch.bool, device="cuda")
    keep[1, 32:64] = False
    assert bool(got[keep].isfinite().all())


# ---------------------------------------------------------------------------
# Weight gradient
# ---------------------------------------------------------------------------

def check_wgrad(tokens, n_out, n_in, dtype, out, seed=0, view=False):
    g = gen(tokens + n_out + n_in + seed)
    x = normal(g, tokens, n_in, dtype=dtype, scale=2)
    up = (n_out + 7) // 8 * 8 + (24 if view else 0)
    buf = torch.full((tokens, up), math.nan, dtype=dtype, device="cuda")  # what lies past a row is not used
    buf[:, :n_out] = normal(g, tokens, n_out)
    dy = buf[:, :n_out]
    p = block.PackedActivation(tokens, n_in).save(x)
    dw = block.weight_grad(dy, p, dtype=out)
    xr = p.restore(dtype).double()
    want = dy.double().t() @ xr
    size = dy.double().abs().t() @ xr.abs()
    tol = (tokens / 8 + 32) * 2 * ref.E * size
    ref.close(dw, want, tol + ref.U[out] * (want.abs() + tol) + ref.TINY[out], "dw")
    return dy, p, dw


@pytest.mark.parametrize("tokens,n_out,n_in", [
    (1, 1, 1), (1, 16, 64), (3, 8, 40), (16, 17, 33), (63, 64, 64), (64, 128, 256), (65, 129, 257), (257, 16, 2048),
    (1000, 200, 328), (2049, 136, 1000), (4097, 256, 264), (300, 1000, 72), (130, 2048, 1024)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_weight_grad(tokens, n_out, n_in, dtype):
    for out in (F32, dtype):
        check_wgrad(tokens, n_out, n_in, dtype, out)


@pytest.mark.parametrize("tokens,n_out,n_in", [(20000, 64, 96), (9000, 520, 1032), (515, 5000, 1024)])
def test_weight_grad_long(tokens, n_out, n_in):
    check_wgrad(tokens, n_out, n_in, BF16, F32)
    check_wgrad(tokens, n_out, n_in, BF16, BF16, view=True)


@pytest.mark.parametrize("tokens", [1, 63, 65, 130, 321, 450])
@pytest.mark.parametrize("n_out,n_in,dtype", [(8200, 5000, BF16), (6000, 8192, F16), (40000, 264, BF16)])
def test_weight_grad_many_tiles(tokens, n_out, n_in, dtype):
    """More tiles than multiprocessors, of one step to several."""
    check_wgrad(tokens, n_out, n_in, dtype, dtype)


def test_weight_grad_exact():
    """Small whole numbers: every product and sum is exact, so is the result."""
    g = gen(11)
    for tokens, n_out, n_in in ((200, 130, 260), (5000, 72, 128)):
        dy = torch.randint(-2, 3, (tokens, n_out + (-n_out) % 8), generator=g, device="cuda").to(BF16)[:, :n_out]
        x = torch.randint(-64, 65, (tokens, n_in), generator=g, device="cuda").to(BF16)
        x[:, ::32] = 64  # fixes every group's scale at 1
        p = block.PackedActivation(tokens, n_in).save(x)
        dw = block.weight_grad(dy, p, dtype=F32)
        assert torch.equal(dw.double(), dy.double().t() @ x.double())


def test_weight_grad_accumulates_and_repeats():
    dy, p, dw = check_wgrad(700, 136, 520, BF16, F32)
    main = normal(gen(8), 136, 520)
    total = block.weight_grad(dy, p, out=main.clone(), accumulate=True)
    assert torch.equal(total, main + dw)
    for _ in range(3):
        assert torch.equal(block.weight_grad(dy, p, dtype=F32), dw)


def test_weight_grad_no_tokens():
    p = block.PackedActivation(0, 64)
    dy = torch.empty(0, 16, dtype=BF16, device="cuda")
    out = torch.full((16, 64), 3.0, device="cuda")
    assert bool((block.weight_grad(dy, p, out=out.clone(), accumulate=True) == 3).all())
    assert bool((block.weight_grad(dy, p, out=out) == 0).all())


def test_weight_grad_non_finite():
    """A NaN group reaches its 32 columns, an inf in dy its row, nothing else."""
    g = gen(21)
    x, dy = normal(g, 300, 160, dtype=BF16), normal(g, 300, 40, dtype=BF16)
    x[77, 70] = math.inf
    dy[5, 9] = math.inf
    dw = block.weight_grad(dy, block.PackedActivation(300, 160).save(x), dtype=F32)
    bad = torch.zeros(40, 160, dtype=torch.bool, device="cuda")
    bad[:, 64:96] = True
    bad[9] = True
    assert bool((~dw.isfinite() == bad).all())


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------

def attention_case(B, Sq, Sk, H, K, D, dtype, causal, window, ragged, seed=0, layout="bshd", hole=math.nan):
    g = gen(seed + Sq * 31 + Sk + D)
    def make(n, heads, scale=1.0):
        if layout == "bshd":
            return normal(g, B, n, heads, D, dtype=dtype, scale=scale)
        if layout == "bhsd":  # heads outside
            return normal(g, B, heads, n, D, dtype=dtype, scale=scale).transpose(1, 2)
        if layout == "sbhd":  # tokens outside
            return normal(g, n, B, heads, D, dtype=dtype, scale=scale).transpose(0, 1)
        wide = normal(g, B, n, heads + 2, D + 24, dtype=dtype, scale=scale)  # inside wider tensors
        return wide[:, :, 1:heads + 1, 8:D + 8]
    q, k, v, do = make(Sq, H), make(Sk, K, 1.5), make(Sk, K), make(Sq, H, 0.1)
    lengths = None
    if ragged:
        n = torch.randint(1, Sk + 1, (B,), generator=g, device="cuda")
        if B > 1:
            n[-1] = 0
        if B > 2:
            n[-2] = Sk
        lengths = n.to(torch.int32)
        for b in range(B):  # nothing may leak from past the length
            k[b, int(lengths[b]):] = hole
            v[b, int(lengths[b]):] = hole
    return q, k, v, do, lengths


def check_attention(B, Sq, Sk, H, K, D, dtype, causal=False, window=0, ragged=False, seed=0, layout="bshd",
                    scale=None, backward=True):
    q, k, v, do, lengths = attention_case(B, Sq, Sk, H, K, D, dtype, causal, window, ragged, seed, layout)
    s = D ** -0.5 if scale is None else scale
    mask = dict(causal=causal, window=window, key_lengths=lengths, scale=scale)
    o, lse = block.attention_forward(q, k, v, **mask)
    ro, rl, to, tl = ref.attention_forward(q, k, v, causal, window, lengths, s)
    ref.close(lse, rl, tl, "lse")
    ref.close(o, ro, to, "o")
    if not backward:
        return
    grads = block.attention_backward(do, q, k, v, o, lse, **mask)
    want = ref.attention_backward(do, q, k, v, o, lse, causal, window, lengths, s)
    for got, name in zip(grads, ("dq", "dk", "dv")):
        ref.close(got, *want[name], name)
    block.check()


@pytest.mark.parametrize("Sq,Sk", [(1, 1), (1, 2), (2, 1), (1, 300), (300, 1), (17, 64), (64, 64), (127, 127), (128, 128),
                                   (129, 129), (255, 130), (130, 255), (257, 511), (513, 384)])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D,dtype", [(128, BF16), (64, F16)])
def test_attention_lengths(Sq, Sk, causal, D, dtype):
    check_attention(2, Sq, Sk, 4, 2, D, dtype, causal)


@pytest.mark.parametrize("D", [8, 16, 40, 64, 72, 80, 96, 120, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_head_dims(D, dtype):
    check_attention(1, 150, 200, 2, 1, D, dtype, causal=True)


@pytest.mark.parametrize("H,K", [(1, 1), (3, 1), (8, 8), (6, 2), (16, 1), (5, 5)])
def test_attention_heads(H, K):
    check_attention(2, 140, 140, H, K, 64, BF16, causal=True)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("window", [0, 1, 7, 128, 200, 10000])
@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("Sq,Sk", [(300, 300), (100, 400), (400, 100)])
def test_attention_masks(causal, window, ragged, Sq, Sk):
    check_attention(3, Sq, Sk, 4, 2, 64, BF16, causal, window, ragged, seed=window)


@pytest.mark.parametrize("layout", ["bhsd", "sbhd", "inner"])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_layouts(layout, D):
    check_attention(2, 200, 260, 4, 2, D, BF16, causal=True, ragged=True, layout=layout)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_longer(dtype):
    check_attention(1, 1500, 1500, 4, 2, 128, dtype, causal=True)
    check_attention(2, 1100, 1300, 3, 1, 96, dtype, window=300, ragged=True)


@pytest.mark.parametrize("D", [40, 64, 128])
@pytest.mark.parametrize("live", [0, 1, 3])
@pytest.mark.parametrize("Sq", [130, 100])
def test_attention_many_rows_of_which_most_see_nothing(D, live, Sq):
    """Several query tiles for every multiprocessor, with empty ones in runs."""
    B, Sk, H = 400, 140, 3
    q, k, v, do, _ = attention_case(B, Sq, Sk, H, 1, D, BF16, False, 0, False)
    lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
    if live:
        lengths[::live] = torch.randint(1, Sk + 1, (len(range(0, B, live)),), generator=gen(D), device="cuda").int()
        lengths[100:200] = 0
    for b in range(B):
        k[b, int(lengths[b]):] = math.nan
        v[b, int(lengths[b]):] = math.nan
    o, lse = torch.full_like(q, math.nan), torch.full((B, H, Sq), math.nan, device="cuda")
    block.attention_forward(q, k, v, key_lengths=lengths, out=o, lse=lse)
    ro, rl, to, tl = ref.attention_forward(q, k, v, False, 0, lengths, D ** -0.5)
    ref.close(lse, rl, tl, "lse")
    ref.close(o, ro, to, "o")
    out = [torch.full_like(t, math.nan) for t in (q, k, v)]
    block.attention_backward(do, q, k, v, o, lse, key_lengths=lengths, dq=out[0], dk=out[1], dv=out[2])
    want = ref.attention_backward(do, q, k, v, o, lse, False, 0, lengths, D ** -0.5)
    for got, name in zip(out, ("dq", "dk", "dv")):
        ref.close(got, *want[name], name)
    block.check()


@pytest.mark.parametrize("B,Sq,Sk,H,K,causal,window", [
    (500, 100, 100, 1, 1, True, 0), (450, 60, 300, 2, 1, False, 0), (200, 300, 60, 2, 2, True, 0),
    (200, 129, 129, 2, 1, True, 0), (120, 400, 500, 1, 1, True, 20), (150, 700, 100, 1, 1, True, 30),
    (90, 1, 700, 6, 2, True, 0)])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_many_pieces_for_a_block(B, Sq, Sk, H, K, causal, window, D):
    """Pieces of one tile to a few, several for every multiprocessor, some without a key."""
    check_attention(B, Sq, Sk, H, K, D, BF16, causal, window)


def test_attention_scale_and_large_logits():
    check_attention(1, 200, 200, 2, 2, 64, BF16, causal=True, scale=1.0)  # logits of +-50: near one-hot rows
    check_attention(1, 200, 200, 2, 2, 64, BF16, causal=True, scale=1e-4)


def test_attention_running_maximum_rises():
    """Keys that grow along the row move the maximum in every tile."""
    q, k, v, do, _ = attention_case(1, 300, 900, 2, 2, 64, BF16, False, 0, False)
    k = (k.float() * torch.linspace(0.1, 6, 900, device="cuda")[None, :, None, None]).to(BF16)
    o, lse = block.attention_forward(q, k, v)
    ro, rl, to, tl = ref.attention_forward(q, k, v, False, 0, None, 64 ** -0.5)
    ref.close(lse, rl, tl, "lse")
    ref.close(o, ro, to, "o")
    grads = block.attention_backward(do, q, k, v, o, lse)
    want = ref.attention_backward(do, q, k, v, o, lse, False, 0, None, 64 ** -0.5)
    for got, name in zip(grads, ("dq", "dk", "dv")):
        ref.close(got, *want[name], name)


def test_attention_no_keys_and_no_queries():
    q = normal(gen(1), 2, 5, 4, 64, dtype=BF16)
    k = torch.empty(2, 0, 2, 64, dtype=BF16, device="cuda")
    o, lse = block.attention_forward(q, k, k)
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())
    dq, dk, dv = block.attention_backward(q, q, k, k, o, lse)
    assert bool((dq == 0).all()) and dk.shape == k.shape
    none = q[:, :0]
    kk = normal(gen(2), 2, 7, 2, 64, dtype=BF16)
    o, lse = block.attention_forward(none, kk, kk)
    dq, dk, dv = block.attention_backward(none, none, kk, kk, o, lse)
    assert bool((dk == 0).all()) and bool((dv == 0).all())


def test_attention_out_of_range_lengths_are_clamped():
    q, k, v, _, _ = attention_case(2, 50, 60, 2, 2, 64, BF16, False, 0, False)
    far = torch.tensor([1000, -5], dtype=torch.int32, device="cuda")
    near = torch.tensor([60, 0], dtype=torch.int32, device="cuda")
    for a, b in zip(block.attention_forward(q, k, v, key_lengths=far),
                    block.attention_forward(q, k, v, key_lengths=near)):
        assert torch.equal(a, b)


def test_attention_inf_marks_only_its_rows():
    """A non-finite key that a causal query does not see changes nothing for it, and
    reaches the gradients of those that do."""
    q, k, v, do, _ = attention_case(1, 200, 200, 2, 2, 64, BF16, True, 0, False)
    clean, _ = block.attention_forward(q, k, v, causal=True)
    k[0, 150, 0, 3] = math.nan
    o, lse = block.attention_forward(q, k, v, causal=True)
    assert same_bits(o[:, :, 1], clean[:, :, 1])
    assert bool(o[0, 150:, 0].isnan().all()) and bool(lse[0, 0, 150:].isnan().all())
    assert same_bits(o[0, :128, 0], clean[0, :128, 0])
    dq, dk, dv = block.attention_backward(do, q, k, v, o, lse, causal=True)
    assert bool(dq[0, 150:, 0].isnan().any()) and bool(dq[:, :, 1].isfinite().all())
    assert bool(dk[:, :, 1].isfinite().all()) and bool(dv[:, :, 1].isfinite().all())


def test_attention_backward_against_differences():
    """<gradient, direction> against central differences of the loss in 64 bits."""
    q, k, v, do, _ = attention_case(1, 70, 70, 2, 1, 64, F16, True, 0, False)
    o, lse = block.attention_forward(q, k, v, causal=True)
    dq, dk, dv = block.attention_backward(do, q, k, v, o, lse, causal=True)
    want = ref.attention_backward(do, q, k, v, o, lse, True, 0, None, 0.125)

    def loss(a, b, c):
        return (ref_forward64(a, b, c) * do.double()).sum()

    def ref_forward64(a, b, c):
        ok = ref.seen(70, 70, True, 0, 70).cuda()
        w = torch.einsum("bihd,bjd->bhij", a, b[:, :, 0]) * 0.125
        p = torch.softmax(w.masked_fill(~ok, -math.inf), -1)
        return torch.einsum("bhij,bjd->bihd", p, c[:, :, 0])

    x = [t.double() for t in (q, k, v)]
    h = 1e-5
    for n, got in enumerate((dq, dk, dv)):
        d = normal(gen(n + 70), *got.shape).double()
        up, down = list(x), list(x)
        up[n], down[n] = x[n] + h * d, x[n] - h * d
        num = (loss(*up) - loss(*down)) / (2 * h)
        tol = want[("dq", "dk", "dv")[n]][1]
        # o's own rounding moves delta: U |do . o| for every pair's ds
        slack = 8 * ref.U[F16] * float((do.double().abs() * o.double().abs()).sum()) * 4
        assert abs(float((got.double() * d).sum() - num)) < 1e-6 + float((tol * d.abs()).sum()) + slack


def test_attention_batches_far_apart():
    """Element offsets beyond 32 bits."""
    base = torch.empty(2 ** 31 + 2 ** 20, dtype=BF16, device="cuda")
    q, k, v, do, _ = attention_case(2, 100, 100, 2, 1, 64, BF16, True, 0, False)
    far = base.as_strided((2, 100, 1, 64), (2 ** 31 + 64, 64, 64, 1))
    far.copy_(k)
    o, lse = block.attention_forward(q, k, v, causal=True)
    o2, lse2 = block.attention_forward(q, far, v, causal=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    a = block.attention_backward(do, q, k, v, o, lse, causal=True)
    b = block.attention_backward(do, q, far, v, o, lse, causal=True)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_attention_repeats_bit_for_bit():
    q, k, v, do, lengths = attention_case(2, 700, 700, 8, 2, 128, BF16, True, 0, True, hole=0.0)
    o, lse = block.attention_forward(q, k, v, causal=True, key_lengths=lengths)
    first = block.attention_backward(do, q, k, v, o, lse, causal=True, key_lengths=lengths)
    for _ in range(5):
        o2, lse2 = block.attention_forward(q, k, v, causal=True, key_lengths=lengths)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        again = block.attention_backward(do, q, k, v, o, lse, causal=True, key_lengths=lengths)
        assert all(torch.equal(x, y) for x, y in zip(first, again))


# ---------------------------------------------------------------------------
# Streams, graphs, guard bands
# ---------------------------------------------------------------------------

def whole_block(x, res, w, dy, q, k, v, do, stream=None):
    p = block.PackedActivation(x.shape[0], x.shape[1], stream=stream)
    y, s, rstd = block.rmsnorm_forward(x, w, residual=res, packed=p, stream=stream)
    dx, dw = block.rmsnorm_backward(dy, s, w, rstd, stream=stream)
    g = block.weight_grad(dy, p, dtype=F32, stream=stream)
    o, lse = block.attention_forward(q, k, v, causal=True, stream=stream)
    return (y, s, rstd, dx, dw, g, o, lse) + block.attention_backward(do, q, k, v, o, lse, causal=True, stream=stream)


def block_inputs(seed=3):
    g = gen(seed)
    x, res, dy = (normal(g, 300, 256, dtype=BF16) for _ in range(3))
    w = normal(g, 256, dtype=BF16)
    q, k, v, do, _ = attention_case(2, 300, 300, 4, 2, 64, BF16, True, 0, False, seed)
    return x, res, w, dy, q, k, v, do


def test_other_stream():
    args = block_inputs()
    want = whole_block(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        side.wait_stream(torch.cuda.current_stream())
        got = whole_block(*args, stream=side)
        junk = [torch.full((1 << 22,), 1.0, device="cuda") for _ in range(8)]  # takes freed memory, if any
        side.synchronize()
        del junk
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_graph_capture():
    args = block_inputs()
    whole_block(*args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = whole_block(*args)
    for a, b in zip(args, block_inputs(4)):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(whole_block(*args), got))


class Guarded:
    """A tensor of the given shape between two guard regions of a pattern."""

    def __init__(self, shape, dtype):
        n = math.prod(shape) * torch.empty(0, dtype=dtype).element_size()
        self.raw = torch.full((8192 + (n + 15) // 16 * 16,), 0xA5, dtype=torch.uint8, device="cuda")
        self.n = n
        self.t = self.raw[4096:4096 + n].view(dtype).view(shape)

    def intact(self):
        return bool((self.raw[:4096] == 0xA5).all()) and bool((self.raw[4096 + self.n:] == 0xA5).all())


@pytest.mark.parametrize("rows,cols", [(1, 8), (7, 33), (65, 136), (130, 1000), (3, 17000)])
def test_no_write_outside_buffers(rows, cols):
    g = gen(cols)
    x, dy = normal(g, rows, cols, dtype=BF16), normal(g, rows, cols, dtype=BF16)
    w = normal(g, cols, dtype=BF16)
    out = {n: Guarded((rows, cols), BF16) for n in ("y", "s", "dx", "back")}
    pitch = (cols + 127) // 128 * 128
    out["q"], out["scales"] = Guarded((rows, pitch), torch.int8), Guarded((rows, pitch // 32), torch.uint8)
    out["rstd"], out["dw"] = Guarded((rows,), F32), Guarded((cols,), BF16)
    p = block.PackedActivation(rows, cols, q=out["q"].t, scales=out["scales"].t)
    block.rmsnorm_forward(x, w, residual=dy, out=out["y"].t, sum_out=out["s"].t, rstd=out["rstd"].t, packed=p)
    block.rmsnorm_backward(dy, out["s"].t, w, out["rstd"].t, dx=out["dx"].t, dweight=out["dw"].t)
    p.restore(out=out["back"].t)
    p.save(x)
    for dtype in (F32, BF16):
        n_out = 24
        out["g"] = Guarded((n_out, cols), dtype)
        block.weight_grad(normal(g, rows, n_out, dtype=BF16), p, out=out["g"].t)
        assert all(o.intact() for o in out.values())
    B, H, K, D = 2, 3, 1, 72
    q, k, v, do, lengths = attention_case(B, rows, min(cols, 300), H, K, D, BF16, False, 0, True)
    at = {"o": Guarded(q.shape, BF16), "lse": Guarded((B, H, rows), F32), "dq": Guarded(q.shape, BF16),
          "dk": Guarded(k.shape, BF16), "dv": Guarded(k.shape, BF16)}
    block.attention_forward(q, k, v, key_lengths=lengths, out=at["o"].t, lse=at["lse"].t)
    block.attention_backward(do, q, k, v, at["o"].t, at["lse"].t, key_lengths=lengths, dq=at["dq"].t, dk=at["dk"].t,
                             dv=at["dv"].t)
    assert all(o.intact() for o in at.values())


def test_wrong_tensors_are_refused():
    x, w = torch.zeros(4, 64, device="cuda"), torch.ones(64, device="cuda")
    rstd = torch.ones(4, device="cuda")
    q = torch.zeros(1, 4, 2, 64, dtype=BF16, device="cuda")
    k = torch.zeros(1, 4, 1, 64, dtype=BF16, device="cuda")
    lse = torch.zeros(1, 2, 4, device="cuda")
    p = block.PackedActivation(4, 64)
    dy = torch.zeros(4, 16, dtype=BF16, device="cuda")
    for call in (
            lambda: block.rmsnorm_forward(x.double(), w), lambda: block.rmsnorm_forward(x, w[:32]),
            lambda: block.rmsnorm_forward(x.t(), w), lambda: block.rmsnorm_forward(x, w, residual=x.half()),
            lambda: block.rmsnorm_forward(x, w, residual=x[:3]), lambda: block.rmsnorm_forward(x, w, sum_out=x),
            lambda: block.rmsnorm_forward(x, w, want_out=False), lambda: block.rmsnorm_forward(x.cpu(), w),
            lambda: block.rmsnorm_forward(x, w.cpu()),
            lambda: block.rmsnorm_forward(x, w, packed=block.PackedActivation(4, 32)),
            lambda: block.rmsnorm_backward(x[:3], x, w, rstd), lambda: block.rmsnorm_backward(x, x, w, rstd[:3]),
            lambda: block.rmsnorm_backward(x, x, w, rstd, dweight_dtype=torch.float64),
            lambda: p.save(x[:3]), lambda: p.save(x.int()), lambda: p.restore(torch.float64),
            lambda: block.PackedActivation(4, 64, q=p.q[:, :64], scales=p.scales),
            lambda: block.weight_grad(dy.float(), p), lambda: block.weight_grad(dy[:3], p),
            lambda: block.weight_grad(dy, p, accumulate=True), lambda: block.weight_grad(dy.t(), p),
            lambda: block.attention_forward(q.float(), k.float(), k.float()),
            lambda: block.attention_forward(q, k, k[:, :3]), lambda: block.attention_forward(q, k.half(), k),
            lambda: block.attention_forward(q, k, k, key_lengths=torch.zeros(1, device="cuda")),
            lambda: block.attention_forward(q[..., ::2], k[..., ::2], k[..., ::2]),
            lambda: block.attention_backward(q, q, k, k, q, lse[:, :1]),
    ):
        with pytest.raises(ValueError):
            call()
