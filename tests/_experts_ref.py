"""The expert layer's operators and scaled matrices in 64 bits, and how far a
kernel may be from them (U and E as in _block_ref)."""
import numpy as np
import torch

from _block_ref import E, TINY, U

# What one addition to a running sum on the tensor cores may lose, relative to
# the magnitudes summed: they cut where fp32 would round (2^-23, not 2^-24).
CUT = 2.0 ** -23


def route(logits, k, normalize):
    """{name: tensor} by the definition, on the CPU, one token after the other."""
    v = logits.detach().cpu().double().numpy() + 0.0
    T, n = v.shape
    chosen = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    key = np.where(np.isnan(v), np.inf, v)
    for t in range(T):
        # NaN before +inf, then by value, the lower expert first
        order = sorted(range(n), key=lambda e: (not np.isnan(v[t, e]), -key[t, e], e))
        order = [e for e in order if v[t, e] != -np.inf][:k]
        chosen[t, :len(order)] = order
        if not order:
            continue
        among = v[t, order] if normalize else v[t]
        top = v[t, order[0]]
        with np.errstate(invalid="ignore"):
            p = np.exp(among - top)
            w[t, :len(order)] = np.exp(v[t, order] - top) / p.sum()
    flat = chosen.reshape(-1)
    slots = [s for e in range(n) for s in np.flatnonzero(flat == e)]
    source = np.full(T * k, -1, np.int32)
    source[:len(slots)] = slots
    place = np.full(T * k, -1, np.int32)
    place[slots] = np.arange(len(slots))
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(n)])]).astype(np.int32)
    return {"weights": torch.from_numpy(w), "experts": torch.from_numpy(chosen), "offsets": torch.from_numpy(offsets),
            "source": torch.from_numpy(source), "place": torch.from_numpy(place.reshape(T, k))}


def weights_tol(logits, w):
    """exp is good to 2 ulp, its argument to one rounding of the difference; a
    sum of num_experts / 32 + 5 additions; a division."""
    v = logits.detach().cpu().double()
    v = torch.where(v.isfinite(), v, 0.0)
    wide = (v.amax(1) - v.amin(1))[:, None]
    rel = 2 * (wide * E + 4 * E) + (v.shape[1] / 32 + 8) * E
    return rel * w.abs() + 2.0 ** -149


def product_tol(k, size, ref, dtype, out_dtype, per_mma=16, run=None):
    """Of a sum of k products with magnitudes summing to `size`: an addition for
    each MMA of per_mma products (16 more inside the MMAs and around them);
    after `run` products the sum is moved with one fp32 rounding."""
    cuts = k / per_mma
    if run is not None and k > run:
        cuts = run / per_mma + k / run
    return (cuts + 16) * CUT * size + U[out_dtype] * ref.abs() + TINY[out_dtype]


def bounds(offsets, rows):
    o = [min(max(int(x), 0), rows) for x in offsets]
    return [(o[i], max(o[i], o[i + 1])) for i in range(len(o) - 1)]


def forward(x, w, offsets):
    """(y, sum of magnitudes)."""
    y = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64, device=x.device)
    size = torch.zeros_like(y)
    for e, (a, b) in enumerate(bounds(offsets, x.shape[0])):
        xx, ww = x[a:b].double(), w[e].double()
        y[a:b], size[a:b] = xx @ ww.t(), xx.abs() @ ww.abs().t()
    return y, size


def input_grad(dy, w, offsets):
    return forward(dy, w.transpose(1, 2), offsets)


def weight_grad(dy, x, offsets):
    dw = torch.zeros(len(offsets) - 1, dy.shape[1], x.shape[1], dtype=torch.float64, device=x.device)
    size = torch.zeros_like(dw)
    for e, (a, b) in enumerate(bounds(offsets, x.shape[0])):
        d, xx = dy[a:b].double(), x[a:b].double()
        dw[e], size[e] = d.t() @ xx, d.abs().t() @ xx.abs()
    return dw, size


# ---- scaled matrices ----------------------------------------------------------

def e4m3(v):
    """float64 values rounded to e4m3 (nearest even, at most 448)."""
    a = np.abs(v)
    step = np.exp2(np.maximum(np.floor(np.log2(np.where(a == 0, 1, a))), -6) - 3)
    return np.rint(v / step) * step


def scaled(x):
    """(values [rows, cols], scale bytes [rows, scale_pitch]) of x once packed."""
    v = x.detach().cpu().double().numpy()
    rows, cols = v.shape
    blocks = -(-cols // 128)
    out = np.empty_like(v)
    byte = np.full((rows, -(-blocks // 4) * 4), 127, np.uint8)
    for b in range(blocks):
        p = v[:, b * 128:(b + 1) * 128]
        ok = np.isfinite(p)
        top = np.abs(np.where(ok, p, 0)).max(1, initial=0)
        e = np.full(rows, -127)
        guess = np.ceil(np.log2(np.where(top == 0, 1, top) / 448)).astype(int)  # within one of the least power
        e = np.where(top == 0, -127, guess)
        e = np.where((top > 0) & (top > 448 * np.exp2(e.astype(float))), e + 1, e)
        e = np.where((top > 0) & (top <= 448 * np.exp2(e - 1.0)), e - 1, e)
        e = np.maximum(e, -127)
        s = np.exp2(e.astype(float))[:, None]
        out[:, b * 128:(b + 1) * 128] = np.where(ok, e4m3(np.where(ok, p, 0) / s) * s, np.nan)
        byte[:, b] = e + 127
    return torch.from_numpy(out), byte
