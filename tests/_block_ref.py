"""The block operators in 64 bits, and how far a kernel may be from them.

Tolerances follow from the formulas: u(dtype) is a type's rounding error, E =
2^-24 one fp32 rounding, and every sum's error is at most (longest chain of
additions) * E * (sum of magnitudes).
"""
import numpy as np
import torch

E = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}


def close(got, ref, tol, name=""):
    """Every element within tol (a tensor); non-finite ones equal."""
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    g = got.double()
    bad = ~((g - ref).abs() <= tol) & ~((g == ref) | (g.isnan() & ref.isnan()))
    if bool(bad.any()):
        at = bad.nonzero()[0].tolist()
        i = tuple(at)
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} outside; first at {at}: "
                             f"got {g[i].item()}, want {ref[i].item()} +- {float(tol.expand_as(ref)[i])}")


# ---- packed activations -----------------------------------------------------

def pack(x):
    """(codes [rows, pitch], scale bytes) of x [rows, cols], by the definition, in numpy."""
    v = x.detach().cpu().to(torch.float64).numpy()
    rows, cols = v.shape
    pitch = -(-cols // 128) * 128
    p = np.zeros((rows, pitch))
    p[:, :cols] = v
    p = p.reshape(rows, pitch // 32, 32)
    finite = np.isfinite(p).all(-1)
    top = np.where(finite, np.abs(np.where(np.isfinite(p), p, 0)).max(-1), 0.0)
    e = np.where(top > 0, np.frexp(top)[1] - 1 - 6, -127)
    e = np.maximum(e, -127)
    q = np.clip(np.rint(np.where(finite[..., None], p, 0) * np.exp2(-e[..., None].astype(np.float64))),
                -127, 127)
    byte = np.where(finite, e + 127, 255).astype(np.uint8)
    return q.astype(np.int8).reshape(rows, pitch), byte, finite


def restore(q, byte, cols, dtype):
    """Values of codes and scale bytes (numpy) as a torch tensor of dtype."""
    rows = q.shape[0]
    s = np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127))
    v = q.reshape(rows, -1, 32) * s[..., None]
    v = torch.from_numpy(v.reshape(rows, -1)[:, :cols].copy())
    return v.to(torch.float32).to(dtype)  # the fp32 step is exact


# ---- RMSNorm ----------------------------------------------------------------

def row_chain(cols):
    """Longest chain of fp32 additions over a row: a thread's own elements (32
    in a team's registers, cols / 256 element by element), the shuffles and the
    warps, and the few roundings around it."""
    return 64 + cols / 256


def norm_forward(s, w, eps):
    """(y, rstd) in 64 bits of the stored sum s."""
    s = s.double()
    rstd = (s.square().mean(1) + eps) ** -0.5
    return s * rstd[:, None] * w.double(), rstd


def norm_backward(dy, s, w, rstd, dsum):
    """(dx, dw, tolerance of dx without its rounding, sum of magnitudes of dw)."""
    dy, s, w, r = dy.double(), s.double(), w.double(), rstd.double()[:, None]
    xh, g = s * r, dy * w
    m = (g * xh).mean(1, keepdim=True)
    dx = r * (g - xh * m)
    size = r * (g.abs() + (xh * m).abs())
    mean_size = (g * xh).abs().mean(1, keepdim=True)
    if dsum is not None:
        dx = dx + dsum.double()
        size = size + dsum.double().abs()
    tol = 8 * E * size + (row_chain(s.shape[1]) + 4) * E * r * xh.abs() * mean_size
    return dx, (dy * xh).sum(0), tol, (dy * xh).abs().sum(0)


# ---- attention --------------------------------------------------------------

def seen(q_len, k_len, causal, window, length):
    i = np.arange(q_len)[:, None] + (k_len - q_len)
    j = np.arange(k_len)[None, :]
    ok = np.broadcast_to(j < length, (q_len, k_len)).copy()
    if causal:
        ok &= j <= i
    if window:
        ok &= j > i - window
    return torch.from_numpy(ok)


def attention_forward(q, k, v, causal, window, lengths, scale):
    """(o, lse, tolerance of o, tolerance of lse), one head at a time.

    With p the exact probabilities: the products q.k carry head_dim fp32
    additions, so a logit is off by at most d = 2 head_dim E scale max(sum |q k|)
    (twice, for the scaling and the maximum's subtraction) and a probability by
    2 d + 2^-20 relatively (its exp within a few E, the total's sum); then it is
    rounded to the inputs' type for the product with v."""
    dt = q.dtype
    B, Sq, H, D = q.shape
    Sk, K = k.shape[1], k.shape[2]
    o = torch.zeros(B, Sq, H, D, dtype=torch.float64, device=q.device)
    lse = torch.full((B, H, Sq), -np.inf, dtype=torch.float64, device=q.device)
    tol_o, tol_l = torch.zeros_like(o), torch.zeros_like(lse)
    for b in range(B):
        n = Sk if lengths is None else int(lengths[b])
        ok = seen(Sq, Sk, causal, window, n).to(q.device)
        rows = ok.any(1)
        for h in range(H):
            c = h * K // H
            # nothing past the length is read, whatever it holds
            qq, kk, vv = q[b, :, h].double(), k[b, :n, c].double(), v[b, :n, c].double()
            w = (qq @ kk.t() * scale).masked_fill(~ok[:, :n], -np.inf)[rows]
            if w.numel() == 0:
                continue
            size = (qq.abs() @ kk.abs().t() * scale).amax(1)[rows][:, None]
            d = 2 * D * E * size
            lse[b, h, rows] = torch.logsumexp(w, 1)
            tol_l[b, h, rows] = (d + 2 ** -20 + 4 * E * lse[b, h, rows][:, None].abs())[:, 0]
            p = torch.softmax(w, 1)
            o[b, rows, h] = p @ vv
            rel = U[dt] + 2 * d + 2 ** -18
            tol_o[b, rows, h] = rel * (p @ vv.abs()) + U[dt] * o[b, rows, h].abs() + TINY[dt]
            if dt == torch.float16:  # probabilities below fp16's smallest number
                tol_o[b, rows, h] += 2 ** -25 * vv.abs().sum(0)
    return o, lse, tol_o, tol_l


def attention_backward(do, q, k, v, o, lse, causal, window, lengths, scale):
    """{name: (gradient, tolerance)} by the formulas, from the given o and lse.

    p = exp(scale q.k - lse) is off by d + 2^-18 + 4 E |lse| relatively; ds = p (dp
    - delta) scale carries that and the two dot products' errors, and is rounded
    to the inputs' type (as p is for dv) before its product."""
    dt = q.dtype
    B, Sq, H, D = q.shape
    Sk, K = k.shape[1], k.shape[2]
    z = lambda t: torch.zeros(t.shape, dtype=torch.float64, device=t.device)  # noqa: E731
    g = {"dq": z(q), "dk": z(k), "dv": z(v)}
    tol = {"dq": z(q), "dk": z(k), "dv": z(v)}
    for b in range(B):
        n = Sk if lengths is None else int(lengths[b])
        ok = seen(Sq, Sk, causal, window, n).to(q.device)[:, :n]
        rows = ok.any(1)
        if n == 0 or not bool(rows.any()):
            continue
        ok = ok[rows]
        for h in range(H):
            c = h * K // H
            qq, kk, vv = q[b, rows, h].double(), k[b, :n, c].double(), v[b, :n, c].double()
            gg, oo, ll = do[b, rows, h].double(), o[b, rows, h].double(), lse[b, h, rows].double()[:, None]
            size = (qq.abs() @ kk.abs().t() * scale).amax(1, keepdim=True)
            d = 2 * D * E * size + 2 ** -18 + 4 * E * ll.abs()
            p = (qq @ kk.t() * scale - ll).masked_fill(~ok, -np.inf).exp()
            x = gg @ vv.t() - (gg * oo).sum(1, keepdim=True)
            ds = p * x * scale
            dots = 2 * D * E * (gg.abs() @ vv.abs().t() + (gg * oo).abs().sum(1, keepdim=True))
            off = p * scale * (d * x.abs() + 2 * dots) + U[dt] * ds.abs()
            off_p = p * (d + U[dt])
            if dt == torch.float16:
                off = off + 2 ** -25 * max(1.0, scale) * ok
                off_p = off_p + 2 ** -25 * ok
            g["dq"][b, rows, h] = ds @ kk
            tol["dq"][b, rows, h] = off @ kk.abs() + Sk * E * (ds.abs() @ kk.abs())
            g["dk"][b, :n, c] += ds.t() @ qq
            tol["dk"][b, :n, c] += off.t() @ qq.abs() + Sq * E * (ds.abs().t() @ qq.abs())
            g["dv"][b, :n, c] += p.t() @ gg
            tol["dv"][b, :n, c] += off_p.t() @ gg.abs() + Sq * E * (p.t() @ gg.abs())
    return {n: (g[n], tol[n] + U[dt] * g[n].abs() + TINY[dt]) for n in g}
