"""The transformer-block operators, case by case: plain forms and the library's.

Three operators that produce the gradients which the ZeRO step consumes:

- RMSNorm with the residual's addition (forward, optionally with the 8-bit
  packed copy of its output; backward);
- 8-bit packed activations (pack and restore; the weight gradient computed
  from the packed copy);
- attention's training pair (forward with the row statistics; backward, which
  recomputes the probabilities).

``listed()`` names the cases, ``draw()`` gives more of the same ranges,
``prepare()`` makes the inputs, ``run()`` makes one pass: elementary torch in
32 bits, or with ``own`` the calls a user makes of mixed_precision_gb300.block.
``exact()`` is the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
GROUP = 32    # elements that share one scale in a packed activation
PITCH = 128   # a packed row is padded to a multiple of this


def listed():
    return [
        # one short micro-batch through a hidden-1024 block: bound by the call, not by the data
        dict(name="norm_fwd_64x1024", op="norm_fwd", rows=64, cols=1024, dtype="bf16", residual=True, pack=False),
        # a 16k-token micro-batch at the expert model's hidden size, keeping the 8-bit copy for backward
        dict(name="norm_fwd_pack_16384x2048", op="norm_fwd", rows=16384, cols=2048, dtype="bf16", residual=True,
             pack=True),
        # the same kind of norm backward at hidden 1024, with the gradient of the residual stream added
        dict(name="norm_bwd_16384x1024", op="norm_bwd", rows=16384, cols=1024, dtype="bf16", dsum=True),
        # a per-head q norm (head_dim columns, tokens x heads rows) in fp16, odd row count
        dict(name="norm_bwd_heads_65551x128", op="norm_bwd", rows=65551, cols=128, dtype="f16", dsum=False),
        # saving an activation in 8 bits and restoring it in backward, odd rows
        dict(name="pack_restore_8191x2048", op="pack", rows=8191, cols=2048, dtype="f16"),
        # weight gradient of a 16-expert router over a short micro-batch
        dict(name="wgrad_router_257", op="wgrad", tokens=257, n_out=16, n_in=2048, dtype="bf16", out="bf16"),
        # weight gradient of a 1024 -> 2048 projection into an fp32 main gradient
        dict(name="wgrad_proj_8192", op="wgrad", tokens=8192, n_out=2048, n_in=1024, dtype="bf16", out="f32"),
        # weight gradient of the tied embedding / output head
        dict(name="wgrad_head_4096", op="wgrad", tokens=4096, n_out=151936, n_in=1024, dtype="bf16", out="bf16"),
        # a short sequence: one tile, where latency counts
        dict(name="attn_fwd_77", op="attn_fwd", batch=1, q_len=77, k_len=77, heads=16, kv_heads=8, head_dim=128,
             dtype="bf16", causal=True, window=0, ragged=False),
        # an ordinary training micro-batch
        dict(name="attn_fwd_4x2048", op="attn_fwd", batch=4, q_len=2048, k_len=2048, heads=16, kv_heads=8,
             head_dim=128, dtype="bf16", causal=True, window=0, ragged=False),
        # padded batch of odd length with a sliding window, one entry without any valid key
        dict(name="attn_bwd_ragged_6x1021", op="attn_bwd", batch=6, q_len=1021, k_len=1021, heads=12, kv_heads=4,
             head_dim=64, dtype="f16", causal=True, window=256, ragged=True),
        # a long document
        dict(name="attn_bwd_8192", op="attn_bwd", batch=1, q_len=8192, k_len=8192, heads=16, kv_heads=8,
             head_dim=128, dtype="bf16", causal=True, window=0, ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "pack", "wgrad", "attn_fwd", "attn_bwd"])
    if op in ("norm_fwd", "norm_bwd", "pack"):
        cols = _log(rng, 64, 8192)
        if rng.random() < 0.75:
            cols = (cols + 7) // 8 * 8
        rows = _log(rng, 1, min(65536, (1 << 25) // cols))
        case = dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]))
        if op == "norm_fwd":
            case.update(residual=rng.random() < 0.7, pack=rng.random() < 0.5)
        elif op == "norm_bwd":
            case.update(dsum=rng.random() < 0.7)
        return case
    if op == "wgrad":
        n_out = _log(rng, 16, 8192)
        n_in = (_log(rng, 64, 8192) + 7) // 8 * 8
        return dict(op=op, tokens=_log(rng, 1, 16384), n_out=n_out, n_in=n_in, dtype=rng.choice(["bf16", "bf16", "f16"]),
                    out=rng.choice(["f32", "same"]))
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 3, 4])
    head_dim = rng.choice([64, 64, 80, 96, 128, 128, 128])
    # a lone key has probability 1 and passes no gradient to q and k: backward draws start above that
    few = 16 if op == "attn_bwd" else 1
    q_len = _log(rng, few, 4096)
    k_len = q_len if rng.random() < 0.7 else _log(rng, few, 4096)
    most = max(1, int(2.5e8 // (heads * q_len * k_len)))
    return dict(op=op, batch=rng.randint(1, min(8, most)), q_len=q_len, k_len=k_len, heads=heads, kv_heads=kv,
                head_dim=head_dim, dtype=rng.choice(["bf16", "bf16", "f16"]), causal=rng.random() < 0.7,
                window=rng.choice([0, 0, 0, 100, 512]), ragged=rng.random() < 0.4)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, rows, cols):
    """Hidden states: every channel has a scale of its own, a few are outliers."""
    scale = torch.exp(0.5 * _normal(g, cols))
    scale = torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, scale * 20, scale)
    return _normal(g, rows, cols) * scale


def _up(n, a):
    return (n + a - 1) // a * a


def _pack(x):
    """Packed form of x [rows, cols] (fp32 values): int8 [rows, pitch] and one biased power-of-two
    exponent for each 32 elements, uint8 [rows, pitch / 32]. The exponent is floor(log2(largest
    magnitude)) - 6, so the largest code is 64..127; codes are rounded to nearest even."""
    rows, cols = x.shape
    pitch = _up(cols, PITCH)
    v = torch.zeros(rows, pitch, dtype=torch.float32, device=x.device)
    v[:, :cols] = x
    v = v.view(rows, pitch // GROUP, GROUP)
    top = v.abs().amax(-1)
    e = torch.frexp(top)[1] - 1 - 6
    e = torch.where(top == 0, torch.full_like(e, -127), e).clamp(-127, 127)
    # two exact steps: 2^-e alone may not be an fp32 number
    half = torch.div(e, 2, rounding_mode="floor")
    one = torch.ones((), device=x.device)
    q = v * torch.ldexp(one, -half)[..., None] * torch.ldexp(one, -(e - half))[..., None]
    q = q.round().clamp(-127, 127).to(torch.int8)
    return q.view(rows, pitch), (e + 127).to(torch.uint8)


def _unpack(q, scales, cols):
    rows = q.shape[0]
    v = q.view(rows, -1, GROUP).float() * torch.ldexp(torch.ones((), device=q.device), scales.int() - 127)[..., None]
    return v.view(rows, -1)[:, :cols]


def _lengths(case, g):
    """Valid keys of each batch entry: half of them at least; the last of several entries has none."""
    if not case["ragged"]:
        return None
    n = case["k_len"] * (1 + torch.rand(case["batch"], generator=g, device="cuda")) / 2
    n = n.ceil().clamp(max=case["k_len"]).to(torch.int32)
    if case["batch"] > 1:
        n[-1] = 0
    return n


def _valid(case, lengths):
    """Which keys each query sees, [batch or 1, q_len, k_len]."""
    i = torch.arange(case["q_len"], device="cuda")[:, None] + (case["k_len"] - case["q_len"])
    j = torch.arange(case["k_len"], device="cuda")[None, :]
    ok = torch.ones(1, case["q_len"], case["k_len"], dtype=torch.bool, device="cuda")
    if case["causal"]:
        ok = ok & (j <= i)
    if case["window"]:
        ok = ok & (j > i - case["window"])
    if lengths is not None:
        ok = ok & (j < lengths[:, None, None])
    return ok


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    op = case["op"]
    dt = DTYPES[case["dtype"]]
    if op in ("norm_fwd", "norm_bwd", "pack"):
        rows, cols = case["rows"], case["cols"]
        s["x"] = _activations(g, rows, cols).to(dt)
        if op == "pack":
            return s
        s["weight"] = (1 + 0.1 * _normal(g, cols)).to(dt)
        s["eps"] = 1e-6
        if op == "norm_fwd":
            s["residual"] = _activations(g, rows, cols).to(dt) if case["residual"] else None
        else:
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(-1) + s["eps"])
            s["dy"] = (1e-2 * _normal(g, rows, cols)).to(dt)
            s["dsum"] = (1e-2 * _normal(g, rows, cols)).to(dt) if case["dsum"] else None
    elif op == "wgrad":
        x = _activations(g, case["tokens"], case["n_in"]).to(dt).float()
        s["q"], s["scales"] = _pack(x)
        # rows of dy start on 16-byte boundaries, as a projection's padded output has them
        dy = torch.zeros(case["tokens"], _up(case["n_out"], 8), dtype=dt, device="cuda")
        dy[:, :case["n_out"]] = 1e-2 * _normal(g, case["tokens"], case["n_out"])
        s["dy"] = dy[:, :case["n_out"]]
    else:
        B, H, K, D = case["batch"], case["heads"], case["kv_heads"], case["head_dim"]
        s["q"] = _normal(g, B, case["q_len"], H, D).to(dt)
        s["k"] = (1.5 * _normal(g, B, case["k_len"], K, D)).to(dt)
        s["v"] = _normal(g, B, case["k_len"], K, D).to(dt)
        s["lengths"] = _lengths(case, g)
        if op == "attn_bwd":
            o, s["lse"] = _attention(s, torch.float32)
            s["o"] = o.to(dt)
            s["do"] = (0.1 * _normal(g, B, case["q_len"], H, D)).to(dt)
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _heads(x, kv, real):
    """[batch, len, heads, dim] -> [batch, kv, heads / kv, len, dim]."""
    b, n, h, d = x.shape
    return x.to(real).view(b, n, kv, h // kv, d).permute(0, 2, 3, 1, 4)


def _tokens(x, dt):
    """The inverse, in type dt."""
    b, kv, r, n, d = x.shape
    return x.permute(0, 3, 1, 2, 4).reshape(b, n, kv * r, d).to(dt)


def _attention(s, real):
    """Output in `real` and the rows' log-sum-exp [batch, heads, q_len]."""
    case = s["case"]
    kv = case["kv_heads"]
    q, k, v = (_heads(s[n], kv, real) for n in "qkv")
    ok = _valid(case, s["lengths"])[:, None, None]
    w = (q @ k.transpose(-1, -2)) * case["head_dim"] ** -0.5
    w = w.masked_fill_(~ok, -math.inf)
    top = w.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    w = w.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    o = (w @ v) / torch.where(total == 0, 1.0, total)
    lse = (top + total.log()).squeeze(-1)
    return _tokens(o, real), lse.reshape(lse.shape[0], -1, lse.shape[-1])


def _plain_norm_fwd(s):
    x, case = s["x"], s["case"]
    out = {}
    if s["residual"] is not None:
        x = (x.float() + s["residual"].float()).to(x.dtype)
        out["sum"] = x
    v = x.float()
    out["rstd"] = torch.rsqrt(v.square().mean(-1) + s["eps"])
    out["y"] = (v * out["rstd"][:, None] * s["weight"].float()).to(x.dtype)
    if case["pack"]:
        out["restored"] = _unpack(*_pack(out["y"].float()), case["cols"]).to(x.dtype)
    return out


def _plain_norm_bwd(s):
    x, dy, w, r = s["x"].float(), s["dy"].float(), s["weight"].float(), s["rstd"][:, None]
    xhat = x * r
    g = dy * w
    dx = r * (g - xhat * (g * xhat).mean(-1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xhat).sum(0)}


def _out_dtype(case):
    return torch.float32 if case["out"] == "f32" else DTYPES[case["dtype"]]


def _plain_wgrad(s):
    x = _unpack(s["q"], s["scales"], s["case"]["n_in"])
    return (s["dy"].float().t() @ x).to(_out_dtype(s["case"]))


def _plain_attn_bwd(s):
    case = s["case"]
    kv, dt, scale = case["kv_heads"], s["q"].dtype, case["head_dim"] ** -0.5
    q, k, v, o, do = (_heads(s[n], kv, torch.float32) for n in ("q", "k", "v", "o", "do"))
    lse = s["lse"].view(q.shape[:-1])[..., None]
    ok = _valid(case, s["lengths"])[:, None, None]
    p = ((q @ k.transpose(-1, -2)) * scale).sub_(torch.where(lse == -math.inf, 0.0, lse)).exp_()
    p = p.masked_fill_(~ok, 0.0)
    dv = (p.transpose(-1, -2) @ do).sum(2, keepdim=True)
    ds = (do @ v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    dk = (ds.transpose(-1, -2) @ q).sum(2, keepdim=True)
    return {"dq": _tokens(ds @ k, dt), "dk": _tokens(dk, dt), "dv": _tokens(dv, dt)}


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    op = case["op"]
    if op == "norm_fwd":
        return _plain_norm_fwd(state)
    if op == "norm_bwd":
        return _plain_norm_bwd(state)
    if op == "pack":
        x = state["x"]
        return {"restored": _unpack(*_pack(x.float()), case["cols"]).to(x.dtype)}
    if op == "wgrad":
        return {"dweight": _plain_wgrad(state)}
    if op == "attn_fwd":
        o, lse = _attention(state, torch.float32)
        return {"o": o.to(state["q"].dtype), "lse": lse}
    return _plain_attn_bwd(state)


# ---------------------------------------------------------------------------
# The library's operators
# ---------------------------------------------------------------------------

def _run_own(s):
    from mixed_precision_gb300 import block
    case = s["case"]
    op = case["op"]
    if op == "norm_fwd":
        packed = block.PackedActivation(case["rows"], case["cols"]) if case["pack"] else None
        y, total, rstd = block.rmsnorm_forward(s["x"], s["weight"], s["eps"], residual=s["residual"], packed=packed)
        out = {"y": y, "rstd": rstd}
        if s["residual"] is not None:
            out["sum"] = total
        if packed is not None:
            out["restored"] = packed.restore(s["x"].dtype)
        return out
    if op == "norm_bwd":
        dx, dw = block.rmsnorm_backward(s["dy"], s["x"], s["weight"], s["rstd"], dsum=s["dsum"],
                                        dweight_dtype=torch.float32)
        return {"dx": dx, "dweight": dw}
    if op == "pack":
        packed = block.PackedActivation(case["rows"], case["cols"])
        packed.save(s["x"])
        return {"restored": packed.restore(s["x"].dtype)}
    if op == "wgrad":
        packed = block.PackedActivation(case["tokens"], case["n_in"], q=s["q"], scales=s["scales"])
        return {"dweight": block.weight_grad(s["dy"], packed, dtype=_out_dtype(case))}
    mask = dict(causal=case["causal"], window=case["window"], key_lengths=s["lengths"])
    if op == "attn_fwd":
        o, lse = block.attention_forward(s["q"], s["k"], s["v"], **mask)
        return {"o": o, "lse": lse}
    dq, dk, dv = block.attention_backward(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], **mask)
    return {"dq": dq, "dk": dk, "dv": dv}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def _pairs(case):
    """Query-key pairs that the causal and window masks leave, of one head (lengths counted full)."""
    n, off = 0, case["k_len"] - case["q_len"]
    for i in range(case["q_len"]):
        hi = min(case["k_len"] - 1, i + off) if case["causal"] else case["k_len"] - 1
        lo = max(0, i + off - case["window"] + 1) if case["window"] else 0
        n += max(0, hi - lo + 1)
    return n


def work(case):
    op = case["op"]
    b = BYTES[case["dtype"]]
    if op == "norm_fwd":
        n = case["rows"] * case["cols"]
        tensors = 4 if case["residual"] else 2
        packed = 2 * (1 + 1 / GROUP) + b if case["pack"] else 0  # written, read back and restored
        return {"bytes": n * (tensors * b + packed) + 4 * case["rows"] + b * case["cols"], "flops": 5 * n}
    if op == "norm_bwd":
        n = case["rows"] * case["cols"]
        return {"bytes": n * b * (4 if case["dsum"] else 3) + 4 * case["rows"] + (b + 4) * case["cols"], "flops": 9 * n}
    if op == "pack":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (2 * b + 2 * (1 + 1 / GROUP)), "flops": 3 * n}
    if op == "wgrad":
        t, m, n = case["tokens"], case["n_out"], case["n_in"]
        out = 4 if case["out"] == "f32" else b
        return {"bytes": t * (m * b + n * (1 + 1 / GROUP)) + out * m * n, "flops": 2 * t * m * n}
    q = case["batch"] * case["q_len"] * case["heads"] * case["head_dim"] * b
    kv = case["batch"] * case["k_len"] * case["kv_heads"] * case["head_dim"] * b
    lse = 4 * case["batch"] * case["heads"] * case["q_len"]
    product = 2 * case["batch"] * case["heads"] * case["head_dim"] * _pairs(case)
    if op == "attn_fwd":
        return {"bytes": 2 * q + 2 * kv + lse, "flops": 2 * product}
    return {"bytes": 4 * q + 4 * kv + lse, "flops": 5 * product}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm_fwd":
        x = s["x"].double()
        out = {}
        if s["residual"] is not None:
            x = x + s["residual"].double()
            out["sum"] = x
            x = x.to(s["x"].dtype).double()  # the norm is taken of the stored sum
        size = torch.linalg.vector_norm(x, dim=1, keepdim=True)
        rms = (size * size / case["cols"] + s["eps"]).sqrt()
        out["rstd"] = 1 / rms[:, 0]
        out["y"] = x / rms * s["weight"].double()
        if case["pack"]:
            out["restored"] = out["y"]  # what the packed copy stands for
        return out
    if op == "norm_bwd":
        # y_t = x_t r_t w, r_t = (mean(x_t^2) + eps)^(-1/2): the products with the Jacobian, written out
        x, dy, w, r = (s[n].double() for n in ("x", "dy", "weight", "rstd"))
        along = torch.einsum("tc,tc,c->t", dy, x, w)
        dx = torch.einsum("tc,c,t->tc", dy, w, r) - torch.einsum("tc,t->tc", x, along * r ** 3 / case["cols"])
        if s["dsum"] is not None:
            dx = dx + s["dsum"].double()
        return {"dx": dx, "dweight": torch.einsum("tc,tc,t->c", dy, x, r)}
    if op == "pack":
        return {"restored": s["x"].double()}
    if op == "wgrad":
        x = s["q"].double() * torch.exp2(s["scales"].double() - 127).repeat_interleave(GROUP, 1)
        return {"dweight": torch.einsum("to,ti->oi", s["dy"].double(), x[:, :case["n_in"]].contiguous())}
    # attention, one head at a time
    B, H, K, D = case["batch"], case["heads"], case["kv_heads"], case["head_dim"]
    off = case["k_len"] - case["q_len"]
    at_q = torch.arange(case["q_len"], device="cuda").view(-1, 1)
    at_k = torch.arange(case["k_len"], device="cuda").view(1, -1)
    o = torch.zeros(B, case["q_len"], H, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, case["q_len"]), -math.inf, dtype=torch.float64, device="cuda")
    grads = {"dq": torch.zeros_like(o)}
    grads["dk"] = torch.zeros(B, case["k_len"], K, D, dtype=torch.float64, device="cuda")
    grads["dv"] = torch.zeros_like(grads["dk"])
    for b in range(B):
        n = case["k_len"] if s["lengths"] is None else int(s["lengths"][b])
        seen = (at_k < n).expand(case["q_len"], -1)
        if case["causal"]:
            seen = seen & (at_k - off <= at_q)
        if case["window"]:
            seen = seen & (at_k - off + case["window"] > at_q)
        rows = seen.any(1)
        if not bool(rows.any()):
            continue
        for h in range(H):
            c = h * K // H
            q, k, v = s["q"][b, :, h].double(), s["k"][b, :, c].double(), s["v"][b, :, c].double()
            w = torch.where(seen, torch.einsum("id,jd->ij", q, k) / math.sqrt(D), -math.inf)[rows]
            lse[b, h, rows] = torch.logsumexp(w, 1)
            p = torch.softmax(w, 1)
            if op == "attn_fwd":
                o[b, rows, h] = p @ v
                continue
            do = s["do"][b, :, h].double()[rows]
            dp = do @ v.t()
            dw = p * (dp - (p * dp).sum(1, keepdim=True)) / math.sqrt(D)
            grads["dv"][b, :, c] += p.t() @ do
            grads["dk"][b, :, c] += dw.t() @ q[rows]
            grads["dq"][b, rows, h] = dw @ k
    return {"o": o, "lse": lse} if op == "attn_fwd" else grads
