"""The expert layer's operators and 8-bit floating-point products, case by case.

Three operators of a mixture-of-experts layer's training step:

- routing: the choice of k experts for each token, the rows' order by expert,
  their copy in that order, and the weighted way back with its gradients;
- the experts' products over ragged runs of rows: forward, input gradient and
  weight gradient;
- products of e4m3 matrices with a power-of-two scale for each 128 elements
  along the contraction, packing included, for a linear layer and for experts.

``listed()`` names the cases, ``draw()`` gives more of the same ranges,
``prepare()`` makes the inputs, ``run()`` makes one pass: elementary torch in
32 bits, or with ``own`` the calls a user makes of mixed_precision_gb300.experts
and mixed_precision_gb300.float8. ``exact()`` is the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = 128   # elements along the contraction that share one scale
TOP = 448.0   # the largest e4m3 number


def listed():
    return [
        # the end of a batch: few tokens through a 16-expert router, where the calls count
        dict(name="route_33x16", op="route", tokens=33, experts=16, k=2, hidden=2048, dtype="bf16", logits="f32",
             normalize=True, padded=False),
        # an ordinary micro-batch of the expert model
        dict(name="route_8192x16", op="route", tokens=8192, experts=16, k=2, hidden=2048, dtype="bf16", logits="f32",
             normalize=True, padded=False),
        # backward of the way back and of the router: many small experts, odd count, padding tokens
        dict(name="combine_bwd_8191x128", op="combine_bwd", tokens=8191, experts=128, k=8, hidden=1024, dtype="f16",
             logits="f32", normalize=False, padded=True),
        # gate and up of 16 experts as one product, two rows a token of an 8192-token micro-batch
        dict(name="up_fwd_16384", op="fwd", rows=16384, experts=16, n_out=2048, n_in=2048, dtype="bf16"),
        # down projection of a few tokens: bound by the experts' weights
        dict(name="down_fwd_74", op="fwd", rows=74, experts=16, n_out=2048, n_in=1024, dtype="bf16"),
        # input gradient of the down projection in fp16, odd sizes, idle experts
        dict(name="down_dgrad_16381", op="dgrad", rows=16381, experts=16, n_out=2048, n_in=1024, dtype="f16"),
        # weight gradient of gate and up into fp32 main gradients
        dict(name="up_wgrad_16384", op="wgrad", rows=16384, experts=16, n_out=2048, n_in=2048, dtype="bf16", out="f32"),
        # weight gradients of many small experts: few rows each, sizes that fill no tile
        dict(name="wgrad_fine_8190x64", op="wgrad", rows=8190, experts=64, n_out=520, n_in=1000, dtype="f16", out="same"),
        # a 1024 -> 2048 projection in 8 bits: its input packed, then the product
        dict(name="f8_linear_8192", op="f8", tokens=8192, experts=0, n_out=2048, n_in=1024, dtype="bf16"),
        # a large linear layer, bound by the tensor cores
        dict(name="f8_large_8192", op="f8", tokens=8192, experts=0, n_out=8192, n_in=4096, dtype="bf16"),
        # weight gradient of a linear layer in 8 bits: both inputs packed along the tokens, odd count, fp32 out
        dict(name="f8_wgrad_4097", op="f8_wgrad", tokens=4097, n_out=2048, n_in=2048, dtype="bf16", out="f32"),
        # gate and up of 16 experts in 8 bits
        dict(name="f8_experts_16384", op="f8", tokens=16384, experts=16, n_out=2048, n_in=2048, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _eights(rng, lo, hi):
    return (_log(rng, lo, hi) + 7) // 8 * 8


def draw(rng):
    op = rng.choice(["route", "combine", "combine_bwd", "fwd", "dgrad", "wgrad", "f8", "f8_wgrad"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op in ("route", "combine", "combine_bwd"):
        experts = _log(rng, 2, 256)
        hidden = _eights(rng, 64, 4096)
        # a lone choice has a normalised weight of 1, which passes nothing back: not drawn
        k = rng.randint(2, min(8, experts))
        tokens = _log(rng, 1, min(32768, (1 << 27) // (hidden * k)))
        return dict(op=op, tokens=tokens, experts=experts, k=k, hidden=hidden, dtype=dtype,
                    logits=rng.choice(["f32", "bf16"]), normalize=rng.random() < 0.6, padded=rng.random() < 0.3)
    n_out, n_in = _log(rng, 16, 4096), _eights(rng, 64, 4096)
    if op == "f8_wgrad":
        return dict(op=op, tokens=_log(rng, 1, 16384), n_out=n_out, n_in=n_in, dtype=dtype, out=rng.choice(["f32", "same"]))
    experts = min(_log(rng, 1, 128), (1 << 28) // (n_out * n_in))
    rows = _log(rng, 1, 16384)
    if op == "f8":
        return dict(op=op, tokens=rows, experts=rng.choice([0, experts]), n_out=n_out, n_in=n_in, dtype=dtype)
    case = dict(op=op, rows=rows, experts=experts, n_out=n_out, n_in=n_in, dtype=dtype)
    if op == "wgrad":
        case.update(out=rng.choice(["f32", "same"]))
    return case


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


def _rows16(x, dt):
    """x in type dt, its rows starting on 16-byte boundaries as a padded projection's do."""
    out = torch.zeros(x.shape[0], (x.shape[1] + 7) // 8 * 8, dtype=dt, device=x.device)
    out[:, :x.shape[1]] = x
    return out[:, :x.shape[1]]


def _runs(g, rows, experts):
    """Where each expert's run of rows starts, [experts + 1]: some experts are much asked for, every
    eighth one is idle."""
    share = torch.exp(0.5 * _normal(g, experts))
    share[7::8] = 0
    at = share.cumsum(0) / share.sum() * rows
    at = at.round().to(torch.int32)
    at[-1] = rows
    return torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), at])


def _pack(x):
    """x [..., rows, cols] (fp32 values) as e4m3 codes [..., rows, cols up to a multiple of 128] and the
    biased exponents of the scales [..., rows, blocks up to a multiple of 4]: the smallest power of two that
    brings a block's largest magnitude to 448 or below."""
    cols = x.shape[-1]
    blocks = (cols + BLOCK - 1) // BLOCK
    v = torch.zeros(*x.shape[:-1], blocks * BLOCK, dtype=torch.float32, device=x.device)
    v[..., :cols] = x
    v = v.view(*x.shape[:-1], blocks, BLOCK)
    m, e = torch.frexp(v.abs().amax(-1))  # top = m 2^e, m in [0.5, 1): 448 = 0.875 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(m == 0, torch.full_like(e, -127), e).clamp(-127, 127)
    half = torch.div(e, 2, rounding_mode="floor")  # 2^-e alone may not be an fp32 number
    one = torch.ones((), device=x.device)
    v = v * torch.ldexp(one, -half)[..., None] * torch.ldexp(one, half - e)[..., None]
    q = v.to(torch.float8_e4m3fn).view(*x.shape[:-1], blocks * BLOCK)
    scales = torch.full((*x.shape[:-1], (blocks + 3) // 4 * 4), 127, dtype=torch.uint8, device=x.device)
    scales[..., :blocks] = (e + 127).to(torch.uint8)
    return q, scales


def _unpack(q, scales, cols):
    blocks = q.shape[-1] // BLOCK
    s = torch.ldexp(torch.ones((), device=q.device), scales[..., :blocks].int() - 127)
    v = q.float().view(*q.shape[:-1], blocks, BLOCK) * s[..., None]
    return v.view(*q.shape[:-1], blocks * BLOCK)[..., :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    op = case["op"]
    dt = DTYPES[case["dtype"]]
    if op in ("route", "combine", "combine_bwd"):
        T, E, k, H = case["tokens"], case["experts"], case["k"], case["hidden"]
        logits = 1.5 * _normal(g, T, E) + 0.5 * _normal(g, E)
        if case["padded"]:  # the batch's padding goes to no expert
            logits[torch.rand(T, generator=g, device="cuda") < 0.1] = -math.inf
        s["logits"] = logits.to(DTYPES[case["logits"]])
        if op == "route":
            s["x"] = _activations(g, T, H).to(dt)
            return s
        s["routing"] = _route(s["logits"], k, case["normalize"])
        s["y"] = _normal(g, T * k, H).to(dt)
        if op == "combine_bwd":
            s["dout"] = (1e-2 * _normal(g, T, H)).to(dt)
        return s
    n_out, n_in, E = case["n_out"], case["n_in"], case.get("experts", 0)
    rows = case["rows"] if "rows" in case else case["tokens"]
    if E:
        s["offsets"] = _runs(g, rows, E)
        s["bounds"] = s["offsets"].tolist()
    if op in ("fwd", "dgrad", "f8"):
        w = _normal(g, *([E] if E else []), n_out, n_in) * n_in ** -0.5
        if op == "f8":
            s["w8"], s["w8_scales"] = _pack(w)
        else:
            s["w"] = w.to(dt)
        del w
    if op in ("fwd", "wgrad", "f8", "f8_wgrad"):
        s["x"] = _rows16(_activations(g, rows, n_in), dt)
    if op in ("dgrad", "wgrad", "f8_wgrad"):
        s["dy"] = _rows16(1e-2 * _normal(g, rows, n_out), dt)
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _route(logits, k, normalize):
    """The choice and the order: the k largest logits of each token (ties: the lower expert; -inf is never
    chosen: expert -1), softmax weights, and the chosen slots t * k + j sorted by expert."""
    T, E = logits.shape
    v = logits.float()
    left = v.clone()
    at = torch.arange(E, device=v.device)
    chosen = []
    for _ in range(k):
        top = left.amax(1, keepdim=True)
        i = torch.where(left == top, at, E).amin(1, keepdim=True)
        chosen.append(torch.where(top == -math.inf, -1, i))
        left = left.scatter(1, i, -math.inf)
    experts = torch.cat(chosen, 1)
    ok = experts >= 0
    top = v.amax(1, keepdim=True)
    p = torch.where(v == -math.inf, 0.0, torch.exp(v - top))
    w = torch.where(ok, p.gather(1, experts.clamp(min=0)), 0.0)
    total = (w if normalize else p).sum(1, keepdim=True)
    w = torch.where(ok, w / total, 0.0)
    flat = torch.where(ok, experts, E).view(-1)
    hits = flat[:, None] == at
    counts = hits.sum(0)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=v.device)
    offsets[1:] = counts.cumsum(0)
    rank = hits.to(torch.int32).cumsum(0).gather(1, flat.clamp(max=E - 1)[:, None])[:, 0] - 1
    place = torch.where(ok.view(-1), offsets[flat.clamp(max=E - 1)] + rank, -1)
    source = torch.full((T * k + 1,), -1, dtype=torch.int64, device=v.device)
    source[torch.where(place < 0, T * k, place)] = torch.arange(T * k, device=v.device)
    source[T * k] = -1
    i32 = torch.int32
    return {"weights": w, "experts": experts.to(i32), "offsets": offsets.to(i32), "source": source[:-1].to(i32),
            "place": place.view(T, k).to(i32)}


def _gather(x, source, k):
    rows = x[torch.div(source, k, rounding_mode="floor").clamp(min=0).long()]
    return torch.where((source >= 0)[:, None], rows, torch.zeros((), dtype=x.dtype, device=x.device))


def _placed(y, place):
    """[tokens, k, hidden] in fp32: the rows at `place`, zero where it is -1."""
    return torch.where((place >= 0)[..., None], y[place.clamp(min=0).long()].float(), 0.0)


def _plain_combine(s):
    r = s["routing"]
    return (_placed(s["y"], r["place"]) * r["weights"][..., None]).sum(1).to(s["y"].dtype)


def _plain_combine_bwd(s):
    r, case, d = s["routing"], s["case"], s["dout"].float()
    k, source = case["k"], r["source"].long()
    w = r["weights"].view(-1)[source.clamp(min=0)]
    dy = d[torch.div(source, k, rounding_mode="floor").clamp(min=0)] * w[:, None]
    dy = torch.where((source >= 0)[:, None], dy, 0.0).to(s["y"].dtype)
    dw = (_placed(s["y"], r["place"]) * d[:, None]).sum(-1)
    along = (r["weights"] * dw).sum(1, keepdim=True)
    at = torch.where(r["experts"] < 0, case["experts"], r["experts"]).long()
    wide = torch.zeros(d.shape[0], case["experts"] + 1, device=d.device)
    if case["normalize"]:
        dlogits = wide.scatter(1, at, r["weights"] * (dw - along))[:, :-1]
    else:
        v = s["logits"].float()
        top = v.amax(1, keepdim=True)
        p = torch.where(v == -math.inf, 0.0, torch.exp(v - torch.where(top == -math.inf, 0.0, top)))
        total = p.sum(1, keepdim=True)
        p = p / torch.where(total == 0, 1.0, total)
        dlogits = wide.scatter(1, at, r["weights"] * dw)[:, :-1] - p * along
    return {"dy": dy, "dweights": dw, "dlogits": dlogits.to(s["logits"].dtype)}


def _out_dtype(case):
    return torch.float32 if case["out"] == "f32" else DTYPES[case["dtype"]]


def _plain_products(s):
    case = s["case"]
    op, dt, at = case["op"], DTYPES[case["dtype"]], s["bounds"]
    if op == "wgrad":
        out = torch.zeros(case["experts"], case["n_out"], case["n_in"], dtype=_out_dtype(case), device="cuda")
    else:
        out = torch.zeros(case["rows"], case["n_out" if op == "fwd" else "n_in"], dtype=dt, device="cuda")
    for e in range(case["experts"]):
        run = slice(at[e], at[e + 1])
        if at[e] == at[e + 1]:
            continue
        if op == "fwd":
            out[run] = (s["x"][run].float() @ s["w"][e].float().t()).to(dt)
        elif op == "dgrad":
            out[run] = (s["dy"][run].float() @ s["w"][e].float()).to(dt)
        else:
            out[e] = (s["dy"][run].float().t() @ s["x"][run].float()).to(out.dtype)
    return out


def _plain_f8(s):
    case = s["case"]
    dt = DTYPES[case["dtype"]]
    x = _unpack(*_pack(s["x"].float()), case["n_in"])
    w = _unpack(s["w8"], s["w8_scales"], case["n_in"])
    if not case["experts"]:
        return {"restored": x.to(dt), "y": (x @ w.t()).to(dt)}
    y = torch.zeros(case["tokens"], case["n_out"], dtype=dt, device="cuda")
    at = s["bounds"]
    for e in range(case["experts"]):
        if at[e] < at[e + 1]:
            y[at[e]:at[e + 1]] = (x[at[e]:at[e + 1]] @ w[e].t()).to(dt)
    return {"restored": x.to(dt), "y": y}


def _plain_f8_wgrad(s):
    case = s["case"]
    dy = _unpack(*_pack(s["dy"].float().t()), case["tokens"])
    x = _unpack(*_pack(s["x"].float().t()), case["tokens"])
    return {"dweight": (dy @ x.t()).to(_out_dtype(case))}


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    op = case["op"]
    if op == "route":
        r = _route(state["logits"], case["k"], case["normalize"])
        return {**r, "rows": _gather(state["x"], r["source"], case["k"])}
    if op == "combine":
        return {"out": _plain_combine(state)}
    if op == "combine_bwd":
        return _plain_combine_bwd(state)
    if op == "f8":
        return _plain_f8(state)
    if op == "f8_wgrad":
        return _plain_f8_wgrad(state)
    return {"out": _plain_products(state)}


# ---------------------------------------------------------------------------
# The framework's operators
# ---------------------------------------------------------------------------

_FIELDS = ("weights", "experts", "offsets", "source", "place")


def _run_own(s):
    from mixed_precision_gb300 import experts, float8
    case = s["case"]
    op = case["op"]
    if op == "route":
        r = experts.route(s["logits"], case["k"], normalize=case["normalize"])
        return {**{n: getattr(r, n) for n in _FIELDS}, "rows": experts.gather(s["x"], r)}
    if op in ("combine", "combine_bwd"):
        r = experts.Routing(case["experts"], case["normalize"], **s["routing"])
        if op == "combine":
            return {"out": experts.combine(s["y"], r)}
        dy, dw = experts.combine_backward(s["dout"], s["y"], r)
        return {"dy": dy, "dweights": dw, "dlogits": experts.route_backward(dw, s["logits"], r)}
    if op == "fwd":
        return {"out": experts.forward(s["x"], s["w"], s["offsets"])}
    if op == "dgrad":
        return {"out": experts.input_grad(s["dy"], s["w"], s["offsets"])}
    if op == "wgrad":
        return {"out": experts.weight_grad(s["dy"], s["x"], s["offsets"], dtype=_out_dtype(case))}
    if op == "f8_wgrad":
        _, dy = float8.pack(s["dy"], direct=False, transposed=True)
        _, x = float8.pack(s["x"], direct=False, transposed=True)
        return {"dweight": float8.matmul(dy, x, dtype=_out_dtype(case))}
    w = float8.Float8Matrix(case["n_out"], case["n_in"], case["experts"] or None, q=s["w8"], scales=s["w8_scales"])
    x, _ = float8.pack(s["x"])
    return {"restored": x.restore(s["x"].dtype), "y": float8.matmul(x, w, s.get("offsets"), dtype=s["x"].dtype)}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op, b = case["op"], BYTES[case["dtype"]]
    if op in ("route", "combine", "combine_bwd"):
        T, E, k, H = case["tokens"], case["experts"], case["k"], case["hidden"]
        choice = T * E * BYTES[case["logits"]]
        if op == "route":
            return {"bytes": choice + 16 * T * k + 4 * (E + 1) + (1 + k) * T * H * b, "flops": T * E * (k + 4)}
        if op == "combine":
            return {"bytes": 8 * T * k + (1 + k) * T * H * b, "flops": 2 * T * k * H}
        return {"bytes": 2 * choice + 20 * T * k + (1 + 2 * k) * T * H * b, "flops": 3 * T * k * H}
    n_out, n_in = case["n_out"], case["n_in"]
    rows = case["rows"] if "rows" in case else case["tokens"]
    E = case.get("experts", 0)
    weights = max(E, 1) * n_out * n_in
    if E:  # idle experts' weights are not read
        weights = min(E - E // 8, rows) * n_out * n_in
    flops = 2 * rows * n_out * n_in
    if op in ("fwd", "dgrad"):
        return {"bytes": b * (rows * (n_out + n_in) + weights) + 4 * (E + 1), "flops": flops}
    if op == "wgrad":
        out = 4 if case["out"] == "f32" else b
        return {"bytes": b * rows * (n_out + n_in) + out * E * n_out * n_in, "flops": flops}
    f8 = 1 + 1 / BLOCK
    if op == "f8":  # x read, its packed copy written and read back twice (product, restored), restored and y written
        return {"bytes": rows * (n_in * (2 * b + 3 * f8) + n_out * b) + f8 * weights, "flops": flops}
    out = 4 if case["out"] == "f32" else b
    return {"bytes": rows * (n_out + n_in) * (b + 2 * f8) + out * n_out * n_in, "flops": flops}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_route(logits, k, normalize):
    T, E = logits.shape
    v = logits.double()
    order = torch.sort(v, dim=1, descending=True, stable=True)[1][:, :k]
    picked = v.gather(1, order)
    taken = picked > -math.inf
    experts = torch.where(taken, order, -1)
    rest = picked if normalize else v
    w = torch.where(taken, torch.exp(picked - torch.logsumexp(rest, 1, keepdim=True)), 0.0)
    flat = torch.where(taken, order, E).reshape(-1)
    by_expert = torch.sort(flat, stable=True)[1]
    n = int(taken.sum())
    source = torch.where(torch.arange(T * k, device=v.device) < n, by_expert, -1)
    place = torch.full((T * k,), -1, dtype=torch.int64, device=v.device)
    place[by_expert[:n]] = torch.arange(n, device=v.device)
    offsets = torch.searchsorted(flat[by_expert], torch.arange(E + 1, device=v.device))
    i32 = torch.int32
    return {"weights": w, "experts": experts.to(i32), "offsets": offsets.to(i32), "source": source.to(i32),
            "place": place.view(T, k).to(i32)}


def _exact_blocks(x):
    """What x [rows, cols] stands for once packed: every element rounded to e4m3 at its block's scale."""
    x = x.double()
    out = torch.empty_like(x)
    for c in range(0, x.shape[1], BLOCK):
        v = x[:, c:c + BLOCK]
        top = v.abs().amax(1, keepdim=True)
        e = torch.ceil(torch.log2(torch.where(top == 0, 1.0, top) / TOP))
        # log2 of a quotient next to a power of two may round to the wrong side of it
        e = torch.where(top > TOP * torch.exp2(e), e + 1, e)
        e = torch.where(top <= TOP * torch.exp2(e - 1), e - 1, e).clamp(min=-127)
        scaled = v / torch.exp2(e)
        size = scaled.abs()
        step = torch.exp2(torch.floor(torch.log2(torch.where(size == 0, 1.0, size))).clamp(min=-6) - 3)
        out[:, c:c + BLOCK] = torch.round(scaled / step) * step * torch.exp2(e)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        r = _exact_route(s["logits"], case["k"], case["normalize"])
        rows = torch.zeros(r["source"].shape[0], case["hidden"], dtype=torch.float64, device="cuda")
        n = int(r["offsets"][-1])
        rows[:n] = s["x"].double().index_select(0, r["source"][:n].long() // case["k"])
        return {**r, "rows": rows}
    if op in ("combine", "combine_bwd"):
        T, k, E = case["tokens"], case["k"], case["experts"]
        r = {n: t.double() if n == "weights" else t.long() for n, t in s["routing"].items()}
        y, n = s["y"], int(r["offsets"][-1])
        slot = r["source"][:n]
        token, w = slot // k, r["weights"].view(-1)[slot]
        if op == "combine":
            out = torch.zeros(T, case["hidden"], dtype=torch.float64, device="cuda")
            return {"out": out.index_add_(0, token, y[:n].double() * w[:, None])}
        dy = torch.zeros(y.shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros(T * k, dtype=torch.float64, device="cuda")
        for at in range(0, n, 1 << 14):
            to = min(n, at + (1 << 14))
            d = s["dout"].double()[token[at:to]]
            dy[at:to] = w[at:to, None] * d
            dw[slot[at:to]] = torch.einsum("rh,rh->r", d, y[at:to].double())
        dw = dw.view(T, k)
        # weights as a function of all logits: dw_j / dl_i = w_j (delta_ij - q_i), q the softmax over those
        # in the total
        taken = r["experts"] >= 0
        column = torch.where(taken, r["experts"], E)
        q = torch.zeros(T, E + 1, dtype=torch.float64, device="cuda")
        own_part = torch.zeros_like(q).scatter_add_(1, column, torch.where(taken, r["weights"] * dw, 0.0))
        if case["normalize"]:
            q.scatter_(1, column, r["weights"])
        else:
            q[:, :E] = torch.nan_to_num(torch.softmax(s["logits"].double(), 1), nan=0.0)
        dl = own_part - q * torch.where(taken, r["weights"] * dw, 0.0).sum(1, keepdim=True)
        return {"dy": dy, "dweights": dw, "dlogits": dl[:, :E]}
    if op == "f8_wgrad":
        dy, x = _exact_blocks(s["dy"].t()), _exact_blocks(s["x"].t())
        return {"dweight": torch.einsum("ot,it->oi", dy, x)}
    experts = case["experts"]
    at = s.get("bounds")
    if op == "f8":
        x = _exact_blocks(s["x"])
        exponents = s["w8_scales"].double().repeat_interleave(BLOCK, -1)[..., :s["w8"].shape[-1]] - 127
        w = (s["w8"].double() * torch.exp2(exponents))[..., :case["n_in"]]
        if not experts:
            return {"restored": x, "y": torch.einsum("ti,oi->to", x, w)}
        y = [torch.einsum("ti,oi->to", x[at[e]:at[e + 1]], w[e]) for e in range(experts)]
        return {"restored": x, "y": torch.cat(y)}
    runs = [slice(at[e], at[e + 1]) for e in range(experts)]
    if op == "fwd":
        parts = [torch.einsum("ti,oi->to", s["x"][t].double(), s["w"][e].double()) for e, t in enumerate(runs)]
        return {"out": torch.cat(parts)}
    if op == "dgrad":
        parts = [torch.einsum("to,oi->ti", s["dy"][t].double(), s["w"][e].double()) for e, t in enumerate(runs)]
        return {"out": torch.cat(parts)}
    return {"out": torch.stack([torch.einsum("to,ti->oi", s["dy"][t].double(), s["x"][t].double()) for t in runs])}
