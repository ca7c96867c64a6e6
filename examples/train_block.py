"""A transformer block trained with the block operators and the ZeRO step.

One pre-norm decoder block (grouped-query attention, SwiGLU) on synthetic data
over W simulated data-parallel ranks. What the backward pass needs of the
activations is kept small, as a ZeRO user wants it:

- the inputs of the projections are kept in 8 bits (the norms' packed output,
  or PackedActivation.save) and the weight gradients are taken from them;
- attention keeps its output and one number a row, and recomputes the
  probabilities;
- the gate and up activations are kept in 8 bits and restored.

Every gradient is written where the step reads it: into the rank's flat
gradient buffer. Plain products (x W^T, dy W) are torch matmuls.

    python examples/train_block.py [--steps 40]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from mixed_precision_gb300 import _abi as abi  # noqa: E402
from mixed_precision_gb300 import block  # noqa: E402
from mixed_precision_gb300.engine import Hparams, ZeroStep  # noqa: E402

HIDDEN, HEADS, KV_HEADS, HEAD_DIM, FFN = 256, 4, 2, 64, 640
NAMES = ("norm1", "wq", "wk", "wv", "wo", "norm2", "gate", "up", "down")
SHAPES = ((HIDDEN,), (HEADS * HEAD_DIM, HIDDEN), (KV_HEADS * HEAD_DIM, HIDDEN), (KV_HEADS * HEAD_DIM, HIDDEN),
          (HIDDEN, HEADS * HEAD_DIM), (HIDDEN,), (FFN, HIDDEN), (FFN, HIDDEN), (HIDDEN, FFN))
EPS = 1e-6


def forward_backward(p, g, x, target, lengths):
    """The loss of one rank's batch, its gradients written into g.

    p, g: dicts of bf16 parameters and gradient views. x, target: [batch,
    length, hidden] bf16; lengths: valid tokens of each entry (int32)."""
    batch, length, _ = x.shape
    tokens = batch * length
    h0 = x.reshape(tokens, HIDDEN)

    # ---- forward
    in1 = block.PackedActivation(tokens, HIDDEN)
    y1, _, rstd1 = block.rmsnorm_forward(h0, p["norm1"], EPS, packed=in1)
    q, k, v = ((y1 @ p[n].t()).view(batch, length, -1, HEAD_DIM) for n in ("wq", "wk", "wv"))
    mask = dict(causal=True, key_lengths=lengths)
    o, lse = block.attention_forward(q, k, v, **mask)
    flat_o = o.view(tokens, -1)
    in_o = block.PackedActivation(tokens, flat_o.shape[1]).save(flat_o)
    in2 = block.PackedActivation(tokens, HIDDEN)
    y2, h1, rstd2 = block.rmsnorm_forward(flat_o @ p["wo"].t(), p["norm2"], EPS, residual=h0, packed=in2)
    gate, up = y2 @ p["gate"].t(), y2 @ p["up"].t()
    kept_gate = block.PackedActivation(tokens, FFN).save(gate)
    kept_up = block.PackedActivation(tokens, FFN).save(up)
    out = h1 + (torch.nn.functional.silu(gate) * up) @ p["down"].t()
    del y1, y2, gate, up

    # mean squared error over the valid tokens
    valid = (torch.arange(length, device=x.device) < lengths[:, None]).reshape(tokens, 1)
    diff = (out.float() - target.reshape(tokens, HIDDEN).float()) * valid
    count = valid.sum() * HIDDEN
    loss = diff.square().sum() / count

    # ---- backward
    d_out = (2 * diff / count).to(x.dtype)
    gate, up = kept_gate.restore(x.dtype).float(), kept_up.restore(x.dtype).float()
    sig = torch.sigmoid(gate)
    act = block.PackedActivation(tokens, FFN).save((gate * sig * up).to(x.dtype))
    block.weight_grad(d_out, act, out=g["down"])
    d_act = (d_out @ p["down"]).float()
    d_gate = (d_act * up * sig * (1 + gate * (1 - sig))).to(x.dtype)
    d_up = (d_act * gate * sig).to(x.dtype)
    block.weight_grad(d_gate, in2, out=g["gate"])
    block.weight_grad(d_up, in2, out=g["up"])
    d_y2 = d_gate @ p["gate"] + d_up @ p["up"]
    d_h1, _ = block.rmsnorm_backward(d_y2, h1, p["norm2"], rstd2, dsum=d_out, dweight=g["norm2"])
    block.weight_grad(d_h1, in_o, out=g["wo"])
    d_o = (d_h1 @ p["wo"]).view_as(o)
    d_q, d_k, d_v = (t.view(tokens, -1) for t in block.attention_backward(d_o, q, k, v, o, lse, **mask))
    d_y1 = d_q @ p["wq"] + d_k @ p["wk"] + d_v @ p["wv"]
    for name, d in (("wq", d_q), ("wk", d_k), ("wv", d_v)):
        block.weight_grad(d, in1, out=g[name])
    block.rmsnorm_backward(d_y1, h0, p["norm1"], rstd1, dsum=d_h1, dweight=g["norm1"])
    return loss


def reference_loss(p, x, target, lengths):
    """The same loss in plain torch, for autograd."""
    def norm(h, w):
        return h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * w

    batch, length, _ = x.shape
    y = norm(x, p["norm1"])
    q, k, v = ((y @ p[n].t()).view(batch, length, -1, HEAD_DIM).transpose(1, 2) for n in ("wq", "wk", "wv"))
    k, v = (t.repeat_interleave(HEADS // KV_HEADS, 1) for t in (k, v))
    at = torch.arange(length, device=x.device)
    seen = (at[None, :] <= at[:, None]) & (at[None, None, :] < lengths[:, None, None])
    w = (q @ k.transpose(-1, -2) * HEAD_DIM ** -0.5).masked_fill(~seen[:, None], -1e30)
    o = (torch.softmax(w, -1) @ v).transpose(1, 2).reshape(batch, length, -1)
    h = x + o @ p["wo"].t()
    y = norm(h, p["norm2"])
    out = h + (torch.nn.functional.silu(y @ p["gate"].t()) * (y @ p["up"].t())) @ p["down"].t()
    valid = (at < lengths[:, None])[..., None]
    return ((out - target) * valid).square().sum() / (valid.sum() * HIDDEN)


def setup(world=2, batch=4, length=200, seed=0):
    """(the step's layout with its state, per-rank data, per-rank flat gradient buffers)."""
    z = ZeroStep(SHAPES, world, 2, grad_dtype=abi.ZERO_BF16, param_dtype=abi.ZERO_BF16)
    z.allocate()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    master = torch.zeros(z.np, device="cuda")
    for i, s in enumerate(SHAPES):
        z.param_view(master, i).copy_(torch.ones(s) if len(s) == 1 else normal(*s) * s[1] ** -0.5)
    z.init(master)
    data = []
    for _ in range(world):
        lengths = torch.randint(length // 2, length + 1, (batch,), generator=gen, device="cuda").to(torch.int32)
        data.append((normal(batch, length, HIDDEN).to(torch.bfloat16), normal(batch, length, HIDDEN).to(torch.bfloat16),
                     lengths))
    grads = [torch.zeros(z.np, dtype=torch.bfloat16, device="cuda") for _ in range(world)]
    return z, data, grads


def named(z, flat):
    return {n: z.param_view(flat, i) for i, n in enumerate(NAMES)}


def train(steps=40, **kw):
    """The mean loss before each step."""
    z, data, grads = setup(**kw)
    losses = []
    for _ in range(steps):
        p = named(z, z.params_flat)
        losses.append(sum(forward_backward(p, named(z, g), *d) for g, d in zip(grads, data)) / len(data))
        z.step(grads, Hparams(lr=3e-3, weight_decay=0.0))
    block.check()
    z.close()
    return [float(x) for x in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=40)
    for i, loss in enumerate(train(ap.parse_args().steps)):
        print(f"step {i:3d}  loss {loss:.4f}")
