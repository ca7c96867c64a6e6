"""The block operators' host side, without a GPU: sizes that the library
reports, calls with nothing to do, and every refusal, all before any device
call. The pointers are made-up addresses that are never read."""
import ctypes

import pytest

P = 1 << 20  # an aligned address


@pytest.fixture(scope="module")
def z():
    from mixed_precision_gb300 import build
    build.build()
    import mixed_precision_gb300 as mp
    return mp


def norm(z, **over):
    f = dict(rows=4, cols=64, x_stride=64, residual_stride=64, dy_stride=64, dtype=2, weight_dtype=2, eps=1e-6)
    f.update(over)
    return z.zero_rmsnorm_desc(**f)


def attention(z, **over):
    f = dict(batch=2, q_len=10, k_len=12, q_heads=4, kv_heads=2, head_dim=64, dtype=2, causal=1, reserved=0, window=0,
             scale=0.125)
    q, k = (10 * 256, 256, 64), (12 * 128, 128, 64)
    for n in "q o do dq".split():
        f[n + "_strides"] = q
    for n in "k v dk dv".split():
        f[n + "_strides"] = k
    f.update(over)
    for n in list(f):
        if n.endswith("_strides"):
            f[n] = (ctypes.c_int64 * 3)(*f[n])
    return z.zero_attention_desc(**f)


def refused(z, call, *args):
    with pytest.raises(z.ZeroError) as e:
        call(*args)
    assert e.value.code == 1 and len(str(e.value)) > 20


def test_act_layout(z):
    assert z.zero_act_layout(3, 1) == (128, 384, 12)
    assert z.zero_act_layout(5, 128) == (128, 640, 20)
    assert z.zero_act_layout(7, 129) == (256, 7 * 256, 56)
    assert z.zero_act_layout(0, 64) == (128, 0, 0)
    for rows, cols in ((-1, 8), (1, 0), (1, 1 << 31), (1 << 41, 8)):
        refused(z, z.zero_act_layout, rows, cols)


def test_workspaces(z):
    assert z.zero_rmsnorm_backward_workspace(norm(z)) >= 64 * 4
    assert z.zero_rmsnorm_backward_workspace(norm(z, rows=0)) >= 0
    assert z.zero_attention_backward_workspace(attention(z)) >= 2 * 4 * 10 * 4
    assert z.zero_act_weight_grad_workspace(100, 64, 64) >= 0
    # large enough at every size that the same descriptor may be used with
    assert z.zero_rmsnorm_backward_workspace(norm(z, rows=1 << 30)) < 1 << 30


def test_nothing_to_do(z):
    z.zero_rmsnorm_forward(norm(z, rows=0), 0, 0, 0, 0, 0, 0, 0, 0, 0)
    z.zero_act_pack(0, 64, 0, 64, 2, 0, 0, 0)
    z.zero_act_unpack(0, 0, 0, 64, 0, 64, 2, 0)
    z.zero_attention_forward(attention(z, batch=0), 0, 0, 0, 0, 0, 0, 0)
    z.zero_attention_forward(attention(z, q_len=0), 0, 0, 0, 0, 0, 0, 0)
    z.zero_attention_backward(attention(z, q_len=0, k_len=0), 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0)


@pytest.mark.parametrize("over", [dict(rows=-1), dict(cols=0), dict(cols=65537), dict(x_stride=63), dict(residual_stride=0),
                                  dict(dy_stride=-64), dict(dtype=3), dict(dtype=-1), dict(weight_dtype=9), dict(eps=-1.0),
                                  dict(eps=float("nan")), dict(eps=float("inf")), dict(rows=1 << 41),
                                  dict(x_stride=1 << 41)])
def test_norm_descriptors(z, over):
    d = norm(z, **over)
    refused(z, z.zero_rmsnorm_forward, d, P, 0, P, 0, P, 0, 0, P, 0)
    refused(z, z.zero_rmsnorm_backward_workspace, d)
    refused(z, z.zero_rmsnorm_backward, d, P, P, P, P, 0, 2 * P, P, 2, P, 1 << 30, 0)


def test_norm_pointers(z):
    good = dict(x=P, res=0, w=P, s=0, y=P, q=0, scales=0, rstd=P)
    for over in (dict(x=0), dict(x=P + 2), dict(w=0), dict(w=P + 8), dict(y=P + 4), dict(rstd=P + 4), dict(s=P),
                 dict(res=P), dict(res=P + 2, s=P), dict(res=P, s=P + 2), dict(q=P), dict(scales=P),
                 dict(q=P + 1, scales=P), dict(q=P, scales=P + 4), dict(y=0)):
        a = {**good, **over}
        refused(z, z.zero_rmsnorm_forward, norm(z), a["x"], a["res"], a["w"], a["s"], a["y"], a["q"], a["scales"],
                a["rstd"], 0)
    # in place only over rows without gaps
    refused(z, z.zero_rmsnorm_forward, norm(z, x_stride=72), P, 2 * P, P, P, 3 * P, 0, 0, P, 0)
    refused(z, z.zero_rmsnorm_forward, norm(z, residual_stride=72), P, 2 * P, P, 2 * P, 3 * P, 0, 0, P, 0)
    good = dict(dy=P, x=2 * P, w=P, rstd=P, dsum=0, dx=3 * P, dw=P, dt=2, ws=P, nb=1 << 30)
    for over in (dict(dy=0), dict(dy=P + 2), dict(x=0), dict(w=0), dict(rstd=0), dict(dsum=P + 2), dict(dx=0), dict(dw=0),
                 dict(dt=5), dict(ws=0), dict(nb=0), dict(dx=2 * P), dict(ws=P + 4)):
        a = {**good, **over}
        refused(z, z.zero_rmsnorm_backward, norm(z), a["dy"], a["x"], a["w"], a["rstd"], a["dsum"], a["dx"], a["dw"],
                a["dt"], a["ws"], a["nb"], 0)
    refused(z, z.zero_rmsnorm_backward, norm(z, dy_stride=72), P, 2 * P, P, P, 0, P, P, 2, P, 1 << 30, 0)
    refused(z, z.zero_rmsnorm_backward_workspace, None)


def test_act_arguments(z):
    for a in ((0, 64, 4, 64, 2, P, P), (P + 2, 64, 4, 64, 2, P, P), (P, 63, 4, 64, 2, P, P), (P, 64, -1, 64, 2, P, P),
              (P, 64, 4, 0, 2, P, P), (P, 64, 4, 64, 3, P, P), (P, 64, 4, 64, 2, 0, P), (P, 64, 4, 64, 2, P, P + 1)):
        refused(z, z.zero_act_pack, *a, 0)
    for a in ((0, P, 4, 64, P, 64, 2), (P, 0, 4, 64, P, 64, 2), (P, P, -4, 64, P, 64, 2), (P, P, 4, 64, 0, 64, 2),
              (P, P, 4, 64, P + 2, 64, 2), (P, P, 4, 64, P, 60, 2), (P, P, 4, 64, P, 64, 7)):
        refused(z, z.zero_act_unpack, *a, 0)
    good = dict(dy=P, st=64, dt=2, q=P, sc=P, t=10, no=64, ni=64, dw=P, dwt=0, acc=0, ws=P, nb=1 << 40)
    for over in (dict(dy=0), dict(dy=P + 2), dict(st=56), dict(st=68), dict(dt=0), dict(q=0), dict(sc=0), dict(t=-1),
                 dict(no=0), dict(ni=0), dict(ni=1 << 31), dict(dw=0), dict(dw=P + 4), dict(dwt=1), dict(dwt=5),
                 dict(dwt=2, acc=1)):
        a = {**good, **over}
        refused(z, z.zero_act_weight_grad, a["dy"], a["st"], a["dt"], a["q"], a["sc"], a["t"], a["no"], a["ni"], a["dw"],
                a["dwt"], a["acc"], a["ws"], a["nb"], 0)


@pytest.mark.parametrize("over", [
    dict(batch=-1), dict(q_len=-1), dict(k_len=1 << 29), dict(q_heads=0), dict(kv_heads=3), dict(head_dim=4),
    dict(head_dim=60), dict(head_dim=136), dict(dtype=0), dict(dtype=4), dict(window=-1), dict(scale=0.0),
    dict(scale=float("nan")), dict(q_strides=(2560, 256, 60)), dict(q_strides=(2560, 256, 32)),
    dict(k_strides=(1 << 41, 128, 64)), dict(v_strides=(-1536, 128, 64)), dict(o_strides=(2560, 252, 64)),
    dict(dk_strides=(1536, 128, 56))])
def test_attention_descriptors(z, over):
    d = attention(z, **over)
    if "dk_strides" not in over:
        refused(z, z.zero_attention_forward, d, P, P, P, 0, P, P, 0)
    refused(z, z.zero_attention_backward_workspace, d)
    refused(z, z.zero_attention_backward, d, P, P, P, P, P, P, 0, P, P, P, P, 1 << 30, 0)


@pytest.mark.parametrize("name", ["o", "dq", "dk", "dv"])
def test_attention_outputs_may_not_overlap(z, name):
    strides = (64, 256, 64) if name in ("o", "dq") else (64, 128, 64)
    d = attention(z, **{name + "_strides": strides})
    if name == "o":
        refused(z, z.zero_attention_forward, d, P, P, P, 0, P, P, 0)
    else:
        refused(z, z.zero_attention_backward, d, P, P, P, P, P, P, 0, P, P, P, P, 1 << 30, 0)


def test_attention_pointers(z):
    good = dict(q=P, k=P, v=P, n=0, o=P, lse=P)
    for over in (dict(q=0), dict(k=0), dict(v=P + 2), dict(n=P + 2), dict(o=0), dict(o=P + 8), dict(lse=0)):
        a = {**good, **over}
        refused(z, z.zero_attention_forward, attention(z), a["q"], a["k"], a["v"], a["n"], a["o"], a["lse"], 0)
    good = dict(do=P, q=P, k=P, v=P, o=P, lse=P, n=0, dq=P, dk=P, dv=P, ws=P, nb=1 << 30)
    for over in (dict(do=0), dict(q=P + 2), dict(k=0), dict(v=0), dict(o=0), dict(lse=0), dict(n=P + 1), dict(dq=0),
                 dict(dk=0), dict(dv=P + 2), dict(ws=0), dict(nb=16)):
        a = {**good, **over}
        refused(z, z.zero_attention_backward, attention(z), a["do"], a["q"], a["k"], a["v"], a["o"], a["lse"], a["n"],
                a["dq"], a["dk"], a["dv"], a["ws"], a["nb"], 0)
