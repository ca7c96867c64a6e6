"""The expert layer's and the scaled products' host side, without a GPU: sizes,
calls with nothing to do, and every refusal, before any device call. The pointers
are made-up addresses that are never read."""
import pytest

from test_block_host import P, refused, z  # noqa: F401
from test_block_host_edges import accepted

F = 1 << 32  # between buffers


def experts_desc(z, **over):  # noqa: F811
    f = dict(rows=10, n_out=64, n_in=32, x_stride=32, y_stride=64, w_stride=64 * 32, w_row_stride=32, experts=4, dtype=2)
    f.update(over)
    return z.zero_experts_desc(**f)


def scaled_desc(z, **over):  # noqa: F811
    f = dict(rows=10, n=64, k=200, out_stride=64, experts=0, out_dtype=2, accumulate=0, reserved=0)
    f.update(over)
    return z.zero_scaled_desc(**f)


def call(z, name, **over):  # noqa: F811
    """An entry point's call with sound arguments, but for those given."""
    a = dict(
        zero_route=dict(logits=F, stride=16, tokens=10, experts=16, k=2, dtype=0, normalize=1, weights=2 * F, chosen=3 * F,
                        offsets=4 * F, source=5 * F, place=6 * F, ws=7 * F, nb=1 << 20, stream=0),
        zero_route_backward=dict(dweights=F, weights=2 * F, chosen=3 * F, logits=4 * F, stride=16, tokens=10, experts=16,
                                 k=2, dtype=0, normalize=0, dlogits=5 * F, stream=0),
        zero_experts_gather=dict(x=F, stride=64, tokens=10, k=2, hidden=64, dtype=2, place=2 * F, source=3 * F, rows=4 * F,
                                 stream=0),
        zero_experts_combine=dict(y=F, stride=64, tokens=10, k=2, hidden=64, dtype=2, place=2 * F, weights=3 * F,
                                  out=4 * F, stream=0),
        zero_experts_combine_backward=dict(dout=F, dout_stride=64, y=2 * F, y_stride=64, tokens=10, k=2, hidden=64,
                                           dtype=2, place=3 * F, source=4 * F, weights=5 * F, dy=6 * F, dweights=7 * F,
                                           stream=0),
        zero_experts_forward=dict(desc=experts_desc(z), x=F, w=2 * F, offsets=3 * F, y=4 * F, stream=0),
        zero_experts_input_grad=dict(desc=experts_desc(z), dy=F, w=2 * F, offsets=3 * F, dx=4 * F, stream=0),
        zero_experts_weight_grad=dict(desc=experts_desc(z), dy=F, x=2 * F, offsets=3 * F, dw=4 * F, dwt=2, acc=0, stream=0),
        zero_scaled_pack=dict(x=F, bs=6400, stride=200, batch=2, rows=32, cols=200, dtype=2, q=2 * F, s=3 * F, qt=4 * F,
                              st=5 * F, stream=0),
        zero_scaled_unpack=dict(q=F, s=2 * F, rows=10, cols=200, out=3 * F, stride=200, dtype=2, stream=0),
        zero_scaled_matmul=dict(desc=scaled_desc(z), a=F, sa=2 * F, b=3 * F, sb=4 * F, offsets=0, out=5 * F, stream=0),
    )[name]
    assert set(over) <= set(a), over
    return (getattr(z, name), *{**a, **over}.values())


NAMES = ["zero_route", "zero_route_backward", "zero_experts_gather", "zero_experts_combine",
         "zero_experts_combine_backward", "zero_experts_forward", "zero_experts_input_grad", "zero_experts_weight_grad",
         "zero_scaled_pack", "zero_scaled_unpack", "zero_scaled_matmul"]


@pytest.mark.parametrize("name", NAMES)
def test_sound_calls_pass_the_checks(z, name):  # noqa: F811
    accepted(z, *call(z, name))


def test_sizes(z):  # noqa: F811
    assert z.zero_scaled_layout(3, 1) == (128, 4)
    assert z.zero_scaled_layout(0, 512) == (512, 4)
    assert z.zero_scaled_layout(5, 513) == (640, 8)
    for rows, cols in ((-1, 8), (1, 0), (1, 1 << 31), (1 << 32, 8)):
        refused(z, z.zero_scaled_layout, rows, cols)
    assert z.zero_route_workspace(0, 16, 2) == 0
    assert 0 < z.zero_route_workspace(1, 16, 2) <= z.zero_route_workspace(1 << 20, 16, 2) < 1 << 20
    for t, e, k in ((-1, 16, 2), (1, 0, 1), (1, 1025, 2), (1, 16, 0), (1, 16, 17), (1, 64, 33), (1 << 30, 16, 2)):
        refused(z, z.zero_route_workspace, t, e, k)


def test_nothing_to_do(z):  # noqa: F811
    z.zero_route_backward(0, 0, 0, 0, 16, 0, 16, 2, 0, 0, 0, 0)
    z.zero_experts_gather(0, 64, 0, 2, 64, 2, 0, 0, 0, 0)
    z.zero_experts_combine(0, 64, 0, 2, 64, 2, 0, 0, 0, 0)
    z.zero_experts_combine_backward(0, 64, 0, 64, 0, 2, 64, 2, 0, 0, 0, 0, 0, 0)
    z.zero_experts_forward(experts_desc(z, rows=0), 0, 0, 0, 0, 0)
    z.zero_experts_input_grad(experts_desc(z, rows=0), 0, 0, 0, 0, 0)
    z.zero_scaled_pack(0, 0, 64, 1, 0, 64, 2, 0, 0, 0, 0, 0)
    z.zero_scaled_pack(0, 64, 64, 0, 1, 64, 2, 0, 0, 0, 0, 0)
    z.zero_scaled_unpack(0, 0, 0, 64, 0, 64, 2, 0)
    z.zero_scaled_matmul(scaled_desc(z, rows=0), 0, 0, 0, 0, 0, 0, 0)


@pytest.mark.parametrize("name,over", [
    ("zero_route", o) for o in (dict(logits=0), dict(logits=F + 2), dict(stride=15), dict(tokens=-1), dict(tokens=1 << 31),
                                dict(experts=0), dict(experts=1025), dict(k=0), dict(k=17), dict(dtype=3), dict(weights=0),
                                dict(chosen=3 * F + 4), dict(offsets=0), dict(source=0), dict(place=0), dict(ws=0),
                                dict(nb=15), dict(weights=3 * F), dict(source=F), dict(place=4 * F + 16),
                                dict(ws=F + 16))] + [
    ("zero_route_backward", o) for o in (dict(dweights=0), dict(weights=0), dict(chosen=0), dict(logits=0), dict(stride=8),
                                         dict(tokens=-1), dict(k=33), dict(dtype=-1), dict(dlogits=0),
                                         dict(dlogits=4 * F), dict(dlogits=F - 16))] + [
    ("zero_experts_gather", o) for o in (dict(x=0), dict(x=F + 8), dict(stride=63), dict(tokens=-1), dict(k=0), dict(k=33),
                                         dict(tokens=1 << 30), dict(hidden=0), dict(hidden=1 << 31), dict(dtype=5),
                                         dict(place=0), dict(source=0), dict(rows=0), dict(rows=F), dict(rows=F + 1264),
                                         dict(rows=2 * F - 2544))] + [
    ("zero_experts_combine", o) for o in (dict(y=0), dict(stride=0), dict(k=-1), dict(hidden=-8), dict(dtype=3),
                                          dict(place=0), dict(weights=3 * F + 4), dict(out=0), dict(out=F + 1280),
                                          dict(out=3 * F))] + [
    ("zero_experts_combine_backward", o) for o in (
        dict(dout=0), dict(y=0), dict(dout_stride=60), dict(y_stride=60), dict(place=0), dict(source=0), dict(weights=0),
        dict(dy=0), dict(dweights=0), dict(dy=F), dict(dy=2 * F + 16), dict(dweights=6 * F + 16), dict(dweights=5 * F))] + [
    (n, o) for n in ("zero_experts_forward", "zero_experts_input_grad") for o in (
        dict(w=0), dict(w=2 * F + 2), dict(offsets=0), dict(offsets=3 * F + 4), dict(desc=None))] + [
    ("zero_experts_forward", o) for o in (dict(x=0), dict(x=F + 8), dict(y=0), dict(y=4 * F + 1), dict(y=F), dict(y=2 * F + 512), dict(y=3 * F))] + [
    ("zero_experts_input_grad", o) for o in (dict(dy=0), dict(dx=0), dict(dx=F + 16), dict(dx=2 * F))] + [
    ("zero_experts_weight_grad", o) for o in (dict(dy=0), dict(x=0), dict(offsets=0), dict(dw=0), dict(dwt=1), dict(dwt=5),
                                              dict(acc=1), dict(dw=F), dict(dw=2 * F), dict(desc=None))] + [
    ("zero_scaled_pack", o) for o in (
        dict(x=0), dict(x=F + 8), dict(stride=199), dict(bs=6399), dict(batch=-1), dict(batch=65536), dict(rows=-1),
        dict(cols=0), dict(cols=65535 * 128 + 1), dict(dtype=4), dict(q=0), dict(s=0), dict(qt=0), dict(st=0),
        dict(q=0, s=0, qt=0, st=0), dict(q=2 * F + 1), dict(st=5 * F + 4), dict(q=F), dict(qt=2 * F + 16384 - 16),
        dict(s=5 * F), dict(rows=1 << 30, batch=2))] + [
    ("zero_scaled_unpack", o) for o in (dict(q=0), dict(s=0), dict(out=0), dict(rows=-1), dict(cols=0), dict(stride=100),
                                        dict(dtype=3), dict(out=F), dict(out=2 * F + 16))] + [
    ("zero_scaled_matmul", o) for o in (dict(a=0), dict(sa=0), dict(b=0), dict(sb=0), dict(out=0), dict(offsets=6 * F),
                                        dict(out=F), dict(out=4 * F + 16), dict(b=3 * F + 8), dict(desc=None))])
def test_refusals(z, name, over):  # noqa: F811
    refused(z, *call(z, name, **over))


@pytest.mark.parametrize("over", [
    dict(rows=-1), dict(rows=1 << 31), dict(n_out=0), dict(n_in=0), dict(n_in=(1 << 24) + 8), dict(experts=0),
    dict(experts=1025), dict(dtype=0), dict(dtype=3), dict(x_stride=24), dict(y_stride=56), dict(w_row_stride=24),
    dict(w_stride=64 * 32 - 8), dict(x_stride=1 << 41), dict(w_stride=-8)])
def test_experts_descriptors(z, over):  # noqa: F811
    d = experts_desc(z, **over)
    for name in ("zero_experts_forward", "zero_experts_input_grad", "zero_experts_weight_grad"):
        refused(z, *call(z, name, desc=d))


def test_experts_strides(z):  # noqa: F811
    """Inputs' rows start on 16 bytes; outputs' need not. A lone expert's stride is not looked at."""
    odd = dict(forward=("x_stride", "w_stride", "w_row_stride"), input_grad=("y_stride", "w_stride", "w_row_stride"),
               weight_grad=("x_stride", "y_stride"))
    for name, inputs in odd.items():
        for field, step in (("x_stride", 33), ("y_stride", 67), ("w_stride", 64 * 40 + 2), ("w_row_stride", 33)):
            d = experts_desc(z, **{"w_stride": 64 * 40, field: step})
            (refused if field in inputs else accepted)(z, *call(z, "zero_experts_" + name, desc=d))
        accepted(z, *call(z, "zero_experts_" + name, desc=experts_desc(z, experts=1, w_stride=0)))


@pytest.mark.parametrize("over", [
    dict(rows=-1), dict(rows=1 << 31), dict(n=0), dict(k=0), dict(n=1 << 25), dict(k=1 << 25), dict(out_stride=63),
    dict(experts=-1), dict(experts=1025), dict(out_dtype=3), dict(accumulate=1)])
def test_scaled_descriptors(z, over):  # noqa: F811
    refused(z, *call(z, "zero_scaled_matmul", desc=scaled_desc(z, **over)))


def test_scaled_matmul_experts(z):  # noqa: F811
    d = scaled_desc(z, experts=3)
    refused(z, *call(z, "zero_scaled_matmul", desc=d))
    accepted(z, *call(z, "zero_scaled_matmul", desc=d, offsets=6 * F))
    refused(z, *call(z, "zero_scaled_matmul", desc=d, offsets=6 * F, out=3 * F + 2 * 64 * 256))
    accepted(z, *call(z, "zero_scaled_matmul", desc=scaled_desc(z, accumulate=1, out_dtype=0)))


def test_far_strides_do_not_wrap(z):  # noqa: F811
    """A span beyond 64 bits of bytes still counts as one that reaches everything behind it."""
    far = 1 << 38
    refused(z, *call(z, "zero_experts_gather", stride=far, tokens=1 << 29, rows=9 * F))
    refused(z, *call(z, "zero_experts_forward", desc=experts_desc(z, rows=1 << 30, x_stride=far), y=9 * F))
