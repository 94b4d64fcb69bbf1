"""Host-side refusals of the layer products, the top logits and the
distillation loss: found before anything is enqueued, so made-up device
addresses and a machine without a GPU do."""
import ctypes

import pytest
import torch

from gradient_compression_dnn_amd import binding as B
from gradient_compression_dnn_amd import workloads as W

P = ctypes.c_void_p
NAN, INF = float("nan"), float("inf")


def _plan():
    # a segment of 7 elements, a matrix of 10 x 12, its bias, 5 more elements
    return B.Plan(W.make_table([7, 120, 10, 5], [1] * 4, [1] * 4, [0, 0, 3, 0]))


def _at(i):
    return P((i + 1) << 20)


def _layer(seg=1, rows=10, bias=2, type=B.GC_BF16, reserved=0):
    l = B.gc_linear(seg, rows, bias, type)
    l.reserved[1] = reserved
    return l


LAYER = [
    (dict(seg=-1), B.GC_EINVAL), (dict(seg=4), B.GC_EINVAL), (dict(rows=0), B.GC_EINVAL), (dict(rows=7), B.GC_EINVAL),
    (dict(bias=-2), B.GC_EINVAL), (dict(bias=4), B.GC_EINVAL), (dict(bias=1), B.GC_EINVAL), (dict(bias=3), B.GC_EINVAL),
    (dict(type=3), B.GC_EINVAL), (dict(type=-1), B.GC_EINVAL), (dict(reserved=1), B.GC_EINVAL),
]
ANY = [(dict(n=1 << 28), B.GC_ERANGE), (dict(ws=None), B.GC_EINVAL), (dict(short=1), B.GC_ECAPACITY), (dict(n=0), B.GC_OK)]


def _need(p, layer, n):
    return B.load().gc_linear_workspace_bytes(p.handle, ctypes.byref(layer), n) if n < 1 << 28 else 1 << 40


def _forward(p, layer, n=50, w=_at(0), x=_at(1), xs=12, act=0, r=_at(2), rs=10, z=_at(3), zs=10, y=_at(4), ys=10, ws=_at(5), short=0):
    need = _need(p, layer, n)
    return B.load().gc_linear_forward(p.handle, ctypes.byref(layer), w, x, xs, n, act, r, rs, z, zs, y, ys, ws, max(need - short, 0), None)


FORWARD = [
    (dict(w=None), B.GC_EINVAL), (dict(x=None), B.GC_EINVAL), (dict(y=None), B.GC_EINVAL),
    (dict(act=5), B.GC_EINVAL), (dict(act=-1), B.GC_EINVAL), (dict(xs=11), B.GC_EINVAL), (dict(rs=9), B.GC_EINVAL),
    (dict(zs=9), B.GC_EINVAL), (dict(ys=9), B.GC_EINVAL), (dict(xs=1 << 45), B.GC_ERANGE), (dict(ys=1 << 45), B.GC_ERANGE),
    (dict(x=P(3)), B.GC_EINVAL), (dict(y=P(1)), B.GC_EINVAL), (dict(r=P(1)), B.GC_EINVAL), (dict(z=P(1)), B.GC_EINVAL), (dict(w=P(1)), B.GC_EINVAL),
    (dict(y=_at(1)), B.GC_EINVAL), (dict(y=_at(0)), B.GC_EINVAL), (dict(y=_at(3)), B.GC_EINVAL), (dict(z=_at(1)), B.GC_EINVAL),
    (dict(z=_at(2)), B.GC_EINVAL), (dict(y=_at(2), ys=12), B.GC_EINVAL), (dict(n=0, w=None, x=None, y=None, ws=None), B.GC_OK),
]


@pytest.mark.parametrize("kw,code", LAYER)
def test_layer_refusals(kw, code):
    p, layer = _plan(), _layer(**kw)
    assert _forward(p, layer) == code and B.gc_last_error() != ""
    assert _input(p, layer) == code and _weight(p, layer) == code
    assert B.load().gc_linear_workspace_bytes(p.handle, ctypes.byref(layer), 50) == 0


@pytest.mark.parametrize("kw,code", FORWARD + ANY)
def test_forward_refusals(kw, code):
    assert _forward(_plan(), _layer(), **kw) == code
    assert (B.gc_last_error() != "") == (code != B.GC_OK)


def _input(p, layer, n=50, w=_at(0), dz=_at(1), ds=10, a=_at(2), als=12, act=2, z=_at(3), zs=12, dx=_at(4), xs=12, dzx=_at(5), gs=12,
           ws=_at(6), short=0):
    need = _need(p, layer, n)
    return B.load().gc_linear_grad_input(p.handle, ctypes.byref(layer), w, dz, ds, n, a, als, act, z, zs, dx, xs, dzx, gs, ws, max(need - short, 0), None)


INPUT = [
    (dict(w=None), B.GC_EINVAL), (dict(dz=None), B.GC_EINVAL), (dict(dx=None, dzx=None), B.GC_EINVAL), (dict(z=None), B.GC_EINVAL),
    (dict(act=9), B.GC_EINVAL), (dict(ds=9), B.GC_EINVAL), (dict(als=11), B.GC_EINVAL), (dict(zs=11), B.GC_EINVAL),
    (dict(xs=11), B.GC_EINVAL), (dict(gs=11), B.GC_EINVAL), (dict(ds=1 << 45), B.GC_ERANGE), (dict(dz=P(1)), B.GC_EINVAL),
    (dict(dx=_at(5)), B.GC_EINVAL), (dict(dx=_at(1)), B.GC_EINVAL), (dict(dzx=_at(3)), B.GC_EINVAL), (dict(dx=_at(0)), B.GC_EINVAL),
    (dict(a=_at(4), als=13), B.GC_EINVAL), (dict(a=_at(5), als=13), B.GC_EINVAL),
]


@pytest.mark.parametrize("kw,code", INPUT + ANY)
def test_input_refusals(kw, code):
    assert _input(_plan(), _layer(), **kw) == code


def _weight(p, layer, n=50, dz=_at(0), ds=10, x=_at(1), xs=12, g=_at(2), add=1, ws=_at(3), short=0):
    need = _need(p, layer, n)
    return B.load().gc_linear_grad_weight(p.handle, ctypes.byref(layer), dz, ds, x, xs, n, g, add, ws, max(need - short, 0), None)


WEIGHT = [
    (dict(dz=None), B.GC_EINVAL), (dict(x=None), B.GC_EINVAL), (dict(g=None), B.GC_EINVAL), (dict(g=P(2)), B.GC_EINVAL),
    (dict(ds=9), B.GC_EINVAL), (dict(xs=11), B.GC_EINVAL), (dict(xs=1 << 45), B.GC_ERANGE), (dict(x=P(1)), B.GC_EINVAL),
    (dict(g=_at(0)), B.GC_EINVAL), (dict(g=_at(1)), B.GC_EINVAL),
]


@pytest.mark.parametrize("kw,code", WEIGHT + ANY)
def test_weight_refusals(kw, code):
    assert _weight(_plan(), _layer(), **kw) == code


def test_null_plan_layer_and_sizes():
    lib, p, layer = B.load(), _plan(), _layer()
    ref = ctypes.byref(layer)
    for plan, l in ((None, ref), (p.handle, None)):
        assert lib.gc_linear_workspace_bytes(plan, l, 5) == 0
        assert lib.gc_linear_forward(plan, l, _at(0), _at(1), 12, 5, 0, None, 0, None, 0, _at(4), 10, _at(5), 1 << 30, None) == B.GC_EINVAL
        assert lib.gc_linear_grad_input(plan, l, _at(0), _at(1), 10, 5, None, 0, 0, None, 0, _at(4), 12, None, 0, _at(5), 1 << 30, None) == B.GC_EINVAL
        assert lib.gc_linear_grad_weight(plan, l, _at(0), 10, _at(1), 12, 5, _at(2), 0, _at(5), 1 << 30, None) == B.GC_EINVAL
    assert lib.gc_linear_workspace_bytes(p.handle, ref, 1 << 28) == 0
    assert lib.gc_linear_workspace_bytes(p.handle, ref, 50) > 0
    # 2^20 columns: 2^15 tokens reach 2^35 elements, one more passes it
    wide = B.Plan(W.make_table([1 << 22], [1], [1]))
    l4 = _layer(0, 4, -1)
    for n, ok in ((1 << 15, True), ((1 << 15) + 1, False)):
        assert (lib.gc_linear_workspace_bytes(wide.handle, ctypes.byref(l4), n) > 0) == ok


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), B.GC_EINVAL), (dict(act=7), B.GC_EINVAL), (dict(n=1 << 28), B.GC_ERANGE), (dict(cols=1 << 34), B.GC_ERANGE),
    (dict(dy=None), B.GC_EINVAL), (dict(z=None), B.GC_EINVAL), (dict(dz=None), B.GC_EINVAL), (dict(ys=8), B.GC_EINVAL),
    (dict(zs=8), B.GC_EINVAL), (dict(ds=8), B.GC_EINVAL), (dict(ds=1 << 47), B.GC_ERANGE), (dict(dz=P(2)), B.GC_EINVAL),
    (dict(dz=_at(0), ds=10), B.GC_EINVAL), (dict(dz=_at(1), ds=10), B.GC_EINVAL), (dict(n=0, dy=None), B.GC_OK), (dict(cols=0, z=None), B.GC_OK),
])
def test_act_grad_refusals(kw, code):
    a = dict(dy=_at(0), ys=9, z=_at(1), zs=9, act=2, type=0, n=6, cols=9, dz=_at(2), ds=9)
    a.update(kw)
    assert B.load().gc_act_grad(a["dy"], a["ys"], a["z"], a["zs"], a["act"], a["type"], a["n"], a["cols"], a["dz"], a["ds"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), B.GC_EINVAL), (dict(k=0), B.GC_EINVAL), (dict(k=1025), B.GC_ENOTSUP), (dict(vocab=0), B.GC_EINVAL),
    (dict(vocab=(1 << 20) + 1, stride=1 << 21), B.GC_ENOTSUP), (dict(stride=99), B.GC_EINVAL), (dict(n=1 << 22), B.GC_ERANGE),
    (dict(stride=1 << 47), B.GC_ERANGE), (dict(t=0.0), B.GC_EINVAL), (dict(t=-1.0), B.GC_EINVAL), (dict(t=NAN), B.GC_EINVAL),
    (dict(t=INF), B.GC_EINVAL), (dict(t=1e-40), B.GC_EINVAL), (dict(t=3.2e-39), B.GC_EINVAL), (dict(z=None), B.GC_EINVAL), (dict(idx=None), B.GC_EINVAL),
    (dict(val=None), B.GC_EINVAL), (dict(z=P(1)), B.GC_EINVAL), (dict(idx=P(2)), B.GC_EINVAL), (dict(val=P(2)), B.GC_EINVAL),
    (dict(lse=P(2)), B.GC_EINVAL), (dict(n=0, z=None), B.GC_OK),
])
def test_top_logits_refusals(kw, code):
    a = dict(z=_at(0), type=1, stride=100, n=6, vocab=100, k=5, t=1.0, idx=_at(1), val=_at(2), lse=None)
    a.update(kw)
    assert B.load().gc_top_logits(a["z"], a["type"], a["stride"], a["n"], a["vocab"], a["k"], a["t"], a["idx"], a["val"], a["lse"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), B.GC_EINVAL), (dict(it=2), B.GC_EINVAL), (dict(tt=3), B.GC_EINVAL), (dict(mode=2), B.GC_EINVAL), (dict(mode=-1), B.GC_EINVAL),
    (dict(reserved=1), B.GC_EINVAL), (dict(T=0.0), B.GC_EINVAL), (dict(T=INF), B.GC_EINVAL), (dict(T=1e30, kd=1.0), B.GC_EINVAL),
    (dict(kd=NAN), B.GC_EINVAL), (dict(ce=INF), B.GC_EINVAL), (dict(scale=NAN), B.GC_EINVAL), (dict(vocab=0), B.GC_EINVAL),
    (dict(vocab=(1 << 20) + 1, stride=1 << 21), B.GC_ENOTSUP), (dict(k=1025), B.GC_ENOTSUP), (dict(n=1 << 22), B.GC_ERANGE),
    (dict(z=None), B.GC_EINVAL), (dict(idx=None), B.GC_EINVAL), (dict(t=None), B.GC_EINVAL), (dict(loss=None), B.GC_EINVAL),
    (dict(lse=None), B.GC_EINVAL), (dict(stride=99), B.GC_EINVAL), (dict(ds=99), B.GC_EINVAL), (dict(xs=4), B.GC_EINVAL), (dict(ts=4), B.GC_EINVAL),
    (dict(stride=1 << 47), B.GC_ERANGE), (dict(xs=1 << 47), B.GC_ERANGE), (dict(z=P(1)), B.GC_EINVAL), (dict(idx=P(4), it=1), B.GC_EINVAL), (dict(t=P(2)), B.GC_EINVAL),
    (dict(labels=P(2)), B.GC_EINVAL), (dict(weights=P(2)), B.GC_EINVAL), (dict(lse=P(2)), B.GC_EINVAL), (dict(loss=P(2)), B.GC_EINVAL), (dict(d=P(1)), B.GC_EINVAL),
    (dict(d=_at(0), ds=101), B.GC_EINVAL), (dict(n=0, z=None, idx=None, loss=None), B.GC_OK),
])
def test_distill_refusals(kw, code):
    a = dict(z=_at(0), type=1, stride=100, n=6, vocab=100, idx=_at(1), it=0, xs=5, t=_at(2), tt=0, ts=5, k=5, lse=_at(3), labels=None,
             weights=None, loss=_at(4), d=_at(5), ds=100, T=2.0, kd=1.0, ce=0.5, scale=1.0, mode=1, reserved=0)
    a.update(kw)
    opt = B.gc_distill_options(a["T"], a["kd"], a["ce"], a["scale"], a["mode"])
    opt.reserved[2] = a["reserved"]
    assert B.load().gc_distill_loss(a["z"], a["type"], a["stride"], a["n"], a["vocab"], a["idx"], a["it"], a["xs"], a["t"], a["tt"], a["ts"],
                                    a["k"], a["lse"], a["labels"], a["weights"], ctypes.byref(opt), a["loss"], a["d"], a["ds"], None) == code


def test_binding_refusals():
    """The binding checks what the library cannot see: shapes, types, devices."""
    p, layer = _plan(), B.linear_layer(1, 10, torch.bfloat16, 2)
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)
    w, ws = t(p.n_total), t(64, dtype=torch.uint8)
    good = dict(w=w, x=t(4, 12), y=t(4, 10), ws=ws)
    for bad in (dict(x=t(4, 11)), dict(y=t(4, 12)), dict(y=t(5, 10)), dict(x=t(4, 12, dtype=torch.float16)), dict(r=t(4, 9)), dict(z=t(3, 10)),
                dict(x=t(4, 24)[:, ::2]), dict(x=None), dict(y=t(1, 10).expand(4, 10)), {}):  # the last: CPU tensors
        with pytest.raises(ValueError):
            B.gc_linear_forward(p, layer, **{**good, **bad})
    with pytest.raises(ValueError):
        B.gc_linear_grad_input(p, layer, w, t(4, 10), t(4, 10), ws)
    with pytest.raises(ValueError):
        B.gc_linear_grad_weight(p, layer, t(4, 10), t(5, 12), t(p.n_total, dtype=torch.float32), False, ws)
    with pytest.raises(ValueError):
        B.gc_linear_forward(p, B.linear_layer(1, 7, torch.bfloat16), w, t(4, 12), t(4, 7), ws)
    with pytest.raises(ValueError):
        B.linear_layer(1, 10, torch.float64)
    with pytest.raises(ValueError):
        B.gc_act_grad(t(4, 6), t(4, 5), B.GC_ACT_GELU, t(4, 6))
    z, i32 = t(3, 50), lambda *s: torch.zeros(*s, dtype=torch.int32)
    f32 = lambda *s: torch.zeros(*s)
    for idx, val in ((i32(3, 4), f32(3, 5)), (i32(2, 4), f32(2, 4)), (i32(3, 0), f32(3, 0)), (i32(3, 4).long(), f32(3, 4)), (i32(3, 4), f32(3, 4))):
        with pytest.raises(ValueError):
            B.gc_top_logits(z, idx, val)
    opt = B.distill_options()
    for idx, val, loss, kw in ((i32(3, 4), f32(3, 5), f32(3), {}), (f32(3, 4), f32(3, 4), f32(3), {}), (i32(3, 4), f32(3, 4), f32(2), {}),
                               (i32(3, 4), f32(3, 4), f32(3), dict(labels=torch.zeros(3, dtype=torch.int64))),
                               (i32(3, 4), f32(3, 4), f32(3), dict(dlogits=f32(3, 50))), (i32(3, 4), f32(3, 4), f32(3), {})):
        with pytest.raises(ValueError):
            B.gc_distill_loss(z, idx, val, opt, loss, **kw)
