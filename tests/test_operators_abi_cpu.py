"""Host-side refusals of the embedding and matrix-update calls: every bad
argument is found before anything is enqueued, so made-up device addresses
and a machine without a GPU do."""
import ctypes

import numpy as np
import pytest
import torch

from gradient_compression_dnn_amd import binding as B
from gradient_compression_dnn_amd import workloads as W

FAKE = ctypes.c_void_p(1 << 20)


def _plan():
    # a segment of 7 elements, an embedding of 10 x 12, a gap, a matrix of 6 x 4
    return B.Plan(W.make_table([7, 120, 24], [1, 1, 1], [1, 1, 1], [0, 0, 5]))


def _lookup(plan, seg=1, rows=10, w=FAKE, tokens=FAKE, tt=0, n=5, scale=1.0, y=FAKE, yt=0, stride=12):
    return B.load().gc_embed_lookup(plan.handle if plan else None, seg, rows, w, tokens, tt, n, scale, y, yt, stride,
                                    None)


@pytest.mark.parametrize("kw,code", [
    (dict(seg=-1), B.GC_EINVAL), (dict(seg=3), B.GC_EINVAL), (dict(rows=0), B.GC_EINVAL), (dict(rows=7), B.GC_EINVAL),
    (dict(w=None), B.GC_EINVAL), (dict(tokens=None), B.GC_EINVAL), (dict(y=None), B.GC_EINVAL),
    (dict(tt=2), B.GC_EINVAL), (dict(tt=-1), B.GC_EINVAL), (dict(yt=3), B.GC_EINVAL), (dict(stride=11), B.GC_EINVAL),
    (dict(scale=float("nan")), B.GC_EINVAL), (dict(scale=float("inf")), B.GC_EINVAL),
    (dict(n=1 << 28), B.GC_ERANGE), (dict(n=(1 << 28) - 1, stride=1 << 30), B.GC_ERANGE),
    (dict(tokens=ctypes.c_void_p(2)), B.GC_EINVAL), (dict(tokens=ctypes.c_void_p(4), tt=1), B.GC_EINVAL),
    (dict(y=ctypes.c_void_p(2)), B.GC_EINVAL), (dict(y=ctypes.c_void_p(1), yt=1), B.GC_EINVAL),
    (dict(n=0), B.GC_OK), (dict(n=0, w=None, tokens=None, y=None), B.GC_OK),
])
def test_lookup_refusals(kw, code):
    assert _lookup(_plan(), **kw) == code
    assert (B.gc_last_error() != "") == (code != B.GC_OK)


def test_embed_null_plan_and_sizes():
    lib = B.load()
    assert _lookup(None) == B.GC_EINVAL
    assert lib.gc_embed_grad(None, 0, 1, None, 0, 1, None, 0, 1, 1.0, None, 0, None, 0, None) == B.GC_EINVAL
    assert lib.gc_embed_message(None, 0, 1, None, 0, 1, None, 0, 1, 1.0, None, None, 0, None) == B.GC_EINVAL
    assert lib.gc_embed_workspace_bytes(None, 0, 1, 1) == 0 and lib.gc_embed_message_cap(None, 0, 1, 1) == 0
    p = _plan()
    assert B.gc_embed_workspace_bytes(p, 1, 7, 10) == 0  # 7 does not divide 120
    assert B.gc_embed_workspace_bytes(p, 1, 10, 1 << 28) == 0
    assert B.gc_embed_message_cap(p, 1, 10, 3) == 36 and B.gc_embed_message_cap(p, 1, 10, 300) == 120
    small, big = (B.gc_embed_workspace_bytes(p, 1, 10, n) for n in (1, 100_000))
    assert 0 < small < big


@pytest.mark.parametrize("kw,code", [
    (dict(g=None), B.GC_EINVAL), (dict(ws=None), B.GC_EINVAL), (dict(short=1), B.GC_ECAPACITY),
    (dict(dy=None), B.GC_EINVAL), (dict(dt=7), B.GC_EINVAL), (dict(stride=3), B.GC_EINVAL),
    (dict(scale=float("nan")), B.GC_EINVAL), (dict(n=1 << 28), B.GC_ERANGE),
])
def test_grad_refusals(kw, code):
    p = _plan()
    a = dict(g=FAKE, ws=FAKE, short=0, dy=FAKE, dt=0, stride=12, scale=1.0, n=50)
    a.update(kw)
    need = B.gc_embed_workspace_bytes(p, 1, 10, 50) - a["short"]
    lib = B.load()
    for acc in (0, 1):
        assert lib.gc_embed_grad(p.handle, 1, 10, a["dy"], a["dt"], a["stride"], FAKE, 0, a["n"], a["scale"], a["g"],
                                 acc, a["ws"], need, None) == code
    cap = 120
    msg = B.gc_sparse(FAKE.value if a["g"] else None, FAKE.value, FAKE.value, None, cap)
    assert lib.gc_embed_message(p.handle, 1, 10, a["dy"], a["dt"], a["stride"], FAKE, 0, a["n"], a["scale"],
                                ctypes.byref(msg), a["ws"], need, None) == code


def test_batches_of_too_many_elements():
    # 2^20 columns: 2^15 tokens reach 2^35 elements, one more passes it
    p = B.Plan(W.make_table([1 << 22], [1], [1]))
    for n, code in ((1 << 15, B.GC_ECAPACITY), ((1 << 15) + 1, B.GC_ERANGE)):
        assert B.load().gc_embed_grad(p.handle, 0, 4, FAKE, 0, 1 << 20, FAKE, 0, n, 1.0, FAKE, 0, FAKE, 0, None) == code


def test_message_refuses_a_short_message():
    p = _plan()
    need = B.gc_embed_workspace_bytes(p, 1, 10, 3)
    lib = B.load()
    for msg, code in ((B.gc_sparse(FAKE.value, FAKE.value, FAKE.value, None, 35), B.GC_ECAPACITY),
                      (B.gc_sparse(FAKE.value, None, FAKE.value, None, 36), B.GC_EINVAL),
                      (B.gc_sparse(FAKE.value, FAKE.value, None, None, 36), B.GC_EINVAL)):
        assert lib.gc_embed_message(p.handle, 1, 10, FAKE, 0, 12, FAKE, 0, 3, 1.0, ctypes.byref(msg), FAKE, need,
                                    None) == code
    assert lib.gc_embed_message(p.handle, 1, 10, FAKE, 0, 12, FAKE, 0, 3, 1.0, None, FAKE, need, None) == B.GC_EINVAL


def test_binding_refuses_cpu_and_misshapen_tensors():
    p = _plan()
    w = torch.zeros(p.n_total)
    t = torch.zeros(5, dtype=torch.int64)
    with pytest.raises(ValueError):
        B.gc_embed_lookup(p, 1, 10, w, t, 1.0, torch.zeros(5, 12))
    with pytest.raises(ValueError):
        B.gc_embed_grad(p, 1, 10, torch.zeros(5, 12), t, 1.0, w, False, torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(ValueError):
        B.gc_embed_lookup(p, 5, 10, w, t, 1.0, torch.zeros(5, 12))
    with pytest.raises(ValueError):
        B.MatrixPlan(p, [0, 10])  # one count per segment
    with pytest.raises(ValueError):
        B.MatrixPlan(p, [0, -1, 6])
    with pytest.raises(ValueError):
        B.orth_options(steps=3, coef=((1, 2, 3), (1, 2, 3)))


# ------------------------------------------------------------ matrix plans
@pytest.mark.parametrize("lengths,rows,code", [
    ([7, 120, 24], [0, 10, 6], B.GC_OK), ([7, 120, 24], [7, 1, 24], B.GC_OK), ([7, 120, 24], [0, 0, 0], B.GC_EINVAL),
    ([7, 120, 24], [0, 11, 6], B.GC_EINVAL), ([(1 << 20) + 1], [1], B.GC_ENOTSUP), ([(1 << 20) + 1], [(1 << 20) + 1], B.GC_ENOTSUP),
    ([1 << 20], [1], B.GC_OK),
])
def test_matrix_plan_validation(lengths, rows, code):
    p = B.Plan(W.make_table(lengths, [1] * len(lengths)))
    if code == B.GC_OK:
        m = B.MatrixPlan(p, rows)
        assert m.workspace_bytes() > 0
        del p  # the matrix plan keeps nothing of the plan
        assert m.workspace_bytes() > 0
    else:
        with pytest.raises(B.GCError) as e:
            B.MatrixPlan(p, rows)
        assert e.value.status == code


def test_matrix_plan_null_arguments():
    lib = B.load()
    p = _plan()
    h = ctypes.c_void_p()
    assert lib.gc_matrix_plan_create(None, (ctypes.c_uint32 * 3)(), ctypes.byref(h)) == B.GC_EINVAL
    assert lib.gc_matrix_plan_create(p.handle, None, ctypes.byref(h)) == B.GC_EINVAL
    assert lib.gc_matrix_plan_create(p.handle, (ctypes.c_uint32 * 3)(0, 0, 6), None) == B.GC_EINVAL
    assert lib.gc_matrix_plan_upload(None) == B.GC_EINVAL
    assert lib.gc_matrix_plan_workspace_bytes(None) == 0
    lib.gc_matrix_plan_destroy(None)
    assert lib.gc_orthogonalize(None, None, None, None, None, 0, None) == B.GC_EINVAL
    assert lib.gc_muon_step(None, None, None, None, None, None, 0, None) == B.GC_EINVAL


def _set(o, **kw):
    for k, v in kw.items():
        setattr(o, k, v)
    return o


def _coef(o, *abc):
    o.coef[0][:] = abc
    return o


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("opt,code", [
    (lambda: _set(B.orth_options(), steps=0), B.GC_EINVAL), (lambda: _set(B.orth_options(), steps=17), B.GC_EINVAL),
    (lambda: _set(B.orth_options(), steps=-1), B.GC_EINVAL), (lambda: B.orth_options(eps=-1.0), B.GC_EINVAL),
    (lambda: B.orth_options(eps=NAN), B.GC_EINVAL), (lambda: B.orth_options(eps=INF), B.GC_EINVAL),
    (lambda: _coef(B.orth_options(), NAN, 0, 0), B.GC_EINVAL), (lambda: _coef(B.orth_options(), 1, NAN, 0), B.GC_EINVAL),
    (lambda: _coef(B.orth_options(), 1, 0, INF), B.GC_EINVAL), (lambda: _coef(B.orth_options(), 1e13, 0, 0), B.GC_EINVAL),
    (lambda: _coef(B.orth_options(), 0, 0, 0), B.GC_EINVAL),  # X vanishes
    (lambda: B.orth_options(steps=16, coef=(3.0, 0.0, 3.0)), B.GC_EINVAL),  # grows without bound
    # a schedule that takes 0.47 to 1.3, 1.9, 6.5 and 4000
    (lambda: B.orth_options(4, ((4.0, -6.0, 2.9), (3.5, -5.0, 2.2), (2.0, -1.5, 0.5), (1.875, -1.25, 0.375))), B.GC_EINVAL),
    (lambda: (lambda o: (o.reserved.__setitem__(0, 1), o)[1])(B.orth_options()), B.GC_EINVAL),
    (lambda: B.orth_options(), B.GC_ECAPACITY),  # the workspace is what is short then
])
def test_orthogonalize_refusals(opt, code):
    p = _plan()
    m = B.MatrixPlan(p, [0, 10, 6])
    o = opt()
    lib = B.load()
    short = m.workspace_bytes() - 1
    assert lib.gc_orthogonalize(m.handle, FAKE, FAKE, ctypes.byref(o), FAKE, short, None) == code
    mo = B.muon_options(0.9, 0.1)
    mo.orth = o
    far = ctypes.c_void_p(FAKE.value + (1 << 20))
    assert lib.gc_muon_step(m.handle, FAKE, far, ctypes.c_void_p(FAKE.value + (2 << 20)), ctypes.byref(mo), FAKE, short,
                            None) == code


def test_matrix_update_buffers_and_options():
    p = _plan()
    m = B.MatrixPlan(p, [0, 10, 6])
    lib = B.load()
    need = m.workspace_bytes()
    o = B.orth_options()
    a, b, c = (ctypes.c_void_p(FAKE.value + k * 65536) for k in range(3))
    inside = ctypes.c_void_p(a.value + 4 * (p.n_total - 1))
    orth = lambda d, out, ws=FAKE: lib.gc_orthogonalize(m.handle, d, out, ctypes.byref(o), ws, need, None)  # noqa: E731
    assert orth(None, a) == B.GC_EINVAL and orth(a, None) == B.GC_EINVAL and orth(a, b, None) == B.GC_EINVAL
    assert orth(a, inside) == B.GC_EINVAL and orth(inside, a) == B.GC_EINVAL
    assert lib.gc_orthogonalize(m.handle, a, b, None, FAKE, need, None) == B.GC_EINVAL

    def muon(g=a, u=b, w=c, **kw):
        mo = _set(B.muon_options(0.9, 0.1), **kw)
        return lib.gc_muon_step(m.handle, g, u, w, ctypes.byref(mo), FAKE, need, None)

    for kw in (dict(g=None), dict(u=None), dict(w=None), dict(u=a), dict(w=a), dict(w=b), dict(w=inside),
               dict(momentum=1.0), dict(momentum=-0.1), dict(momentum=NAN), dict(lr=NAN), dict(lr=INF),
               dict(weight_decay=-1.0), dict(weight_decay=INF), dict(momentum_kind=2), dict(scale=3), dict(scale=-1),
               dict(reserved=1)):
        assert muon(**kw) == B.GC_EINVAL, kw


def test_option_structs_match_the_header():
    # the sizes and offsets a C caller compiles
    assert ctypes.sizeof(B.gc_orth_options) == 8 + 16 * 12 + 8
    assert B.gc_muon_options.momentum.offset == ctypes.sizeof(B.gc_orth_options)
    assert ctypes.sizeof(B.gc_muon_options) == ctypes.sizeof(B.gc_orth_options) + 24
    o = B.orth_options(steps=2, coef=((1, 2, 3), (4, 5, 6)), eps=0.5)
    assert list(o.coef[1]) == [4, 5, 6] and o.steps == 2 and o.eps == 0.5
    assert np.allclose(list(B.orth_options(steps=3).coef[2]), (3.4445, -4.7750, 2.0315))


@pytest.mark.parametrize("op,cols,n", [
    ("message", (1 << 30) + 1, 1), ("message", 1_100_000_000, 16), ("message", (1 << 26) + 1, 256),
    ("add", (1 << 30) + 1, 16), ("add", 1 << 27, 256), ("dense", 1 << 30, 16),
    # the sums alone fit a launch, with the clearing beside them they do not
    ("dense", 1_062_400_000, 1),
])
def test_short_batches_of_more_columns_than_a_launch_has_threads(op, cols, n):
    """A workgroup of 1,024 threads for every 256 columns of every 16 tokens,
    and for every 16,384 elements that are cleared: 2^32 threads or more are
    refused before anything is enqueued."""
    groups = -(-n // 16) * -(-cols // 256) + (-(-cols // 16384) if op == "dense" else 0)
    assert groups * 1024 >= 1 << 32 and n * cols <= 1 << 35
    p = B.Plan(W.make_table([cols], [1]))
    need = B.gc_embed_workspace_bytes(p, 0, 1, n)
    lib = B.load()
    if op == "message":
        msg = B.gc_sparse(FAKE.value, FAKE.value, FAKE.value, None, cols)
        code = lib.gc_embed_message(p.handle, 0, 1, FAKE, 0, cols, FAKE, 0, n, 1.0, ctypes.byref(msg), FAKE, need, None)
    else:
        code = lib.gc_embed_grad(p.handle, 0, 1, FAKE, 0, cols, FAKE, 0, n, 1.0, FAKE, int(op == "add"), FAKE, need, None)
    assert code == B.GC_ERANGE, B.gc_last_error()


# Schedules that are steep at the top of their range: singular values of at
# most 1 stay below 2 at every step.  Published for six steps and more, as they
# are and with their arguments divided by 1.01, and one of five steps.
SIX = ((8.28721, -23.59589, 17.30039), (4.10706, -2.94785, 0.54484), (3.94869, -2.90890, 0.55182),
       (3.31842, -2.48849, 0.51005), (2.30065, -1.66890, 0.41881), (1.89130, -1.26800, 0.37680))
DIVIDED = tuple((a / 1.01, b / 1.01 ** 3, c / 1.01 ** 5) for a, b, c in SIX)
FIVE = ((8.1566, -22.4833, 15.8788), (4.0429, -2.8089, 0.5000), (3.8917, -2.7725, 0.5061), (3.2858, -2.3681, 0.4645),
        (2.3465, -1.6998, 0.4232))
LAST = (1.875, -1.25, 0.375)


@pytest.mark.parametrize("coef,code", [
    (SIX[:3], B.GC_ECAPACITY), (SIX, B.GC_ECAPACITY), (DIVIDED[:4], B.GC_ECAPACITY), (DIVIDED, B.GC_ECAPACITY),
    (DIVIDED + (LAST,) * 10, B.GC_ECAPACITY), (FIVE, B.GC_ECAPACITY), (FIVE + (LAST,), B.GC_ECAPACITY),
    # on either side of the largest X, B and result
    (((7.99, 0, 0), (1, 0, 0)), B.GC_ECAPACITY), (((8.01, 0, 0), (1, 0, 0)), B.GC_EINVAL),
    (((1, 0, 0), (16380, 0, 0)), B.GC_ECAPACITY), (((1, 0, 0), (16390, 0, 0)), B.GC_EINVAL),
    (((0, 0, 7.99), (1, 0, 0)), B.GC_ECAPACITY), (((0, 0, -8.01), (1, 0, 0)), B.GC_EINVAL),
    (((0, 7.99, 0), (0.125, 0, 0)), B.GC_ECAPACITY), (((0, -8.01, 0), (0.125, 0, 0)), B.GC_EINVAL),
    # the largest value inside the range: 8.08 and 7.97 at about 1/2
    (((23.9, -31.0, 0), (0.125, 0, 0)), B.GC_EINVAL), (((23.5, -30.3, 0), (0.125, 0, 0)), B.GC_ECAPACITY),
])
def test_schedules_at_the_edge_of_the_range(coef, code):
    """Refused only where singular values of at most 1 really pass 8 before the
    last step: a short workspace is what an accepted call is refused for."""
    x = np.linspace(0, 1, 20001)
    most = []
    for a, b, c in coef:
        x = np.abs(a * x + b * x ** 3 + c * x ** 5)
        most.append(x.max())
    p = _plan()
    m = B.MatrixPlan(p, [0, 10, 6])
    o = B.orth_options(len(coef), coef)
    lib = B.load()
    assert lib.gc_orthogonalize(m.handle, FAKE, FAKE, ctypes.byref(o), FAKE, m.workspace_bytes() - 1, None) == code, most


@pytest.mark.parametrize("off", [1, 2, 3])
def test_misaligned_embedding_and_message_buffers(off):
    """Every buffer of a call, not only the batch's."""
    p = _plan()
    lib = B.load()
    bad = ctypes.c_void_p(FAKE.value + off)
    need = B.gc_embed_workspace_bytes(p, 1, 10, 5)
    assert _lookup(p, w=bad) == B.GC_EINVAL
    for acc in (0, 1):
        assert lib.gc_embed_grad(p.handle, 1, 10, FAKE, 0, 12, FAKE, 0, 5, 1.0, bad, acc, FAKE, need, None) == B.GC_EINVAL
        # an empty batch still clears
        assert lib.gc_embed_grad(p.handle, 1, 10, None, 0, 12, None, 0, 0, 1.0, bad, acc, None, 0, None) == B.GC_EINVAL
    for k in range(3):
        at = [bad.value if i == k else FAKE.value for i in range(3)]
        msg = B.gc_sparse(at[0], at[1], at[2], None, 60)
        assert lib.gc_embed_message(p.handle, 1, 10, FAKE, 0, 12, FAKE, 0, 5, 1.0, ctypes.byref(msg), FAKE, need,
                                    None) == B.GC_EINVAL
