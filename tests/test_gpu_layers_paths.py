"""The layer products at sizes that take their other tiles, cuts and ways into
LDS, rows far apart, and logits of the largest vocabularies: against 64 bits, with the
bounds of the tests of small sizes."""
import numpy as np
import pytest
import torch

from gradient_compression_dnn_amd import binding as B
from gradient_compression_dnn_amd import workloads as W
from tests.gpu_util import say
from tests.layer_util import ACTS, DTYPES, GUARD, U32, Layer, Rows, act64, act_error
from tests.test_gpu_distill import reference
from tests.test_gpu_linear import normal, sum_bound, within

pytestmark = pytest.mark.gpu

# tokens, rows, columns, offset of the layer, elements between rows: tiles that fill the chip and more, aligned and
# not, with sums that end inside a stage; long sums of few tiles, in parts; few tokens; one token
SIZES = [(4100, 4104, 200, 0, 0), (4099, 4097, 203, 3, 5), (2050, 1030, 1000, 8, 8), (300, 200, 3001, 0, 0), (60, 130, 5000, 0, 8),
         (33, 2000, 2048, 1, 0), (9, 5000, 1037, 0, 3), (16, 4096, 512, 0, 0), (16, 8192, 512, 0, 0), (4, 33, 20001, 5, 1), (1, 3001, 4096, 0, 0)]


def each_call(n, rows, cols, lead, pitch, dtype, seed):
    """Every direction with everything in its epilogue, against 64 bits."""
    D = DTYPES[dtype]
    L = Layer(rows, cols, dtype, lead, True, seed)
    ws = L.ws(n)
    w64, b64 = L.weights().double(), L.bias().double()
    x, r, z, y = (Rows(n, c, D, pitch, None if v is None else normal(n, c, v)) for c, v in ((cols, 1), (rows, 2), (rows, None), (rows, None)))
    B.gc_linear_forward(L.plan, L.layer, L.w, x.t, y.t, ws, act=B.GC_ACT_GELU, r=r.t, z=z.t)
    z64 = x.f64() @ w64.T + b64
    bound = sum_bound(x.f64(), w64.T, cols)
    bound = bound + U32 * (z64.abs() + bound)
    within(z.t, z64, bound, D, "z")
    want = act64(z64, "gelu")[0] + r.f64()
    bound = 1.2 * bound + act_error(z64, "gelu")
    within(y.t, want, bound + U32 * (want.abs() + bound), D, "y")
    assert y.guards_kept() and z.guards_kept()
    del z64, want, bound
    dz = Rows(n, rows, D, pitch, normal(n, rows, 3))
    a, zx, dx, dzx = (Rows(n, cols, D, pitch, None if v is None else normal(n, cols, v)) for v in (4, 5, None, None))
    B.gc_linear_grad_input(L.plan, L.layer, L.w, dz.t, dx.t, ws, a=a.t, act=B.GC_ACT_SILU, z=zx.t, dzx=dzx.t)
    g = dz.f64() @ w64 + a.f64()
    bound = sum_bound(dz.f64(), w64, rows)
    bound = bound + U32 * (g.abs() + bound)
    within(dx.t, g, bound, D, "dx")
    slope, err = act64(zx.f64(), "silu")[1], act_error(zx.f64(), "silu")
    within(dzx.t, g * slope, bound * (slope.abs() + err) + g.abs() * err + 2 * U32 * (g * slope).abs(), D, "dzx")
    assert dx.guards_kept() and dzx.guards_kept()
    del g, bound
    g0 = normal(1, L.plan.n_total, 6)[0]
    for add in (False, True):
        g = g0.clone()
        B.gc_linear_grad_weight(L.plan, L.layer, dz.t, x.t, g, add, ws)
        for part, old, want, bound in ((L.weights(g), L.weights(g0), dz.f64().T @ x.f64(), sum_bound(dz.f64().T, x.f64(), n)),
                                       (L.bias(g), L.bias(g0), dz.f64().sum(0), (2 * n + 8) * U32 * dz.f64().abs().sum(0))):
            within(part, want + (old.double() if add else 0.0), bound, torch.float32, "g")
        assert torch.equal(L.outside(g), L.outside(g0))


@pytest.mark.parametrize("n,rows,cols,lead,pitch", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_tiles_and_cuts(n, rows, cols, lead, pitch, dtype):
    say(f"layer {n}x{rows}x{cols} {dtype} lead={lead} pitch={pitch}")
    each_call(n, rows, cols, lead, pitch, dtype, 7)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_same_bits_again_and_in_any_workspace(dtype):
    n, rows, cols = 300, 700, 3000
    L = Layer(rows, cols, dtype, 0, True)
    x, dz = normal(n, cols, 1).to(DTYPES[dtype]), normal(n, rows, 2).to(DTYPES[dtype])
    kept = None
    for fill in (0x00, 0xFF, 0x7F):  # zeros, NaNs, large numbers
        need = B.gc_linear_workspace_bytes(L.plan, L.layer, n)
        ws = torch.full((need + 9,), fill, dtype=torch.uint8, device="cuda")[9:]  # any alignment
        y, dx, g = torch.empty_like(dz), torch.empty_like(x), torch.zeros(L.plan.n_total, device="cuda")
        B.gc_linear_forward(L.plan, L.layer, L.w, x, y, ws)
        B.gc_linear_grad_input(L.plan, L.layer, L.w, dz, dx, ws)
        B.gc_linear_grad_weight(L.plan, L.layer, dz, x, g, False, ws)
        if kept:
            assert all(torch.equal(a, b) for a, b in zip(kept, (y, dx, g)))
        kept = (y, dx, g)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(700, 3000), (64, 20000), (5000, 300)])
def test_a_workspace_serves_every_smaller_batch(rows, cols, dtype):
    """Smaller batches may be cut into more parts; the bytes for the largest hold them."""
    L = Layer(rows, cols, dtype, 0, True)
    most = 3000
    need = B.gc_linear_workspace_bytes(L.plan, L.layer, most)
    guard = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    ws = guard[:need]
    for n in (1, 5, 16, 17, 64, 65, 100, 128, 129, 300, 512, 1000, 2048, most):
        assert B.gc_linear_workspace_bytes(L.plan, L.layer, n) <= need
        x, dz = normal(n, cols, 1).to(DTYPES[dtype]), normal(n, rows, 2).to(DTYPES[dtype])
        y, dx, g = torch.empty_like(dz), torch.empty_like(x), torch.zeros(L.plan.n_total, device="cuda")
        B.gc_linear_forward(L.plan, L.layer, L.w, x, y, ws)
        B.gc_linear_grad_input(L.plan, L.layer, L.w, dz, dx, ws)
        B.gc_linear_grad_weight(L.plan, L.layer, dz, x, g, False, ws)
        within(y, x.double() @ L.weights().double().T + L.bias().double(), 1.1 * sum_bound(x.double(), L.weights().double().T, cols) + 8 * U32, DTYPES[dtype], "y")
        within(dx, dz.double() @ L.weights().double(), sum_bound(dz.double(), L.weights().double(), rows), DTYPES[dtype], "dx")
        within(L.weights(g), dz.double().T @ x.double(), sum_bound(dz.double().T, x.double(), n), torch.float32, "g")
    assert bool((guard[need:] == 0x5A).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_far_apart(dtype):
    """Offsets past 2^32 bytes and elements: every array's rows 2^31 + 8 elements apart."""
    D = DTYPES[dtype]
    n, rows, cols = 3, 40, 130
    step = (1 << 31) + 8
    L = Layer(rows, cols, dtype, 0, True)
    size = 2 * step + 400
    base = torch.empty(size, dtype=D, device="cuda")
    at = lambda first, c: torch.as_strided(base, (n, c), (step, 1), first)
    x, y, dz, dx = at(0, cols), at(130, rows), at(170, rows), at(210, cols)
    x.copy_(normal(n, cols, 1))
    dz.copy_(normal(n, rows, 2))
    say(f"rows far apart {dtype}")
    B.gc_linear_forward(L.plan, L.layer, L.w, x, y, L.ws(n))
    B.gc_linear_grad_input(L.plan, L.layer, L.w, dz, dx, L.ws(n))
    g = torch.zeros(L.plan.n_total, device="cuda")
    B.gc_linear_grad_weight(L.plan, L.layer, dz, x, g, False, L.ws(n))
    yy, dd, gg = torch.empty(n, rows, dtype=D, device="cuda"), torch.empty(n, cols, dtype=D, device="cuda"), torch.zeros_like(g)
    xc, zc = x.contiguous(), dz.contiguous()
    w64 = L.weights().double()
    within(y, xc.double() @ w64.T + L.bias().double(), 1.1 * sum_bound(xc.double(), w64.T, cols) + 4 * U32, D, "y")
    within(dx, zc.double() @ w64, sum_bound(zc.double(), w64, rows), D, "dx")
    within(L.weights(g), zc.double().T @ xc.double(), sum_bound(zc.double().T, xc.double(), n), torch.float32, "g")
    if dtype == "bf16":  # logits as far apart, loss and top
        V = 400
        z = torch.as_strided(base, (n, V), (step, 1), 0)
        z.copy_(normal(n, V, 5))
        idx, val, lse = torch.empty(n, 9, dtype=torch.int32, device="cuda"), torch.empty(n, 9, device="cuda"), torch.empty(n, device="cuda")
        B.gc_top_logits(z, idx, val, lse)
        i2, v2, l2 = torch.empty_like(idx), torch.empty_like(val), torch.empty_like(lse)
        B.gc_top_logits(z.contiguous(), i2, v2, l2)
        assert torch.equal(idx, i2) and torch.equal(val, v2)
        loss, near, dn = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty(n, V, dtype=D, device="cuda")
        opt = B.distill_options(2.0, 1.0, 0.5, 8.0, tail=True)
        zc = z.contiguous()
        B.gc_distill_loss(zc, idx, val + 0.5, opt, near, dn, t_lse=lse, labels=idx[:, 3].contiguous())
        B.gc_distill_loss(z, idx, val + 0.5, opt, loss, z, t_lse=lse, labels=idx[:, 3].contiguous())
        assert torch.equal(loss, near) and torch.equal(z, dn)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_largest_vocabulary(dtype):
    """2^20 columns, 1,024 entries, the rest held: the most LDS a call takes."""
    n, V, k, T = 2, B.GC_MAX_VOCAB, B.GC_MAX_TOP_LOGITS, 2.0
    z = normal(n, V, 1, 3.0).to(DTYPES[dtype])
    idx, val, lse = torch.empty(n, k, dtype=torch.int32, device="cuda"), torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")
    say(f"largest vocabulary {dtype}")
    B.gc_top_logits(z, idx, val, lse, temperature=T)
    s, j = torch.sort(z.double() + 0.0, dim=1, descending=True, stable=True)
    assert torch.equal(idx, j[:, :k].int()) and torch.equal(val.double(), s[:, :k])
    assert bool(((lse.double() - torch.logsumexp(z.double() / T, 1)).abs() <= 1000 * 2.0 ** -23).all())
    tv = val + 0.25 * normal(n, k, 2)
    for tail in (True, False):
        loss, dz = torch.empty(n, device="cuda"), torch.empty_like(z)
        B.gc_distill_loss(z, idx, tv, B.distill_options(T, 1.0, 0.5, 1e3, tail=tail), loss, dz, t_lse=lse, labels=idx[:, 7].contiguous())
        want_l, want_g = reference(z.double(), idx, tv.double(), T, 1.0, 0.5, 1e3, tail, lse, idx[:, 7], None)
        # the bounds of the small sizes' tests: (|d| + 1000) 2^-23 of each term, |d| <= 40 here
        eq = 1100 * 2.0 ** -23
        assert bool(((loss.double() - want_l).abs() <= 4 * T * T * eq * 40 + 8 * U32 * want_l.abs()).all())
        p, p1 = torch.softmax(z.double() / T, 1), torch.softmax(z.double(), 1)
        room = 1e3 * (4 * T * p * 3 * eq + p1 * eq) + 0.0
        room.scatter_add_(1, idx.long(), torch.full((n, k), 1e3 * T * 2 * eq, dtype=torch.float64, device="cuda"))
        room = room + (torch.finfo(z.dtype).eps / 2) * (want_g.abs() + room) + 1e-30
        assert bool(((dz.double() - want_g).abs() <= room).all())


def test_entries_past_the_threads_of_a_row():
    """More entries than the 256 threads of a short row: every entry counts, named twice or not."""
    n, V, T = 3, 700, 1.0
    for k in (256, 257, 700):
        z = normal(n, V, 3, 2.0)
        idx = torch.stack([torch.randperm(V, device="cuda")[:k] for _ in range(n)])
        idx[:, k - 1] = idx[:, 0]
        t = normal(n, k, 4, 2.0)
        tl = torch.logsumexp(t, 1) + 0.5
        for tail in (False, True):
            loss, dz = torch.empty(n, device="cuda"), torch.empty_like(z)
            B.gc_distill_loss(z, idx, t, B.distill_options(T, tail=tail), loss, dz, t_lse=tl)
            want_l, want_g = reference(z.double(), idx, t.double(), T, 1.0, 0.0, 1.0, tail, tl, None, None)
            assert bool(((loss.double() - want_l).abs() <= 4 * 1200 * 2.0 ** -23 * 20).all())
            assert bool(((dz.double() - want_g).abs() <= 4 * 1200 * 2.0 ** -23 * (want_g.abs() + 0.1)).all())


def test_samples_that_miss():
    """Rows whose largest logits all lie in one place, that rise to their end, and
    that repeat one value: the list fills, and the row is read digit by digit."""
    V, k = 131071, 64
    z = normal(6, V, 9)
    z[0, 70000:72000] += 50
    z[1] = torch.arange(V, device="cuda").float()
    z[2] = 1.0
    z[3, ::2] = 3.0
    z[4, 131000:] = float("inf")
    z[5] = torch.round(z[5])
    for D in (torch.float32, torch.bfloat16):
        y = z.to(D)
        idx, val = torch.empty(6, k, dtype=torch.int32, device="cuda"), torch.empty(6, k, device="cuda")
        B.gc_top_logits(y, idx, val)
        s, j = torch.sort(y.double() + 0.0, dim=1, descending=True, stable=True)
        assert torch.equal(idx, j[:, :k].int()) and torch.equal(val.double(), s[:, :k])


def test_outlier_columns_in_fp32():
    """fp32 products keep fp32's range inside a row: a column 2^60 larger than the
    others, where W is 0, costs the others nothing; the largest numbers do not
    overflow, and an Inf makes its row's sums NaN or that Inf, no other's."""
    n, rows, cols = 200, 260, 300
    L = Layer(rows, cols, "f32", 0, False)
    x = normal(n, cols, 1)
    x[:, 7] = 2.0 ** 60
    L.weights()[:, 7] = 0.0
    y = torch.empty(n, rows, device="cuda")
    B.gc_linear_forward(L.plan, L.layer, L.w, x, y, L.ws(n))
    within(y, x.double() @ L.weights().double().T, sum_bound(x.double(), L.weights().double().T, cols), torch.float32, "y")
    x[3, 9], x[4, 9], x[5, 9] = float("inf"), float("-inf"), torch.finfo(torch.float32).max
    L.weights()[:, 9] = 0.5
    L.weights()[11, 9] = 0.0
    B.gc_linear_forward(L.plan, L.layer, L.w, x, y, L.ws(n))
    keep = torch.arange(rows, device="cuda") != 11
    assert bool((torch.isnan(y[3]) | (y[3] == float("inf"))).all()) and bool((torch.isnan(y[4]) | (y[4] == float("-inf"))).all())
    assert bool((y[5, keep] > 1e38).all()) and bool(torch.isfinite(y[5]).all()) and bool(torch.isfinite(y[6:]).all())


def test_more_entries_than_columns():
    z = torch.tensor([[1.0, 3.0, 2.0, -float("inf"), 3.0]], device="cuda")
    idx, val = torch.empty(1, 9, dtype=torch.int32, device="cuda"), torch.empty(1, 9, device="cuda")
    B.gc_top_logits(z, idx, val)
    assert idx.tolist() == [[1, 4, 2, 0, -1, -1, -1, -1, -1]]
    assert val.tolist() == [[3.0, 3.0, 2.0, 1.0] + [-float("inf")] * 5]
