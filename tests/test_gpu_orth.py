"""The orthogonalised update on the GPU against 64 bits.

Tolerance.  The operands of a product hold 22 bits where fp32 holds 24, and
sums are fp32 in both, so an error grows to at most 4 times that of the same
recurrence in fp32; both take the same path through the steps, since the map
of a step is the same.  The fp32 recurrence is run on the CPU for each case,
its error against 64 bits taken (a sum over thousands of roundings, so it
varies little from one input to the next) and 4 times it allowed, plus 2^-20
for small matrices, where fp32's own error can be near zero by chance (four
operand roundings of 2^-22 each)."""
import numpy as np
import pytest
import torch

from gradient_compression_dnn_amd import binding as B
from gradient_compression_dnn_amd import workloads as W
from tests.gpu_util import dev, same_bits, say, ulp_report
from tests.test_operators_abi_cpu import DIVIDED, FIVE, LAST, SIX

pytestmark = pytest.mark.gpu

COEF = (3.4445, -4.7750, 2.0315)


def recurrence(D, steps, coef, eps, dtype):
    X = torch.from_numpy(np.ascontiguousarray(D)).double()
    norm = torch.linalg.vector_norm(X)
    X = (X / (norm + eps)).to(dtype) if norm > 0 else X.to(dtype)
    flip = X.shape[0] > X.shape[1]
    X = X.T.contiguous() if flip else X
    for k in range(steps):
        a, b, c = coef if np.ndim(coef) == 1 else coef[k]
        A = X @ X.T
        X = a * X + (b * A + c * (A @ A)) @ X
    return (X.T if flip else X).numpy()


def rel(x, y):
    n = np.linalg.norm(y)
    d = np.linalg.norm(x.astype(np.float64) - y)
    return d / n if n else d


def check(got, D, steps=5, coef=COEF, eps=1e-7):
    want = recurrence(D, steps, coef, eps, torch.float64)
    plain = recurrence(D, steps, coef, eps, torch.float32)
    tol = 4 * rel(plain, want) + 2.0 ** -20
    err = rel(got, want)
    assert err <= tol, f"{D.shape}: {err:.3g} > {tol:.3g}"


def matrix(rng, r, c, kind):
    if kind == "gauss":
        return rng.normal(0, 1e-3, (r, c)).astype(np.float32)
    if kind == "rank1":
        return (rng.normal(size=(r, 1)) * rng.normal(size=(1, c))).astype(np.float32)
    if kind == "heavy":  # rows of very different size
        return (rng.normal(size=(r, c)) * np.exp(2 * rng.normal(size=(r, 1)))).astype(np.float32)
    if kind == "ortho":
        return np.linalg.qr(rng.normal(size=(max(r, c), min(r, c))))[0].reshape(r, c) if r >= c else matrix(rng, c, r, "ortho").T
    if kind == "sparse":
        return (rng.normal(size=(r, c)) * (rng.random((r, c)) < 0.02)).astype(np.float32)
    raise KeyError(kind)


class Mats:
    """A flat buffer of matrices, a gap and a vector that is no matrix."""

    def __init__(self, shapes, lead=3):
        lens = [r * c for r, c in shapes] + [11]
        self.shapes = shapes
        self.table = W.make_table(lens, [1] * len(lens), None, [lead] + [0] * (len(lens) - 1))
        self.plan = B.Plan(self.table)
        self.m = B.MatrixPlan(self.plan, [r for r, _ in shapes] + [0])
        self.n = self.plan.n_total

    def flat(self, mats, rng):
        x = rng.normal(size=self.n).astype(np.float32)
        for (o, n, _, _), m in zip(self.table, mats):
            x[o:o + n] = m.reshape(-1)
        return x

    def parts(self, x):
        return [x[o:o + n].reshape(s) for (o, n, _, _), s in zip(self.table, self.shapes)]

    def outside(self, x):
        keep = np.ones(self.n, bool)
        for (o, n, _, _), _ in zip(self.table, self.shapes):
            keep[o:o + n] = False
        return x[keep]

    def ws(self):
        return torch.full((self.m.workspace_bytes(),), 0xFF, dtype=torch.uint8, device=dev())  # NaN in every type


def to_dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(dev())


SHAPES = [(1, 1), (1, 7), (9, 1), (2, 2), (31, 33), (32, 64), (127, 129), (128, 128), (129, 127), (300, 70), (65, 513),
          (256, 384), (400, 400), (29, 1600), (200, 1000)]


@pytest.mark.parametrize("kind", ["gauss", "heavy", "rank1", "sparse"])
def test_orthogonalize_shapes(kind):
    rng = np.random.default_rng(17)
    for shape in SHAPES:
        say(f"orthogonalize {shape} {kind}")
        ms = Mats([shape])
        D = matrix(rng, *shape, kind)
        x = ms.flat([D], rng)
        O = to_dev(np.full(ms.n, 5.0))
        B.gc_orthogonalize(ms.m, to_dev(x), O, B.orth_options(), ms.ws())
        got = O.cpu().numpy()
        check(ms.parts(got)[0], D)
        assert (ms.outside(got) == 5.0).all()


def test_many_matrices_in_one_call():
    rng = np.random.default_rng(18)
    shapes = [(64, 147), (64, 64), (256, 64), (29, 1600), (1, 50), (130, 257), (513, 40)]
    ms = Mats(shapes)
    mats = [matrix(rng, *s, k) for s, k in zip(shapes, ["gauss", "heavy", "gauss", "sparse", "gauss", "rank1", "gauss"])]
    x = to_dev(ms.flat(mats, rng))
    O, ws = torch.zeros_like(x), ms.ws()
    say("orthogonalize many")
    B.gc_orthogonalize(ms.m, x, O, B.orth_options(), ws)
    for got, D in zip(ms.parts(O.cpu().numpy()), mats):
        check(got, D)
    # in place, on a used workspace: the same bits
    B.gc_orthogonalize(ms.m, x, x, B.orth_options(), ws)
    for a, b in zip(ms.parts(x.cpu().numpy()), ms.parts(O.cpu().numpy())):
        assert same_bits(a, b), ulp_report(a, b)


@pytest.mark.parametrize("steps,coef", [
    (1, COEF), (2, COEF), (3, (1.5, -0.5, 0.0)), (16, (1.875, -1.25, 0.375)), (3, (1.0, 0.0, 0.0)),
    (4, ((4.0, -6.0, 2.5), (3.5, -4.0, 1.25), (1.875, -1.25, 0.375), (1.875, -1.25, 0.375))), (2, (0.25, 0.5, -0.125)),
    (3, (-2.0, 1.0, 0.5)),
])
def test_steps_and_coefficients(steps, coef):
    rng = np.random.default_rng(19)
    for shape, kind in (((90, 200), "gauss"), ((200, 90), "ortho")):
        ms = Mats([shape])
        D = matrix(rng, *shape, kind).astype(np.float32)
        O = torch.zeros(ms.n, device=dev())
        say(f"steps {steps} coef {coef} {shape}")
        B.gc_orthogonalize(ms.m, to_dev(ms.flat([D], rng)), O, B.orth_options(steps, coef), ms.ws())
        check(ms.parts(O.cpu().numpy())[0], D, steps, coef)


def test_extreme_gradients():
    rng = np.random.default_rng(20)
    shape = (40, 130)
    base = matrix(rng, *shape, "gauss") * 1000
    ms = Mats([shape] * 7)
    nan, inf = base.copy(), base.copy()
    nan[3, 5], inf[39, 129] = np.nan, -np.inf
    one = np.zeros(shape, np.float32)
    one[7, 100] = -3.0
    mats = [base * np.float32(1e-42), base * np.float32(1e35), np.zeros(shape, np.float32), nan, inf, one, base]
    x = ms.flat(mats, rng)
    O = torch.zeros(ms.n, device=dev())
    say("extreme gradients, eps 0")
    B.gc_orthogonalize(ms.m, to_dev(x), O, B.orth_options(eps=0.0), ms.ws())
    got = ms.parts(O.cpu().numpy())
    for k in (0, 1, 5, 6):
        check(got[k], mats[k], eps=0.0)
    assert (got[2] == 0).all() and np.isnan(got[3]).all() and np.isnan(got[4]).all()
    # eps at work: a gradient of its size is halved at the start
    eps = float(np.linalg.norm(base.astype(np.float64)))
    B.gc_orthogonalize(ms.m, to_dev(x), O, B.orth_options(eps=eps, steps=2), ms.ws())
    check(ms.parts(O.cpu().numpy())[6], base, 2, COEF, float(np.float32(eps)))


@pytest.mark.parametrize("nesterov", [False, True])
@pytest.mark.parametrize("scale", [0, 1, 2])
def test_muon_steps(nesterov, scale):
    rng = np.random.default_rng(21)
    shapes = [(70, 200), (333, 100), (64, 64)]
    ms = Mats(shapes)
    m, lr, wd = np.float32(0.95), np.float32(0.02), np.float32(0.1)
    U, Wt = np.zeros(ms.n, np.float32), rng.normal(0, 0.02, ms.n).astype(np.float32)
    Ud, Wd = to_dev(U), to_dev(Wt)
    opt = B.muon_options(0.95, 0.02, weight_decay=0.1, nesterov=nesterov, scale=scale)
    ws = ms.ws()
    inside = np.ones(ms.n, bool)
    for step in range(3):
        G = ms.flat([matrix(rng, *s, "gauss") for s in shapes], rng)
        say(f"muon step {step} nesterov={nesterov} scale={scale}")
        W0 = Wd.cpu().numpy()
        B.gc_muon_step(ms.m, to_dev(G), Ud, Wd, opt, ws)
        U1, W1 = Ud.cpu().numpy(), Wd.cpu().numpy()
        for (o, n, _, _), (r, c) in zip(ms.table, shapes):
            s = slice(o, o + n)
            U[s] = m * U[s] + G[s]
            D = m * U[s] + G[s] if nesterov else U[s]
            inside[s] = False
            assert same_bits(U1[s], U[s]), ulp_report(U1[s], U[s])
            O64 = recurrence(D.reshape(r, c), 5, COEF, 1e-7, torch.float64).reshape(-1)
            O32 = recurrence(D.reshape(r, c), 5, COEF, 1e-7, torch.float32).reshape(-1)
            f = [1.0, max(1.0, r / c) ** 0.5, 0.2 * max(r, c) ** 0.5][scale]
            decay, l = np.float32(1.0 - float(lr) * float(wd)), np.float32(float(lr) * f)
            want = float(decay) * W0[s].astype(np.float64) - float(l) * O64
            # the update's own tolerance, and three roundings of W's size
            tol = float(l) * (4 * rel(O32, O64) + 2.0 ** -20) * np.linalg.norm(O64) + 3 * 2.0 ** -24 * np.linalg.norm(want)
            assert np.linalg.norm(W1[s] - want) <= tol
        assert same_bits(W1[inside], W0[inside]) and same_bits(U1[inside], U[inside])


def test_same_bits_every_time_and_on_two_streams():
    rng = np.random.default_rng(22)
    ms = Mats([(500, 700), (300, 2000)])
    x = to_dev(ms.flat([matrix(rng, *s, "gauss") for s in ms.shapes], rng))
    ref = torch.zeros_like(x)
    B.gc_orthogonalize(ms.m, x, ref, B.orth_options(), ms.ws())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs, spaces = [torch.zeros_like(x) for _ in streams], [ms.ws() for _ in streams]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, o, w in zip(streams, outs, spaces):
            with torch.cuda.stream(s):
                B.gc_orthogonalize(ms.m, x, o, B.orth_options(), w)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, ref)


def test_graph_replays():
    rng = np.random.default_rng(23)
    ms = Mats([(200, 300), (50, 129)])
    ms.m.upload()
    G = torch.zeros(ms.n, device=dev())
    U, Wt = torch.zeros_like(G), to_dev(rng.normal(0, 0.02, ms.n))
    Ue, We = U.clone(), Wt.clone()
    ws, wse = ms.ws(), ms.ws()
    opt = B.muon_options(0.9, 0.05)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    say("muon graph capture (the plan's first call)")
    with torch.cuda.graph(graph):
        B.gc_muon_step(ms.m, G, U, Wt, opt, ws)
    for t in range(4):
        g = to_dev(ms.flat([matrix(rng, *s, "gauss") for s in ms.shapes], rng))
        G.copy_(g)
        say(f"muon graph replay {t}")
        graph.replay()
        torch.cuda.synchronize()
        B.gc_muon_step(ms.m, g, Ue, We, opt, wse)
        torch.cuda.synchronize()
        assert torch.equal(U, Ue) and torch.equal(Wt, We)
        _ = (G * 2).sum().item()


def test_decoded_update_of_learners_into_weights():
    """The run as a training step makes it: learners' DGC messages and
    embedding messages are decoded into one dense update, which the matrices
    take orthogonalised and the embedding as it is."""
    rng = np.random.default_rng(24)
    rows, cols, mr, mc = 90, 16, 48, 80
    table = W.make_table([rows * cols, mr * mc, 33], [50] * 3, [rows * cols, 400, 33])
    plan = B.Plan(table)
    mplan = B.MatrixPlan(plan, [0, mr, 0])
    n = plan.n_total
    dense = torch.zeros(n, device=dev())
    emb, dgc, dense64 = [], [], np.zeros(n)
    body = B.Plan(table[1:], n)  # DGC on everything but the embedding
    for j in range(2):
        g = rng.normal(0, 1e-3, n).astype(np.float32)
        U, V = torch.zeros(n, device=dev()), torch.zeros(n, device=dev())
        msg = B.Sparse.empty(body, body.total_k, dev())
        B.gc_dgc_step(body, to_dev(g), U, V, 0.0, 0.0, 1, msg, body.workspace(B.GC_OP_DGC, dev()))
        dgc.append(msg)
        idx, val, _, _ = msg.host()
        dense64[idx] += val.astype(np.float64) / 2
        keys = rng.integers(-1, rows, 60)
        dy = rng.normal(size=(60, cols)).astype(np.float32)
        e = B.Sparse.empty(plan, B.gc_embed_message_cap(plan, 0, rows, 60), dev())
        ws = torch.empty(B.gc_embed_workspace_bytes(plan, 0, rows, 60), dtype=torch.uint8, device=dev())
        B.gc_embed_message(plan, 0, rows, to_dev(dy), torch.from_numpy(keys).to(dev()), 1.0, e, ws)
        emb.append(e)
        np.add.at(dense64[:rows * cols].reshape(rows, cols), keys[keys >= 0], dy[keys >= 0].astype(np.float64) / 2)
    say("decode, then the matrices' step")
    B.gc_decompress_accumulate(plan, emb, dense, B.GC_AVG, False, plan.workspace(B.GC_OP_DECODE, dev()))
    B.gc_decompress_accumulate(body, dgc, dense, B.GC_AVG, False, body.workspace(B.GC_OP_DECODE, dev()))
    assert np.abs(dense.cpu().numpy() - dense64).max() <= 80 * 2.0 ** -24 * np.abs(dense64).max() + 2.0 ** -20 * 4
    Wt = to_dev(rng.normal(0, 0.02, n))
    W0, U = Wt.cpu().numpy(), torch.zeros(n, device=dev())
    B.gc_muon_step(mplan, dense, U, Wt, B.muon_options(0.0, 0.1, nesterov=False), mplan.workspace(dev()))
    o = rows * cols
    D = dense.cpu().numpy()[o:o + mr * mc].reshape(mr, mc)
    assert same_bits(U.cpu().numpy()[o:o + mr * mc], D.reshape(-1))
    O64, O32 = (recurrence(D, 5, COEF, 1e-7, t) for t in (torch.float64, torch.float32))
    want = W0[o:o + mr * mc].astype(np.float64) - float(np.float32(0.1)) * O64.reshape(-1)
    tol = 0.1 * (4 * rel(O32, O64) + 2.0 ** -20) * np.linalg.norm(O64) + 3 * 2.0 ** -24 * np.linalg.norm(want)
    W1 = Wt.cpu().numpy()
    assert np.linalg.norm(W1[o:o + mr * mc] - want) <= tol
    assert same_bits(W1[:o], W0[:o]) and same_bits(W1[o + mr * mc:], W0[o + mr * mc:])


@pytest.mark.parametrize("shapes", [
    [(1100, 1500)],                      # tiles cut to fill the units
    [(2600, 600)], [(513, 2000)] * 3,    # the same, transposed and several at once
    [(1030, 1030)], [(511, 1800)],       # square, and fewer rows than steps in pairs need
    [(700, 900), (30, 40), (129, 3001)],  # few rows beside many
    [(128, 9000)], [(5, 6000), (100, 100), (1, 3)],  # few rows only: several slabs a workgroup and parts
])
@pytest.mark.parametrize("steps", [1, 4, 5])
def test_every_schedule(shapes, steps):
    rng = np.random.default_rng(25)
    ms = Mats(shapes)
    kinds = ["gauss", "heavy", "rank1"]
    mats = [matrix(rng, *s, kinds[k % 3]) + matrix(rng, *s, "gauss") for k, s in enumerate(shapes)]
    x = ms.flat(mats, rng)
    O = torch.full((ms.n,), 5.0, device=dev())
    say(f"schedules {shapes} steps {steps}")
    B.gc_orthogonalize(ms.m, to_dev(x), O, B.orth_options(steps), ms.ws())
    got = O.cpu().numpy()
    for o, D in zip(ms.parts(got), mats):
        check(o, D, steps)
    assert (ms.outside(got) == 5.0).all()


@pytest.mark.parametrize("scale", [1e-9, 1e-12])
def test_a_norm_far_below_eps(scale):
    """X_0's entries are near fp16's last bits then.  Every X_k is stored with
    an absolute error of up to 2^-40 an entry or a relative one of 2^-23, and
    the products that make the next one are off by the roundings of B's and
    X's entries (2^-23 each), the dropped product of two low parts (2^-22 at
    most) and the result's (2^-24): less than 2^-21 of |a X_k|, since a X is
    nearly all of the next X while X is small.  An error grows by at most the
    step's largest slope, 3.9 (|p'| on [0, 1.2]).  So after 5 steps
    ||dO|| <= 3.9^5 (1 + 1/3.9 + ...) 2^-40 sqrt(m n) + 5 2^-21 ||O||,
    the geometric sum being at most 1.35."""
    rng = np.random.default_rng(26)
    for shape in ((40, 130), (200, 300)):
        D = (matrix(rng, *shape, "gauss") * np.float32(scale)).astype(np.float32)
        ms = Mats([shape])
        O = torch.zeros(ms.n, device=dev())
        B.gc_orthogonalize(ms.m, to_dev(ms.flat([D], rng)), O, B.orth_options(), ms.ws())
        want = recurrence(D, 5, COEF, 1e-7, torch.float64)
        err = np.linalg.norm(ms.parts(O.cpu().numpy())[0] - want)
        assert err <= 1.35 * 3.9 ** 5 * 2.0 ** -40 * (shape[0] * shape[1]) ** 0.5 + 5 * 2.0 ** -21 * np.linalg.norm(want)


def test_padded_and_gapped_buffers_are_left_alone():
    """Only the matrices' elements are written: a buffer whose gaps and tail
    are NaN keeps them bit for bit, in place too."""
    rng = np.random.default_rng(27)
    shapes = [(64, 147), (300, 520)]
    lens = [r * c for r, c in shapes]
    table = W.make_table([7, lens[0], 3, lens[1]], [1] * 4, None, [2, 5, 0, 9])
    plan = B.Plan(table, W.table_extent(table) + 13)
    m = B.MatrixPlan(plan, [0, 64, 0, 300])
    x = np.full(plan.n_total, np.nan, np.float32)
    for (o, n, _, _), s in ((table[1], shapes[0]), (table[3], shapes[1])):
        x[o:o + n] = matrix(rng, *s, "gauss").reshape(-1)
    inside = np.zeros(plan.n_total, bool)
    for o, n, _, _ in (table[1], table[3]):
        inside[o:o + n] = True
    d, ws = to_dev(x), m.workspace(dev())
    B.gc_orthogonalize(m, d, d, B.orth_options(), ws)
    got = d.cpu().numpy()
    assert same_bits(got[~inside], x[~inside]) and np.isfinite(got[inside]).all()
    U, Wt = to_dev(x * 0), to_dev(x)
    B.gc_muon_step(m, to_dev(x), U, Wt, B.muon_options(0.9, 0.1), ws)
    U, Wt = U.cpu().numpy(), Wt.cpu().numpy()
    assert np.isnan(U[~inside]).all() and same_bits(Wt[~inside], x[~inside])
    assert np.isfinite(U[inside]).all() and np.isfinite(Wt[inside]).all()


def test_refused_calls_touch_nothing():
    ms = Mats([(20, 30)])
    x = torch.ones(ms.n, device=dev())
    O = torch.full((ms.n,), 3.0, device=dev())
    for opt in (B.orth_options(eps=-1.0), B.orth_options(1, (float("nan"), 0, 0))):
        with pytest.raises(B.GCError):
            B.gc_orthogonalize(ms.m, x, O, opt, ms.ws())
    with pytest.raises(B.GCError):
        B.gc_orthogonalize(ms.m, x, O, B.orth_options(), ms.ws()[:100])
    with pytest.raises(ValueError):
        B.gc_orthogonalize(ms.m, x.cpu(), O, B.orth_options(), ms.ws())
    with pytest.raises(ValueError):
        B.gc_orthogonalize(ms.m, x[:-1], O, B.orth_options(), ms.ws())
    torch.cuda.synchronize()
    assert bool((O == 3.0).all())


STEEP = [SIX[:3], SIX, DIVIDED, DIVIDED + (LAST,) * 2, FIVE, ((7.9, 0.0, 0.0), (0.1, 0.0, 0.0))]


@pytest.mark.parametrize("coef", STEEP)
def test_steep_schedules(coef):
    """Schedules whose polynomials are steep where the singular values are
    largest.  The matrices have many singular values, which share the error."""
    rng = np.random.default_rng(28)
    for shape, kind in (((40, 130), "gauss"), ((90, 200), "gauss"), ((200, 90), "ortho"), ((29, 1600), "gauss"),
                        ((300, 520), "gauss"), ((520, 300), "sparse"), ((600, 640), "gauss")):
        D = matrix(rng, *shape, kind).astype(np.float32)
        ms = Mats([shape])
        O = torch.zeros(ms.n, device=dev())
        say(f"steep schedule of {len(coef)} steps {shape} {kind}")
        B.gc_orthogonalize(ms.m, to_dev(ms.flat([D], rng)), O, B.orth_options(len(coef), coef), ms.ws())
        check(ms.parts(O.cpu().numpy())[0], D, len(coef), coef)


@pytest.mark.parametrize("coef", STEEP + [(COEF,) * 5])
def test_a_vector_runs_through_the_polynomials(coef):
    """The one singular value of a vector is 1 at the start and then p(1),
    p(p(1)), ...  X_0 is off by 2^-22 of itself.  A step is off by its
    roundings, 2^-19 of the sizes of its terms (an operand by 2^-23, A by 2^-21,
    c A^2 by 2^-19) and as much again for up to 32 additions of a sum, 2^-24
    each; and by what it was off before times the slope at its value, or p(s) / s,
    whichever is larger.  Half as much again for the second order, which is below
    that while the error is below 0.01."""
    rng = np.random.default_rng(29)
    s, err = 1.0, 2.0 ** -22
    for a, b, c in coef:
        slope = max(abs(a + 3 * b * s ** 2 + 5 * c * s ** 4), abs(a + b * s ** 2 + c * s ** 4))
        err = slope * err + 2.0 ** -18 * (abs(a) * s + abs(b) * s ** 3 + abs(c) * s ** 5)
        s = abs(a * s + b * s ** 3 + c * s ** 5)
    for shape in ((1, 1), (1, 7), (9, 1), (1, 1000), (1000, 1)):
        D = rng.normal(0, 1e-2, shape).astype(np.float32)
        ms = Mats([shape])
        O = torch.zeros(ms.n, device=dev())
        say(f"vector {shape} of {len(coef)} steps")
        B.gc_orthogonalize(ms.m, to_dev(ms.flat([D], rng)), O, B.orth_options(len(coef), coef, eps=0.0), ms.ws())
        got = ms.parts(O.cpu().numpy())[0]
        assert np.isfinite(got).all()
        want = recurrence(D, len(coef), coef, 0.0, torch.float64)
        assert abs(np.linalg.norm(want) - s) <= 1e-6 * s  # the coefficients in fp32 and in 64 bits
        if err < 0.01 * s:
            assert np.linalg.norm(got - want) <= 1.5 * err
        else:  # no digits are left; the bounds the call chose its exponents by still hold
            assert np.linalg.norm(got) <= 8.0
