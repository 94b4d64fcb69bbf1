"""The paths that only large matrices take: steps in pairs, symmetric products
on large tiles, and the order of the common index; and what the split operands
themselves cost, by an emulation of the same roundings.

References run in 64 and 32 bits on the GPU.  Where a test says nothing else, an
error may be 4 times that of the recurrence in fp32 products plus 2^-20, as in
the tests of single steps."""
import math

import pytest
import torch

from gradient_compression_dnn_amd import binding as B
from tests.gpu_util import dev, say
from tests.test_gpu_orth import COEF, Mats
from tests.test_operators_abi_cpu import DIVIDED, FIVE, LAST

pytestmark = pytest.mark.gpu

CUBIC = (1.5, -0.5, 0.0)
FALLING = ((4.0, -6.0, 2.5), (3.5, -4.0, 1.25), LAST, LAST)


def matrix(gen, r, c, lead=True):
    """Noise, and a direction a few times larger in front of it."""
    x = torch.randn(r, c, device=dev(), generator=gen)
    if lead:
        x += 0.2 * torch.randn(r, 1, device=dev(), generator=gen) * torch.randn(1, c, device=dev(), generator=gen)
    return x * 1e-3


def start(D, eps=1e-7):
    """X_0 with fewer rows than columns, in 64 bits."""
    X = D.double() / (torch.linalg.vector_norm(D.double()) + eps)
    return X.T.contiguous() if D.shape[0] > D.shape[1] else X


def recurrence(D, coef, dtype):
    X = start(D).to(dtype)
    for a, b, c in coef:
        A = X @ X.T
        X = a * X + (b * A + c * (A @ A)) @ X
    return X.T if D.shape[0] > D.shape[1] else X


def rel(x, want):
    return float(torch.linalg.vector_norm(x.double() - want) / torch.linalg.vector_norm(want))


class Call:
    """The matrices of one plan in a flat buffer with a gap, and one call."""

    def __init__(self, shapes, gen, lead=True):
        self.ms = Mats(shapes)
        self.D = [matrix(gen, r, c, lead) for r, c in shapes]
        self.x = torch.randn(self.ms.n, device=dev(), generator=gen)
        for (o, n, _, _), d in zip(self.ms.table, self.D):
            self.x[o:o + n] = d.reshape(-1)
        self.ws = self.ms.ws()

    def parts(self, flat):
        return [flat[o:o + n].view(s) for (o, n, _, _), s in zip(self.ms.table, self.ms.shapes)]

    def orthogonalize(self, coef):
        """The results, and how many products of pairs the call launched."""
        O = torch.full((self.ms.n,), 5.0, device=dev())
        B.gc_timing_enable(["orth_pair"])
        try:
            B.gc_orthogonalize(self.ms.m, self.x, O, B.orth_options(len(coef), coef), self.ws)
            launched = B.gc_timing_take("orth_pair")[1]
        finally:
            B.gc_timing_enable(None)
        keep = torch.ones(self.ms.n, dtype=torch.bool, device=dev())
        for o, n, _, _ in self.ms.table[:len(self.D)]:
            keep[int(o):int(o + n)] = False
        assert bool((O[keep] == 5.0).all())
        return self.parts(O), launched


def check(got, D, coef):
    want = recurrence(D, coef, torch.float64)
    tol = 4 * rel(recurrence(D, coef, torch.float32), want) + 2.0 ** -20
    err = rel(got, want)
    assert err <= tol, f"{tuple(D.shape)}: {err:.3g} > {tol:.3g}"


PAIRED = [
    [(768, 8000)], [(8000, 768)],          # small tiles, cut along the common index
    [(520, 4000)] * 6, [(2500, 900)] * 9,  # several matrices; symmetric products that are not cut
    [(2000, 5000), (600, 2000)],           # X X^T on large tiles, the squares on small ones
    [(2000, 5000), (2048, 700)],           # everything on large tiles, matrices both ways round
]


@pytest.mark.parametrize("shapes", PAIRED)
@pytest.mark.parametrize("coef", [
    (COEF,) * 2, (COEF,) * 3, (COEF,) * 4, (COEF,) * 5, (COEF,) * 6, (COEF,) * 16, (CUBIC,) * 6, (LAST,) * 7, FALLING,
    FALLING + (CUBIC,), DIVIDED, FIVE,
], ids=lambda c: f"{len(c)}of{c[0][0]:.3g}")
def test_steps_in_pairs(shapes, coef):
    """Every plan here pairs: three products more than single steps' for each
    pair are counted.  An odd step goes first."""
    gen = torch.Generator(device=dev()).manual_seed(len(coef) + shapes[0][0])
    call = Call(shapes, gen)
    say(f"pairs of {shapes[:2]} x {len(shapes)}, {len(coef)} steps")
    got, launched = call.orthogonalize(coef)
    assert launched == 3 * (len(coef) // 2)
    for o, D in zip(got, call.D):
        check(o, D, coef)


@pytest.mark.parametrize("shapes", [
    [(2048, 2048)], [(2300, 2300)],          # a single large matrix: every product on large tiles, cut
    [(2400, 2400), (100, 5000)], [(2100, 2100)] * 2,
])
@pytest.mark.parametrize("coef", [(COEF,), (COEF,) * 2, (COEF,) * 5, (CUBIC,) * 6, FIVE], ids=lambda c: f"{len(c)}of{c[0][0]:.3g}")
def test_single_steps_on_large_tiles(shapes, coef):
    gen = torch.Generator(device=dev()).manual_seed(len(coef) + shapes[0][0])
    call = Call(shapes, gen)
    say(f"large tiles {shapes}, {len(coef)} steps")
    got, launched = call.orthogonalize(coef)
    assert launched == 0
    for o, D in zip(got, call.D):
        check(o, D, coef)


def test_a_muon_step_in_pairs_captured_and_beside_one_that_is_not_finite():
    """Two graphs that share a workspace full of NaN, replayed in turn, give
    the bits of eager calls; a matrix with an Inf becomes NaN and leaves the
    others their bits."""
    gen = torch.Generator(device=dev()).manual_seed(5)
    shapes = [[(640, 900)] * 4 + [(520, 9000)] * 2, [(768, 8000)]]
    calls = [Call(s, gen) for s in shapes]
    ws = torch.full((max(c.ms.m.workspace_bytes() for c in calls),), 0xFF, dtype=torch.uint8, device=dev())
    opt = B.muon_options(0.9, 0.05, weight_decay=0.1)
    new = lambda c: [torch.zeros_like(c.x), torch.randn(c.ms.n, device=dev(), generator=gen) * 0.02]  # noqa: E731
    states = [new(c) for c in calls]
    twins = [[t.clone() for t in s] for s in states]
    for c in calls:
        c.ms.m.upload()
    torch.cuda.synchronize()
    graphs = []
    for c, (U, Wt) in zip(calls, states):
        say(f"capture of {c.ms.shapes[:1]}")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            B.gc_muon_step(c.ms.m, c.x, U, Wt, opt, ws)
        graphs.append(graph)
    for t in range(4):
        for c in calls:
            c.x.mul_(0.5).add_(torch.randn(c.ms.n, device=dev(), generator=gen), alpha=1e-3)
        say(f"replay {t}")
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for c, (U, Wt), (Ue, We) in zip(calls, states, twins):
            W0 = We.clone()
            B.gc_muon_step(c.ms.m, c.x, Ue, We, opt, c.ws)
            torch.cuda.synchronize()
            assert torch.equal(U, Ue) and torch.equal(Wt, We)
            # the formula, on the first matrix
            o, n = int(c.ms.table[0][0]), int(c.ms.table[0][1])
            r, k = c.ms.shapes[0]
            D = (0.9 * Ue[o:o + n] + c.x[o:o + n]).view(r, k)
            O64, O32 = (recurrence(D, (COEF,) * 5, d) for d in (torch.float64, torch.float32))
            lr = 0.05 * max(1.0, r / k) ** 0.5
            want = (1 - 0.05 * 0.1) * W0[o:o + n].double() - lr * O64.reshape(-1)
            # three roundings of W's size, and d and l in fp32
            tol = (lr * (4 * rel(O32, O64) + 2.0 ** -20 + 2.0 ** -24) * float(torch.linalg.vector_norm(O64))
                   + 4 * 2.0 ** -24 * float(torch.linalg.vector_norm(W0[o:o + n].double())))
            assert float(torch.linalg.vector_norm(We[o:o + n].double() - want)) <= tol
    c = calls[0]
    good = c.parts(torch.empty_like(c.x).copy_(c.x))
    ref, _ = c.orthogonalize((COEF,) * 5)
    o, n = int(c.ms.table[4][0]), int(c.ms.table[4][1])
    c.x[o + n - 1] = float("inf")
    got, launched = c.orthogonalize((COEF,) * 5)
    assert launched == 6
    for k in range(len(good)):
        assert bool(torch.isnan(got[k]).all()) if k == 4 else torch.equal(got[k], ref[k])


# -------------------------------------------------- the roundings themselves
def split(v):
    hi = v.half()
    return hi.float(), (v - hi.float()).half().float()


def product(P, Q, turn, tile, ordered):
    """P Q^T of split operands in fp32 sums, stages of 32 of the common index one
    after the other; turn 1 or 2: each tile of rows or columns starts behind its
    own and ends with them, if `ordered`."""
    (ph, pl), (qh, ql) = P, Q
    stages = (ph.shape[1] + 31) // 32
    whole = slice(None)

    def sums(r, c, first):
        acc = torch.zeros(ph[r].shape[0], qh[c].shape[0], device=dev())
        for s in range(stages):
            k = 32 * ((first + s) % stages)
            k = slice(k, k + 32)
            acc = torch.addmm(acc, ph[r][:, k], ql[c][:, k].T)
            acc = torch.addmm(acc, pl[r][:, k], qh[c][:, k].T)
            acc = torch.addmm(acc, ph[r][:, k], qh[c][:, k].T)
        return acc

    if not turn or not ordered:
        return sums(whole, whole, 0)
    blocks = range(0, (ph if turn == 1 else qh).shape[0], tile)
    at = [(slice(i, i + tile), (i + tile) // 32) for i in blocks]
    return torch.cat([sums(r, whole, f) for r, f in at]) if turn == 1 else torch.cat([sums(whole, c, f) for c, f in at], 1)


def emulated(D, coef, pairs, tile=128, ordered=True):
    """The call's result as its number formats give it."""
    def power(bound):  # keeps values up to the bound inside fp16
        return 2.0 ** math.floor(math.log2(60000.0 / (1.02 * bound)))

    top, bounds = 1.0, []
    for a, b, c in coef:
        x = torch.linspace(0, top, 100_001, dtype=torch.float64)
        q = a + b * x ** 2 + c * x ** 4
        bounds.append((top, float(q.abs().max())))
        top = float((q * x).abs().max())
    bounds.append((top, 0.0))
    X, sx, k = start(D), power(1.0), 0
    eye = torch.eye(X.shape[0], device=dev())
    X = split((X * sx).float())

    def poly(A, sa, abc, sb):
        a, b, c = abc
        return split(product(A, A, 0, tile, ordered) * (c * sb / sa ** 2) + (A[0] + A[1]) * (b * sb / sa) + eye * (a * sb))

    while k < len(coef):
        (t, pb), (t2, pb2) = bounds[k], bounds[k + 1]
        sa, sp = power(t * t), power(pb)
        A = split(product(X, X, 0, tile, ordered) * (sa / sx ** 2))
        P, step = poly(A, sa, coef[k], sp), 1
        if pairs and (len(coef) - k) % 2 == 0:
            ss, sa2, sp2, sq = power(t * t2), power(t2 * t2), power(pb2), power(pb * pb2)
            S = split(product(P, A, 1, tile, ordered) * (ss / sp / sa))
            A = split(product(S, P, 2, tile, ordered) * (sa2 / ss / sp))
            P2 = poly(A, sa2, coef[k + 1], sp2)
            P, sp, step = split(product(P2, P, 1, tile, ordered) * (sq / sp2 / sp)), sq, 2
        k += step
        sn = 1.0 if k == len(coef) else power(bounds[k][0])
        Y = product(P, tuple(v.T.contiguous() for v in X), 1, tile, ordered) * (sn / sp / sx)
        X, sx = split(Y), sn
    return Y.T if D.shape[0] > D.shape[1] else Y


@pytest.mark.parametrize("shape,coef,pairs", [
    ((29, 1600), (COEF,), False), ((29, 1600), (COEF,) * 3, False), ((100, 700), (COEF,) * 2, False),
    ((100, 700), (CUBIC,) * 6, False), ((200, 1000), (COEF,), False), ((200, 1000), (CUBIC,) * 6, False),
    ((900, 600), (COEF,) * 2, False), ((600, 900), (COEF,) * 3, False), ((600, 900), (CUBIC,) * 6, False),
    ((768, 8000), (COEF,) * 2, True), ((768, 8000), (COEF,) * 3, True), ((4100, 1030), (CUBIC,) * 2, False),
])
def test_what_the_split_operands_cost(shape, coef, pairs):
    """Few or gentle steps, where fp32 products lose little and 22 bits show.
    The emulation makes the same roundings; only the 32 products of a stage are
    added in another order.  An error here is a sum of more than 10^4 roundings,
    so twice the emulation's is what another order may give, and a part of a
    product that is left out (2^-12 of it at least) is far above."""
    gen = torch.Generator(device=dev()).manual_seed(shape[0])
    call = Call([shape], gen, lead=False)
    say(f"roundings of {shape}, {len(coef)} steps")
    (got,), launched = call.orthogonalize(coef)
    assert (launched > 0) == pairs
    want = recurrence(call.D[0], coef, torch.float64)
    err, cost = rel(got, want), rel(emulated(call.D[0], coef, pairs), want)
    say(f"  error {err:.3g}, emulated {cost:.3g}, fp32 {rel(recurrence(call.D[0], coef, torch.float32), want):.3g}")
    assert err <= 2 * cost


@pytest.mark.parametrize("shape,pairs", [((2048, 2048), False), ((2400, 2400), False), ((2000, 5000), True)])
def test_the_diagonals_terms_are_added_last(shape, pairs):
    """Sums stay small until the diagonal's terms come, which about halves the
    error of two steps.  The emulation gives both orders' errors; the call's has
    to be nearer to the first (by their ratios)."""
    gen = torch.Generator(device=dev()).manual_seed(shape[1])
    call = Call([shape], gen, lead=False)
    coef = (COEF,) * 2
    say(f"order of the common index {shape}")
    (got,), launched = call.orthogonalize(coef)
    assert (launched > 0) == pairs
    want = recurrence(call.D[0], coef, torch.float64)
    last, plain = (rel(emulated(call.D[0], coef, pairs, 256, o), want) for o in (True, False))
    say(f"  error {rel(got, want):.3g}, diagonal last {last:.3g}, plain order {plain:.3g}")
    assert rel(got, want) <= math.sqrt(last * plain)
