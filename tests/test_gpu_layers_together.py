"""The layer products, the top logits and the distillation loss as a learner uses
them with the embedding, the compression and the matrix updates: gradients
of the whole model against 64 bits, graphs that share a workspace, streams, threads."""
import threading

import numpy as np
import pytest
import torch

from gradient_compression_dnn_amd import binding as B
from gradient_compression_dnn_amd import workloads as W
from tests.gpu_util import say
from tests.layer_util import act64

pytestmark = pytest.mark.gpu


class Student:
    """Embedding (V x E), a block h = e + gelu(e W1^T + b1) W2^T, logits h Wo^T + bo
    over the vocabulary; a teacher of fixed logits sends its top k."""

    def __init__(self, V, E, H, n, k, dtype, seed, T=2.0, ce=0.5):
        rng = np.random.default_rng(seed)
        self.V, self.E, self.H, self.n, self.k, self.T, self.ce, self.dtype = V, E, H, n, k, T, ce, dtype
        self.lens = [V * E, H * E, H, E * H, V * E, V]
        self.plan = B.Plan(W.make_table(self.lens, [50] * 6))
        self.mplan = B.MatrixPlan(self.plan, [0, H, 0, E, 0, 0])
        self.plan.upload()
        self.mplan.upload()
        self.l1, self.l2, self.lo = (B.linear_layer(s, r, dtype, b) for s, r, b in ((1, H, 2), (3, E, -1), (4, V, 5)))
        w = np.concatenate([rng.normal(0, s, m) for s, m in zip((1, E ** -0.5, 0.1, H ** -0.5, E ** -0.5, 0.1), self.lens)])
        self.w0 = torch.from_numpy(w.astype(np.float32)).cuda()
        self.tokens = torch.from_numpy(rng.integers(-1, V + 1, n)).cuda()
        self.labels = torch.from_numpy(rng.integers(-1, V, n)).cuda().int()
        self.teacher = torch.from_numpy(rng.normal(0, 2, (n, V)).astype(np.float32)).cuda().to(dtype)
        self.need = max([B.gc_embed_workspace_bytes(self.plan, 0, V, n), self.mplan.workspace_bytes(), self.plan.workspace_bytes(B.GC_OP_DGC),
                         self.plan.workspace_bytes(B.GC_OP_DECODE)] + [B.gc_linear_workspace_bytes(self.plan, l, n) for l in (self.l1, self.l2, self.lo)])
        self.opt = B.distill_options(T, 1.0, ce, 1.0, tail=True)
        self.muon = B.muon_options(0.0, 0.02)

    def state(self):
        e = lambda c, d=self.dtype: torch.zeros(self.n, c, dtype=d, device="cuda")
        N = self.plan.n_total
        z = lambda: torch.zeros(N, device="cuda")
        return dict(w=self.w0.clone(), wt=torch.zeros(N, dtype=self.dtype, device="cuda"), e=e(self.E), z1=e(self.H), y1=e(self.H), h=e(self.E),
                    logits=e(self.V), idx=torch.zeros(self.n, self.k, dtype=torch.int32, device="cuda"), val=e(self.k, torch.float32),
                    lse=torch.zeros(self.n, device="cuda"), loss=torch.zeros(self.n, device="cuda"), dz=e(self.V), dh=e(self.E), dz1=e(self.H),
                    de=e(self.E), G=z(), U=z(), V=z(), M=z(), D=z(), msg=B.Sparse.empty(self.plan, self.plan.total_k, "cuda"))

    def gradients(self, s, ws):
        """The flat gradient of the sum of the rows' losses, in s["G"]."""
        s["wt"].copy_(s["w"])
        B.gc_embed_lookup(self.plan, 0, self.V, s["w"], self.tokens, 1.0, s["e"])
        B.gc_linear_forward(self.plan, self.l1, s["wt"], s["e"], s["y1"], ws, act=B.GC_ACT_GELU, z=s["z1"])
        B.gc_linear_forward(self.plan, self.l2, s["wt"], s["y1"], s["h"], ws, r=s["e"])
        B.gc_linear_forward(self.plan, self.lo, s["wt"], s["h"], s["logits"], ws)
        B.gc_top_logits(self.teacher, s["idx"], s["val"], s["lse"], temperature=self.T)
        B.gc_distill_loss(s["logits"], s["idx"], s["val"], self.opt, s["loss"], s["dz"], t_lse=s["lse"], labels=self.labels)
        B.gc_linear_grad_weight(self.plan, self.lo, s["dz"], s["h"], s["G"], False, ws)
        B.gc_linear_grad_input(self.plan, self.lo, s["wt"], s["dz"], s["dh"], ws)
        B.gc_linear_grad_weight(self.plan, self.l2, s["dh"], s["y1"], s["G"], False, ws)
        B.gc_linear_grad_input(self.plan, self.l2, s["wt"], s["dh"], None, ws, act=B.GC_ACT_GELU, z=s["z1"], dzx=s["dz1"])
        B.gc_linear_grad_weight(self.plan, self.l1, s["dz1"], s["e"], s["G"], False, ws)
        B.gc_linear_grad_input(self.plan, self.l1, s["wt"], s["dz1"], s["de"], ws, a=s["dh"])
        B.gc_embed_grad(self.plan, 0, self.V, s["de"], self.tokens, 1.0, s["G"], False, ws)

    def step(self, s, ws):
        self.gradients(s, ws)
        B.gc_dgc_step(self.plan, s["G"], s["U"], s["V"], 0.9, 0.0, 1, s["msg"], ws)
        B.gc_decompress_accumulate(self.plan, [s["msg"]], s["D"], B.GC_SUM, False, ws)
        B.gc_muon_step(self.mplan, s["D"], s["M"], s["w"], self.muon, ws)

    def reference(self):
        """Loss and flat gradient in 64 bits by autograd, on the CPU."""
        w = self.w0.double().cpu().requires_grad_(True)
        E, W1, b1, W2, Wo, bo = [p.view(*s) for p, s in zip(torch.split(w, self.lens), ((self.V, self.E), (self.H, self.E), (self.H,), (self.E, self.H), (self.V, self.E), (self.V,)))]
        t = self.tokens.cpu()
        ok = (t >= 0) & (t < self.V)
        e = E[torch.where(ok, t, 0)] * ok[:, None]
        z1 = e @ W1.T + b1
        h = e + act64(z1, "gelu")[0] @ W2.T
        z = h @ Wo.T + bo
        top, idx = torch.sort(self.teacher.double().cpu(), dim=1, descending=True, stable=True)
        lse = torch.logsumexp(top / self.T, 1, keepdim=True)
        q, idx = torch.exp(top[:, :self.k] / self.T - lse), idx[:, :self.k]
        held = 1 - q.sum(1)
        logp = torch.log_softmax(z / self.T, 1)
        inside = torch.zeros_like(logp, dtype=torch.bool).scatter_(1, idx, True)
        logr = torch.logsumexp(logp.masked_fill(inside, -float("inf")), 1)
        kl = (q * (q.log() - logp.gather(1, idx))).sum(1) + held * (held.log() - logr)
        lab = self.labels.long().cpu()
        nll = -torch.log_softmax(z, 1).gather(1, lab.clamp(min=0)[:, None])[:, 0]
        loss = self.T ** 2 * kl + self.ce * torch.where(lab >= 0, nll, 0.0 * nll)
        loss.sum().backward()
        return loss.detach(), w.grad


@pytest.mark.parametrize("dtype,rel", [
    # bf16 rounds e, y1, z1, h, the logits and five gradients by 2^-8 at most each, of which a handful follow one another
    # on any path, and W by the same; fp32 loses some 2^-20 a product.  In the 2-norm, of the whole gradient.
    (torch.float32, 2e-5), (torch.bfloat16, 12 * 2.0 ** -8)])
def test_a_students_gradient(dtype, rel):
    st = Student(900, 72, 200, 130, 24, dtype, 1)
    s = st.state()
    st.gradients(s, torch.full((st.need,), 0xFF, dtype=torch.uint8, device="cuda"))
    loss, grad = st.reference()
    got = s["G"].double().cpu()
    assert float((s["loss"].double().cpu() - loss).norm() / loss.norm()) < rel
    for part, want in zip(torch.split(got, st.lens), torch.split(grad, st.lens)):
        assert float((part - want).norm() / want.norm()) < rel
    # padding tokens' rows have no gradient, and rows without a token are 0
    used = torch.zeros(st.V, dtype=torch.bool)
    t = st.tokens.cpu()
    used[t[(t >= 0) & (t < st.V)]] = True
    assert bool((got[:st.V * st.E].view(st.V, st.E)[~used] == 0).all())


STUDENTS = [(300, 40, 64, 33, 8, torch.bfloat16, 11), (1000, 100, 300, 500, 40, torch.float32, 12), (5000, 64, 96, 7, 3, torch.float16, 13)]
KEPT = ("w", "logits", "loss", "G", "U", "V", "D", "idx", "val")


def same(a, b):
    for k in KEPT:
        assert torch.equal(a[k], b[k]), k


def test_two_graphs_that_share_a_workspace():
    sts = [Student(*a) for a in STUDENTS]
    ws = torch.full((max(t.need for t in sts),), 0xFF, dtype=torch.uint8, device="cuda")
    states, graphs = [t.state() for t in sts], []
    eager, own = [t.state() for t in sts], [torch.full((t.need,), 0xFF, dtype=torch.uint8, device="cuda") for t in sts]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i, (t, s) in enumerate(zip(sts, states)):
        say(f"capture of student {i}")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            t.step(s, ws)
        graphs.append(graph)
    for turn in range(3):
        for i, graph in enumerate(graphs):
            say(f"replay {turn} of student {i}")
            graph.replay()
        torch.cuda.synchronize()
        for t, s, w in zip(sts, eager, own):
            t.step(s, w)
        torch.cuda.synchronize()
        for a, b in zip(states, eager):
            same(a, b)
            assert bool(torch.isfinite(a["w"]).all()) and bool(torch.isfinite(a["loss"]).all())


def test_students_on_their_own_streams_and_threads():
    sts = [Student(*a) for a in STUDENTS]
    spaces = [torch.full((t.need,), 0xFF, dtype=torch.uint8, device="cuda") for t in sts]
    alone, streamed, threaded = ([t.state() for t in sts] for _ in range(3))
    torch.cuda.synchronize()
    for t, s, w in zip(sts, alone, spaces):
        for _ in range(2):
            t.step(s, w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sts]
    say("three students at once")
    for _ in range(2):
        for t, s, w, st in zip(sts, streamed, spaces, streams):
            with torch.cuda.stream(st):
                t.step(s, w)
    torch.cuda.synchronize()
    errors = []

    def work(t, s, w, st):
        try:
            with torch.cuda.stream(st):
                for _ in range(2):
                    t.step(s, w)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    say("three threads")
    threads = [threading.Thread(target=work, args=a) for a in zip(sts, threaded, spaces, streams)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert not errors
    for a, b, c in zip(alone, streamed, threaded):
        same(a, b)
        same(a, c)


def test_a_learning_student():
    """Some steps run, and stay finite; how far the loss falls is not the kernels' matter."""
    st = Student(400, 48, 96, 64, 16, torch.bfloat16, 21)
    s, ws = st.state(), torch.empty(st.need, dtype=torch.uint8, device="cuda")
    for _ in range(5):
        st.step(s, ws)
        s["w"][:st.lens[0]] -= 0.1 * s["D"][:st.lens[0]]
    assert bool(torch.isfinite(s["loss"]).all()) and bool(torch.isfinite(s["w"]).all())
