"""Rows that count, whose entries' own terms are all 0: the teacher's mass lies
outside of them (GC_DISTILL_REST), or nowhere that the student can take it."""
import pytest
import torch

from gradient_compression_dnn_amd import binding as B
from tests.gpu_util import say
from tests.layer_util import DTYPES

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1.0, 2.0])
def test_no_finite_loss_without_a_distribution(dtype, T):
    """q = exp(t / T - t_lse) below every float.  A row with NaN or +Inf, or of nothing but masked columns, has loss
    and gradient NaN all the same; where the entries name every column that is not masked, no mass is left to hold: 0."""
    V = 40
    z = torch.zeros(7, V)
    z[:, 2:] += torch.arange(V - 2) / 8
    z[0] = -INF                    # nothing to choose from
    z[1, 1], z[2, 30], z[3, 0] = float("nan"), float("nan"), INF
    z[4, 2:] = -INF                # the entries name all that is left
    z[5, 2:], z[5, 1] = -INF, float("nan")
    z = z.to(DTYPES[dtype]).cuda()
    idx = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda").repeat(7, 1)
    t, tlse = torch.tensor([[1.0, 0.5]], device="cuda").repeat(7, 1), torch.full((7,), 500.0, device="cuda")
    for ce in (0.0, 0.5):
        say(f"distill rest {dtype} T={T} ce={ce}")
        labels = torch.ones(7, dtype=torch.int32, device="cuda") if ce else None
        loss, dz = torch.full((7,), 9.0, device="cuda"), torch.full_like(z, 9.0)
        B.gc_distill_loss(z, idx, t, B.distill_options(T, 1.0, ce, 1.0, tail=True), loss, dz, t_lse=tlse, labels=labels)
        nan = torch.tensor([0, 1, 2, 3, 5], device="cuda")
        assert bool(torch.isnan(loss[nan]).all()) and bool(torch.isnan(dz[nan]).all())
        assert bool(torch.isfinite(loss[[4, 6]]).all()) and bool(torch.isfinite(dz[[4, 6]]).all())
        if not ce:
            assert float(loss[4]) == 0.0 and bool((dz[4] == 0).all())
        # all of the teacher's mass on the rest: -T^2 log p_r, and the gradient T (p - p_r's softmax)
        z6 = z[6].double()
        logp, log1 = torch.log_softmax(z6 / T, 0), torch.log_softmax(z6, 0)
        want = -T * T * torch.logsumexp(logp[2:], 0) - ce * log1[1]
        g = T * logp.exp() + ce * log1.exp()
        g[2:] -= T * torch.softmax(z6[2:] / T, 0)
        g[1] -= ce
        # a probability is off by (|d| + 1000) 2^-23 of itself with |d| <= 5, a logarithm of one by 1000 2^-23 and |d| 2^-22
        room = (T * T + ce) * 1100 * 2.0 ** -23
        assert abs(float(loss[6]) - float(want)) <= room
        bound = 3 * (T + ce) * 1100 * 2.0 ** -23
        bound = bound + torch.finfo(z.dtype).eps / 2 * (g.abs() + bound)
        assert bool(((dz[6].double() - g).abs() <= bound).all())
