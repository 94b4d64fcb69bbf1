"""What the scalars of a row cost: rows whose sums of exponentials are exact (equal
logits, up to 2^20 of them), so that the logarithms and what they are combined
with are all that is left.

A logarithm is log(m) + e log 2 with m in [0.70, 1.42): the function is within 2
steps of a value below 0.35, 2^-24, and the rest is formed in double."""
import math

import pytest
import torch

from gradient_compression_dnn_amd import binding as B
from tests.gpu_util import say
from tests.layer_util import DTYPES, U32
from tests.test_gpu_distill import reference

pytestmark = pytest.mark.gpu

WIDTHS = [3, 70, 1001, 1777, 5000, 12345, 20011, 50021, 65535, 99991, 131071, 262145, 1000003]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1.0, 3.0, 0.7])
def test_log_sum_exp_of_equal_logits(dtype, T):
    """z / T + log V, rounded once: half a step, and the logarithm's 2^-24."""
    for V in WIDTHS:
        say(f"lse {dtype} V={V} T={T}")
        z = torch.tensor([0.0, 1.375, -7.53125, 25.25, -63.5], device="cuda").to(DTYPES[dtype])[:, None].expand(5, V).contiguous()
        idx, val, lse = torch.zeros(5, 1, dtype=torch.int32, device="cuda"), torch.zeros(5, 1, device="cuda"), torch.zeros(5, device="cuda")
        B.gc_top_logits(z, idx, val, lse, temperature=T)
        want = z[:, 0].double() / float(torch.tensor(T)) + math.log(V)
        room = U32 + U32 * (want.abs() + U32)  # half a step is 2^-24 of the value at most
        assert bool(((lse.double() - want).abs() <= room).all()), (V, (lse.double() - want).abs() / room)


@pytest.mark.parametrize("T", [1.0, 8.0, 3.0])
def test_a_student_close_to_its_teacher(T):
    """Both nearly uniform over the row: KL is small beside its terms, which are as large as log V.  The logarithms of the
    row's sum, of the rest's and of the mass held cost 2^-24 each, that mass' rounding as much; the entries' q, off by
    6e-7 of themselves, weigh k / V, times terms that differ by 0.1 at most."""
    k, n = 8, 16
    for V in WIDTHS[2:]:
        say(f"close V={V} T={T}")
        z = torch.full((n, V), 2.5, device="cuda")
        g = torch.Generator(device="cuda").manual_seed(V)
        idx = torch.randint(0, V // k, (n, k), generator=g, device="cuda", dtype=torch.int32) + torch.arange(k, device="cuda", dtype=torch.int32) * (V // k)
        t = torch.full((n, k), 0.75, device="cuda")
        tlse = (0.75 / T + math.log(V) + 0.1 * (torch.rand(n, generator=g, device="cuda") - 0.5)).float()
        loss = torch.zeros(n, device="cuda")
        B.gc_distill_loss(z, idx, t, B.distill_options(T, tail=True), loss, t_lse=tlse)
        want, _ = reference(z.double(), idx, t.double(), T, 1.0, 0.0, 1.0, True, tlse.double(), None, None)
        room = T * T * (4 * U32 + k / V * 0.1 * 7e-7 + 2 * k / V * U32 * 20) + U32 * want.abs()
        assert bool(((loss.double() - want).abs() <= room).all()), (V, float(((loss.double() - want).abs() / room).max()))


def test_labels_of_equal_logits():
    """log V, whatever the logits are: the logarithm's 2^-24 and one rounding."""
    for V in WIDTHS:
        z = torch.full((3, V), 17.25, device="cuda")
        labels = torch.tensor([0, V // 2, V - 1], device="cuda")
        idx, t = torch.empty(3, 0, dtype=torch.int64, device="cuda"), torch.empty(3, 0, device="cuda")
        for T in (1.0, 2.0):
            loss = torch.zeros(3, device="cuda")
            B.gc_distill_loss(z, idx, t, B.distill_options(T, 1.0, 1.0), loss, labels=labels)
            assert bool(((loss.double() - math.log(V)).abs() <= U32 + U32 * math.log(V) * (1 + U32)).all()), V
