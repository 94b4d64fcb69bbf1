"""The top logits of rows that hold very low finite logits, as masks of the
type's lowest value are: those are candidates as any other, exactly, however few
columns are left beside them."""
import pytest
import torch

from gradient_compression_dnn_amd import binding as B
from tests.gpu_util import say
from tests.layer_util import DTYPES, Rows
from tests.test_gpu_distill import SIZES, logits

pytestmark = pytest.mark.gpu

INF = float("inf")


def check(z, k):
    n = z.n
    idx, val = torch.full((n, k), -7, dtype=torch.int32, device="cuda"), torch.full((n, k), 7.0, device="cuda")
    B.gc_top_logits(z.t, idx, val)
    v = z.f64() + 0.0
    v = torch.where(torch.isnan(v), torch.full_like(v, -INF), v)
    s, j = torch.sort(v, dim=1, descending=True, stable=True)
    pad = max(0, k - s.shape[1])
    s, j = torch.nn.functional.pad(s, (0, pad), value=-INF)[:, :k], torch.nn.functional.pad(j, (0, pad))[:, :k]
    assert torch.equal(idx, torch.where(s > -INF, j, -1).int())
    assert torch.equal(val.double(), torch.where(s > -INF, torch.gather(z.f64(), 1, j), s)) and z.guards_kept()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,vocab,k", SIZES)
def test_lowest_values_in_every_fifth_column(n, vocab, k, dtype):
    for pitch in (0, 5):
        say(f"top wide {n}x{vocab} k={k} {dtype} pitch={pitch}")
        check(logits(n, vocab, dtype, "wide", pitch, 3), k)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab,k", [(32, 32), (32, 40), (33, 9), (70, 70), (1000, 256), (1000, 1000), (4097, 700), (20001, 1024)])
def test_fewer_than_k_columns_beside_low_ones(vocab, k, dtype):
    """k entries of a row whose vectors are fewer than k: nothing bounds them."""
    D = DTYPES[dtype]
    lowest = torch.finfo(D).min
    for mask in (lowest, lowest / 2, lowest / 512, -1e4):
        for keep in (0, 1, 3, max(1, min(k, vocab) - 3), vocab - min(3, vocab)):
            say(f"top low {vocab} k={k} {dtype} mask={mask} keep={keep}")
            g = torch.Generator(device="cuda").manual_seed(vocab + keep)
            n = 4
            z = torch.full((n, vocab), mask, dtype=torch.float64, device="cuda")
            where = torch.rand(n, vocab, generator=g, device="cuda").argsort(1)[:, :keep]
            z.scatter_(1, where, torch.randn(n, keep, generator=g, device="cuda").double())
            z[1, ::7] = -INF
            z[2, ::3] = float("nan")
            check(Rows(n, vocab, D, 3, z), k)


def test_three_lowest_logits_of_a_short_row():
    z = torch.arange(32, device="cuda").float().repeat(2, 1)
    z[0, [3, 13, 30]] = -1e36
    z[1, [3, 13, 30]] = torch.finfo(torch.float32).min
    idx, val = torch.empty(2, 32, dtype=torch.int32, device="cuda"), torch.empty(2, 32, device="cuda")
    B.gc_top_logits(z, idx, val)
    assert idx[:, 29:].tolist() == [[3, 13, 30]] * 2 and torch.equal(val, z.sort(1, descending=True).values)
