"""The distillation loss at widths around every change of its variant, with rows
at every distance from 16 bytes: against 64 bits, with guards behind each row.

Bounds (those of the tests of other sizes): an exponential of d = (z - max) / T
costs at most (|d| + 4) 2^-23 of itself, a sum of its terms 600 2^-24 of itself,
a logarithm 4 steps; so a probability is off by (|d| + 1000) 2^-23 of itself, a
teacher's (|t / T - lse| <= 130) by 1130 2^-23, and log p by 1000 2^-23 + |d| 2^-22."""
import pytest
import torch

from gradient_compression_dnn_amd import binding as B
from tests.gpu_util import say
from tests.layer_util import DTYPES, U32, Rows, half_step
from tests.test_gpu_distill import Case, reference

pytestmark = pytest.mark.gpu

EQ, ELOG = 1130 * 2.0 ** -23, 1000 * 2.0 ** -23


def bounds(z, c, T, kd, ce, rest, w, scale, want_l, want_g, dtype):
    """What the loss and the gradient may be off by, of entries that name a column once."""
    d = z.amax(1, keepdim=True) - z
    vocab = z.shape[1]
    deepest = torch.gather(d, 1, c.idx.t.long().clamp(0, vocab - 1)).amax(1)
    lab_d = torch.gather(d, 1, c.labels.long().clamp(0, vocab - 1)[:, None])[:, 0]
    loss = w * (kd * T * T * 2 * ((EQ + ELOG) * (170 + deepest / T) + deepest / T * 2.0 ** -21) + ce * (ELOG + lab_d * 2.0 ** -21)) + 8 * U32 * want_l.abs()
    ep = lambda x: (x + 1000) * 2.0 ** -23
    named = torch.zeros_like(z).scatter_add_(1, c.idx.t.long().clamp(0, vocab - 1), torch.ones_like(c.t.f64()))
    room = kd * T * (2 * torch.softmax(z / T, 1) * (ep(d / T) + 2 * EQ) + 2 * EQ * named) + ce * (torch.softmax(z, 1) * ep(d) + 4 * U32)
    if rest:  # the softmax over the rest, at its own maximum, times a mass of at most 1
        lr = torch.where(named > 0, torch.full_like(z, -float("inf")), z / T)
        pr = torch.softmax(lr, 1)
        room = room + kd * T * pr * (ep(torch.where(named > 0, torch.zeros_like(z), lr.amax(1, keepdim=True) - lr)) + 2 * EQ)
    room = (w * scale)[:, None] * room
    return loss, room + half_step(dtype) * (want_g.abs() + room) + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps


@pytest.mark.parametrize("vectors", [256 * 4, 256 * 8, 256 * 16, 512 * 16])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_widths_around_a_change_of_variant(dtype, vectors):
    D = DTYPES[dtype]
    N = 16 // D.itemsize
    n, k, kd, scale = 9, 5, 0.8, 64.0
    for vocab in sorted({vectors * N + o for o in (-2 * N + 1, -N, -N + 1, -N + 2, -1, 0, 1, 2, N)}):
        for pitch, T, rest, ce in ((0, 1.0, False, 0.0), (3, 2.0, True, 0.5)):
            say(f"distill widths {dtype} {vocab} pitch={pitch}")
            c = Case(n, vocab, k, dtype, "normal", T, vocab % 97, pitch=pitch)
            c.z.t[:, :N] += 15.0  # what stands behind the row before would count
            labels, tlse = c.labels if ce else None, c.tlse if rest else None
            opt = B.distill_options(T, kd, ce, scale, tail=rest)
            kw = dict(t_lse=tlse, labels=labels)
            loss, dz = torch.full((n,), 7.0, device="cuda"), Rows(n, vocab, D, pitch)
            B.gc_distill_loss(c.z.t, c.idx.t, c.t.t, opt, loss, dz.t, **kw)
            want_l, want_g = reference(c.z.f64(), c.idx.t, c.t.f64(), T, kd, ce, scale, rest, tlse, labels, None)
            w = torch.ones(n, dtype=torch.float64, device="cuda")
            room_l, room_g = bounds(c.z.f64(), c, T, kd, ce, rest, w, scale, want_l, want_g, D)
            assert bool(((loss.double() - want_l).abs() <= room_l).all()), (loss, want_l, room_l)
            off = (dz.f64() - want_g).abs()
            assert bool((off <= room_g).all()), float((off / room_g).max())
            assert dz.guards_kept() and c.z.guards_kept()
            # the loss alone, and in place of the logits: the same bits
            loss2 = torch.zeros_like(loss)
            B.gc_distill_loss(c.z.t, c.idx.t, c.t.t, opt, loss2, None, **kw)
            assert torch.equal(loss, loss2)
            B.gc_distill_loss(c.z.t, c.idx.t, c.t.t, opt, loss2, c.z.t, **kw)
            assert torch.equal(c.z.t, dz.t) and torch.equal(loss, loss2) and c.z.guards_kept()
