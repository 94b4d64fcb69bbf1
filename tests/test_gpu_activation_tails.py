"""The activations and their slopes relative to themselves, far into the tail where
an absolute bound says nothing: every output is a value within the stated error of
the formula's, rounded once.

Bounds.  With a the exponent that the formula forms (z^2 / 2, |2 u| or |z|), the
relative errors of its roundings, at most 6 of 2^-24 and as many of constants and
of the scaling to base 2, come out of the exponential a times as large: 4 a 2^-23.
The exponential, erfc (16 steps), the reciprocal, the sums and products add 20
2^-23, the 16-bit types' Phi 2^-16.8.  An exponential or a quotient below 2^-126 may
be 0, which stands beside |z| <= 90: 2^-119.  A slope is a sum of two terms and is
off by that part of their sizes."""
import math

import pytest
import torch

from gradient_compression_dnn_amd import binding as B
from tests.gpu_util import say
from tests.layer_util import ACTS, DTYPES, Layer, act64, half_step

pytestmark = pytest.mark.gpu

FAST = 2.0 ** -16.8


def relative(z, act, dtype):
    """The error of act, as a part of it."""
    c = 2 * math.sqrt(2 / math.pi)
    a = {"gelu": z * z / 2, "gelu_tanh": (c * (z + 0.044715 * z ** 3)).abs(), "silu": z.abs()}[act].clamp(max=128.0)
    return (4 * a + 20) * 2.0 ** -23 + (FAST if act == "gelu" and dtype is not torch.float32 else 0.0)


def sizes(z, act):
    """The sizes of the slope's two terms."""
    if act == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z.abs() * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    v, d = (z, 1.0) if act == "silu" else (2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3), 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z))
    s = torch.sigmoid(v)
    return s + z.abs() * s * torch.sigmoid(-v) * d


def points(dtype):
    z = torch.cat([torch.linspace(-16, 16, 6143, dtype=torch.float64), torch.linspace(-100, -10, 1500, dtype=torch.float64),
                   torch.tensor([0.0, -0.0, 1e-6, -1e-6, 30.0, 100.0, -5.5, -6.0, -8.0, -10.0], dtype=torch.float64)])
    z = torch.cat([z, torch.zeros(-z.numel() % 128, dtype=torch.float64)])
    return z.to(dtype).cuda().view(-1, 128)


def within(got, want, err, dtype, what, z):
    off = (got.double() - want).abs()
    room = err + half_step(dtype) * (want.abs() + err) + torch.finfo(dtype).smallest_normal * half_step(dtype) + 2.0 ** -119
    bad = ~(off <= room)
    assert not bad.any(), f"{what}: {int(bad.sum())} off, by up to {float((off / room)[bad].max())} of the bound, at {float(z[bad][0])}"


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_relative_to_themselves(act, dtype):
    D = DTYPES[dtype]
    z = points(D)
    z64 = z.double()
    say(f"tails {act} {dtype}")
    want, slope = act64(z64, act)
    # y = act(z) through a layer whose matrix is the identity, few tokens and many
    L = Layer(128, 128, dtype, 0, False)
    L.weights().copy_(torch.eye(128))
    for n in (3, z.shape[0]):
        y = torch.empty_like(z[:n])
        B.gc_linear_forward(L.plan, L.layer, L.w, z[:n], y, L.ws(n), act=ACTS[act])
        within(y, want[:n], relative(z64[:n], act, D) * want[:n].abs(), D, "act", z[:n])
    err = relative(z64, act, D) * sizes(z64, act)
    one, dz, dzx = torch.ones_like(z), torch.empty_like(z), torch.empty_like(z)
    B.gc_act_grad(one, z, ACTS[act], dz)
    within(dz, slope, err, D, "slope", z)
    B.gc_linear_grad_input(L.plan, L.layer, L.w, one, None, L.ws(z.shape[0]), act=ACTS[act], z=z, dzx=dzx)
    assert torch.equal(dz, dzx)


@pytest.mark.parametrize("act", ["gelu_tanh", "silu"])
def test_slopes_where_the_sigmoid_is_nearly_1(act):
    """s + z s (1 - s) d in fp32: 1 - s keeps its relative precision, so the two terms cost 16 roundings of themselves,
    and the exponent's error, 4 a 2^-23, what it changes: s (1 - s) (1 + |z| d)."""
    z = torch.linspace(-20, 20, 1 << 14, dtype=torch.float64).float().cuda().view(128, 128)
    z64 = z.double()
    v, d = (z64, 1.0) if act == "silu" else (2 * math.sqrt(2 / math.pi) * (z64 + 0.044715 * z64 ** 3), 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z64 * z64))
    s, rest = torch.sigmoid(v), torch.sigmoid(-v)
    want = s + z64 * s * rest * d
    assert float((act64(z64, act)[1] - want).abs().max()) < 1e-12
    room = 16 * 2.0 ** -24 * (s + z64.abs() * s * rest * d) + 4 * v.abs().clamp(max=128.0) * 2.0 ** -23 * s * rest * (1 + z64.abs() * d) + 2.0 ** -119
    dz = torch.empty_like(z)
    say(f"slopes {act}")
    B.gc_act_grad(torch.ones_like(z), z, ACTS[act], dz)
    off = (dz.double() - want).abs()
    assert bool((off <= room).all()), float((off / room).max())
