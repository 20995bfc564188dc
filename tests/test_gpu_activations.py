"""GPU: GELU, SiLU and their slopes relative to their own size, also in the
negative tail, where an absolute tolerance would pass zeros.

Counted in half steps of fp32 (2^-24): Phi's polynomial is fitted to 1.6, its
argument is off by 3.5 (a reciprocal of one unit, a multiply-add, a constant),
which its slope d ln P / d ln t raises 3.4 times at most, 8 steps of Horner's
scheme add about 6, the exponential 3.5, products 3: below 32.  The sigmoid:
exponential 3.5, sum 1, reciprocal 2, product 1: below 16.  bf16 forms its
exponents without compensation, 8e-6 at the far end, and is rounded to 2^-9."""

import math

import pytest
import torch

import learn_ref as ref
import weighted_model_update_amd as fa

pytestmark = pytest.mark.gpu


def points(t, low, high):
    z = torch.cat([torch.linspace(low, high, 40001), -torch.logspace(-6, math.log10(-low), 5000), torch.zeros(1)])
    return z.to(t)


def phi(z):
    return 0.5 * torch.erfc(-z / math.sqrt(2))


def forward(z, act):
    return fa.linear_forward(z.cuda()[:, None], torch.ones(1, 1, dtype=z.dtype, device="cuda"), act=act)[:, 0]


def slope(z, act):
    one = torch.ones(1, 1, dtype=z.dtype, device="cuda")
    zc = z.cuda()[:, None].contiguous()
    return fa.linear_backward(torch.ones_like(zc), torch.ones_like(zc), one, act=act, preact=zc, dx=True, dw=None)[0][:, 0]


def steps(t, n):
    return n * ref.U32 if t == torch.float32 else 140 * ref.U32


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_gelu_and_its_slope(t):
    z = points(t, -13.0, 13.0)
    d = ref.d(z)
    want = d * phi(d)
    ref.within(forward(z, "gelu"), want, steps(t, 32) * want.abs(), t, "gelu")
    dens = torch.exp(-d * d / 2) / math.sqrt(2 * math.pi)
    ref.within(slope(z, "gelu"), phi(d) + d * dens, steps(t, 32) * (phi(d) + d.abs() * dens), t, "slope")


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_silu_and_its_slope(t):
    z = points(t, -87.0, 87.0)
    d = ref.d(z)
    s = torch.sigmoid(d)
    ref.within(forward(z, "silu"), d * s, steps(t, 16) * (d * s).abs(), t, "silu")
    # 1 - s is off by what s is
    ref.within(slope(z, "silu"), s + d * s * (1 - s), (steps(t, 24) + steps(t, 12) * d.abs()) * s, t, "slope")


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_far_ends(t):
    inf, big = float("inf"), torch.finfo(t).max
    z = torch.tensor([inf, big, 1e30, 300.0, 1e4, 0.0, -300.0, -1e4, -1e30, -big, float("nan")]).to(t)
    for act in ("gelu", "silu"):
        y = forward(z, act).cpu()
        assert torch.equal(y[:5], z[:5]) and bool((y[5:10] == 0).all()) and bool(torch.isnan(y[10]))
        g = slope(z, act).cpu()
        assert bool((g[1:5] == 1).all()) and float(g[5]) == 0.5 and bool((g[6:10] == 0).all()) and bool(torch.isnan(g[10]))
