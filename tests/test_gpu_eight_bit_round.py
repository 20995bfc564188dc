"""GPU: the example of federated rounds with 8-bit frozen layers and an
orthogonalised server step runs and repeats itself; its gradients agree with a
float64 autograd, its server step with the formulas."""

import os
import sys

import pytest
import torch

import learn_ref as ref
import weighted_model_update_amd as fa
from test_gpu_orthogonal import QUINTIC, formula

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import eight_bit_round as ex  # noqa: E402

pytestmark = pytest.mark.gpu


def test_the_rounds_run_and_repeat():
    kw = dict(blocks=2, hidden=96, rank=8, tokens=50, clients=3, rounds=2, steps=2)
    weights, server, _ = ex.run(**kw)
    again, server2, _ = ex.run(**kw)
    assert torch.equal(server.flat, server2.flat)
    for a, b in zip(weights, again):
        assert all(torch.equal(s, t) for s, t in zip(a, b)) and bool(a[2].isfinite().all())


def rnd(shape, seed, scale, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def values(q, s):
    return ref.d(q) * ref.d(s)[:, None]


def through_8_bits(x):
    """x as the call's own 8 bits hold it, with the gradient of the identity."""
    q, s = fa.quantize_rows(x.detach().to(torch.bfloat16).cuda())
    return x + (values(q, s) - x).detach()


def test_the_gradient_of_the_chain():
    """Two blocks against float64 autograd on the same 8-bit weights.  Every
    intermediate is rounded to bf16 (2^-8 at most, 2^-8 / sqrt(3) in the norm),
    and a token's 8 bits move by a step of 1 / 127 of its largest value where
    such a rounding carries it over a tie, which for values spread as here is
    1 / 127 / sqrt(12) of three standard deviations, 0.7%, of all values at most;
    a dozen of the former and four of the latter enter the first block's
    gradients, whose slopes amplify them by less than two."""
    blocks, hidden, rank, tokens = 2, 64, 8, 40
    frozen = [ex.Frozen(rnd((4 * hidden, hidden), 10 * i, hidden ** -0.5, torch.float32), rnd((4 * hidden,), 10 * i + 1, 0.1),
                        rnd((hidden, 4 * hidden), 10 * i + 2, 0.5 * (4 * hidden) ** -0.5, torch.float32)) for i in range(blocks)]
    a, grad = ex.Adapters(blocks, hidden, rank, torch.bfloat16), ex.Adapters(blocks, hidden, rank, torch.bfloat16)
    a.flat.copy_(rnd(a.flat.shape, 77, 0.1))
    x, dy = rnd((tokens, hidden), 78, 1.0), rnd((tokens, hidden), 79, 1.0)
    y, saved = ex.forward(frozen, a, x)
    dx = ex.backward(dy, frozen, a, saved, grad)

    x64 = ref.d(x).requires_grad_()
    down, up = (ref.d(t).requires_grad_() for t in (a.down, a.up))
    v = x64
    for i, f in enumerate(frozen):
        h = ref.act(through_8_bits(v) @ values(f.q1, f.s1).t() + ref.d(f.b1), "gelu")
        v = v + through_8_bits(h) @ values(f.q2, f.s2).t() + (h @ down[i].t()) @ up[i].t()
    (v * ref.d(dy)).sum().backward()
    tol = 2 * (12 * 2.0 ** -8 / 3 ** 0.5 + 4 * 0.007)
    for got, want in ((y, v.detach()), (dx, x64.grad), (grad.down, down.grad), (grad.up, up.grad)):
        off = float((ref.d(got) - want).norm() / want.norm())
        assert off < tol, off


def test_the_server_step():
    sizes = (3, 48, 16)
    server, momentum = (ex.Adapters(*sizes, torch.float32) for _ in range(2))
    server.flat.copy_(rnd(server.flat.shape, 1, 0.1, torch.float32))
    momentum.flat.copy_(rnd(server.flat.shape, 2, 1e-3, torch.float32))
    weights = [(None, None, rnd((48, 192), 3 + i, 0.1, torch.float32)) for i in range(3)]
    before, m0, s0 = [ref.d(w[2]) for w in weights], ref.d(momentum.flat), ref.d(server.flat)
    sent, n = [rnd(server.flat.shape, 10 + c, 1e-3, torch.float32) for c in range(3)], [5, 7, 9]
    ex.server_step(weights, server, momentum, sent, n, 0.02)

    mean = sum(k * ref.d(t) for k, t in zip(n, sent)) / sum(n)
    beta = float(torch.tensor(0.95))
    m = beta * m0 + mean
    t = mean + beta * m
    # The mean is a sum of products w_k t_k with w_k = n_k / sum n rounded (1 half
    # step, 2 if by a reciprocal) and three roundings of partial sums, each of which
    # is at most S = sum w_k |t_k|: off by (2 + 3) half steps of S, which where the
    # t_k cancel is more than any number of half steps of the mean itself.  beta m is
    # rounded once more, the sum is `within`'s own.
    spread = sum(k * ref.d(t).abs() for k, t in zip(n, sent)) / sum(n)
    ref.within(momentum.flat, m, ref.U32 * (5 * spread + m0.abs()), torch.float32, "momentum")
    want = ex.Adapters(*sizes, torch.float64, (s0 * 1.0).cuda())
    arg = ex.Adapters(*sizes, torch.float64, t.cuda())
    for w, u in ((want.down, arg.down), (want.up, arg.up)):
        w += 0.02 * formula(u, QUINTIC, 5, torch.float64)
    # three roundings of the argument, which the steps enlarge by at most 4 each
    slack = 0.02 * 3 * ref.U32 * 4.0 ** 5 + 4 * ref.U32
    assert float((ref.d(server.down) - want.down.cpu()).abs().max()) < slack
    assert bool((server.up == 0).all())
    for w, b, down, up in zip(weights, before, want.down.cpu(), want.up.cpu()):
        prod = up @ down
        off = (ref.d(w[2]) - (b + prod)).abs().max()
        assert float(off) < slack * float(down.abs().sum(0).max() + up.abs().sum(1).max()) + 32 * ref.U32
    # and into 8 bits: every weight within half a step of its row's scale
    for w in weights:
        q, s = fa.quantize_rows(w[2])
        assert bool(((values(q, s) - ref.d(w[2])).abs() <= ref.d(s)[:, None] * 0.5001).all())
