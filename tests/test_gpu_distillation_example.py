"""GPU: the example round (clients' adapters and top logits, the server's
average and distillation) runs, learns, and its first gradient agrees with a
float64 autograd of the same round."""

import os
import sys

import pytest
import torch

import learn_ref as ref
import weighted_model_update_amd as fa

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import federated_distillation as ex  # noqa: E402

pytestmark = pytest.mark.gpu


def test_the_round_learns_and_repeats():
    kw = dict(tokens=96, vocab=1000, hidden=256, rank=16, clients=3, k=20, steps=15)
    server, losses, token = ex.run(**kw)
    assert all(l == l and l > 0 for l in losses)
    assert losses[-1] < 0.8 * losses[0]
    assert 0 <= int(token) < 1000
    again, losses2, token2 = ex.run(**kw)
    assert losses == losses2 and torch.equal(again.flat, server.flat) and int(token) == int(token2)


def test_the_gradient_of_the_chain():
    """Adapter, head and loss chained, against float64 autograd on the same
    bf16 weights.  Every intermediate is rounded to bf16 (half a step of 2^-8
    each: h, y, z, dz, dy, dh and the gradient itself), so the chain is off by
    about 7 half steps relative to the gradient's norm; three times that
    covers what the layers amplify."""
    hidden, rank, tokens, vocab, k, tau = 128, 16, 64, 500, 20, 2.0
    g = torch.Generator().manual_seed(3)

    def rnd(*shape, scale):
        return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16).cuda()

    x, head = rnd(tokens, hidden, scale=1.0), rnd(vocab, hidden, scale=hidden ** -0.5)
    a, grad = ex.Adapter(hidden, rank), ex.Adapter(hidden, rank)
    a.down.copy_(rnd(rank, hidden, scale=hidden ** -0.5)); a.up.copy_(rnd(hidden, rank, scale=rank ** -0.5))
    a.b1.copy_(rnd(rank, scale=0.3)); a.b2.copy_(rnd(hidden, scale=0.3))
    sent = [fa.logits_topk(rnd(tokens, vocab, scale=2.0), k, tau=tau) for _ in range(2)]
    n = [3, 5]
    y, saved = a.forward(x)
    z = fa.linear_forward(y, head)
    loss, _, dz = fa.distill_loss(z, [s[0] for s in sent], [s[1] for s in sent], n, tau=tau, dz=True)
    dy, _, _ = fa.linear_backward(dz, y, head, dw=None)
    a.backward(dy, saved, grad)

    w = {name: ref.d(getattr(a, name)).requires_grad_() for name in ("down", "b1", "up", "b2")}
    x64 = ref.d(x)
    h64 = ref.act(x64 @ w["down"].t() + w["b1"], "gelu")
    z64 = (h64 @ w["up"].t() + w["b2"] + x64) @ ref.d(head).t()
    logp = torch.log_softmax(z64 / tau, 1)
    want = 0
    for (i, v, _), nc in zip(sent, n):
        lq = torch.log_softmax(ref.d(v) / tau, 1)
        want = want + nc / sum(n) * tau ** 2 * (lq.exp() * (lq - logp.gather(1, i.cpu().long()))).sum()
    want.backward()
    for name, t in w.items():
        got = ref.d(getattr(grad, name))
        off = float((got - t.grad).norm() / t.grad.norm())
        assert off < 3 * 7 * 2.0 ** -8, (name, off)
    want = float(want.detach())
    assert abs(float(loss.sum()) - want) < 3 * 3 * 2.0 ** -8 * want
