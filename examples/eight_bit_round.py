"""Federated rounds with frozen layers in 8 bits and an orthogonalised server step.

The model is a stack of residual blocks.  Each is a frozen two-layer network, which
clients hold in 8 bits, with a trainable low-rank adapter on its second layer:

    h = gelu(x W1^T + b1)                           linear_int8_forward
    y = x + h W2^T + (h down^T) up^T                linear_int8_forward, linear_forward
    backwards through all of it                     linear_int8_backward, linear_backward

Clients train their adapters and send the difference.  The server averages the
differences by sample count (fedavg_aggregate), steps its fp32 adapters with the
orthogonalised average and its momentum (orthogonal_step), adds them to its frozen
weights, W2 + up down, and brings these to 8 bits for the next round
(quantize_rows).

Run: python examples/eight_bit_round.py [--blocks 2 --hidden 512 ...]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import weighted_model_update_amd as fa  # noqa: E402


class Adapters:
    """down [rank, 4 hidden] and up [hidden, rank] of every block as views of
    one flat vector, which is what travels."""

    def __init__(self, blocks, hidden, rank, dtype, flat=None):
        self.sizes = (blocks, hidden, rank)
        n = hidden * rank
        self.flat = torch.zeros(blocks * 5 * n, dtype=dtype, device="cuda") if flat is None else flat
        both = self.flat.view(blocks, 5 * n)
        self.down, self.up = both[:, :4 * n].view(blocks, rank, 4 * hidden), both[:, 4 * n:].view(blocks, hidden, rank)


class Frozen:
    """One block's frozen layers in 8 bits."""

    def __init__(self, w1, b1, w2):
        self.q1, self.s1 = fa.quantize_rows(w1)
        self.q2, self.s2 = fa.quantize_rows(w2)
        self.b1 = b1


def forward(frozen, adapters, x):
    saved = []
    for f, down, up in zip(frozen, adapters.down, adapters.up):
        pre = torch.empty(x.shape[0], f.q1.shape[0], dtype=x.dtype, device=x.device)
        h = fa.linear_int8_forward(x, f.q1, f.s1, f.b1, act="gelu", preact=pre)
        y = fa.linear_int8_forward(h, f.q2, f.s2, residual=x)
        low = fa.linear_forward(h, down)
        x = fa.linear_forward(low, up, residual=y, out=y)
        saved.append((pre, h, low))
    return x, saved


def backward(dy, frozen, adapters, saved, grad):
    """Writes the adapters' gradients into `grad`; returns the input's."""
    for i in reversed(range(len(frozen))):
        f, (pre, h, low) = frozen[i], saved[i]
        dlow, _, _ = fa.linear_backward(dy, low, adapters.up[i], dw=grad.up[i])
        dh, _, _ = fa.linear_backward(dlow, h, adapters.down[i], dw=grad.down[i])
        dh += fa.linear_int8_backward(dy, f.q2, f.s2)[0]
        dy = dy + fa.linear_int8_backward(dh, f.q1, f.s1, act="gelu", preact=pre)[0]
    return dy


def client(frozen, start, x, target, steps, lr):
    """The difference that a client's training makes to the adapters, in fp32."""
    master = start.flat.clone()
    local, grad = Adapters(*start.sizes, x.dtype), Adapters(*start.sizes, x.dtype)
    for _ in range(steps):
        local.flat.copy_(master)
        y, saved = forward(frozen, local, x)
        backward((y - target) / x.shape[0], frozen, local, saved, grad)
        master.sub_(grad.flat.float(), alpha=lr)
    return master - start.flat


def server_step(weights, server, momentum, sent, n, rate):
    """The averaged difference, orthogonalised, into the adapters, and these
    into the frozen weights; `up` starts the next round at zero."""
    update = Adapters(*server.sizes, torch.float32)
    fa.fedavg_aggregate(sent, n, update.flat)
    fa.orthogonal_step(server.down, update.down, rate, momentum=momentum.down)
    fa.orthogonal_step(server.up, update.up, rate, momentum=momentum.up)
    for (_, _, w2), down, up in zip(weights, server.down, server.up):
        fa.linear_forward(up, down.t().contiguous(), residual=w2, out=w2)
    server.up.zero_()
    return update


def run(blocks=2, hidden=256, rank=16, tokens=256, clients=3, rounds=2, steps=4, lr=0.005, rate=0.02, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*shape, scale, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    weights = [(rnd(4 * hidden, hidden, scale=hidden ** -0.5), rnd(4 * hidden, scale=0.1, dtype=torch.bfloat16),
                rnd(hidden, 4 * hidden, scale=0.5 * (4 * hidden) ** -0.5)) for _ in range(blocks)]
    server, momentum = (Adapters(blocks, hidden, rank, torch.float32) for _ in range(2))
    server.down.copy_(rnd(*server.down.shape, scale=(4 * hidden) ** -0.5))
    data = [[rnd(tokens + 3 * c, hidden, scale=1.0, dtype=torch.bfloat16) for _ in range(2)] for c in range(clients)]
    n = [x.shape[0] for x, _ in data]
    for _ in range(rounds):
        frozen = [Frozen(*w) for w in weights]
        sent = [client(frozen, server, x, t, steps, lr) for x, t in data]
        server_step(weights, server, momentum, sent, n, rate)
    return weights, server, data


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("blocks", 2), ("hidden", 512), ("rank", 16), ("tokens", 512), ("clients", 4), ("rounds", 3),
                          ("steps", 5)):
        p.add_argument("--" + name, type=int, default=default)
    a = p.parse_args()
    weights, server, data = run(**vars(a))
    x, target = data[0]
    y, _ = forward([Frozen(*w) for w in weights], Adapters(*server.sizes, torch.bfloat16, server.flat.to(torch.bfloat16)), x)
    print(f"mean squared error of the first client's data after {a.rounds} rounds: "
          f"{float((y.float() - target.float()).square().mean()):.4f}")
