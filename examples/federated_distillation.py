"""One round of adapter federation with distilled knowledge.

K clients hold a bottleneck adapter each on a shared frozen backbone.  Every
client sends its adapter and, for a batch of public tokens, its top logits.  The
server averages the adapters by sample count, then distils the clients' top
logits, weighted by the same counts, into the averaged adapter:

    h   = gelu(x down^T + b1)            linear_forward, keeps the pre-activation
    y   = h up^T + b2 + x                linear_forward with the residual
    z   = y head^T                       linear_forward
    loss, dz                             distill_loss, both in one call
    d(y), d(up), d(b2), d(h), ...        linear_backward, layer by layer

Run: python examples/federated_distillation.py [--tokens 512 --vocab 8192 ...]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import weighted_model_update_amd as fa  # noqa: E402


class Adapter:
    """down [rank, hidden], b1, up [hidden, rank], b2 as views of one flat
    bf16 vector, which is what a client sends."""

    def __init__(self, hidden, rank, flat=None):
        self.hidden, self.rank = hidden, rank
        n = 2 * hidden * rank + rank + hidden
        self.flat = torch.zeros(n, dtype=torch.bfloat16, device="cuda") if flat is None else flat
        parts = self.flat.split([rank * hidden, rank, hidden * rank, hidden])
        self.down, self.b1 = parts[0].view(rank, hidden), parts[1]
        self.up, self.b2 = parts[2].view(hidden, rank), parts[3]

    def forward(self, x):
        pre = torch.empty(x.shape[0], self.rank, dtype=x.dtype, device=x.device)
        h = fa.linear_forward(x, self.down, self.b1, act="gelu", preact=pre)
        y = fa.linear_forward(h, self.up, self.b2, residual=x)
        return y, (x, pre, h)

    def backward(self, dy, saved, grad):
        """Writes the gradients into the adapter `grad`."""
        x, pre, h = saved
        dh, _, _ = fa.linear_backward(dy, h, self.up, dw=grad.up, db=grad.b2)
        fa.linear_backward(dh, x, self.down, act="gelu", preact=pre, dx=None, dw=grad.down, db=grad.b1)


def clients_round(clients, n, x, head, k, tau):
    """What the clients send: adapters, sample counts and top logits of the
    public tokens x."""
    sent = []
    for c in clients:
        y, _ = c.forward(x)
        sent.append(fa.logits_topk(fa.linear_forward(y, head), k, tau=tau))
    return [c.flat for c in clients], n, sent


def server_round(flats, n, sent, x, head, hidden, rank, tau, steps, lr):
    """The averaged adapter after `steps` of distillation; the mean loss of
    each step."""
    server = Adapter(hidden, rank)
    fa.fedavg_aggregate(flats, n, server.flat)
    master = server.flat.float()                 # fp32 master weights
    grad = Adapter(hidden, rank)
    rows = torch.full((x.shape[0],), 1.0 / x.shape[0], device="cuda")
    idx, val = [s[0] for s in sent], [s[1] for s in sent]
    losses = []
    for _ in range(steps):
        y, saved = server.forward(x)
        z = fa.linear_forward(y, head)
        # the gradient takes the logits' place
        loss, _, dz = fa.distill_loss(z, idx, val, n, tau=tau, row_weight=rows, dz=z)
        losses.append(loss.sum())
        dy, _, _ = fa.linear_backward(dz, y, head, dw=None)
        server.backward(dy, saved, grad)
        master.sub_(grad.flat.float(), alpha=lr)
        server.flat.copy_(master)
    return server, [float(v) for v in losses]


def next_token(server, x, head):
    """The most likely token after one position: single-row calls."""
    y, _ = server.forward(x)
    return fa.logits_topk(fa.linear_forward(y, head), 1)[0]


def run(tokens=512, vocab=8192, hidden=1024, rank=64, clients=4, k=32, tau=2.0, steps=20, lr=0.5, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*shape, scale):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    x, head = rnd(tokens, hidden, scale=1.0), rnd(vocab, hidden, scale=hidden ** -0.5)
    # locally trained adapters: a common part and each client's own
    common = [rnd(rank, hidden, scale=hidden ** -0.5), rnd(hidden, rank, scale=2.0 * rank ** -0.5)]
    local = []
    for _ in range(clients):
        a = Adapter(hidden, rank)
        a.down.copy_(common[0] + rnd(rank, hidden, scale=0.5 * hidden ** -0.5))
        a.up.copy_(common[1] + rnd(hidden, rank, scale=rank ** -0.5))
        local.append(a)
    n = [100 + 50 * c for c in range(clients)]
    flats, n, sent = clients_round(local, n, x, head, k, tau)
    server, losses = server_round(flats, n, sent, x, head, hidden, rank, tau, steps, lr)
    return server, losses, next_token(server, x[:1], head)


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("tokens", 512), ("vocab", 8192), ("hidden", 1024), ("rank", 64), ("clients", 4), ("k", 32),
                          ("steps", 20)):
        p.add_argument("--" + name, type=int, default=default)
    p.add_argument("--lr", type=float, default=0.5)
    a = p.parse_args()
    _, losses, token = run(**vars(a))
    print(f"distillation loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps; next token {int(token)}")
