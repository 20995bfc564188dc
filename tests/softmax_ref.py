"""Float64 forms of the softmax, the top logits' normaliser and the
distillation taken relative to each row's maximum, so that they hold for rows
of any offset and for any temperature, with the rounding errors that a result
in fp32 may carry.  For tests of large offsets, masks and temperatures."""

import numpy as np
import torch

from learn_ref import U32


def f32(v):
    """The value that a float argument has in the library."""
    return float(np.float32(v))


class Row:
    """Statistics of one row of logits: d = (z - max) / tau, log s, p, log p,
    lse, and `off`, what lse may be off by before its own rounding."""

    def __init__(self, z, tau):
        V = z.numel()
        self.m = z.max()
        self.d = (z - self.m) / tau
        e = torch.exp(self.d)
        self.logs = torch.log(e.sum())
        self.p = e / e.sum()
        self.logp = self.d - self.logs
        self.lse = self.m / tau + self.logs
        # exponents are rounded a few times relative to |d|, sums at most
        # V / 256 + 40 times; entries far below the maximum add nothing
        spread = float((self.p * self.d.clamp(min=-200).abs()).sum())
        self.sum_off = (V / 256 + 48 + 8 * spread) * U32
        self.off = self.sum_off + 4 * U32 * float((self.m / tau).abs())


def distill_row(z, lists, n, tau, g, teacher_lse=None, given_lse=False):
    """(loss, its slack, dz, its slack) of one row of float64 logits; lists:
    per client (indices, float64 values), all valid and not empty.  With
    given_lse the gradient is formed from the stored normaliser, whose
    magnitude up to 128 its error scales with."""
    row = Row(z, tau)
    V = z.numel()
    W = sum(n)
    loss = loss_off = 0.0
    Q, Qoff = torch.zeros(V).double(), torch.zeros(V).double()
    for c, (i, v) in enumerate(lists):
        k = len(i)
        if teacher_lse is None:
            dv = (v - v.max()) / tau
            lq = dv - torch.logsumexp(dv, 0)
            steps = k + 60 + 8 * dv.abs().clamp(max=200)
        else:
            lq = v / tau - teacher_lse[c]
            steps = k + 60 + 8 * (v / tau).abs() + 8 * abs(float(teacher_lse[c]))
        w = n[c] / W
        q = torch.exp(lq)
        steps = steps + len(n)
        keep = q != 0
        qk, lk, pk, sk, dk = q[keep], lq[keep], row.logp[i][keep], steps[keep], row.d[i][keep]
        loss = loss + w * float((qk * (lk - pk)).sum())
        loss_off = loss_off + w * float((qk * (1 + lk.abs() + pk.abs()) * (sk * U32 + row.sum_off)).sum()) \
            + w * float((8 * U32 * qk * dk.abs()).sum())
        Q[i] += w * q
        Qoff[i] += w * q * steps * U32
    mass, mass_off = Q.sum(), Qoff.sum()
    dz = g * tau * (mass * row.p - Q)
    rel = row.sum_off + 8 * U32 * row.d.abs().clamp(max=200) + 8 * U32
    if given_lse:
        rel = rel + 8 * U32 * min(abs(float(row.lse)), 128.0)
    off = abs(g) * tau * (mass * row.p * rel + mass_off * row.p + Qoff + 8 * U32 * Q + 2.4e-38 * mass)
    return g * tau * tau * loss, abs(g) * tau * tau * loss_off, dz, off
