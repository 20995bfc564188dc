"""Plain float64 forms of the linear layer, the top logits of rows and the
distillation loss, on the CPU, for the GPU tests.  They share no code with the
library or the measured cases."""

import math

import torch

U32 = 2.0 ** -24  # half a step of fp32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def d(t):
    return t.detach().cpu().double()


def act(z, name):
    if name == "relu":
        return torch.clamp(z, min=0)
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def act_slope(z, name):
    if name == "relu":
        return (z > 0).double()
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1 - s)
    return torch.ones_like(z)


def linear(x, w, bias, name, residual, alpha):
    """(out, z, sum of magnitudes that entered) in float64."""
    x, w = d(x), d(w)
    z = alpha * (x @ w.t())
    mag = abs(alpha) * (x.abs() @ w.abs().t())
    if bias is not None:
        z, mag = z + d(bias), mag + d(bias).abs()
    y = act(z, name)
    if residual is not None:
        y, mag = y + d(residual), mag + d(residual).abs()
    return y, z, mag


def within(got, want, slack, dtype, what=""):
    """got was rounded once to dtype from a value at most `slack` off want."""
    got = d(got)
    tol = half_step(dtype) * (want.abs() + slack) + slack + 1e-38
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float(((got - want).abs() / tol)[bad].max()):.3g} x tolerance at {bad.nonzero()[0].tolist()}")


def top_rows(x, k):
    """Indices (ascending) and values of the k largest of each row: by value,
    NaN first, then by lower index."""
    x = x.detach().cpu().float()
    idx = []
    for row in x.tolist():
        order = sorted(range(len(row)), key=lambda i: (0 if row[i] != row[i] else 1,
                                                       -row[i] if row[i] == row[i] else 0.0, i))
        idx.append(sorted(order[:k]))
    idx = torch.tensor(idx, dtype=torch.int64).reshape(x.shape[0], k)
    return idx, x.gather(1, idx)


def lse_of(x, tau):
    return torch.logsumexp(d(x) / tau, dim=1)


def distill(z, idx, val, n, tau, teacher_lse=None, row_weight=None):
    """loss [R], lse [R], dz [R, V] in float64, row by row and client by
    client from the definition; flawed lists count as not sent.  Also the
    magnitude that rounding errors of the loss scale with."""
    zz = d(z)
    R, V = zz.shape
    loss, lse_o, dz, mag = torch.zeros(R).double(), torch.zeros(R).double(), torch.zeros(R, V).double(), torch.zeros(R).double()
    flawed = False
    for r in range(R):
        g = 1.0 if row_weight is None else float(row_weight[r])
        for c in range(len(n)):
            if int(n[c]) > 0 and g != 0:
                li = [int(i) for i in idx[c][r]]
                m = next((j for j, i in enumerate(li) if i < 0), len(li))
                flawed |= any(i >= V for i in li[:m]) or any(a >= b for a, b in zip(li[:m], li[1:m]))
        if g == 0:
            continue
        y = zz[r] / tau
        lse = torch.logsumexp(y, 0) if V else torch.tensor(-math.inf).double()
        lse_o[r] = lse
        if lse == -math.inf:
            continue
        sent = []
        for c in range(len(n)):
            if int(n[c]) == 0:
                continue
            li = [int(i) for i in idx[c][r]]
            m = next((j for j, i in enumerate(li) if i < 0), len(li))
            li = li[:m]
            if any(i >= V for i in li) or any(a >= b for a, b in zip(li, li[1:])):
                continue
            v = d(val[c])[r, :m] / tau
            if m == 0 or bool((v == -math.inf).all()):
                continue
            L = torch.logsumexp(v, 0) if teacher_lse is None else d(teacher_lse[c])[r]
            sent.append((c, li, v - L))
        W = sum(int(n[c]) for c, _, _ in sent)
        Q = torch.zeros(V).double()
        for c, li, lq in sent:
            q = torch.exp(lq)
            lp = y[li] - lse
            wc = int(n[c]) / W
            keep = q != 0
            loss[r] += wc * (q[keep] * (lq[keep] - lp[keep])).sum()
            mag[r] += wc * (q[keep] * (1 + lq[keep].abs() + lp[keep].abs())).sum()
            Q[li] += wc * q
        if sent:
            dz[r] = g * tau * (Q.sum() * torch.exp(y - lse) - Q)
        loss[r] *= g * tau * tau
        mag[r] *= abs(g) * tau * tau
    return loss, lse_o, dz, mag, flawed
