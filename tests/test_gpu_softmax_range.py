"""GPU: normalisers of rows with large offsets, whole rows under finite masks
and extreme temperatures, against float64 relative to the row's maximum.
Every finite row whose normaliser fp32 can hold has a finite one."""

import pytest
import torch

import learn_ref as ref
import softmax_ref as sref
import weighted_model_update_amd as fa

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def rnd(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g) * scale


def offset_rows(V, t):
    """Rows of one value, of a value with others next to it, and rows that
    finite masks cover in whole or in part."""
    low = torch.finfo(t).min
    rows = [torch.full((V,), v) for v in (-1e9, -1e10, -3e10, 1e10, 1e20, -1e25, low, -low, 3000.0, -200.0)]
    for at in (1e4, -1e6, 1e9, 4e9, -3e10):
        x = torch.full((V,), at).to(t).float()
        x[::3] = torch.nextafter(x.to(t), torch.tensor(float("inf"), dtype=t))[::3].float()
        rows.append(x)
    for mask in (-1e4, -1e9, -1e10, low):
        x = rnd((V,), 17, 2.5)
        x[V // 3:] = mask
        rows.append(x)
        y = torch.full((V,), mask)      # ordinary logits at the end, after every thread has met the mask
        y[-5:] = torch.tensor([1.0, 2.0, 3.0, 2.0, 1.0])
        rows.append(y)
    x = torch.arange(V).float() * 1e7   # the maximum rises from entry to entry
    rows += [x, -x]
    return torch.stack(rows).to(t)


def check_lse(lse, x, tau):
    want = [sref.Row(z, sref.f32(tau)) for z in ref.d(x)]
    exact = torch.stack([r.lse for r in want])
    assert bool(torch.isfinite(lse).all())
    ref.within(lse, exact, torch.tensor([r.off for r in want]).double(), torch.float32, f"lse at tau {tau}")


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("V", [70, 3001, 40003])
def test_normaliser_of_rows_with_large_offsets(V, dt):
    x = offset_rows(V, DTYPES[dt])
    for k in (0, 3):
        check_lse(fa.logits_topk(x.cuda(), k, tau=1.0)[2], x, 1.0)
    idx, val = torch.zeros(x.shape[0], 1, dtype=torch.int32, device="cuda"), torch.zeros(x.shape[0], 1, device="cuda")
    check_lse(fa.distill_loss(x.cuda(), [idx], [val], [1])[1], x, 1.0)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("tau", [1e-20, 1e-12, 1e-10, 1e-9, 1e-8, 1e-6, 1e-4, 1e-2, 1e6, 1e20])
def test_normaliser_at_extreme_temperatures(tau, dt):
    # many rows, and few that are split into pieces
    for R, V in ((300, 700), (2, 50001)):
        x = rnd((R, V), 5, 2.5).to(DTYPES[dt])
        check_lse(fa.logits_topk(x.cuda(), 2, tau=tau)[2], x, tau)
        idx, val = torch.zeros(R, 1, dtype=torch.int32, device="cuda"), torch.zeros(R, 1, device="cuda")
        check_lse(fa.distill_loss(x.cuda(), [idx], [val], [1], tau=tau)[1], x, tau)
