"""GPU: loss and gradient of the distillation for rows with large offsets,
rows under finite masks and extreme temperatures, against float64 relative to
the row's maximum."""

import pytest
import torch

import learn_ref as ref
import softmax_ref as sref
import weighted_model_update_amd as fa
from test_gpu_softmax_range import offset_rows, rnd

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def lists_of(R, V, ks, seed, first=0):
    """Per client [R, k] ascending places, the first `first` of the row and
    random ones among the others, and values."""
    g = torch.Generator().manual_seed(seed)
    idx, val = [], []
    for k in ks:
        rest = [first + torch.randperm(V - first, generator=g)[:k - first].sort().values for _ in range(R)]
        idx.append(torch.stack([torch.cat([torch.arange(first), r]) for r in rest]).int())
        val.append(torch.randn(R, k, generator=g) * 2)
    return idx, val


def want_of(z, idx, val, n, tau, teacher_lse=None, given_lse=False):
    zz, t = ref.d(z), sref.f32(tau)
    rows = [sref.distill_row(zz[r], [(i[r].long(), ref.d(v[r])) for i, v in zip(idx, val)], n, t, 1.0,
                             None if teacher_lse is None else [ref.d(l)[r] for l in teacher_lse], given_lse)
            for r in range(z.shape[0])]
    return [torch.stack([torch.as_tensor(r[j]).double() for r in rows]) for j in range(4)]


def cuda(ts):
    return [t.cuda() for t in ts]


def check_dz(z, idx, val, n, tau):
    _, _, dz, off = want_of(z, idx, val, n, tau)
    zc, args = z.cuda(), (cuda(idx), cuda(val), n)
    _, lse, got = fa.distill_loss(zc, *args, tau=tau, dz=True)
    ref.within(got, dz, off, z.dtype, "dz")
    off = want_of(z, idx, val, n, tau, given_lse=True)[3]
    back = fa.distill_backward(zc, lse, *args, tau=tau)
    ref.within(back, dz, off, z.dtype, "dz of the backward call")
    place = zc.clone()
    fa.distill_backward(place, lse, *args, tau=tau, dz=place)
    assert torch.equal(place.view(torch.uint8), back.view(torch.uint8))
    place = zc.clone()
    fa.distill_loss(place, *args, tau=tau, dz=place)
    assert torch.equal(place.view(torch.uint8), got.view(torch.uint8))


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("V", [70, 3001, 40003])
def test_gradient_of_rows_with_large_offsets(V, dt):
    z = offset_rows(V, DTYPES[dt])
    idx, val = lists_of(z.shape[0], V, (20, 7), V)
    check_dz(z, idx, val, [3, 5], 1.0)


@pytest.mark.parametrize("dt", list(DTYPES))
def test_gradient_of_more_rows_than_workgroups_hold_at_once(dt):
    z = offset_rows(9001, DTYPES[dt])
    z = z.repeat(300 // z.shape[0] + 1, 1)[:300]
    idx, val = lists_of(300, 9001, (12,), 3)
    check_dz(z, idx, val, [1], 1.0)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("tau", [1e-9, 1e-8, 1e-6, 1e-5, 1e-3, 0.05, 1e4])
def test_gradient_at_extreme_temperatures(tau, dt):
    for R, V in ((6, 700), (2, 50001)):
        z = rnd((R, V), 5, 2.5).to(DTYPES[dt])
        # equal values: the lists' own softmax is then exact at any temperature
        idx, val = lists_of(R, V, (16, 8), 9)
        val = [torch.full_like(v, 0.5) for v in val]
        check_dz(z, idx, val, [3, 5], tau)

@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("V", [500, 40003])
def test_gradient_where_the_normaliser_passes_fp32(V, dt):
    # the type's lowest and largest value over tau: lse is infinite, p is not
    low = torch.finfo(DTYPES[dt]).min
    z = torch.stack([torch.full((V,), low), torch.full((V,), -low), rnd((V,), 4)])
    z[0, ::2] = -float("inf")
    idx, val = lists_of(3, V, (9,), 2)
    val = [v / 4 for v in val]
    check_dz(z.to(DTYPES[dt]), idx, val, [1], 0.25)


def check_loss(z, idx, val, n, tau, teacher_lse=None):
    loss, off, _, _ = want_of(z, idx, val, n, tau, teacher_lse)
    got = fa.distill_loss(z.cuda(), cuda(idx), cuda(val), n, tau=tau,
                          teacher_lse=None if teacher_lse is None else cuda(teacher_lse))[0]
    ref.within(got, loss, off, torch.float32, "loss")


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("V", [70, 3001, 40003])
def test_loss_of_rows_with_large_offsets(V, dt):
    z = offset_rows(V, DTYPES[dt])
    z = z[[r for r in range(z.shape[0]) if r != 22]]    # its loss, nearly all of fp32's range, may round to infinity
    # places among the ordinary logits of rows whose end is masked, and others
    idx, val = lists_of(z.shape[0], V, (20, 7), V, first=5)
    check_loss(z, idx, val, [3, 5], 1.0)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("tau", [1e-6, 1e-4, 1e-2, 100.0])
def test_loss_at_extreme_temperatures(tau, dt):
    for R, V in ((6, 700), (2, 50001)):
        z = rnd((R, V), 5, 2.5).to(DTYPES[dt])
        idx, val = lists_of(R, V, (16, 8), 9)
        val = [torch.full_like(v, 0.5) for v in val]
        check_loss(z, idx, val, [3, 5], tau)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("tau", [1e-9, 1e-7, 1e-5, 1e-3])
def test_lists_own_softmax_at_small_temperatures(tau, dt):
    """Values of a list in steps of tau upon an offset: their softmax does not
    depend on the offset."""
    R, V = 5, 900
    z = torch.zeros(R, V).to(DTYPES[dt])
    idx, val = lists_of(R, V, (16, 8), 9)
    val = [(v / 2 * tau).float() for v in val]
    at = 2.0 ** 10 * tau
    shifted = [(v + at).float() for v in val]
    for vs in (val, shifted):
        check_loss(z, idx, vs, [3, 5], tau)
        _, _, dz, off = want_of(z, idx, vs, [3, 5], tau)
        ref.within(fa.distill_loss(z.cuda(), cuda(idx), cuda(vs), [3, 5], tau=tau, dz=True)[2], dz, off, z.dtype, "dz")


def test_lists_under_a_finite_mask():
    """Lists whose values are all one large number are uniform."""
    R, V, k = 4, 500, 12
    z = rnd((R, V), 3)
    idx, val = lists_of(R, V, (k,), 5)
    for r, v in enumerate((-1e9, -1e10, 1e20, torch.finfo(torch.float32).min)):
        val[0][r] = v
    check_dz(z, idx, val, [1], 1.0)
    check_loss(z, idx, val, [1], 1.0)


@pytest.mark.parametrize("tau", [1e-25, 1e-21, 1e-15])
def test_loss_at_temperatures_whose_square_is_below_fp32(tau):
    # loss = tau^2 * kl and kl grows as 1 / tau: the product is a number
    R, V = 3, 300
    z = rnd((R, V), 5, 2.5)
    idx, val = lists_of(R, V, (1,), 9)
    check_loss(z, idx, val, [1], tau)


@pytest.mark.parametrize("tau", [0.5, 1e-3])
def test_loss_of_listed_logits_under_the_lowest_value_at_small_temperatures(tau):
    # log p is about 1e38 / tau, the loss tau^2 times that
    z = rnd((2, 400), 5, 2.5)
    z[:, 200:] = torch.finfo(torch.float32).min
    idx, val = lists_of(2, 400, (30,), 9)
    val = [v * tau for v in val]
    check_loss(z, idx, val, [1], tau)


def test_loss_of_listed_logits_all_under_the_lowest_value():
    # each client's mass times 3.4e38, of which tau and the shares leave less
    z = rnd((64, 40), 5, 2.5)
    z[:, 8:] = torch.finfo(torch.float32).min
    idx, val = lists_of(64, 40, (9, 6, 12), 3)
    idx = [torch.stack([8 + torch.randperm(32, generator=torch.Generator().manual_seed(r))[:i.shape[1]].sort().values
                        for r in range(64)]).int() for i in idx]
    check_loss(z, idx, val, [3, 4, 5], 0.5)
