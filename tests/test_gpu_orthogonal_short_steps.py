"""GPU: the orthogonalised matrix of short sides after more steps than a Gram matrix
carries in fp64, against the formula in float64."""

import pytest
import torch

import learn_ref as ref
import weighted_model_update_amd as fa
from test_gpu_orthogonal import DTYPES, QUINTIC, check, formula, off, rnd
from test_gpu_orthogonal_steps import low_rank

pytestmark = pytest.mark.gpu

# one launch, three, many parts, tall and wide
SHORT = [(12, 14), (16, 200), (200, 16), (16, 400), (400, 16), (48, 200), (200, 48), (64, 1000), (1000, 64), (3, 20, 90), (130, 8, 300)]


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("steps", [6, 8, 9, 16, 17, 32])
@pytest.mark.parametrize("shape", SHORT, ids=str)
def test_short_sides(shape, steps, dt):
    x = rnd(shape, DTYPES[dt], 31)
    check(x, fa.orthogonalize(x, steps=steps), steps=steps)


@pytest.mark.parametrize("steps", [8, 9, 12, 16, 18, 20])
@pytest.mark.parametrize("shape", SHORT, ids=str)
def test_short_sides_of_low_rank(shape, steps):
    """Each of a step's three products rounds by at most s 2^-53 of its factors (G
    and X to 1.5, H to 3), and what that leaves in directions which the matrix does
    not have grows by 3.4 in every later step: 10 s 2^-53 3.4^steps in all, both here
    and in the formula."""
    x = low_rank(shape, 3, 32)
    s = min(shape[-2:])
    want = formula(x, QUINTIC, steps, torch.float64)
    slack = 2 * 10 * s * 2.0 ** -53 * QUINTIC[0] ** steps + 1e-8
    for dtype in (torch.float32, torch.bfloat16):
        out = fa.orthogonalize(x.to(dtype), steps=steps)
        ref.within(out, want.cpu(), slack + 3 * ref.U32 * want.abs().cpu(), dtype, "O")


@pytest.mark.parametrize("shape", SHORT, ids=str)
def test_short_sides_of_low_rank_at_the_largest_number_of_steps(shape):
    """Rounding fills the missing directions by then (2^-53 3.4^32 = 17), so the
    values are left open; they go through the same steps and stay below 1.21."""
    x = low_rank(shape, 3, 33)
    out = fa.orthogonalize(x, steps=32)
    assert bool(out.isfinite().all())
    assert float(torch.linalg.matrix_norm(out.double().cpu(), 2).max()) <= 1.21


@pytest.mark.parametrize("shape", [(16, 200), (48, 200), (400, 16)], ids=str)
def test_short_sides_with_zero_rows_and_columns(shape):
    x = rnd(shape, torch.float32, 34)
    x[3], x[:, 5] = 0, 0
    out = fa.orthogonalize(x, steps=24)
    check(x, out, steps=24)
    assert bool((out[3] == 0).all()) and bool((out[:, 5] == 0).all())
    x.zero_()
    assert bool((fa.orthogonalize(x, steps=24) == 0).all())
    x[2, 1] = float("nan")
    assert bool(fa.orthogonalize(x, steps=24).isnan().all())


@pytest.mark.parametrize("steps", [12, 24])
@pytest.mark.parametrize("shape", [(16, 200), (300, 10), (64, 450), (3, 48, 450), (450, 64), (5, 20, 30), (2, 40, 9000)], ids=str)
def test_in_place_views_and_momentum(shape, steps):
    x = rnd(shape, torch.float32, 35)
    want = fa.orthogonalize(x, steps=steps)
    y = x.clone()
    fa.orthogonalize(y, steps=steps, out=y)
    assert torch.equal(y, want)
    # columns of a wider buffer, its gap untouched
    wide = torch.full((*shape[:-1], shape[-1] + 3), -9.0, device="cuda")
    part = wide[..., 1:-2]
    part.copy_(x)
    fa.orthogonalize(part, steps=steps, out=part)
    assert torch.equal(part, want)
    part.fill_(-9.0)
    assert bool((wide == -9.0).all())
    for dtype in (torch.float32, torch.bfloat16):
        u, m0, w = x.to(dtype), rnd(shape, torch.float32, 36), rnd(shape, dtype, 37)
        mom, w0 = m0.clone(), w.clone()
        fa.orthogonal_step(w, u, rate=0.5, momentum=mom, beta=0.5, steps=steps)
        # the momentum is stepped once; t is formed of it as a fused product is
        m = (0.5 * m0.double() + u.double()).float()
        assert torch.equal(mom, m)
        t = (0.5 * m.double() + u.double()).float()
        o = formula(t, QUINTIC, steps, torch.float64)
        ref.within(w, (w0.double() + 0.5 * o).cpu(), 1e-8 + 4 * ref.U32 * (o.abs() + w0.double().abs()).cpu(), dtype, "weights")


def test_batches_of_more_than_a_pass_holds():
    x = rnd((75, 64, 4096), torch.float32, 38)
    x[7], x[40, 3, 3] = 0, float("inf")
    out = fa.orthogonalize(x, steps=12)
    assert bool((out[7] == 0).all()) and bool(out[40].isnan().all())
    for b in (0, 31, 32, 64, 74):
        check(x[b], out[b], steps=12)
    y = x.clone()
    assert torch.equal(fa.orthogonalize(y, steps=12, out=y).view(torch.int32), out.view(torch.int32))


@pytest.mark.parametrize("shape", [(16, 200), (3, 64, 450), (100, 110)], ids=str)
def test_many_steps_captured_and_replayed(shape):
    x, out = rnd(shape, torch.float32, 39), torch.empty(shape, device="cuda")
    ws = torch.empty(fa.orthogonalize_workspace_size(shape[0] if len(shape) == 3 else 1, *shape[-2:]), dtype=torch.uint8, device="cuda")
    call = lambda: fa.orthogonalize(x, steps=20, out=out, workspace=ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in range(4):
        x.copy_(rnd(shape, torch.float32, 40 + k))
        graph.replay()
        got = out.clone()
        torch.cuda.synchronize()
        out.zero_()
        ws.fill_(255)
        call()
        assert torch.equal(got, out)


def test_groups_end_alike_for_every_number_of_steps():
    """A step more is the next step of the formula, also where a group ends."""
    for shape in ((16, 200), (48, 300), (300, 33)):
        x = rnd(shape, torch.float32, 50)
        for steps in range(1, 33):
            check(x, fa.orthogonalize(x, steps=steps), steps=steps)


@pytest.mark.parametrize("steps", [5, 6, 7, 8])
@pytest.mark.parametrize("shape", [(48, 200), (200, 48), (64, 1000), (33, 90), (16, 400)], ids=str)
def test_one_gram_matrix_of_low_rank(shape, steps):
    """Up to 8 steps on one Gram matrix: the result's rounding, and, as for
    test_short_sides_of_low_rank, 10 s 2^-53 3.4^steps here and in the formula."""
    for rank in (2, 3, 8):
        x = low_rank(shape, rank, 51)
        want = formula(x, QUINTIC, steps, torch.float64)
        out = fa.orthogonalize(x, steps=steps)
        assert off(out, want) <= 2.0 ** -24 + 2 * 10 * min(shape) * 2.0 ** -53 * QUINTIC[0] ** steps


def test_singular_values_of_every_size():
    """From 1 to 1e-9 of the largest.  At the end of a group G's rounding has grown to at
    most 2^-53 1e8 times the steps' five products; X takes it with |b| of 4.8: 3e-7 in the
    one direction of s that has grown as much by then, the result's rounding beside it."""
    for shape in ((16, 400), (64, 1000), (300, 33)):
        m, n = shape
        g = torch.Generator().manual_seed(52)
        k = min(shape)
        u, _ = torch.linalg.qr(torch.randn(m, k, generator=g, dtype=torch.float64))
        v, _ = torch.linalg.qr(torch.randn(n, k, generator=g, dtype=torch.float64))
        x = ((u * torch.logspace(0, -9, k, dtype=torch.float64)) @ v.t()).float().cuda()
        for steps in (5, 8, 9, 12):
            want = formula(x, QUINTIC, steps, torch.float64)
            out = fa.orthogonalize(x, steps=steps)
            assert off(out, want) <= 2.0 ** -24 + 3e-7 / k ** 0.5


@pytest.mark.parametrize("shape", [(20000, 5, 3), (17000, 3, 20), (3500, 40, 33)], ids=str)
def test_large_batches_of_small_matrices(shape):
    x = rnd(shape, torch.float32, 53)
    x[5] = 0
    out = fa.orthogonalize(x, steps=12)
    assert bool((out[5] == 0).all())
    for b in (0, 1, shape[0] // 2, shape[0] - 1):
        check(x[b], out[b], steps=12)
    # the last ones by themselves, in a pass of their own
    assert torch.equal(out[-100:], fa.orthogonalize(x[-100:], steps=12))
