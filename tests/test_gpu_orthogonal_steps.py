"""GPU: the orthogonalised matrix of long sides after more steps than five, whose
bounds are carried on from step to step, against the formula in float64."""

import math

import pytest
import torch

import learn_ref as ref
import weighted_model_update_amd as fa
from test_gpu_orthogonal import CUBIC, QUINTIC, check, formula, off, rnd, update

pytestmark = pytest.mark.gpu

LONG = [(100, 110), (110, 100), (300, 400), (130, 1000), (1000, 130), (2, 300, 320)]


def low_rank(shape, rank, seed):
    """Whole numbers of exactly that rank, exact in every type."""
    *lead, m, n = shape
    g = torch.Generator().manual_seed(seed)
    a, b = (torch.randint(-2, 3, s, generator=g).float() for s in ((*lead, m, rank), (*lead, rank, n)))
    return (a @ b).cuda()


def carried(x, steps):
    """What unit errors of the singular values after each step come to at the end,
    relative to the result's norm: an error e of v becomes |p'(v)| e in the next,
    with p'(v) = a + 3 b v^2 + 5 c v^4.  Over 32 steps single values reach 1e5, and
    whether the rounding of fp32 products hits these says nothing about others."""
    a, b, c = QUINTIC
    errors, values = 0.0, 0.0
    for t in (x if x.dim() == 3 else x[None]).double().cpu():
        v = torch.linalg.svdvals(t / t.norm())
        v = v[v > 1e-12]  # rows of zeros stay zeros exactly
        e = torch.zeros_like(v)
        for _ in range(steps):
            e = e * (a + 3 * b * v ** 2 + 5 * c * v ** 4).abs() + 1
            v = (a * v + b * v ** 3 + c * v ** 5).abs()
        errors, values = errors + float(e.square().sum()), values + float(v.square().sum())
    return math.sqrt(errors / values)


def check_carried(x, out, steps):
    """X, G and H round to 24 bits and each product leaves out the product of its low
    halves, 2^-24 of it: independent errors of the entries, below 2^-22 of X in the
    norm of a step, which the later steps enlarge."""
    want = formula(x, QUINTIC, steps, torch.float64)
    assert off(out, want) <= ref.half_step(out.dtype) + 2.0 ** -22 * carried(x, steps)


# ------------------------------------------------------------------ long sides

@pytest.mark.parametrize("steps", [6, 7, 10, 32])
@pytest.mark.parametrize("shape", LONG, ids=str)
def test_long_sides_of_fp32(shape, steps):
    x = rnd(shape, torch.float32, 21)
    check_carried(x, fa.orthogonalize(x, steps=steps), steps)
    x[..., 3, :] = 0
    out = fa.orthogonalize(x, steps=steps)
    check_carried(x, out, steps)
    assert bool((out[..., 3, :] == 0).all())


@pytest.mark.parametrize("steps", [6, 7, 10])
@pytest.mark.parametrize("shape", LONG, ids=str)
def test_long_sides_of_low_rank(shape, steps):
    """Rounding in directions that the matrix does not have grows by 3.4 a step in
    every arithmetic: at most four times that of fp32 products, as at the fifth step."""
    x = low_rank(shape, 4, 22)
    check(x, fa.orthogonalize(x, steps=steps), steps=steps)


@pytest.mark.parametrize("steps", [6, 7, 10, 32])
@pytest.mark.parametrize("shape", [(100, 110), (300, 310), (70, 300), (300, 70), (2, 200, 900), (520, 2100)], ids=str)
def test_long_sides_of_bf16(shape, steps):
    """The singular values of noise lie within a factor of 20, and G's errors grow
    with G but for that factor squared: 2^-22 for each of three products a step, of
    five steps a group, times 400 and H's slope |b| + 2 |c| = 9, in the worst of s
    directions: 0.013 / sqrt(s) of the norm, at most 0.0016 for s = 70."""
    x = rnd(shape, torch.bfloat16, 23)
    want = formula(x, QUINTIC, steps, torch.float64)
    fp32 = off(formula(x, QUINTIC, steps, torch.float32), want)
    got = fa.orthogonalize(x, steps=steps)
    assert off(got, want) <= ref.half_step(torch.bfloat16) + 4 * fp32 + 0.013 / math.sqrt(min(shape[-2:]))
    w = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    fa.orthogonal_step(w, x.float(), rate=1.0, steps=steps)
    assert torch.equal(w, got)


def test_steps_with_other_coefficients_on_long_sides():
    """Steps whose largest value changes from one to the next, a step that ends
    below one and one that starts above."""
    rows = ((8.0, -23.0, 17.0), (0.25, 0.0, 0.0), (3.0, -4.0, 2.0), QUINTIC, QUINTIC, CUBIC, CUBIC, CUBIC, CUBIC)
    for shape in ((100, 110), (110, 100), (130, 1000)):
        x = rnd(shape, torch.float32, 24)
        check(x, fa.orthogonalize(x, steps=len(rows), coef=rows), coef=rows, steps=len(rows))


# ------------------------------------------------------------------ groups of steps

def carried_in_groups(x, rows):
    """A bound of the error of steps on one Gram matrix, relative to the result's norm.
    With l an eigenvalue of G and q = a + b l + c l^2, a step takes l to l q^2 and P to
    q P, and errors e of l and p of P to |q^2 + 2 l q q'| e and |q| p + |P q'| e.
    Every product adds 2^-22 of its largest value (two roundings to 24 bits and the
    low halves' product, 2^-24 each): two for G, one each for H, P and the product with
    X.  A group ends when the largest q^2, with a margin of 5%, have passed 3e4."""
    unit = 2.0 ** -22
    errors, values = 0.0, 0.0
    for t in (x if x.dim() == 3 else x[None]).double().cpu():
        v = torch.linalg.svdvals(t / t.norm())
        dv, top, growth = torch.zeros_like(v), 1.01, 0.0
        for i, (a, b, c) in enumerate(rows):
            if growth == 0.0:
                l, P, growth = v * v, torch.ones_like(v), 1.0
                e, p = torch.full_like(v, unit * float(l.max())), torch.zeros_like(v)
            grid = torch.linspace(0, top ** 2, 2001, dtype=torch.float64)
            q, slope, most = a + (b + c * l) * l, b + 2 * c * l, a + (b + c * grid) * grid
            growth *= max(1.0, float((1.05 * most).abs().max()) ** 2)
            top = float((most * grid.sqrt()).abs().max())
            p = q.abs() * p + P.abs() * (slope.abs() * e + unit * float(((b + c * grid) * grid).abs().max())) + unit * float((q * P).abs().max())
            P, e, l = q * P, (q * q + 2 * l * q * slope).abs() * e + 2 * unit * top ** 2, l * q * q
            if growth > 3e4 or i + 1 == len(rows):
                v, dv, growth = (P * v).abs(), P.abs() * dv + p * v + unit * top, 0.0
        errors, values = errors + float(dv.square().sum()), values + float(v.square().sum())
    return math.sqrt(errors / values)


@pytest.mark.parametrize("shape", [(70, 300), (300, 70), (2, 200, 900), (520, 2100)], ids=str)
@pytest.mark.parametrize("rows", [(QUINTIC,) * 5, (QUINTIC,) * 2, (QUINTIC,) * 10, (CUBIC,) * 20, ((5.0, -9.0, 5.0),) + (CUBIC,) * 4,
                                  ((100.0, 0.0, 0.0),) * 3], ids=["quintic", "two", "ten", "cubic", "steep", "linear"])
def test_groups_of_steps_beside_the_rounding(shape, rows):
    """bf16 rounds to the nearest, so a value d off is rounded to within |want rounded -
    want| + d of itself: the result is off by that and 2 d."""
    x = update(shape, torch.bfloat16, 6)
    want = formula(x, rows, len(rows), torch.float64)
    got = fa.orthogonalize(x, steps=len(rows), coef=rows)
    assert off(got, want) <= off(want.bfloat16(), want) + 2 * carried_in_groups(x, rows)


def left_over(x, steps):
    """What a call with bf16 results is off by, relative to the norm, without the
    rounding of the result: a step whose weights are the rounded result's negative
    leaves the difference, to eight bits of it."""
    want = formula(x, QUINTIC, steps, torch.float64)
    near = want.bfloat16()
    w = -near
    fa.orthogonal_step(w, x, rate=1.0, steps=steps)
    return float((w.double() + near.double() - want).norm() / want.norm())


@pytest.mark.parametrize("rank", [1, 2, 3, 5])
@pytest.mark.parametrize("shape", [(100, 300), (300, 1000), (600, 1000), (1000, 300), (1000, 1300)], ids=str)
def test_groups_of_steps_on_low_rank(shape, rank):
    """Rounding in directions that the matrix does not have grows by 3.4 a step, as
    that of fp32 products does, in a group and outside one: 2^-24 3.4^5 = 3e-5 for each
    of the four roundings of a product (two factors, the low halves' product, the sum)
    and of the up to four products a step, if all are alike; equal rows round alike."""
    for seed in (1, 2, 3):
        x = low_rank(shape, rank, seed).bfloat16()
        assert left_over(x, 5) <= 16 * 2.0 ** -24 * QUINTIC[0] ** 5
