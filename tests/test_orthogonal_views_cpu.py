"""CPU-only: which parts of one buffer a call of the orthogonalised update takes
beside one another.  Calls come without a workspace, so that what is accepted is
refused for that."""

import pytest
import torch

from test_learn_cpu import ARG, WORKSPACE
from test_orthogonal_cpu import orthogonalize, step

BASE = 1 << 44


def place(shape, strides, offset):
    return shape, strides, offset


def overlaps(a, b, shape):
    """By marking the elements."""
    size = max(o + sum((d - 1) * s for d, s in zip(shape, st)) for st, o in (a, b)) + 1
    seen = torch.zeros(size, dtype=torch.bool)
    st, o = a
    torch.as_strided(seen, shape, st, o).fill_(True)
    st, o = b
    return bool(torch.as_strided(seen, shape, st, o).any())


def code(shape, a, b, dtype=0):
    """x at a and out at b: strides of matrix and row, and the first element."""
    B, m, n = shape
    (sx, ldx), (so, ldo) = a[0], b[0]
    return orthogonalize(dtype=dtype, B=B, m=m, n=n, x=BASE + a[1] * 4, ldx=ldx, sx=sx, out=BASE + b[1] * 4, ldo=ldo, so=so, ws=None)


def check(shape, a, b):
    want = ARG if overlaps((a[0] + (1,), a[1]), (b[0] + (1,), b[1]), shape) else WORKSPACE
    assert code(shape, a, b) == want, (shape, a, b)
    assert code(shape, b, a) == want, (shape, a, b)
    return want


def test_columns_of_one_matrix():
    # buf [8, 40]: columns 0 .. 15 and from s on
    got = {s: check((1, 8, 16), ((0, 40), 0), ((0, 40), s)) for s in range(1, 40)}
    assert got[15] == ARG and got[16] == got[24] == WORKSPACE and got[25] == ARG
    # with strides that a single matrix does not use
    assert code((1, 8, 16), ((320, 40), 0), ((7, 40), 16)) == WORKSPACE


def test_rows_of_one_matrix():
    for s in (1, 7, 8, 9):
        check((1, 8, 16), ((0, 16), 0), ((0, 16), s * 16))


def test_columns_of_every_matrix():
    # buf [3, 8, 40], also with rows between the matrices
    for gap in (0, 2):
        stride = (8 + gap) * 40
        got = {s: check((3, 8, 16), ((stride, 40), 0), ((stride, 40), s)) for s in range(1, 40)}
        assert got[15] == ARG and got[16] == got[24] == WORKSPACE


def test_rows_of_every_matrix():
    # buf [3, 16, 16]: rows 0 .. 7 and 8 .. 15
    for s in (4, 8, 12, 16, 24):
        check((3, 8, 16), ((256, 16), 0), ((256, 16), s * 16))


def test_matrices_that_interleave_by_rows():
    # buf [8, 3 matrices, 40]
    for s in (8, 16, 20, 24, 25, 40):
        check((3, 8, 16), ((40, 120), 0), ((40, 120), s))


def test_single_rows_and_columns():
    for s in (1, 2, 3):
        check((1, 8, 1), ((0, 4), 0), ((0, 4), s))
        check((5, 1, 2), ((6, 2), 0), ((6, 2), 2 * s - 1))
        check((5, 1, 2), ((6, 2), 0), ((6, 2), 2 * s))


def test_what_cannot_be_told_apart_is_refused():
    # pitches that differ: whole extents count
    assert code((1, 8, 16), ((0, 40), 0), ((0, 41), 16)) == ARG


@pytest.mark.parametrize("B,stride", [(1, 0), (3, 8 * 60)])
def test_a_step_on_columns_of_one_buffer(B, stride):
    """Update, momentum and weights in the columns of one fp32 buffer."""
    def call(u, mom, w):
        return step(udtype=0, dtype=0, B=B, m=8, n=16, u=BASE + 4 * u, ldu=60, su=stride, mom=BASE + 4 * mom, ldm=60, sm=stride,
                    w=BASE + 4 * w, ldw=60, sw=stride, ws=None)
    assert call(0, 16, 32) == call(44, 0, 20) == WORKSPACE
    assert call(0, 15, 32) == call(0, 16, 31) == call(0, 16, 8) == call(0, 16, 45) == ARG


def test_the_workspace_lies_apart():
    B, m, n = 1, 8, 16
    # a pitched result and the workspace in its gap: whole extents count, as for every workspace
    assert orthogonalize(dtype=0, B=B, m=m, n=n, x=1 << 40, ldx=16, sx=0, out=BASE, ldo=1 << 12, so=0, ws=BASE + 4 * 16, wsb=4096) == ARG
