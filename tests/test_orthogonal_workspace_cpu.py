"""CPU-only: workspaces of the orthogonalised update by its number of steps."""

import pytest

from test_learn_cpu import ARG, WORKSPACE
from test_orthogonal_cpu import bytes_of, orthogonalize


@pytest.mark.parametrize("B,m,n", [(2, 8, 16), (3, 16, 4096), (5, 64, 300), (1, 300, 64)])
def test_short_sides(B, m, n):
    """A group of steps whose Gram matrix carries them needs what it always did; more
    hold X in fp64 between the groups.  The workspace is not aligned, so that one large
    enough is refused for that."""
    whole = bytes_of(B, m, n)
    assert whole >= 8 * B * m * n
    few = 256 if m <= 16 and n <= 256 else None
    kw = dict(B=B, m=m, n=n, ldx=n, sx=m * n, ldo=n, so=m * n, x=1 << 45, out=1 << 46, ws=(1 << 44) + 8)
    for steps in (1, 5, 8):
        if few:
            assert orthogonalize(steps=steps, wsb=few, **kw) == ARG
    for steps in (9, 12, 32):
        assert orthogonalize(steps=steps, wsb=whole - 1, **kw) == WORKSPACE
        assert orthogonalize(steps=steps, wsb=whole, **kw) == ARG
    # the cubic's steps enlarge rounding by less
    assert orthogonalize(steps=32, coef=(1.5, -0.5, 0.0), wsb=whole - 1, **kw) == WORKSPACE
    if few:
        assert orthogonalize(steps=21, coef=(1.5, -0.5, 0.0), wsb=few, **kw) == ARG


def test_the_held_matrices_are_bounded():
    for B in (1 << 10, 1 << 16):
        assert bytes_of(B, 16, 4096) - bytes_of(B // 2, 16, 4096) < B * 16 * 4096
    assert bytes_of(1, 64, 1 << 20) < 3 * 8 * 64 << 20


def test_large_batches_of_small_matrices():
    for m, n in ((1, 1), (8, 8), (5, 16), (16, 100)):
        assert bytes_of(1 << 20, m, n) <= (1 << 28)
        assert bytes_of(1 << 20, m, n) == bytes_of(1 << 19, m, n)
