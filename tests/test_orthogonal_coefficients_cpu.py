"""CPU-only: the coefficients of the orthogonalised update are read at every call,
in whatever form numbers come."""

import numpy as np
import pytest
import torch

from test_learn_cpu import RANGE
from weighted_model_update_amd import fedavg


def values(coef, steps):
    return list(fedavg._coef_of(coef, steps))


def test_numbers_changed_between_calls_are_read_again():
    a, b, c = (torch.tensor(v, dtype=torch.float64) for v in (3.0, -2.0, 0.5))
    assert values((a, b, c), 2) == [3.0, -2.0, 0.5] * 2
    a.fill_(1.0)
    c.fill_(0.25)
    assert values((a, b, c), 2) == [1.0, -2.0, 0.25] * 2
    rows = [(a, b, c), (b, c, a)]
    assert values(rows, 2) == [1.0, -2.0, 0.25, -2.0, 0.25, 1.0]
    b.fill_(-1.0)
    assert values(rows, 2) == [1.0, -1.0, 0.25, -1.0, 0.25, 1.0]


def test_what_a_call_got_is_not_changed_by_the_next():
    first = fedavg._coef_of((1.0, 0.0, 0.0), 1)
    second = fedavg._coef_of((2.0, 0.0, 0.0), 1)
    assert list(first) == [1.0, 0.0, 0.0] and list(second) == [2.0, 0.0, 0.0]


def test_coefficients_made_on_the_way():
    assert values((v for v in (1.0, 2.0, 3.0)), 2) == [1.0, 2.0, 3.0] * 2
    assert values(((k, 0.0, 1.0) for k in range(3)), 3) == [0.0, 0.0, 1.0, 1.0, 0.0, 1.0, 2.0, 0.0, 1.0]
    assert values((iter((k, 0.0, 1.0)) for k in range(2)), 2) == [0.0, 0.0, 1.0, 1.0, 0.0, 1.0]


ROW, ROWS = [1.5, -0.5, 0.25], [[1.5, -0.5, 0.25], [2.0, -1.0, 0.0]]


@pytest.mark.parametrize("make", [list, tuple, np.array, lambda v: np.array(v, dtype=np.float32), torch.tensor,
                                  lambda v: torch.tensor(v, dtype=torch.float64)],
                         ids=["list", "tuple", "array", "array32", "tensor", "tensor64"])
def test_forms(make):
    assert values(make(ROW), 3) == ROW * 3
    assert values(make(ROWS), 2) == ROWS[0] + ROWS[1]
    assert values([make(r) for r in ROWS], 2) == ROWS[0] + ROWS[1]
    assert values(tuple(make(r) for r in ROWS), 2) == ROWS[0] + ROWS[1]


@pytest.mark.parametrize("coef,steps", [((), 1), ((1.0, 2.0), 2), ((1.0, 2.0, 3.0, 4.0), 4), (np.ones((2, 2)), 2), (np.ones((3, 3)), 2),
                                        (torch.ones(2, 3), 3), ([(1.0, 2.0, 3.0), 4.0], 2), ([1.0, (1.0, 2.0, 3.0), 2.0], 3),
                                        (np.ones((1, 1, 3)), 1)], ids=str)
def test_shapes_that_are_refused(coef, steps):
    with pytest.raises(ValueError, match="three numbers"):
        fedavg._coef_of(coef, steps)


# ------------------------------------------------------------------ what they let X grow to

def accepted(coef, steps):
    """The call's answer for no matrices: coefficients are checked all the same."""
    return fedavg.load().orthogonalize(0, 0, 8, 16, None, 16, 128, fedavg._coef_of(coef, steps), steps, 1.0, None, 16, 128, None, 0,
                                       None)


OK, QUINTIC, CUBIC = 0, fedavg.ORTHO_COEF, (1.5, -0.5, 0.0)


@pytest.mark.parametrize("coef", [QUINTIC, CUBIC, (1.0, 0.0, 0.0), (0.0, 0.0, 0.0), (0.5, 0.0, 0.0)], ids=str)
def test_steps_that_stay_bounded_are_taken_in_any_number(coef):
    """[0, 1.01] goes to [0, 1.2024] under the default and stays there."""
    for steps in range(1, 33):
        assert accepted(coef, steps) == OK


# (3, -4, 2) takes [0, 0.5626] to 1.0882, from where the default returns; (4, -6, 3) to
# 1.3530, from where it goes to 2.0446, 38.8 and the cubic to 2.9e4, 1.2e13
STEEP = ((8.0, -23.0, 17.0), (0.25, 0.0, 0.0))


@pytest.mark.parametrize("rows,code", [
    (STEEP + ((3.0, -4.0, 2.0), QUINTIC, QUINTIC, CUBIC, CUBIC, CUBIC, CUBIC), OK),
    (STEEP + ((4.0, -6.0, 3.0), QUINTIC, QUINTIC, CUBIC), OK),
    (STEEP + ((4.0, -6.0, 3.0), QUINTIC, QUINTIC, CUBIC, CUBIC), RANGE),
    # 1.01e9 and 0.909e9
    (((1.0, 0.0, 0.0), (1e9, 0.0, 0.0)), RANGE), (((0.9, 0.0, 0.0), (1e9, 0.0, 0.0)), OK),
], ids=["back", "before it grows", "grows", "at the end", "below"])
def test_bounds_of_steps_in_turn(rows, code):
    assert accepted(rows, len(rows)) == code


def coefficients_only(coef, steps, m, n, dtype):
    return fedavg.load().orthogonalize(dtype, 0, m, n, None, n, m * n, fedavg._coef_of(coef, steps), steps, 1.0, None, n, m * n, None,
                                       0, None)


# X as small as 1e-26 and a coefficient that would bring its fifth power back: as
# scales in fp32, 1e75 times 2^(111 - 2 * 114)
FAR = ((1e-26, 0.0, 0.0), (1.0, 0.0, 1e75))


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("m,n", [(100, 110), (110, 100), (100, 900)])
def test_scales_that_leave_fp32_are_refused_on_long_sides(m, n, dtype):
    assert coefficients_only(FAR, 2, m, n, dtype) == RANGE
    assert coefficients_only(((0.0, 0.0, 0.0), (1e300, 0.0, 0.0)), 2, m, n, dtype) == RANGE
    assert coefficients_only(((1e-26, 0.0, 0.0), (1.0, 0.0, 1e70)), 2, m, n, dtype) == OK
    # in fp64 they do not
    assert coefficients_only(FAR, 2, 60, n, dtype) == OK
    for steps in range(1, 33):
        for coef in (QUINTIC, CUBIC, (1.0, 0.0, 0.0)):
            assert coefficients_only(coef, steps, m, n, dtype) == OK
