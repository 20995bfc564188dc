"""GPU: the distillation's error flag is set by every call, also where there
are no rows or no columns."""

import pytest
import torch

import weighted_model_update_amd as fa

pytestmark = pytest.mark.gpu


def both(z, idx, want):
    val = torch.zeros(idx.shape, device="cuda")
    for call in ("loss", "gradient"):
        err = torch.full((1,), 5, dtype=torch.int32, device="cuda")
        if call == "loss":
            fa.distill_loss(z, [idx], [val], [1], err_flag=err)
        else:
            dz = fa.distill_backward(z, torch.zeros(z.shape[0], device="cuda"), [idx], [val], [1], err_flag=err)
            assert dz.shape == z.shape
        assert int(err) == want, call


def lists(rows):
    return torch.tensor(rows, dtype=torch.int32, device="cuda")


def test_no_rows():
    both(torch.empty(0, 9, device="cuda"), torch.empty(0, 3, dtype=torch.int32, device="cuda"), 0)
    both(torch.empty(0, 0, device="cuda"), torch.empty(0, 3, dtype=torch.int32, device="cuda"), 0)


def test_no_columns():
    z = torch.empty(3, 0, device="cuda")
    both(z, lists([[-1, -1]] * 3), 0)
    both(z, lists([[-1, -1], [0, 1], [-1, -1]]), -7)


def test_some_of_both():
    z = torch.zeros(2, 7, device="cuda")
    both(z, lists([[1, 6], [2, -1]]), 0)
    both(z, lists([[1, 7], [2, -1]]), -7)
