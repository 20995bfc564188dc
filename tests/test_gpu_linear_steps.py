"""GPU: large products whose sums take every number of steps modulo four, the
turn of the pipelined kernel's buffers, whole and ragged at the end, in all
three products and for each of its tiles."""

import pytest
import torch

import learn_ref as ref
import weighted_model_update_amd as fa
from test_gpu_linear import check_backward, check_forward, rnd

pytestmark = pytest.mark.gpu

# outputs that take 256x256, 128x256, 256x128 and mixed rounds of 128x128 tiles
TILES = [(2041, 2040), (634, 12792), (12792, 634), (2600, 5400)]


def products(P, Q, r, t):
    a, b = rnd((P, r), t, 1), rnd((Q, r), t, 2, r ** -0.5)
    check_forward(a, b, None, "none", None, 1.0, fa.linear_forward(a, b), None)
    dy, w = rnd((P, r), t, 3), rnd((r, Q), t, 4, r ** -0.5)
    got = fa.linear_backward(dy, torch.empty(P, Q, dtype=t, device="cuda"), w, dx=True, dw=None)
    check_backward(dy, torch.zeros(P, Q, dtype=t), w, "none", None, 1.0, got[0], None, None)
    dy, x = rnd((r, P), t, 5), rnd((r, Q), t, 6, r ** -0.5)
    got = fa.linear_backward(dy, x, torch.empty(P, Q, dtype=t, device="cuda"), dx=None, dw=True)
    check_backward(dy, x, torch.zeros(P, Q, dtype=t), "none", None, 1.0, None, got[1], None)


# steps of 32: 1, 2, 4, 6, 8, 9, 10, 12, and 2, 4, 6, 8 whose last is not whole
@pytest.mark.parametrize("r", [32, 64, 128, 192, 256, 288, 320, 384, 40, 120, 184, 248])
def test_bf16(r):
    products(*TILES[0], r, torch.bfloat16)


@pytest.mark.parametrize("r", [128, 192, 256])
@pytest.mark.parametrize("P,Q", TILES[1:], ids=str)
def test_bf16_other_tiles(P, Q, r):
    products(P, Q, r, torch.bfloat16)


# steps of 16: 1, 2, 4, 6, 8, and 4, 6 whose last is not whole
@pytest.mark.parametrize("r", [16, 32, 64, 96, 128, 60, 92])
def test_f32(r):
    products(2996, 3000, r, torch.float32)
