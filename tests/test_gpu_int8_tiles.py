"""GPU: the layer on 8-bit weights where the rule for its tiles changes, against the
plain form in 64 bits."""

import pytest
import torch

import weighted_model_update_amd as fa
from test_gpu_int8 import DTYPES, check_forward, ints, positive, rnd

pytestmark = pytest.mark.gpu


# 512 and 513 or more tiles of 64 x 64; odd rows, which go through registers, with 256
# and more tiles of 128 x 128, and copied with whole rows; one step and several
@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("shape", [(1024, 2048, 64), (1025, 2048, 64), (1090, 2050, 208), (1920, 2048, 272), (300, 8192, 144),
                                   (100, 25088, 64), (300, 8190, 101), (400, 8192, 101), (385, 8193, 67), (500, 12288, 77),
                                   (511, 8192, 501), (513, 8100, 501), (65, 33000, 48), (33000, 65, 33)], ids=str)
def test_forward_around_the_rules(shape, dt):
    M, N, K = shape
    t = DTYPES[dt]
    xq, xs, w, ws = ints((M, K), 1, -128), positive(M, 2, 0.02), ints((N, K), 3, -128), positive(N, 4, 0.02 * K ** -0.5)
    bias, res, pre = rnd((N,), t, 5), rnd((M, N), t, 6), torch.empty(M, N, dtype=t, device="cuda")
    out = fa.linear_int8_forward(xq, w, ws, bias, act="gelu", residual=res, alpha=0.5, x_scale=xs, preact=pre, dtype=t)
    check_forward(xq, xs, w, ws, bias, "gelu", res, 0.5, out, pre)
    # rows by themselves take other tiles
    few = fa.linear_int8_forward(xq[:40], w, ws, bias, act="gelu", residual=res[:40], alpha=0.5, x_scale=xs[:40], dtype=t)
    assert torch.equal(out[:40], few)
