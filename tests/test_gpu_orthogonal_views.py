"""GPU: the orthogonalised update on parts of one buffer that lie beside one
another, against the same call on tensors of their own."""

import pytest
import torch

import weighted_model_update_amd as fa
from test_gpu_orthogonal import rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(20, 33), (40, 16), (100, 70), (3, 20, 33), (2, 70, 130)], ids=str)
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_columns_and_rows_of_one_buffer(shape, dt):
    *lead, m, n = shape
    x = rnd(shape, dt, 1)
    want = fa.orthogonalize(x)
    beside = torch.full((*lead, m, 2 * n + 3), 7.0, dtype=dt, device="cuda")
    beside[..., :n] = x
    fa.orthogonalize(beside[..., :n], out=beside[..., n + 1:2 * n + 1])
    assert torch.equal(beside[..., n + 1:2 * n + 1], want) and torch.equal(beside[..., :n], x)
    assert bool((beside[..., n] == 7).all()) and bool((beside[..., 2 * n + 1:] == 7).all())
    below = torch.full((*lead, 2 * m, n), 7.0, dtype=dt, device="cuda")
    below[..., :m, :] = x
    fa.orthogonalize(below[..., :m, :], out=below[..., m:, :])
    assert torch.equal(below[..., m:, :], want) and torch.equal(below[..., :m, :], x)


@pytest.mark.parametrize("shape", [(20, 33), (100, 70), (3, 20, 33)], ids=str)
def test_a_step_on_columns_of_one_buffer(shape):
    *lead, m, n = shape
    u, mom, w = (rnd(shape, torch.float32, i) for i in (1, 2, 3))
    buf = torch.full((*lead, m, 3 * n + 1), 7.0, device="cuda")
    parts = [buf[..., i * n:(i + 1) * n] for i in range(3)]
    for p, t in zip(parts, (u, mom, w)):
        p.copy_(t)
    fa.orthogonal_step(parts[2], parts[0], 0.1, momentum=parts[1])
    fa.orthogonal_step(w, u, 0.1, momentum=mom)
    for p, t in zip(parts, (u, mom, w)):
        assert torch.equal(p, t)
    assert bool((buf[..., 3 * n:] == 7).all())
