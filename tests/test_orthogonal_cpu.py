"""CPU-only: the orthogonalised matrix and the server's step with it refuse bad
arguments, shared memory and tensors of another device before any device work."""

import ctypes

import pytest
import torch

import weighted_model_update_amd as fa
from test_learn_cpu import ARG, DTYPE, RANGE, WORKSPACE, at
from test_learn_devices_cpu import OnGpu, Stream, current  # noqa: F401
from weighted_model_update_amd import fedavg

BIG = 1 << 34


def lib():
    return fa.load()


def coefficients(c, steps):
    return None if c is None else (ctypes.c_double * (3 * max(steps, 1)))(*(list(c) * max(steps, 1)))


def orthogonalize(dtype=1, B=2, m=8, n=16, x=at(1), ldx=16, sx=128, coef=fa.ORTHO_COEF, steps=5, scale=1.0, out=at(2),
                  ldo=16, so=128, ws=at(12), wsb=1 << 30):
    return lib().orthogonalize(dtype, B, m, n, x, ldx, sx, coefficients(coef, steps), steps, scale, out, ldo, so, ws, wsb,
                               None)


def step(udtype=1, dtype=0, B=2, m=8, n=16, u=at(1), ldu=16, su=128, mom=at(3), ldm=16, sm=128, beta=0.9, nesterov=1,
         coef=fa.ORTHO_COEF, steps=5, rate=0.1, keep=1.0, w=at(2), ldw=16, sw=128, ws=at(12), wsb=1 << 30):
    return lib().orthogonal_step(udtype, dtype, B, m, n, u, ldu, su, mom, ldm, sm, beta, nesterov,
                                 coefficients(coef, steps), steps, rate, keep, w, ldw, sw, ws, wsb, None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("call,kw,code", [
    (orthogonalize, dict(dtype=2), DTYPE), (orthogonalize, dict(B=-1), ARG), (orthogonalize, dict(m=-1), ARG),
    (orthogonalize, dict(B=(1 << 20) + 1), RANGE), (orthogonalize, dict(n=(1 << 20) + 1), RANGE),
    (orthogonalize, dict(m=(1 << 15) + 1, n=(1 << 15) + 1), RANGE), (orthogonalize, dict(B=1 << 10, m=1 << 12, n=1 << 12), RANGE),
    (orthogonalize, dict(steps=0), ARG), (orthogonalize, dict(steps=33), ARG), (orthogonalize, dict(coef=None), ARG),
    (orthogonalize, dict(coef=(1e10, 0, 0)), RANGE), (orthogonalize, dict(coef=(100.0, 0, 0)), RANGE),
    (orthogonalize, dict(coef=(8.0, -23.0, 17.0), steps=6), RANGE),
    (orthogonalize, dict(coef=(1, NAN, 0)), RANGE), (orthogonalize, dict(coef=(1, 0, INF)), RANGE),
    (orthogonalize, dict(x=None), ARG), (orthogonalize, dict(out=None), ARG), (orthogonalize, dict(x=at(1, 1)), ARG),
    (orthogonalize, dict(out=at(2, 1)), ARG), (orthogonalize, dict(ldx=-1), ARG), (orthogonalize, dict(sx=-1), ARG),
    (orthogonalize, dict(ldx=1 << 41), RANGE), (orthogonalize, dict(so=1 << 41), RANGE),
    (orthogonalize, dict(ldo=15), ARG), (orthogonalize, dict(so=127), ARG), (orthogonalize, dict(so=0), ARG),
    (orthogonalize, dict(ldo=17, so=8), ARG),
    (orthogonalize, dict(out=at(1, 256)), ARG), (orthogonalize, dict(out=at(1), ldo=17, so=200), ARG),
    (orthogonalize, dict(out=at(1), so=130), ARG),
    (orthogonalize, dict(ws=None), WORKSPACE), (orthogonalize, dict(wsb=100), WORKSPACE), (orthogonalize, dict(ws=at(12, 8)), ARG),
    (orthogonalize, dict(ws=at(1)), ARG), (orthogonalize, dict(ws=at(2)), ARG),
    (step, dict(udtype=2), DTYPE), (step, dict(dtype=5), DTYPE), (step, dict(beta=-0.1), ARG), (step, dict(beta=1.5), ARG),
    (step, dict(beta=NAN), ARG), (step, dict(n=-3), ARG), (step, dict(steps=-1), ARG),
    (step, dict(u=None), ARG), (step, dict(w=None), ARG), (step, dict(mom=at(3, 2)), ARG), (step, dict(w=at(2, 2)), ARG),
    (step, dict(ldm=12), ARG), (step, dict(sm=100), ARG), (step, dict(ldw=3), ARG),
    (step, dict(w=at(1)), ARG), (step, dict(dtype=1, w=at(1)), ARG), (step, dict(mom=at(1)), ARG), (step, dict(mom=at(2, 1000)), ARG),
    (step, dict(ws=at(3)), ARG), (step, dict(ws=None), WORKSPACE),
], ids=lambda v: getattr(v, "__name__", str(v)))
def test_refusals(call, kw, code):
    assert call(**kw) == code
    assert lib().fedavg_last_error()


def test_an_input_whose_span_leaves_64_bits_is_refused():
    # rows and matrices both 2^40 elements apart, neither within the other: 2^61 elements
    assert orthogonalize(B=1 << 20, m=1 << 10, n=8, ldx=1 << 40, sx=1 << 40, ldo=8, so=1 << 13) == RANGE


@pytest.mark.parametrize("empty", [dict(B=0), dict(m=0), dict(n=0)], ids=str)
def test_nothing_to_do(empty):
    assert orthogonalize(**empty, x=None, out=None, ws=None) == 0
    assert step(**empty, u=None, w=None, mom=None, ws=None) == 0


def bytes_of(B, m, n):
    b = ctypes.c_size_t(77)
    rc = lib().orthogonalize_workspace_size(B, m, n, ctypes.byref(b))
    return b.value if rc == 0 else rc


def test_workspace_sizes():
    assert bytes_of(0, 8, 16) == 0 and bytes_of(3, 0, 16) == 0
    # the polynomial of the Gram matrix, in fp64
    assert bytes_of(5, 16, 300) >= 5 * 256 * 8
    # two X and the two symmetric matrices as pairs of fp16
    assert bytes_of(2, 100, 300) >= 2 * 2 * (2 * 100 * 300 + 2 * 100 * 100) * 2
    assert bytes_of(1, 1 << 20, 1 << 14) == RANGE and bytes_of(-1, 2, 2) == ARG
    assert lib().orthogonalize_workspace_size(1, 2, 2, None) == ARG
    # the largest sizes do not overflow
    assert bytes_of(1, 1 << 13, 1 << 20) >= 8 << 33
    assert bytes_of(1 << 13, 1, 1 << 20) > 0


def args(gpu, **other):
    t = {k: OnGpu((4, 8), other.get(k, gpu)) for k in ("x", "out", "weights", "update", "momentum")}
    t["workspace"] = OnGpu((64,), other.get("workspace", gpu), torch.uint8)
    return t


def o_call(t, **kw):
    fedavg.orthogonalize(t["x"], out=t["out"], workspace=t["workspace"], **kw)


def s_call(t, **kw):
    fedavg.orthogonal_step(t["weights"], t["update"], 0.1, momentum=t["momentum"], workspace=t["workspace"], **kw)


CALLS = [(o_call, ["out", "workspace"]), (s_call, ["update", "momentum", "workspace"])]


@pytest.mark.parametrize("call,name", [(c, n) for c, names in CALLS for n in names],
                         ids=[f"{c.__name__}-{n}" for c, names in CALLS for n in names])
def test_one_tensor_on_another_device(call, name):
    with pytest.raises(ValueError, match="GPU 1|on GPU 0"):
        call(args(0, **{name: 1}))


@pytest.mark.parametrize("call", [c for c, _ in CALLS], ids=lambda c: c.__name__)
def test_devices_and_streams(call):
    with pytest.raises(ValueError, match="current device"):
        call(args(1))
    with pytest.raises(ValueError, match="stream"):
        call(args(0), stream=Stream(1))
    with pytest.raises(AssertionError, match="went on"):
        call(args(0), stream=Stream(0))


def test_shapes_types_and_coefficients():
    t = args(0)
    with pytest.raises(ValueError):
        fedavg.orthogonalize(OnGpu((8,), 0))
    with pytest.raises(ValueError):
        fedavg.orthogonalize(OnGpu((2, 2, 4, 8), 0))
    with pytest.raises(ValueError):
        fedavg.orthogonalize(t["x"], out=OnGpu((8, 4), 0))
    with pytest.raises(TypeError):
        fedavg.orthogonalize(t["x"], out=OnGpu((4, 8), 0, torch.bfloat16))
    with pytest.raises(TypeError):
        fedavg.orthogonalize(OnGpu((4, 8), 0, torch.float16))
    with pytest.raises(TypeError):
        fedavg.orthogonal_step(t["weights"], t["update"], 0.1, momentum=OnGpu((4, 8), 0, torch.bfloat16))
    for kw in (dict(steps=0), dict(steps=33), dict(coef=(1.0, 2.0)), dict(coef=((1.0, 2.0, 3.0),) * 4),
               dict(coef=((1.0, 2.0),) * 5)):
        with pytest.raises(ValueError):
            fedavg.orthogonalize(t["x"], out=t["out"], **kw)
    with pytest.raises(AssertionError, match="went on"):
        fedavg.orthogonalize(t["x"], out=t["out"], steps=2, coef=[[1.0, 2.0, 3.0], (1, 2, 3)])
