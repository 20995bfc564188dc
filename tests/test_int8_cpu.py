"""CPU-only: the calls of the layers on 8-bit weights refuse bad arguments,
shared memory and tensors of another device before any device work."""

import ctypes

import pytest
import torch

import weighted_model_update_amd as fa
from test_learn_cpu import ARG, DTYPE, RANGE, WORKSPACE, at
from test_learn_devices_cpu import OnGpu, Stream, current  # noqa: F401
from weighted_model_update_amd import fedavg


def lib():
    return fa.load()


def quantize(dtype=1, R=4, C=16, x=at(1), ldx=16, q=at(2), ldq=16, scale=at(3)):
    return lib().quantize_rows(x, dtype, R, C, ldx, q, ldq, scale, None)


def forward(dtype=1, M=4, N=8, K=16, x=at(1), ldx=16, xs=at(10), w=at(2), ldw=16, ws=at(11), bias=at(3), act=2, alpha=1.0,
            res=at(4), ldr=8, out=at(5), ldo=8, pre=at(6), ldp=8, work=at(12), workb=1 << 20):
    return lib().linear_int8_forward(dtype, M, N, K, x, ldx, xs, w, ldw, ws, bias, act, alpha, res, ldr, out, ldo, pre,
                                     ldp, work, workb, None)


def backward(dtype=1, M=4, N=8, K=16, dy=at(1), lddy=8, w=at(2), ldw=16, ws=at(11), act=2, alpha=1.0, pre=at(6), ldp=8,
             dx=at(4), lddx=16, db=at(5), work=at(12), workb=1 << 20):
    return lib().linear_int8_backward(dtype, M, N, K, dy, lddy, w, ldw, ws, act, alpha, pre, ldp, dx, lddx, db, work,
                                      workb, None)


BIG = 1 << 17


@pytest.mark.parametrize("call,kw,code", [
    (quantize, dict(dtype=2), DTYPE), (quantize, dict(R=-1), ARG), (quantize, dict(C=-1), ARG),
    (quantize, dict(R=1 << 20, C=1 << 17, ldx=BIG, ldq=BIG), RANGE), (quantize, dict(R=1 << 37), RANGE),
    (quantize, dict(x=None), ARG), (quantize, dict(q=None), ARG), (quantize, dict(scale=None), ARG),
    (quantize, dict(x=at(1, 1)), ARG), (quantize, dict(scale=at(3, 2)), ARG), (quantize, dict(ldx=-16), ARG),
    (quantize, dict(ldq=15), ARG), (quantize, dict(ldx=1 << 41), RANGE),
    (quantize, dict(q=at(1, 100)), ARG), (quantize, dict(scale=at(1, 16)), ARG), (quantize, dict(scale=at(2, 60)), ARG),
    (forward, dict(dtype=2), DTYPE), (forward, dict(act=4), ARG), (forward, dict(M=-1), ARG),
    (forward, dict(K=BIG, ldx=BIG, ldw=BIG), RANGE), (forward, dict(N=(1 << 28) + 1), RANGE),
    (forward, dict(x=None), ARG), (forward, dict(w=None), ARG), (forward, dict(ws=None), ARG), (forward, dict(out=None), ARG),
    (forward, dict(xs=at(10, 2)), ARG), (forward, dict(ws=at(11, 1)), ARG), (forward, dict(bias=at(3, 1)), ARG),
    (forward, dict(ldx=-1), ARG), (forward, dict(ldo=7), ARG), (forward, dict(ldp=0), ARG),
    (forward, dict(xs=None, x=at(1, 1)), ARG), (forward, dict(xs=None, work=None), WORKSPACE),
    (forward, dict(xs=None, workb=100), WORKSPACE), (forward, dict(xs=None, work=at(12, 8)), ARG),
    (forward, dict(out=at(1)), ARG), (forward, dict(out=at(2, 100)), ARG), (forward, dict(out=at(10, 8)), ARG),
    (forward, dict(out=at(11, 28)), ARG), (forward, dict(out=at(3)), ARG), (forward, dict(pre=at(5)), ARG),
    (forward, dict(pre=at(4)), ARG), (forward, dict(out=at(4, 16)), ARG), (forward, dict(pre=at(12)), ARG),
    (forward, dict(work=at(1)), ARG), (forward, dict(work=at(10)), ARG), (forward, dict(work=at(2)), ARG),
    (forward, dict(work=at(11)), ARG), (forward, dict(work=at(3)), ARG), (forward, dict(work=at(4)), ARG),
    (forward, dict(M=20, N=8192, K=16384, ldx=16384, ldw=16384, ldr=8192, ldo=8192, ldp=8192, work=None), WORKSPACE),
    (backward, dict(dtype=2), DTYPE), (backward, dict(act=-1), ARG), (backward, dict(N=-1), ARG),
    (backward, dict(K=BIG, ldw=BIG, lddx=BIG), RANGE), (backward, dict(N=(1 << 22) + 1, lddy=1 << 23, ldp=1 << 23), RANGE),
    (backward, dict(dy=None), ARG), (backward, dict(w=None), ARG), (backward, dict(ws=None), ARG), (backward, dict(pre=None), ARG),
    (backward, dict(dy=at(1, 1)), ARG), (backward, dict(lddx=15), ARG), (backward, dict(lddy=-8), ARG),
    (backward, dict(dx=at(1)), ARG), (backward, dict(dx=at(2)), ARG), (backward, dict(dx=at(11, 4)), ARG),
    (backward, dict(dx=at(6)), ARG), (backward, dict(db=at(1)), ARG), (backward, dict(db=at(4, 32)), ARG),
    (backward, dict(work=None), WORKSPACE), (backward, dict(workb=64), WORKSPACE), (backward, dict(work=at(12, 8)), ARG),
    (backward, dict(work=at(1)), ARG), (backward, dict(work=at(2)), ARG), (backward, dict(work=at(11)), ARG),
    (backward, dict(work=at(6)), ARG), (backward, dict(work=at(4)), ARG),
], ids=lambda v: getattr(v, "__name__", str(v)))
def test_refusals(call, kw, code):
    assert call(**kw) == code
    assert lib().fedavg_last_error()


def test_calls_without_outputs_are_no_ops():
    none = dict(x=None, xs=None, w=None, ws=None, bias=None, res=None, out=None, pre=None, work=None, workb=0)
    assert forward(M=0, **none) == 0 and forward(N=0, **none) == 0
    assert quantize(R=0, x=None, q=None, scale=None) == 0
    assert backward(dx=None, db=None, dy=None, w=None, ws=None, pre=None, work=None) == 0


def bytes_of(M, N, K, dtype=1, quantized=0, backward=0):
    b = ctypes.c_size_t(77)
    rc = lib().linear_int8_workspace_size(dtype, M, N, K, quantized, backward, ctypes.byref(b))
    return b.value if rc == 0 else rc


def test_workspace_sizes():
    assert bytes_of(0, 8, 16) == 0
    # x in 8 bits with its scales
    assert bytes_of(4, 8, 17) >= 4 * 32 + 4 * 4
    assert bytes_of(4, 8, 17, quantized=1) == 0
    # dz and the weights as values
    assert bytes_of(100, 64, 200, dtype=0, backward=1) >= 100 * 64 * 4 + 64 * 200
    assert bytes_of(4, 8, BIG) == RANGE and bytes_of(4, 8, 16, dtype=3) == DTYPE
    assert lib().linear_int8_workspace_size(1, 4, 8, 16, 0, 0, None) == ARG


def i8(shape, gpu=0):
    return OnGpu(shape, gpu, torch.int8)


def f32(shape, gpu=0):
    return OnGpu(shape, gpu)


def args(gpu, **other):
    at_ = lambda name: other.get(name, gpu)  # noqa: E731
    t = {k: f32(s, at_(k)) for k, s in dict(x=(4, 8), w_scale=(6,), x_scale=(4,), bias=(6,), residual=(4, 6), out=(4, 6),
                                            preact=(4, 6), dy=(4, 6), dx=(4, 8), db=(6,), scale=(4,)).items()}
    t.update(w=i8((6, 8), at_("w")), xq=i8((4, 8), at_("xq")), q=i8((4, 8), at_("q")),
             workspace=OnGpu((64,), at_("workspace"), torch.uint8))
    return t


def q_call(t, **kw):
    fedavg.quantize_rows(t["x"], q=t["q"], scale=t["scale"], **kw)


def f_call(t, **kw):
    fedavg.linear_int8_forward(t["xq"], t["w"], t["w_scale"], t["bias"], residual=t["residual"], x_scale=t["x_scale"],
                               out=t["out"], preact=t["preact"], workspace=t["workspace"], **kw)


def b_call(t, **kw):
    fedavg.linear_int8_backward(t["dy"], t["w"], t["w_scale"], act="gelu", preact=t["preact"], dx=t["dx"], db=t["db"],
                                workspace=t["workspace"], **kw)


CALLS = [(q_call, ["q", "scale"]), (f_call, ["w", "w_scale", "x_scale", "bias", "residual", "out", "preact", "workspace"]),
         (b_call, ["w", "w_scale", "preact", "dx", "db", "workspace"])]


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


def test_types_and_shapes():
    t = args(0)
    with pytest.raises(TypeError):
        fedavg.quantize_rows(i8((4, 8)))
    with pytest.raises(TypeError):
        fedavg.linear_int8_forward(t["xq"], t["w"], t["w_scale"])          # 8-bit tokens without their scales
    with pytest.raises(TypeError):
        fedavg.linear_int8_forward(t["x"], t["w"], t["w_scale"], x_scale=t["x_scale"])
    with pytest.raises(TypeError):
        fedavg.linear_int8_forward(t["x"], t["x"], t["w_scale"])
    with pytest.raises(TypeError):
        fedavg.linear_int8_forward(t["x"], t["w"], t["w_scale"], dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        fedavg.linear_int8_forward(t["xq"], t["w"], t["w_scale"], x_scale=t["x_scale"], dtype=torch.float16)
    with pytest.raises(ValueError):
        fedavg.linear_int8_forward(t["x"], t["w"], t["x_scale"])
    with pytest.raises(ValueError):
        fedavg.quantize_rows(t["x"], q=i8((4, 9)))
    with pytest.raises(ValueError):
        fedavg.linear_int8_forward(t["x"], t["w"], t["w_scale"], act="tanh")
