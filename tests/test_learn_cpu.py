"""CPU-only checks of the linear layer's, the top logits' and the distillation
loss's entry points: bad arguments are refused on the host, with the documented
code, before any device work; no-op sizes need no pointers."""

import ctypes

import pytest
import torch

import weighted_model_update_amd as fa

ARG, DTYPE, RANGE, WORKSPACE = -1, -2, -3, -8
P = ctypes.c_void_p
BASE = 1 << 40          # addresses that no refused call may touch


def at(i, off=0):
    return P(BASE + (i << 36) + off)


def forward(dtype=1, M=4, N=8, K=16, x=at(1), ldx=16, w=at(2), ldw=16, bias=at(3), act=2, alpha=1.0, res=at(4), ldr=8,
            out=at(5), ldo=8, pre=at(6), ldp=8, ws=None, wsb=0):
    return fa.load().linear_forward(dtype, M, N, K, x, ldx, w, ldw, bias, act, alpha, res, ldr, out, ldo, pre, ldp, ws,
                                    wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), DTYPE), (dict(act=4), ARG), (dict(act=-1), ARG), (dict(M=-1), ARG), (dict(K=-3), ARG),
    (dict(M=(1 << 30) + 1), RANGE), (dict(N=(1 << 28) + 1, ldo=(1 << 28) + 1, ldr=(1 << 28) + 1, ldp=(1 << 28) + 1), RANGE), (dict(M=1 << 20, N=1 << 20, ldo=1 << 20), RANGE),
    (dict(x=None), ARG), (dict(w=None), ARG), (dict(out=None), ARG),
    (dict(x=at(1, 1)), ARG), (dict(dtype=0, w=at(2, 2)), ARG), (dict(bias=at(3, 1)), ARG),
    (dict(ldx=-1), ARG), (dict(ldo=7), ARG), (dict(ldp=0), ARG), (dict(ldx=1 << 41), RANGE),
    (dict(out=at(1)), ARG), (dict(out=at(2, 32)), ARG), (dict(out=at(3, 8)), ARG), (dict(pre=at(5)), ARG),
    (dict(pre=at(4)), ARG), (dict(out=at(4, 16)), ARG), (dict(out=at(4), ldo=9), ARG),
], ids=str)
def test_forward_refusals(kw, code):
    assert forward(**kw) == code
    assert fa.load().fedavg_last_error()


def test_forward_without_outputs_is_a_no_op():
    none = dict(x=None, w=None, bias=None, res=None, out=None, pre=None)
    assert forward(M=0, **none) == 0
    assert forward(N=0, **none) == 0


def backward(dtype=1, M=4, N=8, K=16, dy=at(1), lddy=8, x=at(2), ldx=16, w=at(3), ldw=16, act=2, alpha=1.0, pre=at(4),
             ldp=8, dx=at(5), lddx=16, dw=at(6), lddw=16, db=at(7), ws=at(8), wsb=1 << 30):
    return fa.load().linear_backward(dtype, M, N, K, dy, lddy, x, ldx, w, ldw, act, alpha, pre, ldp, dx, lddx, dw, lddw,
                                     db, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), DTYPE), (dict(act=9), ARG), (dict(N=-1), ARG), (dict(N=1 << 31), RANGE),
    (dict(dy=None), ARG), (dict(x=None), ARG), (dict(w=None), ARG), (dict(pre=None), ARG),
    (dict(dy=at(1, 1)), ARG), (dict(dw=at(6, 1)), ARG), (dict(db=at(7, 1)), ARG),
    (dict(lddx=15), ARG), (dict(lddw=8), ARG), (dict(lddy=-8), ARG),
    (dict(dx=at(2)), ARG), (dict(dw=at(3)), ARG), (dict(db=at(1)), ARG), (dict(dx=at(6)), ARG), (dict(db=at(5, 32)), ARG),
    (dict(dx=at(8)), ARG), (dict(ws=None), WORKSPACE), (dict(wsb=64), WORKSPACE), (dict(ws=at(8, 8)), ARG),
], ids=str)
def test_backward_refusals(kw, code):
    assert backward(**kw) == code
    assert fa.load().fedavg_last_error()


def test_backward_without_outputs_is_a_no_op():
    assert backward(dx=None, dw=None, db=None, dy=None, x=None, w=None, pre=None, ws=None, wsb=0) == 0


def test_column_slices_of_one_buffer_do_not_overlap_but_shifted_ones_do():
    # x and out are column slices [0, 16) and [16, 24) of rows of 24: only the
    # residual's overlap with out is a fault
    ok = dict(x=at(1), ldx=24, out=at(1, 32), ldo=24, pre=None)
    assert forward(res=at(1, 34), ldr=24, **ok) == ARG
    assert b"residual" in fa.load().fedavg_last_error()
    assert forward(x=at(1), ldx=24, out=at(1, 30), ldo=24, pre=None) == ARG


def topk(x=at(1), dtype=1, R=4, V=100, ldx=100, k=5, tau=1.0, idx=at(2), val=at(3), lse=at(4), ws=at(5), wsb=1 << 34):
    return fa.load().logits_topk(x, dtype, R, V, ldx, k, tau, idx, val, lse, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), DTYPE), (dict(R=-1), ARG), (dict(V=-1), ARG), (dict(k=-1), RANGE), (dict(k=101), RANGE),
    (dict(k=257, V=1000, ldx=1000), RANGE), (dict(V=(1 << 30) + 1), RANGE), (dict(R=1 << 31), RANGE),
    (dict(tau=0.0), ARG), (dict(tau=-1.0), ARG), (dict(tau=float("nan")), ARG), (dict(tau=float("inf")), ARG),
    (dict(tau=1e-45), ARG), (dict(x=None), ARG), (dict(idx=None), ARG), (dict(val=None), ARG), (dict(x=at(1, 1)), ARG),
    (dict(idx=at(2, 2)), ARG), (dict(lse=at(4, 2)), ARG), (dict(ldx=-1), ARG), (dict(idx=at(1)), ARG), (dict(lse=at(1, 8)), ARG),
    (dict(val=at(2, 16)), ARG), (dict(idx=at(5)), ARG),
], ids=str)
def test_topk_refusals(kw, code):
    assert topk(**kw) == code
    assert fa.load().fedavg_last_error()


def test_topk_without_results_is_a_no_op():
    assert topk(R=0, x=None, idx=None, val=None, lse=None, ws=None, wsb=0) == 0
    assert topk(k=0, x=None, idx=None, val=None, lse=None, ws=None, wsb=0) == 0


def ptrs(*v):
    return (P * len(v))(*[p.value if p is not None else None for p in v])


def i64(*v):
    return (ctypes.c_int64 * len(v))(*v)


def distill(loss_call=True, clients=2, idx=(at(1), at(2)), val=(at(3), at(4)), tl=None, k=(5, 6), n=(1, 2), z=at(5), dtype=1,
            R=3, V=100, ldz=100, tau=1.0, rw=at(6), loss=at(7), lse=at(8), dz=at(9), lddz=100, err=at(10), ws=at(11),
            wsb=1 << 34):
    a = [clients, None if idx is None else ptrs(*idx), None if val is None else ptrs(*val), None if tl is None else ptrs(*tl),
         None if k is None else i64(*k), None if n is None else i64(*n), z, dtype, R, V, ldz, tau, rw]
    lib = fa.load()
    if loss_call:
        return lib.distill_loss(*a, loss, lse, dz, lddz, err, ws, wsb, None)
    return lib.distill_backward(*a, lse, dz, lddz, err, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), DTYPE), (dict(R=-1), ARG), (dict(V=-1), ARG), (dict(V=1 << 31), RANGE), (dict(tau=0.0), ARG),
    (dict(tau=float("nan")), ARG), (dict(clients=0), RANGE), (dict(clients=65), RANGE), (dict(idx=None), ARG),
    (dict(val=None), ARG), (dict(k=None), ARG), (dict(n=None), ARG), (dict(n=(1, -1)), RANGE),
    (dict(n=(1, (1 << 24) + 1)), RANGE), (dict(k=(-1, 5)), RANGE), (dict(k=(257, 5)), RANGE),
    (dict(idx=(at(1), None)), ARG), (dict(val=(None, at(4))), ARG), (dict(tl=(at(12), None)), ARG),
    (dict(idx=(at(1, 2), at(2))), ARG), (dict(tl=(at(12), at(13, 1))), ARG), (dict(z=None), ARG), (dict(z=at(5, 1)), ARG),
    (dict(ldz=-2), ARG), (dict(lddz=99), ARG), (dict(dz=at(5, 2)), ARG), (dict(dz=at(5), lddz=104), ARG),
    (dict(rw=at(6, 2)), ARG), (dict(err=at(10, 1)), ARG), (dict(lse=at(8, 2)), ARG), (dict(lse=at(9)), ARG),
    (dict(ws=at(9)), ARG),
], ids=str)
@pytest.mark.parametrize("loss_call", [True, False], ids=["loss", "backward"])
def test_distill_refusals(kw, code, loss_call):
    assert distill(loss_call, **kw) == code
    assert fa.load().fedavg_last_error()


def test_distill_refusals_of_one_call():
    assert distill(True, loss=None) == ARG
    assert distill(True, loss=at(8)) == ARG
    assert distill(True, loss=at(5)) == ARG
    assert distill(False, lse=None) == ARG
    assert distill(False, dz=None) == ARG


def test_distill_refuses_too_many_entries():
    c = 17
    many = dict(clients=c, idx=(at(1),) * c, val=(at(2),) * c, n=(1,) * c)
    assert distill(True, k=(256,) * c, **many) == RANGE
    # clients of weight 0 do not count: the next check is the one that refuses
    assert distill(True, k=(256,) * c, **{**many, "n": (1,) * 16 + (0,)}, loss=None) == ARG


def test_workspace_sizes():
    lib = fa.load()
    b = ctypes.c_size_t(7)
    assert lib.linear_workspace_size(1, 8, 8, 8, 0, 0, None) == ARG
    assert lib.linear_workspace_size(5, 8, 8, 8, 0, 0, ctypes.byref(b)) == DTYPE
    assert lib.linear_workspace_size(1, 8, -8, 8, 0, 1, ctypes.byref(b)) == ARG
    assert lib.linear_workspace_size(1, 8, 8, 8, 7, 1, ctypes.byref(b)) == ARG
    assert lib.linear_workspace_size(1, 8, 8, 1 << 31, 0, 0, ctypes.byref(b)) == RANGE
    assert lib.logits_topk_workspace_size(1, 8, 8, 9, ctypes.byref(b)) == RANGE
    assert lib.logits_topk_workspace_size(1, 8, 8, 8, None) == ARG
    assert lib.distill_workspace_size(1, 8, -1, ctypes.byref(b)) == ARG
    assert lib.distill_workspace_size(1, 8, 8, None) == ARG
    for args in ((0, 0, 0), (1, 1, 1), (1000, 1, 7)):
        assert fa.linear_workspace_size(*args, act="gelu", backward=True) >= args[0] * args[1] * 2


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x, w = torch.zeros(4, 8), torch.zeros(6, 8)
    with pytest.raises(ValueError, match="GPU"):
        fa.linear_forward(x, w)
    with pytest.raises(ValueError, match="matrices"):
        fa.linear_forward(x[0], w)
    with pytest.raises(ValueError, match="act"):
        fa.linear_forward(x, w, act="tanh")
    with pytest.raises(TypeError):
        fa.linear_forward(x.half(), w.half())
    with pytest.raises(ValueError, match="GPU"):
        fa.linear_backward(torch.zeros(4, 6), x, w)
    with pytest.raises(ValueError, match="GPU"):
        fa.logits_topk(x, 2)
    with pytest.raises(ValueError, match="GPU"):
        fa.distill_loss(x, [], [], [])
    with pytest.raises(ValueError, match="matrix"):
        fa.distill_backward(x[0], x[0], [], [], [])
