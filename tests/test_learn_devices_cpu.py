"""CPU-only: the calls of the linear layer, the top logits and the distillation
refuse tensors and streams that are not on the device they would run on.
Stand-ins take the place of GPU tensors; no refused call reaches the library."""

import pytest
import torch

from weighted_model_update_amd import fedavg


class OnGpu:
    """What the checks ask of a contiguous GPU tensor; it has no memory."""

    def __init__(self, shape, gpu, dtype=torch.float32):
        self._t, self._gpu = torch.empty(shape, dtype=dtype, device="meta"), gpu
        self.is_cuda, self.dtype, self.shape = True, dtype, self._t.shape
        self.device = torch.device("cuda", gpu)

    def get_device(self):
        return self._gpu

    def data_ptr(self):
        return 1 << 40

    def __getattr__(self, name):
        return getattr(self._t, name)


class Library:
    def __getattr__(self, name):
        def call(*a):
            raise AssertionError("the call went on")
        return call


class Stream:
    cuda_stream = 0

    def __init__(self, gpu):
        self.device_index = gpu
        self.device = torch.device("cuda", gpu)


@pytest.fixture(autouse=True)
def current(monkeypatch):
    monkeypatch.setattr(fedavg, "load", Library)
    monkeypatch.setattr(fedavg, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(fedavg, "_new", lambda shape, dtype, device, stream: OnGpu(shape, device.index, dtype))
    monkeypatch.setattr(fedavg, "_bytes_of", lambda *a: 0)
    monkeypatch.setattr(fedavg, "_raw_stream", lambda *a: 0)


def args(gpu, **other):
    """Arguments of all calls on `gpu`, but for those in `other`."""
    f = dict(x=(4, 8), w=(6, 8), bias=(6,), residual=(4, 6), out=(4, 6), preact=(4, 6), dy=(4, 6), dx=(4, 8), dw=(6, 8),
             db=(6,), z=(4, 8), loss=(4,), lse=(4,), dz=(4, 8), row_weight=(4,), lse_out=(4,), val_out=(4, 2), val=(4, 2),
             teacher_lse=(4,))
    i = dict(idx_out=(4, 2), idx=(4, 2), err_flag=(1,))
    t = {k: OnGpu(s, other.get(k, gpu)) for k, s in f.items()}
    t.update({k: OnGpu(s, other.get(k, gpu), torch.int32) for k, s in i.items()})
    t["workspace"] = OnGpu((64,), other.get("workspace", gpu), torch.uint8)
    return t


def forward(t, **kw):
    fedavg.linear_forward(t["x"], t["w"], t["bias"], residual=t["residual"], out=t["out"], preact=t["preact"],
                          workspace=t["workspace"], **kw)


def backward(t, **kw):
    fedavg.linear_backward(t["dy"], t["x"], t["w"], act="gelu", preact=t["preact"], dx=t["dx"], dw=t["dw"], db=t["db"],
                           workspace=t["workspace"], **kw)


def topk(t, **kw):
    fedavg.logits_topk(t["x"], 2, idx_out=t["idx_out"], val_out=t["val_out"], lse_out=t["lse_out"], workspace=t["workspace"], **kw)


def loss(t, **kw):
    fedavg.distill_loss(t["z"], [t["idx"]], [t["val"]], [1], teacher_lse=[t["teacher_lse"]], row_weight=t["row_weight"],
                        loss=t["loss"], lse=t["lse"], dz=t["dz"], err_flag=t["err_flag"], workspace=t["workspace"], **kw)


def gradient(t, **kw):
    fedavg.distill_backward(t["z"], t["lse"], [t["idx"]], [t["val"]], [1], teacher_lse=[t["teacher_lse"]],
                            row_weight=t["row_weight"], dz=t["dz"], err_flag=t["err_flag"], workspace=t["workspace"], **kw)


LISTS = ["idx", "val", "teacher_lse", "row_weight", "lse", "dz", "err_flag", "workspace"]
CALLS = [(forward, ["w", "bias", "residual", "out", "preact", "workspace"]),
         (backward, ["dy", "w", "preact", "dx", "dw", "db", "workspace"]),
         (topk, ["idx_out", "val_out", "lse_out", "workspace"]), (loss, ["loss"] + LISTS), (gradient, LISTS)]


@pytest.mark.parametrize("call,name", [(c, n) for c, names in CALLS for n in names],
                         ids=[f"{c.__name__}-{n}" for c, names in CALLS for n in names])
def test_one_tensor_on_another_device(call, name):
    with pytest.raises(ValueError, match="GPU 1|on GPU 0"):
        call(args(0, **{name: 1}))


@pytest.mark.parametrize("call", [c for c, _ in CALLS], ids=lambda c: c.__name__)
def test_all_on_a_device_that_is_not_the_current_one(call):
    with pytest.raises(ValueError, match="current device"):
        call(args(1))


@pytest.mark.parametrize("call", [c for c, _ in CALLS], ids=lambda c: c.__name__)
def test_stream_of_another_device(call):
    with pytest.raises(ValueError, match="stream"):
        call(args(0), stream=Stream(1))


@pytest.mark.parametrize("call", [c for c, _ in CALLS], ids=lambda c: c.__name__)
def test_tensors_and_stream_of_the_current_device_pass_the_checks(call):
    with pytest.raises(AssertionError, match="went on"):
        call(args(0), stream=Stream(0))
