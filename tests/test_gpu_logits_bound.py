"""GPU: rows of up to 16 KB have a bound for every k, FA_MAX_TOP, the number of
threads that share a row, among them.  Without one all entries are candidates
and the k-th is counted out bit by bit: the same result in six to ten times the
time of k = 128, where a bound takes three to four."""

import pytest
import torch

import weighted_model_update_amd as fa

pytestmark = pytest.mark.gpu


def seconds(x, k):
    out = fa.logits_topk(x, k)
    times = []
    for _ in range(7):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(10):
            fa.logits_topk(x, k, idx_out=out[0], val_out=out[1], lse_out=out[2])
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    return sorted(times)[3]


@pytest.mark.parametrize("dt,V", [(torch.bfloat16, 8192), (torch.bfloat16, 4000), (torch.float32, 4096)], ids=str)
def test_time_of_the_largest_k(dt, V):
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randn(4096, V, generator=g, device="cuda").to(dt)
    assert seconds(x, fa.FA_MAX_TOP) < 5.5 * seconds(x, 128)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("k", [203, 204, 205, 206, 230, 255, 256])
def test_values_around_the_number_of_threads(k, dt):
    for V in (513, 2049, 2056, 4000, 4096, 8191, 8192):
        x = torch.randn(9, V, generator=torch.Generator().manual_seed(V + k)).to(dt)
        x[3] = torch.arange(V).to(dt)
        x[4] = 1.0
        x[5, 300:] = -float("inf")
        x[6, ::2] = float("nan")
        idx, val, _ = fa.logits_topk(x.cuda(), k)
        y = torch.where(torch.isnan(x.float()), torch.full((), float("inf")), x.float())
        want = torch.sort(y, dim=1, descending=True, stable=True).indices[:, :k].sort(1).values
        assert torch.equal(idx.cpu().long(), want)
        assert torch.equal(val.cpu().view(torch.int32), x.float().gather(1, want).view(torch.int32))
