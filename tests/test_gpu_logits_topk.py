"""GPU: the top logits of rows against a plain sort, and their normaliser
against float64."""

import pytest
import torch

import learn_ref as ref
import weighted_model_update_amd as fa

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def rnd(shape, seed, scale=3.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g) * scale


def check(x, k, tau=1.0, **kw):
    idx, val, lse = fa.logits_topk(x, k, tau=tau, **kw)
    wi, wv = ref.top_rows(x, k)
    assert idx.dtype == torch.int32 and idx.shape == (x.shape[0], k)
    assert torch.equal(idx.cpu().long(), wi)
    got, want = val.cpu().view(torch.int32), wv.contiguous().view(torch.int32)
    assert torch.equal(got, want)                 # the values themselves, bit for bit
    want = ref.lse_of(x, tau)
    y = ref.d(x).abs() / tau
    top = torch.where(torch.isfinite(y), y, torch.zeros_like(y)).amax(1) if x.shape[1] else torch.zeros(x.shape[0])
    # at most V / 256 + 40 additions one after another, relative to the sum,
    # and a few roundings of the largest exponent
    slack = (x.shape[1] / 256 + 40) * ref.U32 + 16 * ref.U32 * top
    fine = torch.isfinite(want)
    ref.within(lse[fine.cuda()], want[fine], slack[fine], torch.float32, "lse")
    odd = torch.isnan(ref.d(x)).any(1) | (ref.d(x) == float("inf")).any(1)
    assert bool(torch.isnan(lse.cpu()[odd]).all())
    assert bool((lse.cpu()[(want == -float("inf")) & ~odd] == -float("inf")).all())
    return idx, val, lse


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("R,V,k", [(1, 1, 1), (3, 2, 2), (2, 63, 7), (5, 64, 64), (4, 257, 256), (2, 1000, 1), (3, 1025, 33),
                                   (2, 4099, 256), (7, 8192, 64), (2, 32003, 100), (1, 65537, 5), (1, 151936, 50),
                                   (2, 131071, 256)])
def test_random_rows(R, V, k, dt):
    check(rnd((R, V), R + V + k).to(DTYPES[dt]).cuda(), k, tau=2.0)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("V", [300, 5000, 40000])
def test_ties_and_masks(V, dt):
    t = DTYPES[dt]
    x = rnd((12, V), V)
    low = torch.finfo(t).min
    x[0] = 0.25                               # one value everywhere
    x[1] = -float("inf")                      # nothing left
    x[2] = low                                # the type's lowest everywhere
    x[3] = -float("inf"); x[3, V // 2] = 1.0  # one left
    x[4] = low; x[4, -3:] = -5.0
    x[5] = torch.arange(V) % 3                # three values
    x[6, 1::2] = -float("inf")
    x[7] = 0.0; x[7, ::2] = -0.0              # equal zeros of both signs
    x[8] = torch.arange(V).float()            # ascending
    x[9] = -torch.arange(V).float()           # descending
    x[10] = torch.where(torch.arange(V) < 200, 5.0, 4.0)
    x[11, :] = 7.5; x[11, 17] = 8.0
    for k in (1, 50, 256):
        check(x.to(t).cuda(), k)


def test_nan_and_infinities():
    for t in DTYPES.values():
        x = rnd((6, 3000), 5).to(t)
        x[0, 100] = float("nan")
        x[1, [5, 2999]] = float("inf")
        x[2] = float("nan")
        x[3, :300] = float("nan")
        x[4, ::7] = float("inf"); x[4, 3] = float("nan")
        x[5, 10] = -float("nan") if t == torch.float32 else float("nan")
        for k in (1, 64):
            check(x.cuda(), k)


def test_no_entries_and_normaliser_alone():
    x = rnd((5, 700), 1).cuda()
    check(x, 0, tau=4.0)
    for V in (0,):
        idx, val, lse = fa.logits_topk(torch.empty(3, V, device="cuda"), 0)
        assert idx.shape == (3, 0) and bool((lse == -float("inf")).all())
    idx, val, lse = fa.logits_topk(torch.empty(0, 50, device="cuda"), 5)
    assert idx.shape == (0, 5)


@pytest.mark.parametrize("dt", list(DTYPES))
def test_pitched_unaligned_and_repeated_rows(dt):
    t = DTYPES[dt]
    buf = rnd((9 * 5011 + 1,), 3).to(t).cuda()
    for cols in (5003, 5008):
        check(buf[1:].view(9, 5011)[:, :cols], 40)
    check(buf[:40000].view(5, 8000)[:, :7001], 40)
    check(buf[1:6001].view(1, 6000).expand(4, 6000), 10)


def test_outputs_given_and_nothing_else_written():
    x = rnd((4, 2000), 9).cuda()
    idx = torch.full((4 * 20 + 8,), -9, dtype=torch.int32, device="cuda")
    val = torch.full((4 * 20 + 8,), -9.0, device="cuda")
    lse = torch.full((4 + 8,), -9.0, device="cuda")
    check(x, 20, idx_out=idx[:80].view(4, 20), val_out=val[:80].view(4, 20), lse_out=lse[:4])
    assert bool((idx[80:] == -9).all()) and bool((val[80:] == -9).all()) and bool((lse[4:] == -9).all())


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("V,k", [(30000, 20), (66000, 200), (66000, 256), (9000, 256), (400000, 250)])
def test_unsplit_long_rows_and_their_rare_paths(V, k, dt):
    """More rows than CUs.  Among random rows some that rise along the row
    (every bound is too low), some that rise within one thread's share, equal
    values, and rows with fewer values than are asked for."""
    t = DTYPES[dt]
    R = 300 if V < 100000 else 260
    x = rnd((R, V), V + k).to(t)
    i = torch.arange(V)
    x[3] = (i / V * 1000).to(t)
    x[17] = (-i / V * 1000).to(t)
    x[40] = ((i // 8 * 8 % 512 == 0).float() * 50 + i / V).to(t)   # few threads hold all large values
    x[41] = ((i // 4096 % 3 == 0).float() * 50 + torch.randn(V)).to(t)
    x[99] = 2.5
    x[120] = -float("inf"); x[120, V // 3:V // 3 + 10] = 1.0
    x[121] = torch.finfo(t).min; x[121, -5:] = 0.0
    x[200] = (i % 7).to(t)
    idx, val, lse = fa.logits_topk(x.cuda(), k, tau=1.0)
    # a stable descending sort keeps equal values in index order
    want = torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :k].sort(1).values
    assert torch.equal(idx.cpu().long(), want)
    assert torch.equal(val.cpu(), x.float().gather(1, want))
    ex = ref.lse_of(x, 1.0)
    slack = (V / 256 + 40) * ref.U32 + 16 * ref.U32 * ref.d(x).clamp(min=-1e30).abs().amax(1)
    fine = ref.d(x).amax(1) > -1e30
    ref.within(lse.cpu()[fine], ex[fine], slack[fine], torch.float32, "lse")


def test_many_rows():
    x = rnd((5000, 130), 21).to(torch.bfloat16).cuda()
    check(x, 9)


def test_other_stream_and_graph_replays():
    x = rnd((6, 20000), 2).to(torch.bfloat16).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = fa.logits_topk(x, 30, stream=side)
    side.synchronize()
    for u, v in zip(a, fa.logits_topk(x, 30)):
        assert torch.equal(u, v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = fa.logits_topk(x, 30)
    for seed in (1, 2, 3):
        x.copy_(rnd((6, 20000), 100 + seed))
        graph.replay()
        torch.cuda.synchronize()
        for u, v in zip(outs, fa.logits_topk(x, 30)):
            assert torch.equal(u, v)
