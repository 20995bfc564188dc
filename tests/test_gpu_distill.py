"""GPU: the distillation loss and gradient over several clients' top logits
against float64 from the definition, and against differences."""

import pytest
import torch

import learn_ref as ref
import weighted_model_update_amd as fa

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def rnd(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g) * scale


def lists(R, V, ks, seed, holes=True):
    """Ascending random lists, overlapping between clients; with holes, some
    rows end early or are empty."""
    g = torch.Generator().manual_seed(seed)
    idx, val = [], []
    pool = min(V, 2 * max(list(ks) + [1]))
    cand = torch.stack([torch.randperm(V, generator=g)[:pool] for _ in range(R)]) if R else torch.zeros(0, pool)
    for k in ks:
        i = torch.full((R, k), -1, dtype=torch.int32)
        v = torch.randn((R, k), generator=g) * 2
        for r in range(R):
            m = k if not holes or r % 3 else int(torch.randint(0, k + 1, (1,), generator=g))
            pick = torch.randperm(pool, generator=g)[:m]
            i[r, :m] = cand[r][pick].sort().values.to(torch.int32)
        idx.append(i.cuda())
        val.append(v.cuda())
    return idx, val


def check(z, idx, val, n, tau=1.0, teacher_lse=None, row_weight=None, in_place=False, pitched=None):
    err = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    kw = dict(tau=tau, teacher_lse=teacher_lse, row_weight=row_weight)
    want_loss, want_lse, want_dz, mag, flawed = ref.distill(z, idx, val, n, tau, teacher_lse, row_weight)
    loss, lse, dz = fa.distill_loss(z, idx, val, n, dz=True if pitched is None else pitched, err_flag=err, **kw)
    assert int(err) == (-7 if flawed else 0)
    R, V = z.shape
    zd = ref.d(z)
    y = torch.where(torch.isfinite(zd), zd, torch.zeros_like(zd)).abs().amax(1) / tau if V else torch.zeros(R).double()
    vmax = torch.stack([torch.where(torch.isfinite(ref.d(v)), ref.d(v), torch.zeros(()).double()).abs().amax(1) / tau
                        if v.shape[1] else torch.zeros(R).double() for v in val]).amax(0) if len(val) else y
    if teacher_lse is not None:
        vmax = vmax + torch.stack([ref.d(t).abs() for t in teacher_lse]).amax(0)
    # additions in a row: V / 256 + 40 of the softmax, k + clients of the
    # lists; exponents' roundings scale with their size
    h = V / 256 + 40 + sum(i.shape[1] for i in idx) + len(n) + 16 * (1 + y + vmax)
    fine = torch.isfinite(want_lse)
    ref.within(lse.cpu()[fine], want_lse[fine], ((V / 256 + 40) + 16 * y[fine]) * ref.U32, torch.float32, "lse")
    assert torch.equal(lse.cpu().double()[~fine], want_lse[~fine])
    ref.within(loss, want_loss, h * ref.U32 * mag * 2, torch.float32, "loss")
    gt = tau * (torch.ones(R).double() if row_weight is None else ref.d(row_weight).abs())
    p = torch.where(fine[:, None], torch.exp(zd / tau - want_lse[:, None]), torch.zeros_like(zd))
    p = torch.nan_to_num(p)
    mass = torch.zeros(R).double()
    q = torch.zeros(R, V).double()
    # |Q| = |m p - dz / (g tau)|, m = sum of Q; recovered from the exact gradient
    safe = torch.where(gt == 0, torch.ones_like(gt), gt)
    for r in range(R):
        touched = sorted({int(i) for c in range(len(n)) if int(n[c]) for i in idx[c][r] if 0 <= int(i) < V})
        if touched and gt[r] != 0:
            off = [i for i in range(V) if i not in set(touched)]
            pm = float(p[r][off].max()) if off else 0.0
            if pm > 0:
                j = off[int(p[r][off].argmax())]
                mass[r] = abs(float(want_dz[r, j])) / (float(safe[r]) * pm)
            else:
                mass[r] = 1.0 + float(want_dz[r].abs().sum()) / float(safe[r])
    q = (mass[:, None] * p - want_dz / safe[:, None]).abs()
    slack = (h * ref.U32 * 2 * gt)[:, None] * (mass[:, None] * p + q)
    ref.within(dz, want_dz, slack, z.dtype, "dz")
    back = fa.distill_backward(z, lse, idx, val, n, **kw)
    ref.within(back, want_dz, slack, z.dtype, "dz of the backward call")
    l2, e2, _ = fa.distill_loss(z, idx, val, n, **kw)
    assert torch.equal(l2, loss) and torch.equal(e2, lse)
    again = fa.distill_loss(z, idx, val, n, dz=True, **kw)[2]
    assert torch.equal(dz.contiguous().view(torch.uint8), again.view(torch.uint8))
    if in_place:
        zz = z.clone()
        fa.distill_loss(zz, idx, val, n, dz=zz, **kw)
        assert torch.equal(zz.view(torch.uint8), again.view(torch.uint8))
        zz = z.clone()
        fa.distill_backward(zz, lse, idx, val, n, dz=zz, **kw)
        assert torch.equal(zz.view(torch.uint8), back.view(torch.uint8))
    return loss, lse, dz


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("R,V,ks", [(1, 1, [1]), (2, 3, [2, 3]), (4, 64, [8]), (3, 257, [16, 1, 30]), (9, 1000, [20, 20, 20, 20]),
                                    (2, 4099, [256]), (3, 8200, [64] * 16), (2, 32003, [100, 50]), (1, 70001, [32] * 3),
                                    (2, 131073, [200]), (2, 5000, [256] * 16), (2, 300, [3] * 64)])
def test_against_the_definition(R, V, ks, dt):
    z = rnd((R, V), R * V + len(ks), 2.5).to(DTYPES[dt]).cuda()
    idx, val = lists(R, V, ks, 7 + V)
    n = [50 + 31 * c for c in range(len(ks))]
    check(z, idx, val, n, tau=2.0, in_place=True)


@pytest.mark.parametrize("dt", list(DTYPES))
def test_teacher_normalisers_and_row_weights(dt):
    R, V, ks = 8, 3001, [40, 12]
    z = rnd((R, V), 3, 2.0).to(DTYPES[dt]).cuda()
    idx, val = lists(R, V, ks, 4)
    tl = [(torch.logsumexp(v / 1.5, 1) + 0.4).contiguous() for v in val]
    rw = torch.tensor([0.0, 1.0, 0.5, 0.0, -2.0, 3.0, 1e-3, 0.0]).cuda()
    loss, lse, dz = check(z, idx, val, [10, 1000], tau=1.5, teacher_lse=tl, row_weight=rw, in_place=True)
    gone = rw.cpu() == 0
    assert bool((loss.cpu()[gone] == 0).all()) and bool((dz.cpu()[gone] == 0).all()) and bool((lse.cpu()[gone] == 0).all())


def test_rows_of_weight_zero_are_not_read():
    z = rnd((4, 500), 1).cuda()
    z[1] = float("nan")
    idx, val = lists(4, 500, [9], 2, holes=False)
    val[0][1] = float("nan")
    idx[0][1] = 12345                  # flawed, but of a row that is left out
    rw = torch.tensor([1.0, 0.0, 1.0, 1.0]).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, lse, dz = fa.distill_loss(z, idx, val, [5], row_weight=rw, dz=True, err_flag=err)
    assert int(err) == 0
    assert float(loss[1]) == 0 and float(lse[1]) == 0 and bool((dz[1] == 0).all())
    assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(dz).all())


@pytest.mark.parametrize("dt", list(DTYPES))
def test_masked_student_and_unsent_rows(dt):
    t = DTYPES[dt]
    R, V = 8, 900
    z = rnd((R, V), 11, 2.0)
    z[0] = -float("inf")                          # nothing left
    z[1, 300:] = -float("inf")
    z[2] = torch.finfo(t).min                     # the type's lowest everywhere: uniform
    z[3, 300:] = torch.finfo(t).min
    z[4] = -float("inf"); z[4, 7] = 3.0
    idx, val = lists(R, 300, [20, 10], 5)
    idx[0][4] = -1; idx[1][4] = -1                # a row that no client sent
    idx[0][5] = -1                                # one that only the second did
    val[0][6] = -float("inf")                     # entries that are all -inf: not sent
    val[1][7, :3] = -float("inf")                 # some of them
    z[2:4] /= 2                                   # keep sums of the lowest finite
    check(z.to(t).cuda(), idx, val, [3, 4], tau=1.0, in_place=True)


def test_clients_of_weight_zero_are_not_read():
    R, V = 3, 400
    z = rnd((R, V), 2).cuda()
    idx, val = lists(R, V, [9, 9], 3, holes=False)
    a = fa.distill_loss(z, [idx[0], None, idx[1]], [val[0], None, val[1]], [7, 0, 9], dz=True)
    b = fa.distill_loss(z, idx, val, [7, 9], dz=True)
    for u, v in zip(a, b):
        assert torch.equal(u, v)
    loss, _, dz = fa.distill_loss(z, [None], [None], [0], dz=True)
    assert bool((loss == 0).all()) and bool((dz == 0).all())


def test_flawed_lists_are_left_out_and_reported():
    R, V = 6, 700
    z = rnd((R, V), 2).cuda()
    idx, val = lists(R, V, [12, 12], 3, holes=False)
    idx[0][0, 3] = idx[0][0, 2]                   # twice
    idx[0][1, 11] = V                             # past the end
    idx[1][2, 0] = idx[1][2, 5]                   # out of order
    idx[0][3, 6] = 2 ** 31 - 1
    idx[0][4, 6] = -5                             # ends the list, no flaw
    check(z, idx, val, [1, 2], tau=1.0)


def test_nan_and_infinity_propagate_within_their_row():
    R, V = 5, 600
    z = rnd((R, V), 2).cuda()
    z[1, 50] = float("nan")
    z[2, 60] = float("inf")
    idx, val = lists(R, V, [10], 3, holes=False)
    val[0][3, 4] = float("nan")
    loss, lse, dz = fa.distill_loss(z, idx, val, [1], dz=True)
    for r in (1, 2, 3):
        assert not bool(torch.isfinite(loss[r])) and bool(torch.isnan(dz[r]).any())
    for r in (0, 4):
        assert bool(torch.isfinite(loss[r])) and bool(torch.isfinite(dz[r]).all())
    assert bool(torch.isnan(lse[1:3]).all())


@pytest.mark.parametrize("dt", list(DTYPES))
def test_pitched_views_and_untouched_gaps(dt):
    t = DTYPES[dt]
    for shift, ld, V in ((0, 1032, 1000), (1, 1003, 1001), (3, 5000, 4999)):
        R = 4
        z = rnd((R * ld + shift + 8,), 3).to(t).cuda()[shift:shift + R * ld].view(R, ld)[:, :V]
        idx, val = lists(R, V, [15, 15], 4)
        buf = torch.full((R * ld + shift + 8,), -77.0, dtype=t, device="cuda")
        dz = buf[shift:shift + R * ld].view(R, ld)[:, :V]
        check(z, idx, val, [3, 5], tau=2.0, pitched=dz)
        dz.fill_(-77.0)
        assert bool((buf == -77.0).all())


def test_against_differences():
    """Central differences of the fp32 loss along random directions.  With
    step h the third-order term is below h^2 / 6 times m tau^2 (sum |v|^3 /
    tau^3 weighted by p: at most the largest |v| cubed), the loss is rounded
    to half a step of its magnitude, divided by h."""
    R, V, tau = 3, 500, 2.0
    z = rnd((R, V), 2, 2.0).cuda()
    idx, val = lists(R, V, [20, 20, 20], 3, holes=False)
    n = [5, 6, 7]
    loss, lse, dz = fa.distill_loss(z, idx, val, n, tau=tau, dz=True)
    _, _, _, mag, _ = ref.distill(z, idx, val, n, tau)
    h = 2.0 ** -4
    for seed in range(4):
        v = rnd((R, V), 90 + seed).cuda()
        up = fa.distill_loss(z + h * v, idx, val, n, tau=tau)[0].double()
        dn = fa.distill_loss(z - h * v, idx, val, n, tau=tau)[0].double()
        slope = ((up - dn) / (2 * h)).cpu()
        want = (dz.double() * v.double()).sum(1).cpu()
        third = h * h / 6 * 8 * float(v.abs().max()) ** 3 / tau
        noise = 200 * ref.U32 * mag / h
        assert bool(((slope - want).abs() <= third + noise).all()), (slope, want, third, noise)


def test_empty_sizes():
    loss, lse, dz = fa.distill_loss(torch.empty(0, 9, device="cuda"), [torch.empty(0, 3, dtype=torch.int32, device="cuda")],
                                    [torch.empty(0, 3, device="cuda")], [1], dz=True)
    assert loss.shape == (0,) and dz.shape == (0, 9)
    idx = [torch.full((3, 2), -1, dtype=torch.int32, device="cuda")]
    loss, lse, _ = fa.distill_loss(torch.empty(3, 0, device="cuda"), idx, [torch.zeros(3, 2, device="cuda")], [1])
    assert bool((loss == 0).all()) and bool((lse == -float("inf")).all())
    z = rnd((3, 40), 1).cuda()
    loss, _, dz = fa.distill_loss(z, [torch.empty(3, 0, dtype=torch.int32, device="cuda")], [torch.empty(3, 0, device="cuda")],
                                  [1], dz=True)
    assert bool((loss == 0).all()) and bool((dz == 0).all())


@pytest.mark.parametrize("dt", list(DTYPES))
def test_more_rows_than_workgroups_hold_at_once(dt):
    # rows are not split: the paths that keep a row, with long lists, padding
    # rows, and dense clusters of listed indices
    R, V = 300, 9001
    z = rnd((R, V), 5, 2.0).to(DTYPES[dt]).cuda()
    g = torch.Generator().manual_seed(8)
    idx, val = [], []
    for k in (200, 64, 3):
        i = torch.rand(R, 1200, generator=g).topk(k, 1).indices.sort(1).values.to(torch.int32)
        i[::7, k // 2:] = -1
        idx.append((i + torch.where(i >= 0, 4000, 0)).int().cuda())
        val.append(torch.randn(R, k, generator=g).cuda())
    rw = torch.rand(R, generator=g) + 0.5
    rw[::5] = 0.0
    check(z, idx, val, [3, 1, 9], tau=1.5, row_weight=rw.cuda(), in_place=True)


def test_very_long_row():
    # chains of chunks cover several chunks
    R, V = 2, 300007
    z = rnd((R, V), 5, 2.0).to(torch.bfloat16).cuda()
    idx, val = lists(R, V, [256] * 4, 9, holes=False)
    check(z, idx, val, [3, 1, 9, 2], tau=2.0, in_place=True)


def test_many_rows():
    R, V = 6000, 70
    z = rnd((R, V), 2).to(torch.bfloat16).cuda()
    g = torch.Generator().manual_seed(1)
    idx = [torch.rand(R, V, generator=g).topk(5, 1).indices.sort(1).values.to(torch.int32).cuda() for _ in range(2)]
    val = [torch.randn(R, 5, generator=g).cuda() for _ in range(2)]
    check(z, idx, val, [1, 3], tau=1.0)


def test_clients_top_logits_feed_the_loss():
    """The lists logits_topk makes, against a dense Kullback-Leibler loss of
    the same kept entries."""
    R, V, k = 5, 2000, 40
    teachers = [rnd((R, V), 60 + c, 3.0).cuda() for c in range(3)]
    sent = [fa.logits_topk(x, k, tau=2.0) for x in teachers]
    z = rnd((R, V), 70, 2.0).cuda()
    for tl in (None, [s[2] for s in sent]):
        check(z, [s[0] for s in sent], [s[1] for s in sent], [1, 2, 3], tau=2.0, teacher_lse=tl)


def test_other_stream_and_graph_replays():
    R, V = 7, 9001
    z = rnd((R, V), 2, 2.0).to(torch.bfloat16).cuda()
    idx, val = lists(R, V, [30, 30], 3)
    n = [2, 5]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = fa.distill_loss(z, idx, val, n, dz=True, stream=side)
    side.synchronize()
    for u, v in zip(a, fa.distill_loss(z, idx, val, n, dz=True)):
        assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))

    def step():
        loss, lse, dz = fa.distill_loss(z, idx, val, n, dz=True)
        return loss, lse, dz, fa.distill_backward(z, lse, idx, val, n)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in (1, 2, 3):
        z.copy_(rnd((R, V), 100 + seed, 2.0))
        graph.replay()
        torch.cuda.synchronize()
        for u, v in zip(outs, step()):
            assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))
