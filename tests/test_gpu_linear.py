"""GPU: the linear layer (forward, backward) against float64, at the sizes,
pitches and alignments where a tiled kernel can go wrong."""

import pytest
import torch

import learn_ref as ref
import weighted_model_update_amd as fa

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ["none", "relu", "gelu", "silu"]

# one, below, at and above the tile and step sizes; odd in each dimension;
# ranks of adapters; single tokens; long sums
SHAPES = [(1, 1, 1), (1, 16, 8), (3, 5, 7), (16, 16, 64), (17, 33, 65), (128, 128, 64), (129, 257, 130),
          (1, 1000, 4096), (5, 512, 2048), (16, 1030, 520), (33, 96, 72), (300, 16, 1024), (1000, 16, 136), (777, 4, 96),
          (64, 1000, 16), (513, 384, 16), (257, 264, 1000), (256, 256, 512), (300, 520, 264), (2, 40, 9000),
          (700, 513, 257), (520, 1032, 128)]


def rnd(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def padded(rows, cols, ld, shift, dtype, seed, fill=None):
    """A [rows, cols] view with row pitch ld, `shift` elements into its
    buffer; the buffer too."""
    buf = rnd((rows * ld + shift + 8,), dtype, seed) if fill is None else \
        torch.full((rows * ld + shift + 8,), fill, dtype=dtype, device="cuda")
    return buf[shift:shift + rows * ld].view(rows, ld)[:, :cols], buf


def check_forward(x, w, bias, act, residual, alpha, out, pre):
    y, z, mag = ref.linear(x, w, bias, act, residual, alpha)
    # K additions in any order and the epilogue's few roundings, each at most
    # half a step of what entered; the activations' slopes are below 1.13
    slack = 1.2 * (x.shape[1] + 32) * ref.U32 * mag
    ref.within(out, y, slack, x.dtype, "out")
    if pre is not None:
        ref.within(pre, z, slack, x.dtype, "preact")


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, dt):
    M, N, K = shape
    t = DTYPES[dt]
    act = ACTS[(M + N + K) % 4]
    x, w = rnd((M, K), t, 1), rnd((N, K), t, 2, K ** -0.5)
    bias, res = rnd((N,), t, 3), rnd((M, N), t, 4)
    pre = torch.empty(M, N, dtype=t, device="cuda")
    out = fa.linear_forward(x, w, bias, act=act, residual=res, alpha=0.5, preact=pre)
    check_forward(x, w, bias, act, res, 0.5, out, pre)
    plain = fa.linear_forward(x, w)
    check_forward(x, w, None, "none", None, 1.0, plain, None)
    again = fa.linear_forward(x, w)
    assert torch.equal(plain.view(torch.uint8), again.view(torch.uint8))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", list(DTYPES))
def test_forward_activations_over_their_range(dt, act):
    t = DTYPES[dt]
    K = 8
    x = torch.linspace(-30, 30, 4001).to(t).cuda()[:, None].expand(-1, K).contiguous()
    x[:, 1:] = 0
    w = torch.eye(K, dtype=t, device="cuda")[:1].expand(24, K).contiguous()
    out = fa.linear_forward(x, w, act=act)
    y, z, mag = ref.linear(x, w, None, act, None, 1.0)
    # 1 + erf cancels below zero: up to half a step of 1, times |z| / 2
    slack = (16 + K) * ref.U32 * mag
    ref.within(out, y, slack, t, "out")


def shape_views(M, N, K, t, odd):
    pad = 3 if odd else 8
    shift = 1 if odd else 0
    x, _ = padded(M, K, K + pad, shift, t, 11)
    w, _ = padded(N, K, K + 2 * pad, shift, t, 12)
    res, _ = padded(M, N, N + pad, shift, t, 13)
    return x, w, res, pad, shift


@pytest.mark.parametrize("odd", [False, True], ids=["pitch", "unaligned"])
@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("shape", [(1, 40, 64), (19, 72, 200), (140, 136, 72), (300, 24, 512), (300, 520, 136)], ids=str)
def test_forward_pitched_views_and_untouched_gaps(shape, dt, odd):
    M, N, K = shape
    t = DTYPES[dt]
    x, w, res, pad, shift = shape_views(M, N, K, t, odd)
    out, obuf = padded(M, N, N + pad, shift, t, 0, fill=-77.0)
    pre, pbuf = padded(M, N, N + 2 * pad, shift, t, 0, fill=-55.0)
    bias = rnd((N + 1,), t, 14)[1:]
    fa.linear_forward(x, w, bias, act="silu", residual=res, out=out, preact=pre)
    check_forward(x, w, bias, "silu", res, 1.0, out, pre)
    for v, buf, fill in ((out, obuf, -77.0), (pre, pbuf, -55.0)):
        v.fill_(fill)
        assert bool((buf == fill).all())


def test_forward_repeated_rows_and_in_place_residual():
    t = torch.bfloat16
    M, N, K = 70, 136, 96
    x = rnd((1, K), t, 1).expand(M, K)          # pitch 0
    w = rnd((N, K), t, 2, K ** -0.5)
    res = rnd((1, N), t, 3).expand(M, N)
    check_forward(x, w, None, "gelu", res, 1.0, fa.linear_forward(x, w, act="gelu", residual=res), None)
    h = rnd((M, N), t, 4)
    before = h.clone()
    assert fa.linear_forward(x, w, residual=h, out=h) is h
    check_forward(x, w, None, "none", before, 1.0, h, None)


def test_forward_column_slices_of_one_buffer():
    t = torch.float32
    buf = rnd((50, 200), t, 5)
    x, out = buf[:, :96], buf[:, 96:160]
    w = rnd((64, 96), t, 6)
    want = ref.linear(x, w, None, "none", None, 1.0)
    fa.linear_forward(x, w, out=out)
    ref.within(out, want[0], 1.2 * 128 * ref.U32 * want[2], t, "out")


def test_forward_infinities_and_nan_stay_in_their_rows_and_columns():
    for t in DTYPES.values():
        x, w = rnd((40, 72), t, 1), rnd((48, 72), t, 2)
        x[3, 5], x[20, 71] = float("nan"), float("inf")
        w[7, 0] = float("nan")
        out = fa.linear_forward(x, w).cpu()
        good = torch.ones(40, 48, dtype=torch.bool)
        good[3], good[20], good[:, 7] = False, False, False
        assert bool(torch.isfinite(out[good]).all())
        assert bool(torch.isnan(out[3]).all()) and bool(torch.isnan(out[:, 7]).all())
        assert not bool(torch.isfinite(out[20]).any())


def test_empty_sizes():
    for t in DTYPES.values():
        bias, res = rnd((24,), t, 1), rnd((5, 24), t, 2)
        out = fa.linear_forward(torch.empty(5, 0, dtype=t, device="cuda"), torch.empty(24, 0, dtype=t, device="cuda"),
                                bias, act="gelu", residual=res)
        ref.within(out, ref.act(ref.d(bias)[None], "gelu") + ref.d(res), 64 * ref.U32 * 8, t)
        assert fa.linear_forward(torch.empty(0, 8, dtype=t, device="cuda"), rnd((4, 8), t, 3)).shape == (0, 4)
        # no rows: the gradients of the weights are zero
        dx, dw, db = fa.linear_backward(torch.empty(0, 24, dtype=t, device="cuda"),
                                        torch.empty(0, 40, dtype=t, device="cuda"), rnd((24, 40), t, 4), db=True)
        assert dx.shape == (0, 40) and bool((dw == 0).all()) and bool((db == 0).all())
        dx, dw, db = fa.linear_backward(torch.empty(7, 0, dtype=t, device="cuda"), rnd((7, 40), t, 5),
                                        torch.empty(0, 40, dtype=t, device="cuda"), db=True)
        assert bool((dx == 0).all()) and dw.shape == (0, 40)


def check_backward(dy, x, w, act, pre, alpha, dx, dw, db):
    t = x.dtype
    z = ref.d(pre) if pre is not None else torch.zeros(dy.shape).double()
    dz = ref.d(dy) * ref.act_slope(z, act)
    # the slope's own roundings, at most a few steps of 1 + |z|
    size = ref.d(dy).abs() * (1 + z.abs())
    M, N = dy.shape
    held = ref.half_step(t) if pre is not None else 0.0   # dz in the element type
    wx, ww = ref.d(x), ref.d(w)
    if dx is not None:
        m1, m2 = abs(alpha) * (size @ ww.abs()), abs(alpha) * (dz.abs() @ ww.abs())
        ref.within(dx, alpha * (dz @ ww), (N + 48) * ref.U32 * m1 + held * 1.01 * m2, t, "dx")
    if dw is not None:
        m1, m2 = abs(alpha) * (size.t() @ wx.abs()), abs(alpha) * (dz.abs().t() @ wx.abs())
        ref.within(dw, alpha * (dz.t() @ wx), (M + 48) * ref.U32 * m1 + held * 1.01 * m2, t, "dw")
    if db is not None:
        ref.within(db, dz.sum(0), (M + 48) * ref.U32 * size.sum(0), t, "db")


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(shape, dt):
    M, N, K = shape
    t = DTYPES[dt]
    act = ACTS[(M + 2 * N + K) % 4]
    dy, x, w = rnd((M, N), t, 1), rnd((M, K), t, 2), rnd((N, K), t, 3, K ** -0.5)
    pre = rnd((M, N), t, 4, 1.5) if act != "none" else None
    got = fa.linear_backward(dy, x, w, act=act, preact=pre, alpha=2.0, db=True)
    check_backward(dy, x, w, act, pre, 2.0, *got)
    again = fa.linear_backward(dy, x, w, act=act, preact=pre, alpha=2.0, db=True)
    for a, b in zip(got, again):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# enough tiles for the larger tile sizes, ragged at both edges; the last two
# unaligned
LARGE = [(2058, 2184, 72), (2600, 5400, 136), (2600, 136, 5400), (136, 2600, 5400), (2059, 2183, 71), (2601, 5399, 67)]


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("shape", LARGE, ids=str)
def test_large_tiles(shape, dt):
    M, N, K = shape
    t = DTYPES[dt]
    x, w, dy = rnd((M, K), t, 1), rnd((N, K), t, 2, K ** -0.5), rnd((M, N), t, 3)
    bias, res = rnd((N,), t, 4), rnd((M, N), t, 5)
    pre = torch.empty(M, N, dtype=t, device="cuda")
    out = fa.linear_forward(x, w, bias, act="silu", residual=res, preact=pre)
    check_forward(x, w, bias, "silu", res, 1.0, out, pre)
    check_backward(dy, x, w, "none", None, 1.0, *fa.linear_backward(dy, x, w, db=True))


@pytest.mark.parametrize("dt", list(DTYPES))
def test_large_products_of_views_off_16_bytes(dt):
    # sizes that are whole chunks at addresses that are not
    t = DTYPES[dt]
    M, N, K = 2056, 2072, 136
    if dt == "f32":
        M, N = 3000, 3080
    x, _ = padded(M, K, K, 1, t, 1)
    w, _ = padded(N, K, K + 3, 0, t, 2)
    dy, _ = padded(M, N, N, 3, t, 3)
    out, obuf = padded(M, N, N + 1, 1, t, 0, fill=-77.0)
    fa.linear_forward(x, w, out=out)
    check_forward(x, w, None, "none", None, 1.0, out, None)
    out.fill_(-77.0)
    assert bool((obuf == -77.0).all())
    wide = padded(M, N, N, 1, t, 4)[0]       # as the left operand's partner: dx and dw of that size
    g, _ = padded(M, K, K, 1, t, 5)
    dx, dw, _ = fa.linear_backward(g, wide, padded(K, N, N, 1, t, 6)[0])
    check_backward(g, wide, padded(K, N, N, 1, t, 6)[0], "none", None, 1.0, dx, dw, None)


# outputs [P, Q] and sum length r that take each tile, ragged at both edges, in
# all three products: the forward one, dx and dw
@pytest.mark.parametrize("P,Q,r", [(2041, 2040, 136), (634, 12792, 72), (12792, 634, 136), (2600, 5400, 200), (2041, 2040, 72),
                                   (130, 264, 2200), (10, 300, 1544), (1032, 16, 2056), (2041, 2039, 71)], ids=str)
def test_each_tile_in_each_product(P, Q, r):
    t = torch.bfloat16
    a, b = rnd((P, r), t, 1), rnd((Q, r), t, 2, r ** -0.5)
    check_forward(a, b, None, "none", None, 1.0, fa.linear_forward(a, b), None)
    dy, w = rnd((P, r), t, 3), rnd((r, Q), t, 4, r ** -0.5)
    got = fa.linear_backward(dy, torch.empty(P, Q, dtype=t, device="cuda"), w, dx=True, dw=None)
    check_backward(dy, torch.zeros(P, Q, dtype=t), w, "none", None, 1.0, got[0], None, None)
    dy, x = rnd((r, P), t, 5), rnd((r, Q), t, 6, r ** -0.5)
    got = fa.linear_backward(dy, x, torch.empty(P, Q, dtype=t, device="cuda"), dx=None, dw=True)
    check_backward(dy, x, torch.zeros(P, Q, dtype=t), "none", None, 1.0, None, got[1], None)


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("only", ["dx", "dw", "db"])
def test_backward_each_gradient_alone(only, act):
    t = torch.bfloat16
    M, N, K = 150, 72, 88
    dy, x, w = rnd((M, N), t, 1), rnd((M, K), t, 2), rnd((N, K), t, 3)
    pre = rnd((M, N), t, 4) if act != "none" else None
    got = fa.linear_backward(dy, x, w, act=act, preact=pre, dx=only == "dx", dw=only == "dw", db=only == "db")
    assert [g is not None for g in got] == [only == n for n in ("dx", "dw", "db")]
    check_backward(dy, x, w, act, pre, 1.0, *got)


@pytest.mark.parametrize("odd", [False, True], ids=["pitch", "unaligned"])
@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("shape", [(1, 40, 64), (19, 72, 200), (300, 136, 24), (300, 24, 136), (270, 264, 272)], ids=str)
def test_backward_pitched_views_and_untouched_gaps(shape, dt, odd):
    M, N, K = shape
    t = DTYPES[dt]
    x, w, pre, pad, shift = shape_views(M, N, K, t, odd)
    dy, _ = padded(M, N, N + 2 * pad, shift, t, 21)
    dx, xbuf = padded(M, K, K + pad, shift, t, 0, fill=-77.0)
    dw, wbuf = padded(N, K, K + pad, shift, t, 0, fill=-55.0)
    db = torch.empty(N, dtype=t, device="cuda")
    fa.linear_backward(dy, x, w, act="silu", preact=pre, dx=dx, dw=dw, db=db)
    check_backward(dy, x, w, "silu", pre, 1.0, dx, dw, db)
    for v, buf, fill in ((dx, xbuf, -77.0), (dw, wbuf, -55.0)):
        v.fill_(fill)
        assert bool((buf == fill).all())


def test_backward_repeated_gradient_rows():
    # the gradient of a sum over the outputs: one row, and one value, repeated
    t = torch.float32
    M, N, K = 60, 48, 80
    x, w = rnd((M, K), t, 1), rnd((N, K), t, 2)
    dy = rnd((1, N), t, 3).expand(M, N)
    check_backward(dy, x, w, "none", None, 1.0, *fa.linear_backward(dy, x, w, db=True))


@pytest.mark.parametrize("act", ACTS)
def test_backward_against_differences(act):
    """The directional derivative of f = sum(c * out) from the forward kernel.
    With h = 2^-5 and directions of unit size per element the second-order
    term is at most h^2 / 6 times the third derivative (below 4 for these
    activations away from relu's corner), and fp32 rounding of f adds about
    2^-24 sqrt(MN) (K + 32) / h; relu is held away from its corner."""
    t = torch.float32
    M, N, K = 20, 24, 32
    x, w, b = rnd((M, K), t, 1), rnd((N, K), t, 2, K ** -0.5), rnd((N,), t, 3)
    if act == "relu":
        b = torch.where(torch.arange(N, device="cuda") % 2 == 0, 12.0, -12.0).to(t)
    c = rnd((M, N), t, 4)
    h = 2.0 ** -5

    def f(x, w, b):
        return float((c.double() * fa.linear_forward(x, w, b, act=act).double()).sum())

    pre = torch.empty(M, N, dtype=t, device="cuda")
    fa.linear_forward(x, w, b, act=act, preact=pre)
    dx, dw, db = fa.linear_backward(c, x, w, act=act, preact=pre, db=True)
    for which, g in enumerate((dx, dw, db)):
        v = rnd(g.shape, t, 50 + which, 0.2 if which == 0 else 0.2 * K ** -0.5 if which == 1 else 0.2)
        args = [x, w, b]
        plus, minus = list(args), list(args)
        plus[which], minus[which] = args[which] + h * v, args[which] - h * v
        slope = (f(*plus) - f(*minus)) / (2 * h)
        want = float((g.double() * v.double()).sum())
        # change of z per unit step, by which the third-order term scales
        dz = (v @ w.t() if which == 0 else x @ v.t() if which == 1 else v[None].expand(M, N)).double()
        third = 4 * float((c.double().abs() * dz.abs() ** 3).sum()) * h * h / 6
        noise = ref.U32 * (K + 32) * float(c.abs().double().sum()) * 4 / h
        assert abs(slope - want) <= third + noise, (which, slope, want, third, noise)


def test_other_stream_and_graph_replays():
    t = torch.bfloat16
    M, N, K = 130, 256, 192
    x, w, bias, dy = rnd((M, K), t, 1), rnd((N, K), t, 2), rnd((N,), t, 3), rnd((M, N), t, 4)

    def step():
        pre = torch.empty(M, N, dtype=t, device="cuda")
        y = fa.linear_forward(x, w, bias, act="gelu", preact=pre)
        return (y, pre) + fa.linear_backward(dy, x, w, act="gelu", preact=pre, db=True)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z = fa.linear_forward(x, w, bias, stream=side)
    side.synchronize()
    check_forward(x, w, bias, "none", None, 1.0, z, None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in (31, 32, 33):
        x.copy_(rnd((M, K), t, seed))
        dy.copy_(rnd((M, N), t, seed + 10))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, step()):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# odd operands of products long enough for aligned copies beside the partial
# sums of splits; all three products' sums joined in one launch
@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("shape", [(1501, 901, 1603), (301, 5003, 1503), (5001, 301, 1501), (203, 801, 12501)], ids=str)
def test_odd_products_of_small_tiles(shape, dt, act):
    M, N, K = shape
    t = DTYPES[dt]
    x, w, dy = rnd((M, K), t, 1), rnd((N, K), t, 2, K ** -0.5), rnd((M, N), t, 3)
    pre = rnd((M, N), t, 4, 1.5) if act != "none" else None
    check_forward(x, w, None, act, None, 1.0, fa.linear_forward(x, w, act=act), None)
    got = fa.linear_backward(dy, x, w, act=act, preact=pre, db=True)
    check_backward(dy, x, w, act, pre, 1.0, *got)
    again = fa.linear_backward(dy, x, w, act=act, preact=pre, db=True)
    for a, b in zip(got, again):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_rows_too_long_for_a_tile_of_aligned_copies():
    # 256 rows of 2^22 + 1 bf16 span more than 2 GiB
    K = 2 ** 22 + 1
    x = torch.zeros(1, K, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(1, K, dtype=torch.bfloat16, device="cuda")
    for i, k in enumerate((0, 70, 2 ** 21 + 7, K - 1)):
        x[0, k] = 2.0 ** i
        w[0, k] = 1.0
    out = fa.linear_forward(x.expand(2048, K), w.expand(2048, K))
    assert bool((out == 15.0).all())
