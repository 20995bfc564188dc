"""GPU: rows to 8 bits, and the linear layer on 8-bit weights (forward,
backward), against plain forms in 64 bits."""

import numpy as np
import pytest
import torch

import learn_ref as ref
import weighted_model_update_amd as fa

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ["none", "relu", "gelu", "silu"]


def rnd(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def ints(shape, seed, lo=-127, hi=128):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(lo, hi, shape, generator=g, dtype=torch.int8).cuda()


def positive(n, seed, scale):
    g = torch.Generator().manual_seed(seed)
    return ((torch.rand(n, generator=g) + 0.5) * scale).cuda()


def rows_to_8_bits(x):
    """The definition, in IEEE fp32 on the host."""
    x = x.detach().float().cpu().numpy()
    with np.errstate(all="ignore"):
        top = np.abs(x).max(axis=1, initial=0).astype(np.float32)
        bad = ~np.isfinite(x).all(axis=1)
        scale = np.where(bad, np.float32(np.nan), top / np.float32(127))
        live = scale > 0
        q = np.rint(x / np.where(live, scale, 1).astype(np.float32)[:, None])
    q = np.where(live[:, None], np.clip(q, -127, 127), 0)
    return q.astype(np.int8), scale.astype(np.float32)


def check_quantized(x, q, scale):
    wq, ws = rows_to_8_bits(x)
    assert np.array_equal(scale.cpu().numpy(), ws, equal_nan=True)
    assert np.array_equal(q.cpu().numpy(), wq)


# one value, around 16 (a thread's share), the ends of each row form (1024, 4096,
# 16384 values held), rows read twice
@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("shape", [(1, 1), (3, 16), (5, 17), (40, 15), (300, 33), (7, 1000), (17, 1024), (6, 1025), (3, 4096),
                                   (9, 4097), (2, 16384), (3, 16385), (1, 70001), (4000, 8)], ids=str)
def test_quantize(shape, dt):
    x = rnd(shape, DTYPES[dt], sum(shape), 0.02)
    check_quantized(x, *fa.quantize_rows(x))


@pytest.mark.parametrize("dt", list(DTYPES))
def test_quantize_odd_rows(dt):
    x = rnd((14, 100), DTYPES[dt], 1)
    x[1] = 0
    x[2, 3] = float("nan")
    x[3, 99] = float("inf")
    x[4, 0] = float("-inf")
    x[5] *= 1e-38                       # subnormal scale
    x[6] = 0
    x[6, 7] = 1e-45                     # the scale underflows (and bf16 has no such value)
    x[7] *= 1e37
    x[8] = -0.0
    x[9, 1:] = 0
    x[10] = torch.arange(100).to(x.dtype) - 50      # ties: x / (50 / 127) and halves
    x[11] = 1.0
    x[12, ::2], x[12, 1::2] = 2.0, -1.0             # 127 and -63.5
    x[13] = float("nan")
    check_quantized(x, *fa.quantize_rows(x))


@pytest.mark.parametrize("dt", list(DTYPES))
def test_quantize_views_and_untouched_gaps(dt):
    R, C = 9, 77
    x = rnd((R * 90 + 1,), DTYPES[dt], 3)[1:].view(R, 90)[:, 5:5 + C]
    buf = torch.full((R * 83 + 3,), 99, dtype=torch.int8, device="cuda")
    q = buf[3:].view(R, 83)[:, :C]
    scale = torch.full((R + 2,), 5.0, device="cuda")
    fa.quantize_rows(x, q=q, scale=scale[1:R + 1])
    check_quantized(x, q, scale[1:R + 1])
    q.fill_(99)
    assert bool((buf == 99).all()) and float(scale[0]) == 5.0 and float(scale[R + 1]) == 5.0
    repeated = rnd((1, C), DTYPES[dt], 4).expand(R, C)
    check_quantized(repeated, *fa.quantize_rows(repeated))


def test_quantize_no_rows_or_columns():
    q, s = fa.quantize_rows(torch.empty(0, 8, device="cuda"))
    assert q.shape == (0, 8) and s.shape == (0,)
    _, s = fa.quantize_rows(torch.empty(4, 0, device="cuda"))
    assert bool((s == 0).all())


# ------------------------------------------------------------------ forward

def layer(xq, xs, w, ws, bias, act, residual, alpha):
    """(out, z, magnitude) in float64 of 8-bit operands."""
    prod = (ref.d(xq) @ ref.d(w).t()) * ref.d(xs)[:, None] * ref.d(ws)[None, :] * alpha
    z, mag = prod, prod.abs()
    if bias is not None:
        z, mag = z + ref.d(bias), mag + ref.d(bias).abs()
    y = ref.act(z, act)
    if residual is not None:
        y, mag = y + ref.d(residual), mag + ref.d(residual).abs()
    return y, z, mag


def check_forward(xq, xs, w, ws, bias, act, residual, alpha, out, pre):
    y, z, mag = layer(xq, xs, w, ws, bias, act, residual, alpha)
    # the sum's own rounding, the three factors and the bias: 5 half steps; the
    # activations are within 16 half steps of what enters and their slopes
    # below 1.13; the residual one more
    slack = 1.13 * 24 * ref.U32 * mag
    ref.within(out, y, slack, out.dtype, "out")
    if pre is not None:
        ref.within(pre, z, slack, out.dtype, "preact")


# one value; single rows and columns; below, at and above the tiles (16, 64, 128,
# 256) and the steps of 64 and 128 values; sums split over workgroups; odd widths
SHAPES = [(1, 1, 1), (1, 40, 16), (3, 5, 7), (16, 16, 64), (17, 33, 65), (1, 1000, 4096), (2, 130, 9000), (16, 300, 1024),
          (33, 96, 144), (64, 64, 128), (65, 129, 1040), (300, 16, 1024), (1000, 9, 133), (129, 257, 130), (257, 264, 2000),
          (520, 1032, 128), (1100, 1030, 321), (2050, 2100, 208), (4100, 2050, 96), (2050, 4100, 96), (1500, 1400, 1001)]


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, dt):
    M, N, K = shape
    t, act = DTYPES[dt], ACTS[(M + N + K) % 4]
    xq, xs, w, ws = ints((M, K), 1, -128), positive(M, 2, 0.02), ints((N, K), 3, -128), positive(N, 4, 0.02 * K ** -0.5)
    bias, res = rnd((N,), t, 5), rnd((M, N), t, 6)
    pre = torch.empty(M, N, dtype=t, device="cuda")
    out = fa.linear_int8_forward(xq, w, ws, bias, act=act, residual=res, alpha=0.5, x_scale=xs, preact=pre, dtype=t)
    check_forward(xq, xs, w, ws, bias, act, res, 0.5, out, pre)
    plain = fa.linear_int8_forward(xq, w, ws, x_scale=xs, dtype=t)
    check_forward(xq, xs, w, ws, None, "none", None, 1.0, plain, None)
    # x in 8 bits by the call itself
    x = rnd((M, K), t, 7)
    xq, xs = (torch.from_numpy(v).cuda() for v in rows_to_8_bits(x))
    out = fa.linear_int8_forward(x, w, ws, bias, act=act, alpha=2.0)
    check_forward(xq, xs, w, ws, bias, act, None, 2.0, out, None)
    assert torch.equal(out, fa.linear_int8_forward(xq, w, ws, bias, act=act, alpha=2.0, x_scale=xs, dtype=t))


# one launch for few tokens: one to four and five, sums of one step to many
# rounds, the ends of the pieces (4096 values, four in all), odd numbers of columns
@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("shape", [(1, 1, 16), (1, 17, 48), (2, 33, 64), (3, 100, 80), (4, 16, 256), (4, 300, 1040), (5, 300, 1040),
                                   (1, 50, 5008), (2, 40, 8192), (2, 40, 8208), (4, 40, 4096), (4, 40, 4112), (3, 24, 4000), (1, 40, 12304),
                                   (1, 24, 16384), (1, 24, 16400),
                                   (2, 33000, 48), (1, 70001, 16), (3, 20000, 576)], ids=str)
def test_forward_few_tokens(shape, dt):
    M, N, K = shape
    t = DTYPES[dt]
    w, ws, x = ints((N, K), 1, -128), positive(N, 2, 0.02 * K ** -0.5), rnd((M, K), t, 3)
    bias, res, pre = rnd((N,), t, 4), rnd((M, N), t, 5), torch.empty(M, N, dtype=t, device="cuda")
    if M > 1:
        x[1] = 0
    xq, xs = (torch.from_numpy(v).cuda() for v in rows_to_8_bits(x))
    out = fa.linear_int8_forward(x, w, ws, bias, act="silu", residual=res, alpha=0.5, preact=pre)
    check_forward(xq, xs, w, ws, bias, "silu", res, 0.5, out, pre)
    assert torch.equal(out, fa.linear_int8_forward(xq, w, ws, bias, act="silu", residual=res, alpha=0.5, x_scale=xs, dtype=t))
    # the same rows among others, which take another way
    many = torch.cat([x, rnd((20, K), t, 6)])
    assert torch.equal(out, fa.linear_int8_forward(many, w, ws, bias, act="silu", residual=torch.cat([res, rnd((20, N), t, 7)]),
                                                   alpha=0.5)[:M])


@pytest.mark.parametrize("shape", [(1, 64), (3, 20), (20, 3), (70, 200)], ids=str)
def test_forward_the_largest_sums(shape):
    """128 * 128 * (2^17 - 1) = 2^31 - 2^14, of one sign and of both."""
    M, N, K = *shape, (1 << 17) - 1
    x = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    w[::2] = 127
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    out = fa.linear_int8_forward(x, w, one(N), x_scale=one(M), dtype=torch.float32)
    want = torch.where(torch.arange(N) % 2 == 0, -128.0 * 127 * K, 128.0 * 128 * K)
    # whole numbers below 2^31: one rounding to fp32
    assert torch.equal(out.cpu(), want.double().float().expand(M, N))


@pytest.mark.parametrize("odd", [False, True], ids=["pitch", "unaligned"])
@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("shape", [(1, 40, 64), (19, 72, 208), (140, 136, 72), (300, 24, 512), (1100, 1032, 144)], ids=str)
def test_forward_pitched_views_and_untouched_gaps(shape, dt, odd):
    M, N, K = shape
    t, pad, shift = DTYPES[dt], 3 if odd else 16, 1 if odd else 0

    def view(rows, cols, ld, dtype, seed, fill=None):
        n = rows * ld + shift + 8
        buf = torch.full((n,), fill, dtype=dtype, device="cuda") if fill is not None else \
            ints((n,), seed) if dtype is torch.int8 else rnd((n,), dtype, seed)
        return buf[shift:shift + rows * ld].view(rows, ld)[:, :cols], buf

    xq, w = view(M, K, K + pad, torch.int8, 1)[0], view(N, K, K + 2 * pad, torch.int8, 2)[0]
    xs, ws = positive(M, 3, 0.02), positive(N, 4, 0.02 * K ** -0.5)
    x = view(M, K, K + pad, t, 9)[0]
    res = view(M, N, N + pad, t, 5)[0]
    bias = rnd((N + 1,), t, 6)[1:]
    out, obuf = view(M, N, N + pad, t, 0, -77.0)
    pre, pbuf = view(M, N, N + 2 * pad, t, 0, -55.0)
    fa.linear_int8_forward(xq, w, ws, bias, act="silu", residual=res, x_scale=xs, out=out, preact=pre)
    check_forward(xq, xs, w, ws, bias, "silu", res, 1.0, out, pre)
    fa.linear_int8_forward(x, w, ws, bias, act="gelu", out=out)
    q, s = (torch.from_numpy(v).cuda() for v in rows_to_8_bits(x))
    check_forward(q, s, w, ws, bias, "gelu", None, 1.0, out, None)
    for v, buf, fill in ((out, obuf, -77.0), (pre, pbuf, -55.0)):
        v.fill_(fill)
        assert bool((buf == fill).all())


@pytest.mark.parametrize("M", [1, 5, 40, 600])
def test_forward_nan_and_zero_scales(M):
    N, K = 700, 256
    x = rnd((M, K), torch.float32, 1)
    w, ws = ints((N, K), 2), positive(N, 3, 0.01)
    bias = rnd((N,), torch.float32, 4)
    ws[7], ws[9] = float("nan"), 0.0
    x[M // 2, 3] = float("inf")
    out = fa.linear_int8_forward(x, w, ws, bias)
    assert bool(out[:, 7].isnan().all()) and bool(out[M // 2].isnan().all())
    fine = torch.ones(M, dtype=torch.bool, device="cuda")
    fine[M // 2] = False
    assert torch.equal(out[fine][:, 9], bias[9].expand(int(fine.sum())))
    keep = torch.ones(N, dtype=torch.bool, device="cuda")
    keep[7] = False
    assert bool(out[fine][:, keep].isfinite().all())
    x.zero_()
    ws.fill_(0.5)
    assert torch.equal(fa.linear_int8_forward(x, w, ws, bias), bias.expand(M, N))


def test_forward_in_place_residual_repeated_rows_and_empty_sums():
    M, N, K = 70, 136, 96
    x = ints((1, K), 1).expand(M, K)                    # pitch 0
    xs, w, ws = positive(M, 2, 0.02), ints((N, K), 3), positive(N, 4, 0.01)
    h = rnd((M, N), torch.bfloat16, 5)
    before = h.clone()
    assert fa.linear_int8_forward(x, w, ws, residual=h, x_scale=xs, out=h) is h
    check_forward(x, xs, w, ws, None, "none", before, 1.0, h, None)
    bias = rnd((N,), torch.float32, 6)
    none = fa.linear_int8_forward(torch.empty(M, 0, device="cuda"), w[:, :0], ws, bias, act="relu")
    assert torch.equal(none, bias.clamp(min=0).expand(M, N))
    assert fa.linear_int8_forward(torch.empty(0, K, device="cuda"), w, ws).shape == (0, N)
    assert fa.linear_int8_forward(rnd((M, K), torch.float32, 7), w[:0], ws[:0]).shape == (M, 0)


# ------------------------------------------------------------------ backward

def check_backward(dy, w, ws, act, pre, alpha, dx, db):
    dz = ref.d(dy) * (ref.act_slope(ref.d(pre), act) if pre is not None else 1.0)
    # |act'| is below 1.13 and formed within 16 half steps of its own size and of 1
    size = ref.d(dy).abs() * (1.13 if pre is not None else 1.0)
    if dx is not None:
        wv = ref.d(w) * ref.d(ws)[:, None]
        # dz times the scale is held in dtype: half a step; N additions, the
        # slope, the scale and alpha in fp32
        u = ref.half_step(dx.dtype) * 1.01 + 1.2 * (dz.shape[1] + 32) * ref.U32
        slack = u * abs(alpha) * (size @ wv.abs())
        ref.within(dx, alpha * (dz @ wv), slack, dx.dtype, "dx")
    if db is not None:
        slack = 1.2 * (dz.shape[0] + 32) * ref.U32 * size.sum(0)
        ref.within(db, dz.sum(0), slack, db.dtype, "db")


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 5, 7), (1, 1000, 640), (17, 33, 65), (33, 96, 144), (300, 16, 264), (1000, 9, 133),
                                   (64, 1000, 16), (129, 257, 130), (513, 384, 1030), (2050, 130, 2060), (40, 5000, 48), (3, 4096, 1008),
                                   (513, 385, 1040), (130, 9000, 64), (1100, 71, 4112), (2050, 130, 2064)], ids=str)
def test_backward(shape, dt):
    M, N, K = shape
    t, act = DTYPES[dt], ACTS[(M + N + K) % 4]
    dy, w, ws = rnd((M, N), t, 1), ints((N, K), 2, -128), positive(N, 3, 0.01)
    pre = rnd((M, N), t, 4) if act != "none" else None
    dx, db = fa.linear_int8_backward(dy, w, ws, act=act, preact=pre, alpha=0.5, db=True)
    check_backward(dy, w, ws, act, pre, 0.5, dx, db)
    dx2, none = fa.linear_int8_backward(dy, w, ws)
    assert none is None
    check_backward(dy, w, ws, "none", None, 1.0, dx2, None)
    none, db2 = fa.linear_int8_backward(dy, w, None, act=act, preact=pre, dx=None, db=True)
    assert none is None
    check_backward(dy, w, ws, act, pre, 1.0, None, db2)
    again, _ = fa.linear_int8_backward(dy, w, ws, act=act, preact=pre, alpha=0.5)
    assert torch.equal(again, dx)


@pytest.mark.parametrize("odd", [False, True], ids=["pitch", "unaligned"])
@pytest.mark.parametrize("dt", list(DTYPES))
def test_backward_pitched_views_and_untouched_gaps(dt, odd):
    M, N, K, t = 70, 200, 88, DTYPES[dt]
    pad, shift = (3, 1) if odd else (16, 0)
    cut = lambda buf, rows, cols: buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]  # noqa: E731
    dy, pre = cut(rnd((M * (N + pad) + 8,), t, 1), M, N), cut(rnd((M * (N + pad) + 8,), t, 2), M, N)
    w, ws = cut(ints((N * (K + pad) + 8,), 3), N, K), positive(N, 4, 0.01)
    buf = torch.full((M * (K + pad) + 8,), -7.0, dtype=t, device="cuda")
    dx = cut(buf, M, K)
    fa.linear_int8_backward(dy, w, ws, act="gelu", preact=pre, dx=dx)
    check_backward(dy, w, ws, "gelu", pre, 1.0, dx, None)
    dx.fill_(-7.0)
    assert bool((buf == -7.0).all())
    # one gradient for every token: pitch 0
    same = rnd((1, N), t, 5).expand(M, N)
    dx, db = fa.linear_int8_backward(same, w, ws, db=True)
    check_backward(same, w, ws, "none", None, 1.0, dx, db)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("shape", [(5, 300, 64), (700, 200, 1040)], ids=str)
def test_backward_the_whole_range_of_values(shape, dt):
    """Gradients over many orders of magnitude, up to the largest fp32 and down to
    subnormals; NaN and infinities stay in their rows."""
    M, N, K = shape
    t = DTYPES[dt]
    w, ws = ints((N, K), 1, -128), torch.ones(N, device="cuda")
    dy = rnd((M, N), t, 2) * torch.exp2(torch.randint(-100, 90, (M, N), generator=torch.Generator().manual_seed(3)).cuda().float()).to(t)
    dy[1] = 0
    dy[1, 3] = 2e38
    dy[2] = rnd((1, N), t, 4) * 2.0 ** -125
    w[3] = w[3].clamp(-1, 1)
    dx, _ = fa.linear_int8_backward(dy, w, ws)
    check_backward(dy, w, ws, "none", None, 1.0, dx, None)
    want = dx.clone()
    dy[0, 5], dy[4, 7] = float("inf"), float("nan")
    w[5], w[7] = 1, 2
    dx, _ = fa.linear_int8_backward(dy, w, ws)
    assert bool((dx[0] == float("inf")).all()) and bool(dx[4].isnan().all())
    w[5], w[7] = ints((N, K), 1, -128)[5], ints((N, K), 1, -128)[7]
    dx, _ = fa.linear_int8_backward(dy, w, ws)
    assert torch.equal(dx[1:4], want[1:4])


def test_backward_no_tokens_or_channels():
    w, ws = ints((24, 40), 1), positive(24, 2, 0.1)
    dx, db = fa.linear_int8_backward(torch.empty(0, 24, device="cuda"), w, ws, db=True)
    assert dx.shape == (0, 40) and bool((db == 0).all()) and db.shape == (24,)
    dx, db = fa.linear_int8_backward(torch.empty(5, 0, device="cuda"), w[:0], ws[:0], db=True)
    assert bool((dx == 0).all()) and dx.shape == (5, 40) and db.shape == (0,)


@pytest.mark.parametrize("act", ACTS)
def test_backward_against_differences(act):
    """dx along random directions against central differences of the layer in
    float64, on values that 8 bits hold exactly.  The difference's own error:
    |f'''| h^2 / 6 and 2^-53 |f| / h, both below 1e-7 of the gradient's size
    here; the kernel's is fp32's."""
    M, N, K, h = 9, 50, 33, 1e-4
    w, ws = ints((N, K), 1), positive(N, 2, 0.002)
    x = ref.d(rnd((M, K), torch.float32, 3))
    g, bias = rnd((M, N), torch.float32, 4), rnd((N,), torch.float32, 5)
    wv = ref.d(w) * ref.d(ws)[:, None]
    f = lambda v: (ref.act(v @ wv.t() + ref.d(bias), act) * ref.d(g)).sum()  # noqa: E731
    pre = (x @ wv.t() + ref.d(bias)).float().cuda()
    pre = torch.where(pre.abs() < 1e-2, pre.sign() * 1e-2 + pre, pre) if act == "relu" else pre
    if act == "relu":       # keep the kink out of the differences' reach
        bias_of = ref.d(pre) - x @ wv.t()
        f = lambda v: (ref.act(v @ wv.t() + bias_of, act) * ref.d(g)).sum()  # noqa: E731
    dx, _ = fa.linear_int8_backward(g, w, ws, act=act, preact=pre)
    for seed in range(4):
        d = torch.randn(M, K, generator=torch.Generator().manual_seed(10 + seed)).double()
        d /= d.norm()
        want = (f(x + h * d) - f(x - h * d)) / (2 * h)
        got = (ref.d(dx) * d).sum()
        # N + 32 half steps of the sum of magnitudes, as for the formula; 2^-24 of
        # the pre-activation given in fp32
        slack = 1.2 * (N + 40) * ref.U32 * ((ref.d(g).abs() * 1.13) @ wv.abs() * d.abs()).sum() + 1e-6 * float(ref.d(dx).norm())
        assert abs(got - want) < slack


# ------------------------------------------------------------------ streams and graphs

@pytest.mark.parametrize("M", [1, 50, 1100])
def test_calls_captured_and_replayed(M):
    N, K, t = 1030, 512, torch.bfloat16
    x, dy = rnd((M, K), t, 1), rnd((M, N), t, 2)
    wt = rnd((N, K), t, 3, K ** -0.5)
    out, pre, dx = torch.empty(M, N, dtype=t, device="cuda"), torch.empty(M, N, dtype=t, device="cuda"), torch.empty_like(x)
    db, q, s = torch.empty(N, dtype=t, device="cuda"), torch.empty(N, K, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
    ws = torch.empty(max(fa.linear_int8_workspace_size(M, N, K), fa.linear_int8_workspace_size(M, N, K, backward=True)),
                     dtype=torch.uint8, device="cuda")

    def calls():
        fa.quantize_rows(wt, q=q, scale=s)
        fa.linear_int8_forward(x, q, s, act="gelu", out=out, preact=pre, workspace=ws)
        fa.linear_int8_backward(dy, q, s, act="gelu", preact=pre, dx=dx, db=db, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for k in range(3):
        x.copy_(rnd((M, K), t, 20 + k))
        wt.copy_(rnd((N, K), t, 30 + k, K ** -0.5))
        dy.copy_(rnd((M, N), t, 40 + k))
        graph.replay()
        got = [v.clone() for v in (q, s, out, pre, dx, db)]
        for v in (q, s, out, pre, dx, db):
            v.zero_()
        torch.cuda.synchronize()
        calls()
        assert all(torch.equal(a, b) for a, b in zip(got, (q, s, out, pre, dx, db)))


def test_two_streams_at_once():
    N, K, t = 520, 256, torch.bfloat16
    w, ws = ints((N, K), 1), positive(N, 2, 0.01)
    xs = [rnd((300, K), t, 3 + i) for i in range(2)]
    want = [fa.linear_int8_forward(x, w, ws) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[] for _ in xs]
    for _ in range(5):
        for i, s in enumerate(streams):
            got[i].append(fa.linear_int8_forward(xs[i], w, ws, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(v, want[i]) for i in range(2) for v in got[i])
