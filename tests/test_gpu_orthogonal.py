"""GPU: the orthogonalised matrix and the server's step with it, against the
formula in float64."""

import math

import pytest
import torch

import learn_ref as ref
import weighted_model_update_amd as fa

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
QUINTIC, CUBIC = fa.ORTHO_COEF, (1.5, -0.5, 0.0)


def rnd(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def update(shape, dtype, seed):
    """A few strong directions over a background, as averaged updates have."""
    *lead, m, n = shape
    g = torch.Generator().manual_seed(seed)
    r = max(1, min(m, n) // 8)
    low = torch.randn(*lead, m, r, generator=g) @ torch.randn(*lead, r, n, generator=g)
    return ((low / math.sqrt(r) + 0.25 * torch.randn(shape, generator=g)) * 1e-3).to(dtype).cuda()


def formula(x, coef, steps, dtype):
    """O of every matrix of x, evaluated in dtype: fp32 as a stand-in for products
    in that type, fp64 as the reference."""
    rows = coef if isinstance(coef[0], tuple) else [coef] * steps
    out = []
    for t in (x if x.dim() == 3 else x[None]).detach().double():
        tall = t.shape[0] > t.shape[1]
        t = (t.t() if tall else t).contiguous()
        size = t.norm()
        t = (t / size if float(size) != 0 else t * 0).to(dtype)
        for a, b, c in rows:
            gram = t @ t.t().contiguous()
            t = a * t + (b * gram + c * (gram @ gram)) @ t
        out.append(t.t() if tall else t)
    return torch.stack(out).reshape(x.shape)


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


def check(x, out, scale=1.0, coef=QUINTIC, steps=5):
    """Short sides: fp64 throughout, in which rounding grows by a step's largest
    slope squared, 12^5 2^-53 100 < 1e-8, then a rounding to fp32, the scale and
    the result's.  Long sides: halves of 23 bits in the place of fp32's 24 and the
    product of the low halves left out (2^-22) come to at most four times the
    error that fp32 products make on the same matrix, plus a few half steps of
    fp32; every result has its own half step in the norm."""
    want = formula(x, coef, steps, torch.float64) * scale
    if min(x.shape[-2:]) <= 64:
        ref.within(out, want.cpu(), abs(scale) * 1e-8 + 3 * ref.U32 * want.abs().cpu(), out.dtype, "O")
        return
    fp32 = off(formula(x, coef, steps, torch.float32) * scale, want)
    assert off(out, want) <= ref.half_step(out.dtype) + 4 * fp32 + 8 * ref.U32, (off(out, want), fp32)


SHORT = [(1, 1), (1, 5), (5, 1), (2, 3), (16, 16), (17, 33), (33, 17), (48, 200), (200, 48), (64, 64), (64, 1000), (1000, 64),
         (3, 8200), (4100, 16), (63, 65), (65, 63), (16, 4096)]
LONG = [(65, 65), (65, 70), (70, 65), (128, 128), (130, 1000), (1000, 130), (513, 257), (601, 600), (700, 1025), (300, 5000),
        (5001, 300), (1300, 1300)]


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("shape", SHORT + LONG, ids=str)
def test_orthogonalize(shape, dt):
    x = update(shape, DTYPES[dt], sum(shape))
    out = fa.orthogonalize(x)
    check(x, out)
    assert torch.equal(out.view(torch.uint8), fa.orthogonalize(x).view(torch.uint8))
    noise = rnd(shape, DTYPES[dt], 5)
    check(noise, fa.orthogonalize(noise, scale=0.25), scale=0.25)


@pytest.mark.parametrize("shape", [(3, 16, 40), (5, 40, 24), (130, 8, 300), (700, 5, 3), (3, 65, 100), (2, 300, 129), (7, 200, 200),
                                   (48, 512, 520), (40, 600, 512)], ids=str)
def test_batches(shape):
    x = update(shape, torch.float32, 3)
    x[1] = 0
    out = fa.orthogonalize(x)
    assert bool((out[1] == 0).all())
    for b in {0, 2 % shape[0], shape[0] - 1} - {1}:
        check(x[b], out[b])
    # each matrix by itself: the same formula with other splits of the sums
    check(x[0], fa.orthogonalize(x[0]))


def test_the_largest_tiles():
    for shape in ((4100, 4200), (4200, 4100)):
        x = rnd(shape, torch.float32, 1)
        check(x, fa.orthogonalize(x))


@pytest.mark.parametrize("shape", [(20, 50), (50, 20), (70, 90), (300, 200)], ids=str)
@pytest.mark.parametrize("coef,steps", [(QUINTIC, 1), (CUBIC, 8), (((2.0, -1.5, 0.5), (1.5, -0.5, 0.0), (1.0, 0.0, 0.0)), 3),
                                        ((0.5, 0.0, 0.0), 3), ((8.0, -23.0, 17.0), 1), ((100.0, 0.0, 0.0), 2)], ids=str)
def test_coefficients_and_steps(shape, coef, steps):
    x = rnd(shape, torch.float32, 7)
    check(x, fa.orthogonalize(x, steps=steps, coef=coef), coef=coef, steps=steps)


@pytest.mark.parametrize("shape", [(70, 300), (300, 70), (2, 200, 900), (520, 2100)], ids=str)
@pytest.mark.parametrize("coef,steps", [(QUINTIC, 5), (QUINTIC, 2), (CUBIC, 20), (((5.0, -9.0, 5.0),) + (CUBIC,) * 4, 5),
                                        ((100.0, 0.0, 0.0), 3)], ids=["quintic", "two", "cubic", "steep", "linear"])
def test_groups_of_steps(shape, coef, steps):
    """bf16 results of long matrices run several steps on one Gram matrix.  Its
    rounding, half a step of fp32, grows by at most 3e4 in a group, and H takes
    it times |b| of at most 23: in the worst direction 3e4 23 2^-24 = 0.04 of an
    entry, but spread over the s directions of which one in s is that one: its
    share of the norm, 0.04 / sqrt(s), is below 0.005; groups end before that."""
    x = update(shape, torch.bfloat16, 6)
    want = formula(x, coef, steps, torch.float64)
    got = fa.orthogonalize(x, steps=steps, coef=coef)
    assert off(got, want) <= ref.half_step(torch.bfloat16) + 0.04 / math.sqrt(min(shape[-2:]))
    # the same call with fp32 results, rounded afterwards: a step at a time
    alone = fa.orthogonalize(x.float(), steps=steps, coef=coef)
    assert off(got, alone.double()) <= ref.half_step(torch.bfloat16) + 0.04 / math.sqrt(min(shape[-2:]))
    w = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    fa.orthogonal_step(w, x.float(), rate=1.0, steps=steps, coef=coef)
    assert torch.equal(w, got)


@pytest.mark.parametrize("shape", [(40, 60), (60, 40), (100, 80), (80, 300)], ids=str)
def test_the_largest_number_of_steps(shape):
    x = rnd(shape, torch.float32, 8)
    out = fa.orthogonalize(x, steps=32, coef=CUBIC)
    # the cubic converges: singular values of one, vectors kept
    u, _, v = torch.linalg.svd(x.double().cpu(), full_matrices=False)
    assert off(out.cpu(), u @ v) < 4e-6


@pytest.mark.parametrize("scale", [1e-30, 1e30, 1e-42, 1e38], ids=str)
@pytest.mark.parametrize("shape", [(12, 30), (100, 70)], ids=str)
def test_the_size_of_the_input_does_not_matter(shape, scale):
    x = rnd(shape, torch.float32, 9).clamp(-3, 3)
    x = (x.double() * scale).float()
    check(x, fa.orthogonalize(x))


@pytest.mark.parametrize("shape", [(3, 12, 30), (3, 30, 12), (3, 100, 70), (3, 70, 300)], ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")], ids=str)
def test_nan_and_infinities_stay_in_their_matrix(shape, bad):
    x = rnd(shape, torch.float32, 10)
    want = fa.orthogonalize(x)
    x[1, 2, 3] = bad
    out = fa.orthogonalize(x)
    assert bool(out[1].isnan().all())
    assert torch.equal(out[0], want[0]) and torch.equal(out[2], want[2])


@pytest.mark.parametrize("shape", [(20, 50), (50, 20), (100, 130), (130, 100)], ids=str)
def test_rank_one_zero_rows_and_orthogonal_input(shape):
    m, n = shape
    one = rnd((m, 1), torch.float32, 11) @ rnd((1, n), torch.float32, 12)
    check(one, fa.orthogonalize(one, steps=3), steps=3)
    x = rnd(shape, torch.float32, 13)
    x[3], x[:, 5] = 0, 0
    out = fa.orthogonalize(x)
    check(x, out)
    assert bool((out[3] == 0).all()) and bool((out[:, 5] == 0).all())
    eye = torch.zeros(shape, device="cuda")
    eye.fill_diagonal_(2.0)
    check(eye, fa.orthogonalize(eye))


# ------------------------------------------------------------------ views

def spread(B, m, n, ld, stride, shift, dtype, seed=None, fill=0.0):
    size = shift + (B - 1) * stride + (m - 1) * ld + n + 9
    buf = rnd((size,), dtype, seed) if seed is not None else torch.full((size,), fill, dtype=dtype, device="cuda")
    return torch.as_strided(buf, (B, m, n), (stride, ld, 1), shift), buf


@pytest.mark.parametrize("rowwise", [False, True], ids=["matrices", "interleaved"])
@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("shape", [(3, 10, 37), (3, 37, 10), (2, 66, 131), (2, 131, 66)], ids=str)
def test_views_and_untouched_gaps(shape, dt, rowwise):
    B, m, n = shape
    place = dict(ld=B * (n + 3) + 2, stride=n + 3) if rowwise else dict(ld=n + 5, stride=(m + 2) * (n + 5) + 1)
    x, _ = spread(B, m, n, shift=3, dtype=DTYPES[dt], seed=1, **place)
    out, buf = spread(B, m, n, shift=1, dtype=DTYPES[dt], fill=-9.0, **place)
    fa.orthogonalize(x, out=out)
    for b in range(B):
        check(x[b], out[b])
    assert torch.equal(out.contiguous(), fa.orthogonalize(x.contiguous()))
    out.fill_(-9.0)
    assert bool((buf == -9.0).all())
    # a matrix repeated, rows repeated
    same = x[:1].expand(B, m, n)
    check(same[0], fa.orthogonalize(same)[B - 1])
    rows = x[0, :1].expand(m, n)
    check(rows, fa.orthogonalize(rows, steps=2), steps=2)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("shape", [(10, 300), (300, 10), (3, 64, 64), (130, 70), (2, 70, 130), (2, 64, 450), (20, 700), (3, 48, 450), (33, 64),
                                   (2, 40, 9000), (450, 64), (600, 33, 70)], ids=str)
def test_in_place(shape, dt):
    x = rnd(shape, DTYPES[dt], 2)
    want = fa.orthogonalize(x)
    for _ in range(3):
        y = x.clone()
        assert fa.orthogonalize(y, out=y) is y
        assert torch.equal(y, want)


def test_one_update_of_a_flat_model():
    """Matrices of different shapes as views of one flat update and one flat
    weight vector, as the average leaves them."""
    shapes = [(4, 16, 96), (4, 96, 16), (1, 100, 130)]
    sizes = [math.prod(s) for s in shapes]
    flat, weights = rnd((sum(sizes),), torch.float32, 3), rnd((sum(sizes),), torch.float32, 4)
    before = weights.clone()
    for s, u, w, b in zip(shapes, flat.split(sizes), weights.split(sizes), before.split(sizes)):
        fa.orthogonal_step(w.view(s), u.view(s), rate=0.1)
        o = fa.orthogonalize(u.view(s))
        assert torch.allclose(w.view(s), b.view(s) + 0.1 * o, rtol=0, atol=4 * ref.U32 * 6)
    # adapters of one rank that lie side by side in every layer
    layers = rnd((5, 2 * 16 * 40), torch.float32, 5)
    a = layers[:, :16 * 40].view(5, 16, 40)
    check(a[3], fa.orthogonalize(a)[3])


# ------------------------------------------------------------------ the step

def check_step(w0, u, m0, w, mom, rate, keep, beta, nesterov):
    rate, keep, beta = torch.tensor([rate, keep, beta]).tolist()      # the call takes them in fp32
    t = ref.d(u)
    if m0 is not None:
        m = beta * ref.d(m0) + t
        # one rounding of the sum
        ref.within(mom, m, 1e-45, torch.float32, "momentum")
        t = t + beta * m if nesterov else m
    t = t.cuda()
    o = formula(t, QUINTIC, 5, torch.float64)
    want = keep * ref.d(w0).cuda() + rate * o
    got, size = w.double(), float(o.norm()) * abs(rate)
    fp32 = off(formula(t.float(), QUINTIC, 5, torch.float32), o) if min(u.shape[-2:]) > 64 else 1e-8
    # t itself is rounded to fp32 (momentum twice): half a step each, which the
    # formula's steps enlarge by at most 4 each on small singular values; the
    # fp32 form has the same input error
    slack = (4 * fp32 + 16 * ref.U32 + 2 * ref.U32 * (4.0 ** 5 if m0 is not None else 0)) * size
    # keep w, the sum and the weight's own rounding
    slack += (ref.half_step(w.dtype) + 2 * ref.U32) * float(want.norm()) + 2 * ref.U32 * float(ref.d(w0).norm())
    assert float((got - want).norm()) <= slack, (float((got - want).norm()), slack)


@pytest.mark.parametrize("shape", [(7, 5), (16, 200), (2, 200, 48), (90, 130), (3, 130, 90), (400, 513)], ids=str)
@pytest.mark.parametrize("types", [("f32", "f32"), ("bf16", "f32"), ("f32", "bf16"), ("bf16", "bf16")], ids="-".join)
def test_step(shape, types):
    ut, wt = (DTYPES[t] for t in types)
    u, w0 = update(shape, ut, 1), rnd(shape, wt, 2, 0.02)
    w = w0.clone()
    assert fa.orthogonal_step(w, u, rate=0.03, keep=0.9) is w
    check_step(w0, u, None, w, None, 0.03, 0.9, 0.0, False)
    for nesterov in (False, True):
        m0 = update(shape, torch.float32, 3)
        w, mom = w0.clone(), m0.clone()
        fa.orthogonal_step(w, u, rate=-0.5, momentum=mom, beta=0.95, nesterov=nesterov)
        check_step(w0, u, m0, w, mom, -0.5, 1.0, 0.95, nesterov)
        mom2, w2 = m0.clone(), w0.clone()
        fa.orthogonal_step(w2, u, rate=-0.5, momentum=mom2, beta=0.95, nesterov=nesterov)
        assert torch.equal(w, w2) and torch.equal(mom, mom2)


@pytest.mark.parametrize("shape", [(2, 9, 33), (2, 33, 9), (2, 70, 90)], ids=str)
def test_step_views_and_untouched_gaps(shape):
    B, m, n = shape
    w, wbuf = spread(B, m, n, ld=n + 4, stride=(n + 4) * m + 3, shift=1, dtype=torch.bfloat16, seed=1)
    mom, mbuf = spread(B, m, n, ld=n + 2, stride=(n + 2) * m + 5, shift=2, dtype=torch.float32, seed=2)
    u, _ = spread(B, m, n, ld=n + 1, stride=(n + 1) * m, shift=0, dtype=torch.float32, seed=3)
    w0, m0, wb, mb = w.clone(), mom.clone(), wbuf.clone(), mbuf.clone()
    fa.orthogonal_step(w, u, rate=0.5, momentum=mom, beta=0.5)
    check_step(w0, u, m0, w, mom, 0.5, 1.0, 0.5, True)
    w.copy_(w0)
    mom.copy_(m0)
    assert torch.equal(wbuf, wb) and torch.equal(mbuf, mb)


def test_step_without_update_keeps_the_weights():
    for shape in ((8, 24), (100, 70)):
        w = rnd(shape, torch.float32, 1)
        want = w * torch.tensor(0.75)
        fa.orthogonal_step(w, torch.zeros(shape, device="cuda"), rate=3.0, keep=0.75)
        assert torch.equal(w, want)
        mom = torch.zeros(shape, device="cuda")
        fa.orthogonal_step(w, torch.zeros(shape, device="cuda"), rate=3.0, momentum=mom)
        assert torch.equal(w, want) and bool((mom == 0).all())


def test_nothing_to_do():
    for shape in ((0, 5), (5, 0), (0, 4, 4), (3, 0, 4)):
        x = torch.empty(shape, device="cuda")
        assert fa.orthogonalize(x).shape == shape
        fa.orthogonal_step(x, x.clone(), rate=1.0)


# ------------------------------------------------------------------ streams and graphs

@pytest.mark.parametrize("shape", [(4, 16, 200), (60, 50), (2, 100, 300), (520, 513)], ids=str)
def test_calls_captured_and_replayed(shape):
    u, w, mom = update(shape, torch.bfloat16, 1), rnd(shape, torch.float32, 2), torch.zeros(shape, device="cuda")
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    B = shape[0] if len(shape) == 3 else 1
    ws = torch.empty(fa.orthogonalize_workspace_size(B, *shape[-2:]), dtype=torch.uint8, device="cuda")

    def calls():
        fa.orthogonal_step(w, u, rate=0.02, momentum=mom, workspace=ws)
        fa.orthogonalize(u, out=out, workspace=ws)

    start = (w.clone(), mom.clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    w.copy_(start[0]); mom.copy_(start[1])
    w2, mom2 = w.clone(), mom.clone()
    for k in range(4):
        u.copy_(update(shape, torch.bfloat16, 10 + k))
        graph.replay()
        got = [v.clone() for v in (w, mom, out)]
        torch.cuda.synchronize()
        # the same step eagerly, from the same state
        w.copy_(w2); mom.copy_(mom2); out.zero_(); ws.fill_(255)
        calls()
        assert all(torch.equal(a, b) for a, b in zip(got, (w, mom, out)))
        w2, mom2 = w.clone(), mom.clone()


def test_two_streams_at_once():
    xs = [rnd((200, 300), torch.float32, i) for i in range(2)] + [rnd((3, 20, 90), torch.float32, i) for i in range(2)]
    want = [fa.orthogonalize(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[fa.orthogonalize(x, stream=s) for _ in range(4)] for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(v, w) for g, w in zip(got, want) for v in g)
