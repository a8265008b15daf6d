"""Layer norm's forward and backward pass against the definition in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

import rows_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
EPS = 1e-6
# widths on both sides of every lane count and piece count of the kernels
WIDTHS = [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 31, 33, 64, 65, 100, 127, 129, 256, 257, 320, 511,
          513, 768, 1001, 1024, 1030, 1536, 2047, 2048, 2049, 2560, 4096, 4097, 5000, 8192, 8193,
          12288, 16383, 16384]
SHORT = [1, 3, 8, 15, 33, 65, 257, 513, 1001, 1030, 2049, 2560, 4097, 8193, 16383]


@pytest.fixture(scope="module")
def gn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import groupnorm_silu_normalization_amd as gn
    return gn


@pytest.fixture(autouse=True)
def no_grad():
    with torch.no_grad():
        yield


def make(M, C, dtype, adt, seed):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(M, C, generator=gen) * torch.exp(0.3 * torch.randn(C, generator=gen))
         + 0.5 * torch.randn(C, generator=gen)).to(dtype)
    w = (1 + 0.3 * torch.randn(C, generator=gen)).to(adt)
    b = (0.3 * torch.randn(C, generator=gen)).to(adt)
    dy = torch.randn(M, C, generator=gen).to(dtype)
    return x, w, b, dy


def cu(*ts):
    return [None if t is None else t.cuda() for t in ts]


def check_forward(gn, x, w, b, eps, what, **kw):
    xg, wg, bg = cu(x, w, b)
    y, mean, rstd = gn.layer_norm_rows(xg, wg, bg, eps, stats=True, **kw)
    wy, wm, wr, ey, em, er = ref.layer_norm(x, w, b, eps, x.dtype)
    assert y.dtype == x.dtype and y.shape == x.shape and mean.shape == x.shape[:-1]
    ref.check(y, wy, ey, "%s y" % (what,))
    ref.check(mean, wm, em, "%s mean" % (what,))
    ref.check(rstd, wr, er, "%s rstd" % (what,))
    return y, mean, rstd


def check_backward(gn, dy, x, mean, rstd, w, what, saved=None):
    dyg, xg, wg = cu(dy, x, w)
    dx, dw, db = gn.layer_norm_rows_backward(dyg, xg if saved is None else saved, mean, rstd, wg)
    wdt = torch.float32 if w is None else w.dtype
    assert dx.dtype == dy.dtype and dw.dtype == wdt and db.dtype == wdt
    M = dy.numel() // dy.shape[-1]
    # a column's sum: at most M sequential additions of fp32
    wx, ww, wb, ex, ew, eb = ref.layer_norm_backward(dy, x, mean, rstd, w, dy.dtype, wdt,
                                                     min(M, 4096) + 16)
    ref.check(dx, wx, ex, "%s dx" % (what,))
    ref.check(dw, ww, ew, "%s dw" % (what,))
    ref.check(db, wb, eb, "%s db" % (what,))
    return dx, dw, db


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("C", WIDTHS)
def test_forward_and_backward_widths(gn, C, dtype):
    for M, adt in ((1, torch.float32), (5, dtype), (67, torch.float32)):
        print("case layer_norm M=%d C=%d %s affine=%s" % (M, C, dtype, adt), flush=True)
        x, w, b, dy = make(M, C, dtype, adt, 1000 * M + C)
        _, mean, rstd = check_forward(gn, x, w, b, EPS, (M, C, dtype))
        if C > 1:   # one value per row: h is zero, nothing to differentiate but dy's sum
            check_backward(gn, dy, x, mean, rstd, w, (M, C, dtype))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,C", [(2051, 40), (9001, 24), (4099, 257), (1025, 1024), (700, 2560),
                                 (1300, 4096)])
def test_many_rows(gn, M, C, dtype):
    """More rows than one round of workgroups."""
    print("case layer_norm rows M=%d C=%d %s" % (M, C, dtype), flush=True)
    x, w, b, dy = make(M, C, dtype, torch.float32, M + C)
    _, mean, rstd = check_forward(gn, x, w, b, EPS, (M, C, dtype))
    check_backward(gn, dy, x, mean, rstd, w, (M, C, dtype))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("C", SHORT)
def test_saved_input(gn, C, dtype):
    """The forward pass that also writes the checkpoint: y, mean and rstd as
    without it, the checkpoint as checkpoint_rows; the backward pass from it
    as from the values it stands for."""
    M = 37
    print("case layer_norm saved M=%d C=%d %s" % (M, C, dtype), flush=True)
    x, w, b, dy = make(M, C, dtype, torch.float32, 77 + C)
    xg, wg, bg = cu(x, w, b)
    y0, m0, r0 = gn.layer_norm_rows(xg, wg, bg, EPS, stats=True)
    y, mean, rstd, ck = gn.layer_norm_rows(xg, wg, bg, EPS, checkpoint=True)
    for p, q in ((y, y0), (mean, m0), (rstd, r0)):
        assert torch.equal(p, q)
    codes, E, val = ref.checkpoint(x)
    assert torch.equal(ck.codes.cpu().to(torch.int64), codes)
    assert torch.equal(ck.scales.cpu().to(torch.int64), E)
    if C > 1:
        check_backward(gn, dy, val, mean, rstd, w, (M, C, dtype, "saved"), saved=ck)


@pytest.mark.parametrize("which", ["none", "weight", "bias"])
def test_absent_parameters(gn, which):
    x, w, b, dy = make(21, 200, torch.bfloat16, torch.float32, 4)
    w = w if which == "weight" else None
    b = b if which == "bias" else None
    _, mean, rstd = check_forward(gn, x, w, b, EPS, which)
    check_backward(gn, dy, x, mean, rstd, w, which)
    dyg, xg = cu(dy, x)
    full = gn.layer_norm_rows_backward(dyg, xg, mean, rstd)
    alone = gn.layer_norm_rows_backward(dyg, xg, mean, rstd, weight_grad=False)
    assert alone[1] is None and alone[2] is None and torch.equal(alone[0], full[0])


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_far_from_zero_and_outliers(gn, dtype):
    """A mean far above the spread, one channel far above the rest, equal
    values, zeros: what cancels a one-pass variance."""
    C = 1000
    x = make(6, C, dtype, torch.float32, 8)[0].float()
    x[0] += 100.0
    x[1, 17] = 3000.0
    x[2] = 2.0
    x[3] = 0.0
    x[4, 0] = -2000.0
    x = x.to(dtype)
    _, w, b, dy = make(6, C, dtype, torch.float32, 9)
    _, mean, rstd = check_forward(gn, x, w, b, 1e-5, dtype)
    check_backward(gn, dy, x, mean, rstd, w, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("C", [24, 321, 1001, 4096])
def test_infinity_and_nan_stay_in_their_row(gn, C, dtype):
    x, w, b, dy = make(9, C, dtype, torch.float32, 6)
    x[1, 3] = float("inf")
    x[4, C - 1] = float("nan")
    x[6, 0] = float("-inf")
    xg, wg, bg, dyg = cu(x, w, b, dy)
    y, mean, rstd, ck = gn.layer_norm_rows(xg, wg, bg, EPS, checkpoint=True)
    dx, dw, db = gn.layer_norm_rows_backward(dyg, xg, mean, rstd, wg)
    dx8, _, _ = gn.layer_norm_rows_backward(dyg, ck, mean, rstd, wg)
    good = [0, 2, 3, 5, 7, 8]
    y2, m2, r2 = gn.layer_norm_rows(xg[good], wg, bg, EPS, stats=True)
    d2, _, _ = gn.layer_norm_rows_backward(dyg[good], xg[good], m2, r2, wg)
    assert torch.equal(y[good], y2) and torch.equal(dx[good], d2)
    assert bool(torch.isfinite(dx8[good]).all())
    for r in (1, 4, 6):
        # the statistics are not finite, so the whole row is NaN
        assert bool(torch.isnan(y[r]).all()) and bool(torch.isnan(dx[r]).all())
        assert bool(torch.isnan(dx8[r]).all())
    assert bool(torch.isnan(dw).all()) and bool(torch.isfinite(db).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_strides_alignment_and_leading_dimensions(gn, dtype):
    big, w, b, dyb = make(60, 333, dtype, dtype, 12)
    bg, dg = cu(big, dyb)
    for lo, hi in ((0, 333), (3, 331), (5, 261), (1, 2), (8, 264)):
        for shape in ((60, 333), (5, 12, 333), (3, 4, 5, 333)):
            x, dy = big.reshape(shape)[..., lo:hi], dyb.reshape(shape)[..., lo:hi]
            xg, dyg = bg.reshape(shape)[..., lo:hi], dg.reshape(shape)[..., lo:hi]
            print("case layer_norm view %s %s" % (tuple(xg.shape), xg.stride()), flush=True)
            ww, bb = w[lo:hi].contiguous(), b[lo:hi].contiguous()
            wg, wb = cu(ww, bb)
            y, mean, rstd = gn.layer_norm_rows(xg, wg, wb, EPS, stats=True)
            wy, wm, wr, ey, em, er = ref.layer_norm(x, ww, bb, EPS, dtype)
            ref.check(y, wy, ey, "y")
            if hi - lo > 1:
                dx, dw, db = gn.layer_norm_rows_backward(dyg, xg, mean, rstd, wg)
                r = ref.layer_norm_backward(dy, x, mean, rstd, ww, dtype, dtype, 80)
                for got, want, bound in zip((dx, dw, db), r[:3], r[3:]):
                    ref.check(got, want, bound, "gradient")
            # the same through outputs between other data
            wide = torch.full((60, 350), 5.0, dtype=dtype, device="cuda").reshape(
                shape[:-1] + (350,))
            r2 = gn.layer_norm_rows(xg, wg, wb, EPS, out=wide[..., 7:7 + hi - lo])
            assert torch.equal(r2, y)
            assert bool((wide[..., :7] == 5).all()) and bool((wide[..., 7 + hi - lo:] == 5).all())
    one = bg[4].expand(9, 333)      # one row for all (a broadcast input)
    y, mean, rstd = gn.layer_norm_rows(one, None, None, EPS, stats=True)
    assert torch.equal(y, gn.layer_norm_rows(bg[4:5], None, None, EPS).expand(9, 333))
    ga, _, _ = gn.layer_norm_rows_backward(dg[5].expand(9, 333), one, mean, rstd)
    gb, _, _ = gn.layer_norm_rows_backward(dg[5:6], bg[4:5], mean[:1], rstd[:1])
    assert torch.equal(ga, gb.expand(9, 333))
    # parameters at 2 mod 4
    pb = torch.empty(334, dtype=torch.bfloat16, device="cuda")
    pb[1:] = w.to(torch.bfloat16).cuda()
    z = gn.layer_norm_rows(bg, pb[1:], None, EPS)
    assert torch.equal(z, gn.layer_norm_rows(bg, pb[1:].float(), None, EPS))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("C", [24, 321, 1001, 2560, 5001])
def test_in_place(gn, C, dtype):
    x, w, b, dy = make(301, C, dtype, torch.float32, 31)
    xg, wg, bg, dyg = cu(x, w, b, dy)
    y, mean, rstd = gn.layer_norm_rows(xg, wg, bg, EPS, stats=True)
    dx = gn.layer_norm_rows_backward(dyg, xg, mean, rstd, wg)
    for target in ("dy", "x"):
        d2, x2 = dyg.clone(), xg.clone()
        out = d2 if target == "dy" else x2
        r = gn.layer_norm_rows_backward(d2, x2, mean, rstd, wg, out=out)
        for p, q in zip(r, dx):
            assert torch.equal(p, q)
    x2 = xg.clone()
    assert gn.layer_norm_rows(x2, wg, bg, EPS, out=x2) is x2
    assert torch.equal(x2, y)


@pytest.mark.parametrize("M", [301, 1500])
@pytest.mark.parametrize("C", [24, 321, 1001, 2560])
def test_in_place_with_checkpoints(gn, M, C):
    """y in x's place while x is saved; dx in dy's place while x comes saved;
    few rows and many."""
    x, w, b, dy = cu(*make(M, C, torch.bfloat16, torch.float32, 5 * C))
    y, mean, rstd, ck = gn.layer_norm_rows(x, w, b, EPS, checkpoint=True)
    want = gn.layer_norm_rows_backward(dy, ck, mean, rstd, w)
    x2, d2 = x.clone(), dy.clone()
    r = gn.layer_norm_rows(x2, w, b, EPS, checkpoint=True, out=x2)
    assert torch.equal(x2, y) and torch.equal(r[1], mean) and torch.equal(r[2], rstd)
    assert torch.equal(r[3].codes, ck.codes) and torch.equal(r[3].scales, ck.scales)
    got = gn.layer_norm_rows_backward(d2, ck, mean, rstd, w, out=d2)
    for p, q in zip(got, want):
        assert torch.equal(p, q)
    # the saved rows in another type than the gradient's: only the codes count
    ck32 = gn.Checkpoint8(ck.codes, ck.scales, torch.float32)
    for p, q in zip(gn.layer_norm_rows_backward(dy, ck32, mean, rstd, w), want):
        assert torch.equal(p, q)


def test_same_bits_on_every_call_and_stream(gn):
    x, w, b, dy = cu(*make(3001, 1030, torch.bfloat16, torch.float32, 2))
    y, mean, rstd = gn.layer_norm_rows(x, w, b, EPS, stats=True)
    first = gn.layer_norm_rows_backward(dy, x, mean, rstd, w)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        again = gn.layer_norm_rows_backward(dy, x, mean, rstd, w)
        with torch.cuda.stream(other):
            there = gn.layer_norm_rows_backward(dy, x, mean, rstd, w)
            y2 = gn.layer_norm_rows(x, w, b, EPS)
        torch.cuda.synchronize()
        assert torch.equal(y, y2)
        for p, q, r in zip(first, again, there):
            assert torch.equal(p, q) and torch.equal(p, r)


def test_two_captured_graphs_with_eager_work_between(gn):
    """Each captured backward pass has its own workspace: replays in any
    order, on two streams at once, give the eager bits."""
    sets = [cu(*make(513, C, torch.bfloat16, torch.float32, C)) for C in (777, 2304)]
    eager, graphs, outs = [], [], []
    for x, w, b, dy in sets:
        y, mean, rstd = gn.layer_norm_rows(x, w, b, EPS, stats=True)
        eager.append((y,) + gn.layer_norm_rows_backward(dy, x, mean, rstd, w))
    torch.cuda.synchronize()
    for x, w, b, dy in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y, mean, rstd = gn.layer_norm_rows(x, w, b, EPS, stats=True)
            o = (y,) + gn.layer_norm_rows_backward(dy, x, mean, rstd, w)
        graphs.append(g)
        outs.append(o)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(3):
        for o in outs:
            for t in o:
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        x, w, b, dy = sets[turn % 2]
        y, mean, rstd = gn.layer_norm_rows(x, w, b, EPS, stats=True)
        mine = (y,) + gn.layer_norm_rows_backward(dy, x, mean, rstd, w)
        torch.cuda.synchronize()
        for p, q in zip(mine, eager[turn % 2]):
            assert torch.equal(p, q)
        for o, e in zip(outs, eager):
            for p, q in zip(o, e):
                assert torch.equal(p, q)


def test_gradient_against_differences(gn):
    """dx, dw and db against central differences of the forward definition in
    64 bits: f(theta) = sum(v * layer_norm(theta)), along random directions.
    The differences are off by h^2/6 * |f'''|, far below the bound taken from
    the roundings of the fp32 gradients."""
    M, C = 7, 130
    x, w, b, v = make(M, C, torch.float32, torch.float32, 15)
    xg, wg, bg, vg = cu(x, w, b, v)
    _, mean, rstd = gn.layer_norm_rows(xg, wg, bg, EPS, stats=True)
    grads = [t.cpu().double() for t in gn.layer_norm_rows_backward(vg, xg, mean, rstd, wg)]
    theta = [x.double(), w.double(), b.double()]

    def f(t):
        d = t[0] - t[0].mean(-1, keepdim=True)
        h = d / torch.sqrt((d * d).mean(-1, keepdim=True) + EPS)
        return (v.double() * (h * t[1] + t[2])).sum()

    gen = torch.Generator().manual_seed(1)
    for i in range(3):
        for _ in range(4):
            u = torch.randn(theta[i].shape, generator=gen, dtype=torch.float64)
            up, dn = list(theta), list(theta)
            up[i], dn[i] = theta[i] + 1e-5 * u, theta[i] - 1e-5 * u
            num = float((f(up) - f(dn)) / 2e-5)
            ana = float((grads[i] * u).sum())
            # every term of the product off by at most 200 fp32 roundings of its
            # size, the differences by 1e-8 of the terms' sum
            scale = float((grads[i].abs() * u.abs()).sum()) + float(v.abs().sum())
            assert abs(num - ana) <= (200 * ref.U + 1e-7) * scale


def test_no_rows(gn):
    w = torch.ones(40, dtype=torch.bfloat16, device="cuda")
    for shape in ((0, 40), (2, 0, 40)):
        x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        y, mean, rstd, ck = gn.layer_norm_rows(x, w, w, EPS, checkpoint=True)
        assert y.shape == x.shape and mean.shape == shape[:-1] and ck.shape == x.shape
        dx, dw, db = gn.layer_norm_rows_backward(x, x, mean, rstd, w)
        assert dx.shape == x.shape
        assert bool((dw == 0).all()) and bool((db == 0).all()) and dw.dtype == torch.bfloat16
        dx, dw, db = gn.layer_norm_rows_backward(x, ck, mean, rstd, w, weight_grad=False)
        assert dw is None and db is None


def test_offsets_beyond_32_bits(gn):
    """Rows of x, dy and dx that lie beyond 2^31 elements, and beyond 2^32
    bytes, of one buffer."""
    C, step = 64, (1 << 31) // 3 + 7
    buf = torch.zeros(3 * step + C + 64, dtype=torch.bfloat16, device="cuda")
    x, w, b, dy = make(4, C, torch.bfloat16, torch.float32, 3)
    view = torch.as_strided(buf, (4, C), (step, 1))
    view.copy_(x.cuda())
    y, mean, rstd = gn.layer_norm_rows(view, w.cuda(), b.cuda(), EPS, stats=True)
    want = gn.layer_norm_rows(x.cuda(), w.cuda(), b.cuda(), EPS)
    assert torch.equal(y, want)
    out = torch.as_strided(buf, (4, C), (step, 1), 64)
    assert gn.layer_norm_rows(view, w.cuda(), b.cuda(), EPS, out=out) is not None
    assert torch.equal(out, want)
    d1 = gn.layer_norm_rows_backward(dy.cuda(), view, mean, rstd, w.cuda(), out=out)
    d2 = gn.layer_norm_rows_backward(dy.cuda(), x.cuda(), mean, rstd, w.cuda())
    for p, q in zip(d1, d2):
        assert torch.equal(p, q)


def corrected_bounds(x, w, b, eps):
    """ref.layer_norm's values for fp32 rows with the bounds of a mean that is
    corrected by the mean difference from it.  D = ref.ROW_DEPTH + 4 roundings
    stand for a sum of differences, their own rounding and the quotient."""
    y, mean, rstd, _, _, _ = ref.layer_norm(x, w, b, eps, torch.float32)
    U, D = ref.U, ref.ROW_DEPTH + 4
    x = x.double()
    mean, rstd = mean.unsqueeze(-1), rstd.unsqueeze(-1)
    d = x - mean
    var = (d * d).mean(-1, keepdim=True)
    e1 = D * U * x.abs().mean(-1, keepdim=True)             # the first mean
    a = d.abs() + e1                                        # differences from it, at most
    es = D * U * a.mean(-1, keepdim=True)                   # the shift
    ec = es + U * (a + d.abs() + es)                        # the centred values
    dv = (D * U * (a * a).mean(-1, keepdim=True) + 2 * (e1 + es) * es + es * es
          + 3 * U * (e1 + es) ** 2 + U * var)
    assert bool((dv < var + eps).all())
    er = 0.5 * dv * (var + eps - dv) ** -1.5 + 3 * U * rstd
    ey = (w.abs().double() * (rstd * ec + (d.abs() + ec) * er + 2 * U * (d * rstd).abs())
          + U * (y.abs() + b.abs().double()))
    em = es + U * mean.abs()
    return (y, mean.squeeze(-1), rstd.squeeze(-1), 1.01 * ey + ref.rounded(y, torch.float32),
            1.01 * em.squeeze(-1), 1.01 * er.squeeze(-1))


@pytest.mark.parametrize("save", [False, True])
@pytest.mark.parametrize("C", [1, 3, 8, 129, 768, 777, 1001, 4095, 4100, 12288, 16383])
def test_fp32_rows_whose_spread_is_lost_in_their_size(gn, C, save):
    """Equal values, and a spread of a few steps of fp32, far from zero: the
    mean has to be nearer than the roundings of a plain fp32 sum."""
    print("case layer_norm far rows C=%d save=%s" % (C, save), flush=True)
    gen = torch.Generator().manual_seed(C)
    x = torch.empty(6, C)
    x[0], x[1], x[2] = 10000.1, -1000.3, 100.7
    x[3] = 10000.0 + 0.01 * torch.randn(C, generator=gen)
    x[4] = -3000.0 + 0.001 * torch.randn(C, generator=gen)
    x[5] = torch.randn(C, generator=gen)
    w = 1 + 0.3 * torch.randn(C, generator=gen)
    b = 0.3 * torch.randn(C, generator=gen)
    r = gn.layer_norm_rows(*cu(x, w, b), EPS, stats=True, checkpoint=save)
    want = corrected_bounds(x, w, b, EPS)
    for got, v, bound, name in zip(r, want[:3], want[3:], ("y", "mean", "rstd")):
        ref.check(got, v, bound, "C=%d %s" % (C, name))
    assert torch.equal(r[0][:3].cpu(), b.expand(3, C))      # equal values: beta


@pytest.mark.parametrize("C", [5, 777, 1001, 4095, 12288])
def test_fp32_rows_of_equal_values_whose_squares_are_infinite(gn, C):
    """Equal values so large that the squares of a sum's roundings leave fp32:
    the normalised values are still at most a few roundings from zero."""
    b = torch.randn(C, generator=torch.Generator().manual_seed(C))
    # the values above times a power of two: their sums are rounded alike
    x = (torch.tensor([10000.1, -1000.3, 100.7]) * 2.0 ** 90).unsqueeze(1).expand(3, C)
    for save in (False, True):
        r = gn.layer_norm_rows(x.contiguous().cuda(), None, b.cuda(), EPS, stats=True,
                               checkpoint=save)
        y, mean = r[0].cpu(), r[1].cpu()
        # 2^-12, the root of a rounding: y is the rounding of a difference over
        # the root of the rounding of its square, or over infinity
        assert float((y - b).abs().max()) <= 2.0 ** -12
        assert bool(((mean - x[:, 0]).abs() <= 4 * ref.U * x[:, 0].abs()).all())
