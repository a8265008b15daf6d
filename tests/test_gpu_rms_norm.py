"""Root-mean-square norm, forward and backward, and rows in 8 bits against the
definitions in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

import rows8_reference as ref  # noqa: E402
import rows_reference as rows  # noqa: E402

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
EPS = 1e-6
# widths on both sides of every lane count and piece count of the kernels
WIDTHS = [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 31, 33, 64, 65, 100, 127, 129, 256, 257, 320, 511,
          513, 768, 1001, 1024, 1030, 1536, 2047, 2048, 2049, 2560, 4096, 4097, 5000, 8192, 8193,
          12288, 16383, 16384]


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
    x = (torch.randn(M, C, generator=gen) * torch.exp(0.3 * torch.randn(C, generator=gen))).to(dtype)
    r = torch.randn(M, C, generator=gen).to(dtype)
    w = (1 + 0.3 * torch.randn(C, generator=gen)).to(adt)
    dy = torch.randn(M, C, generator=gen).to(dtype)
    return x, r, w, dy


def cu(*ts):
    return [None if t is None else t.cuda() for t in ts]


def check_codes(q, codes, scales, es, what):
    assert torch.equal(q.codes.cpu().to(torch.int64), codes), "%s codes" % (what,)
    rows.check(q.scales, scales, es, "%s scales" % (what,))


def check_forward(gn, x, r, w, eps, what):
    """All four outputs' forms; (h, rstd) on the GPU."""
    xg, rg, wg = cu(x, r, w)
    wh, wy, wr, wq, ws, ey, er, es = ref.rms_norm(x, w, eps, x.dtype, r)
    got = gn.rms_norm_rows(xg, wg, eps, residual=rg, stats=True)
    y, h, rstd = got if r is not None else (got[0], xg, got[1])
    assert y.dtype == x.dtype and y.shape == x.shape and rstd.shape == x.shape[:-1]
    assert torch.equal(h.cpu(), wh), "%s h" % (what,)
    rows.check(y, wy, ey, "%s y" % (what,))
    rows.check(rstd, wr, er, "%s rstd" % (what,))
    got = gn.rms_norm_rows(xg, wg, eps, residual=rg, quantize=True)
    q = got[0] if r is not None else got
    if r is not None:
        assert torch.equal(got[1], h)
    assert isinstance(q, gn.Rows8) and q.shape == x.shape and q.dtype == x.dtype
    check_codes(q, wq, ws, es, what)
    return h, rstd


def check_backward(gn, dy, h, rstd, w, dh, what, saved=None):
    dyg, wg, dhg = cu(dy, w, dh)
    dx, dw = gn.rms_norm_rows_backward(dyg, h.cuda() if saved is None else saved, rstd, wg,
                                       residual_grad=dhg)
    wdt = torch.float32 if w is None else w.dtype
    assert dx.dtype == dy.dtype and dw.dtype == wdt
    M = dy.numel() // dy.shape[-1]
    # a column's sum: at most M sequential additions of fp32
    wx, ww, ex, ew = ref.rms_norm_backward(dy, h, rstd, w, dh, dy.dtype, wdt, min(M, 4096) + 16)
    rows.check(dx, wx, ex, "%s dx" % (what,))
    rows.check(dw, ww, ew, "%s dw" % (what,))
    return dx, dw


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("C", WIDTHS)
def test_widths(gn, C, dtype):
    for M, adt, with_res in ((1, torch.float32, True), (5, dtype, False), (67, torch.float32, True)):
        what = (M, C, dtype, with_res)
        print("case rms_norm %s" % (what,), flush=True)
        x, r, w, dy = make(M, C, dtype, adt, 1000 * M + C)
        h, rstd = check_forward(gn, x, r if with_res else None, w, EPS, what)
        check_backward(gn, dy, h, rstd, w, r if with_res else None, what)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,C", [(2051, 40), (9001, 24), (4099, 257), (1025, 1024), (700, 2560),
                                 (1300, 4096), (3001, 1537), (1111, 5000)])
def test_many_rows(gn, M, C, dtype):
    """More rows than one round of workgroups, from h and from its checkpoint."""
    what = (M, C, dtype)
    print("case rms_norm rows %s" % (what,), flush=True)
    x, r, w, dy = make(M, C, dtype, torch.float32, M + C)
    h, rstd = check_forward(gn, x, r, w, EPS, what)
    check_backward(gn, dy, h, rstd, w, r, what)
    ck = gn.checkpoint_rows(h)
    val = gn.restore_rows(ck, torch.float32)
    check_backward(gn, dy, val, rstd, w, None, what + ("saved",), saved=ck)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,C", [(5000, 2560), (17001, 513), (1500, 9000)])
def test_several_rows_a_slot(gn, M, C, dtype):
    """Forward passes of more rows than the launches' row slots."""
    what = (M, C, dtype)
    print("case rms_norm slots %s" % (what,), flush=True)
    x, r, w, _ = make(M, C, dtype, dtype, M + C)
    check_forward(gn, x, r, w, EPS, what)
    check_forward(gn, x, None, w, EPS, what)
    q = gn.quantize_rows(x.cuda())
    check_codes(q, *ref.quantize(x), what)
    want = q.codes.cpu().double() * q.scales.cpu().double().unsqueeze(-1)
    rows.check(gn.dequantize_rows(q), want, rows.U * want.abs() + rows.rounded(want, dtype),
               "%s widened" % (what,))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("C", [1, 3, 8, 15, 33, 65, 257, 513, 1001, 1030, 2049, 2560, 4097, 8193,
                               16383])
def test_gradient_from_a_checkpoint(gn, C, dtype):
    x, r, w, dy = make(37, C, dtype, dtype, 77 + C)
    xg, wg = cu(x, w)
    _, rstd = gn.rms_norm_rows(xg, wg, EPS, stats=True)
    ck = gn.checkpoint_rows(xg)
    check_backward(gn, dy, rows.checkpoint(x)[2], rstd, w, r, (C, dtype, "saved"), saved=ck)


def test_absent_parameters(gn):
    x, r, w, dy = make(21, 200, torch.bfloat16, torch.float32, 4)
    h, rstd = check_forward(gn, x, r, None, EPS, "no weight")
    check_backward(gn, dy, h, rstd, None, None, "no weight")
    dyg, wg = cu(dy, w)
    full = gn.rms_norm_rows_backward(dyg, h, rstd, wg)
    alone = gn.rms_norm_rows_backward(dyg, h, rstd, wg, weight_grad=False)
    assert alone[1] is None and torch.equal(alone[0], full[0])
    xg, = cu(x)
    assert torch.equal(gn.rms_norm_rows(xg, wg, EPS), gn.rms_norm_rows(xg, wg, EPS, stats=True)[0])


@pytest.mark.parametrize("dtype", DTYPES)
def test_codes_next_to_borders(gn, dtype):
    """Rows whose products with the weight lie on and beside the borders between
    two codes, in both signs, and rows of tiny, huge and equal values."""
    C = 1280
    k = torch.arange(C) % 127
    t = (k + 0.5) * torch.where(torch.arange(C) % 2 == 0, 1.0, -1.0)
    t[0] = 127.0
    x = torch.stack([t, t * 2 ** -7, t * 3, t * 5, t * 7, t * 31, torch.full((C,), -2.5),
                     torch.zeros(C), t * 2.0 ** -20])
    if dtype != torch.float16:
        x = torch.cat([x, torch.stack([t * 2.0 ** -126, t * 2.0 ** -118, t * 2.0 ** 118,
                                       t * 2.0 ** -133])])
    steps = torch.tensor([0.0, 2.0 ** -23, -2.0 ** -23])
    x = torch.cat([x, x[:6] * (1 + steps[torch.arange(C) % 3])]).to(dtype)
    q = gn.quantize_rows(x.cuda())
    check_codes(q, *ref.quantize(x), "quantize")
    w = torch.ones(C)
    w[3::7] = 1 + 2.0 ** -23
    w[4::7] = 1 - 2.0 ** -24
    q = gn.rms_norm_rows(x[:7].cuda(), w.cuda(), 1e-5, quantize=True)
    _, _, _, wq, ws, _, _, es = ref.rms_norm(x[:7], w, 1e-5, dtype)
    check_codes(q, wq, ws, es, "rms_norm")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("C", [24, 321, 1001, 4096, 9000])
def test_infinity_nan_and_zero_stay_in_their_row(gn, C, dtype):
    x, r, w, dy = make(10, C, dtype, torch.float32, 6)
    x[1, 3] = float("inf")
    x[4, C - 1] = float("nan")
    x[6, 0] = float("-inf")
    x[8] = 0.0
    xg, wg, dyg = cu(x, w, dy)
    q = gn.quantize_rows(xg)
    check_codes(q, *ref.quantize(x), "quantize")
    bad = [1, 4, 6]
    assert bool(torch.isnan(gn.dequantize_rows(q)[bad]).all())
    y, rstd = gn.rms_norm_rows(xg, wg, EPS, stats=True)
    n = gn.rms_norm_rows(xg, wg, EPS, quantize=True)
    assert bool(torch.isnan(n.scales[bad]).all()) and not n.codes[bad].any()
    assert not n.codes[8].any() and float(n.scales[8]) == 0.0 and not y[8].any()
    good = [0, 2, 3, 5, 7, 8, 9]
    y2, r2 = gn.rms_norm_rows(xg[good], wg, EPS, stats=True)
    assert torch.equal(y[good], y2)
    dx, _ = gn.rms_norm_rows_backward(dyg, xg, rstd, wg)
    d2, _ = gn.rms_norm_rows_backward(dyg[good], xg[good], r2, wg)
    assert torch.equal(dx[good], d2)


@pytest.mark.parametrize("dtype", DTYPES)
def test_strides_and_what_lies_between_rows(gn, dtype):
    C, M = 333, 40
    x, r, w, dy = make(M, C, dtype, torch.float32, 12)
    xg, rg, wg, dyg = cu(x, r, w, dy)
    wide = [torch.full((M, C + 7), 3.0, dtype=dtype, device="cuda") for _ in range(5)]
    xs, rs, ys, hs, ds = [t[:, 2:2 + C] for t in wide]
    xs.copy_(xg)
    rs.copy_(rg)
    y, h, rstd = gn.rms_norm_rows(xg, wg, EPS, residual=rg, stats=True)
    y2, h2, rstd2 = gn.rms_norm_rows(xs, wg, EPS, residual=rs, stats=True, out=ys, residual_out=hs)
    assert y2 is ys and h2 is hs
    assert torch.equal(y, y2) and torch.equal(h, h2) and torch.equal(rstd, rstd2)
    dx, dw = gn.rms_norm_rows_backward(dyg, h, rstd, wg, residual_grad=rg)
    dx2, dw2 = gn.rms_norm_rows_backward(dyg, hs, rstd, wg, residual_grad=rs, out=ds)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    for t in wide:
        assert bool((t[:, :2] == 3).all()) and bool((t[:, 2 + C:] == 3).all())
    # one row for all, as the residual and as x
    one = rg[:1].expand(M, C)
    a = gn.rms_norm_rows(xg, wg, EPS, residual=one)
    b = gn.rms_norm_rows(xg, wg, EPS, residual=one.contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # through the C entry: codes at their own stride, the bytes between them kept
    codes = torch.full((M, C + 5), 77, dtype=torch.int8, device="cuda")
    scales = torch.empty(M, device="cuda")
    assert gn.gn_quantize_rows(xg.data_ptr(), C, codes.data_ptr(), C + 5, scales.data_ptr(), M, C,
                               gn.dtype_code(dtype),
                               torch.cuda.current_stream().cuda_stream) == gn.GnStatus.OK
    q = gn.quantize_rows(xg)
    assert torch.equal(codes[:, :C], q.codes) and bool((codes[:, C:] == 77).all())
    assert torch.equal(scales, q.scales)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,C", [(3, 77), (64, 1001), (2000, 515), (1500, 4097), (300, 12001)])
def test_in_place(gn, M, C, dtype):
    x, r, w, dy = make(M, C, dtype, dtype, M + C)
    xg, rg, wg, dyg = cu(x, r, w, dy)
    y, h, rstd = gn.rms_norm_rows(xg, wg, EPS, residual=rg, stats=True)
    a, b = xg.clone(), rg.clone()
    y2, h2 = gn.rms_norm_rows(a, wg, EPS, residual=b, out=a, residual_out=b)
    assert y2 is a and h2 is b and torch.equal(y2, y) and torch.equal(h2, h)
    a = xg.clone()
    _, h3 = gn.rms_norm_rows(a, wg, EPS, residual=rg, residual_out=a)
    assert torch.equal(h3, h)
    dx, dw = gn.rms_norm_rows_backward(dyg, h, rstd, wg, residual_grad=rg)
    for which in range(3):      # dx over dy, over h, over the residual's gradient
        args = [dyg.clone(), h.clone(), rg.clone()]
        d2, w2 = gn.rms_norm_rows_backward(args[0], args[1], rstd, wg, residual_grad=args[2],
                                           out=args[which])
        assert d2 is args[which] and torch.equal(d2, dx) and torch.equal(w2, dw)


def test_gradient_against_differences(gn):
    """The gradient of sum(y * dy) + sum(h * dh) by central differences of the
    definition in 64 bits."""
    M, C, d = 3, 19, 1e-5
    x, r, w, dy = make(M, C, torch.float32, torch.float32, 31)
    dh = torch.flip(dy, (0,))
    rstd = gn.rms_norm_rows(x.cuda(), w.cuda(), EPS, stats=True)[1]
    dx, dw = gn.rms_norm_rows_backward(*cu(dy, x), rstd, w.cuda(), residual_grad=dh.cuda())

    def loss(xx, ww):
        n = xx / torch.sqrt((xx * xx).mean(-1, keepdim=True) + EPS)
        return float((n * ww * dy.double()).sum() + (xx * dh.double()).sum())

    x64, w64 = x.double(), w.double()
    for i in range(M):
        for j in range(0, C, 3):
            e = torch.zeros_like(x64)
            e[i, j] = d
            want = (loss(x64 + e, w64) - loss(x64 - e, w64)) / (2 * d)
            # fp32 (2^-20 of the size of the terms) and the difference's own d^2
            assert abs(float(dx[i, j]) - want) < 2e-5 * (1 + abs(want))
    for j in range(C):
        e = torch.zeros_like(w64)
        e[j] = d
        want = (loss(x64, w64 + e) - loss(x64, w64 - e)) / (2 * d)
        assert abs(float(dw[j]) - want) < 2e-5 * (1 + abs(want))


def test_dequantize(gn):
    x, _, _, _ = make(33, 1001, torch.bfloat16, torch.float32, 9)
    q = gn.quantize_rows(x.cuda())
    want = q.codes.cpu().double() * q.scales.cpu().double().unsqueeze(-1)
    for dt in DTYPES:
        got = gn.dequantize_rows(q, dt)
        # the product, and its rounding to the type
        rows.check(got, want, rows.U * want.abs() + rows.rounded(want, dt), str(dt))
    out = torch.full((33, 1010), 5.0, device="cuda")
    assert gn.dequantize_rows(q, out=out[:, :1001]) is not None
    assert bool((out[:, 1001:] == 5).all())
    assert torch.equal(out[:, :1001], gn.dequantize_rows(q, torch.float32))
    assert gn.dequantize_rows(q).dtype == torch.bfloat16
    dense = gn.Rows8(q.codes.contiguous(), q.scales, torch.bfloat16)
    assert torch.equal(gn.dequantize_rows(dense), gn.dequantize_rows(q))


def test_no_rows(gn):
    w = torch.ones(40, device="cuda", dtype=torch.bfloat16)
    x = torch.empty(0, 40, device="cuda", dtype=torch.bfloat16)
    y, h, rstd = gn.rms_norm_rows(x, w, EPS, residual=x, stats=True)
    assert y.shape == (0, 40) and h.shape == (0, 40) and rstd.shape == (0,)
    q = gn.rms_norm_rows(x, w, EPS, quantize=True)
    assert q.shape == (0, 40) and gn.dequantize_rows(q).shape == (0, 40)
    assert gn.quantize_rows(x).shape == (0, 40)
    dx, dw = gn.rms_norm_rows_backward(x, x, rstd, w)
    assert dx.shape == (0, 40) and dw.dtype == torch.bfloat16 and not dw.any()


def test_declined_and_refused_on_the_gpu(gn):
    x = torch.ones(4, 64, device="cuda")
    st = torch.ones(4, device="cuda")
    assert gn.rms_norm_rows(x.double()) is None
    assert gn.rms_norm_rows(x, residual=x.half()) is None
    assert gn.rms_norm_rows(x, torch.ones(64)) is None              # weight on the CPU
    assert gn.rms_norm_rows(x.t()) is None
    assert gn.rms_norm_rows(torch.ones(2, 16385, device="cuda")) is None
    assert gn.quantize_rows(torch.ones(2, 16385, device="cuda")) is None
    assert gn.rms_norm_rows_backward(x, x.half(), st) is None
    assert gn.rms_norm_rows_backward(x, x, st, residual_grad=x.half()) is None
    with torch.enable_grad():
        assert gn.rms_norm_rows(x) is None and gn.quantize_rows(x) is None
    for call in (lambda: gn.rms_norm_rows(x, residual=x[:2]),
                 lambda: gn.rms_norm_rows(x, torch.ones(63, device="cuda")),
                 lambda: gn.rms_norm_rows(x, quantize=True, out=x),
                 lambda: gn.rms_norm_rows(x, residual_out=x),
                 lambda: gn.rms_norm_rows(x, out=x[:2]),
                 lambda: gn.rms_norm_rows(x, eps=-1.0),
                 lambda: gn.rms_norm_rows(x, residual=x, out=(y := x.clone()), residual_out=y),
                 lambda: gn.rms_norm_rows_backward(x, x, st[:3]),
                 lambda: gn.rms_norm_rows_backward(x, x[:2], st),
                 lambda: gn.rms_norm_rows_backward(x, x, st, residual_grad=x[:2])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        gn.rms_norm_rows(x, residual=3.0)


def test_offsets_beyond_32_bits(gn):
    """Rows whose byte and element offsets pass 2^32: the last rows of a wide
    stride (values elsewhere are never touched)."""
    C, M, stride = 1000, 5, (1 << 30) + 8
    buf = torch.empty(4 * stride + C, dtype=torch.bfloat16, device="cuda")
    xs = buf.as_strided((M, C), (stride, 1))
    x, r, w, dy = make(M, C, torch.bfloat16, torch.float32, 3)
    xs.copy_(x)
    wg, rg, dyg = cu(w, r, dy)
    y, h, rstd = gn.rms_norm_rows(xs, wg, EPS, residual=rg, stats=True)
    y2, h2, rstd2 = gn.rms_norm_rows(x.cuda(), wg, EPS, residual=rg, stats=True)
    assert torch.equal(y, y2) and torch.equal(h, h2)
    q = gn.quantize_rows(xs)
    assert torch.equal(q.codes, gn.quantize_rows(x.cuda()).codes)
    dx, dw = gn.rms_norm_rows_backward(dyg, xs, rstd, wg)
    dx2, dw2 = gn.rms_norm_rows_backward(dyg, x.cuda(), rstd, wg)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    del xs, buf


def test_captured_graph(gn):
    M, C = 1500, 1001
    x, r, w, dy = cu(*make(M, C, torch.bfloat16, torch.float32, 5))
    new = cu(*make(M, C, torch.bfloat16, torch.float32, 6))

    def step():
        y, h, rstd = gn.rms_norm_rows(x, w, EPS, residual=r, stats=True)
        q = gn.rms_norm_rows(x, w, EPS, quantize=True)
        dx, dw = gn.rms_norm_rows_backward(dy, h, rstd, w, residual_grad=r)
        return y, h, rstd, q.codes, q.scales, gn.dequantize_rows(q), dx, dw

    step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for k in range(4):
        x.copy_(new[k % 2])
        dy.copy_(new[3] if k < 2 else new[1])
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b)


def test_another_stream_and_bits_alike(gn):
    x, r, w, dy = cu(*make(3000, 515, torch.float16, torch.float16, 8))
    y, h, rstd = gn.rms_norm_rows(x, w, EPS, residual=r, stats=True)
    dx, dw = gn.rms_norm_rows_backward(dy, h, rstd, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y2, h2, rstd2 = gn.rms_norm_rows(x, w, EPS, residual=r, stats=True)
        dx2, dw2 = gn.rms_norm_rows_backward(dy, h2, rstd2, w)
    s.synchronize()
    for a, b in ((y, y2), (h, h2), (rstd, rstd2), (dx, dx2), (dw, dw2)):
        assert torch.equal(a, b)
