"""The backward pass of GroupNorm(+SiLU) and the apply step that saves its
input, against the definition in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

import rows_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
# (N, L, C, G): widths on both sides of the pieces, of one and several column
# blocks, groups inside a piece, across pieces, of more than 64 channels, one
# group, one channel per group; one row and many
SHAPES = [
    (1, 1, 64, 8), (1, 5, 1, 1), (2, 9, 2, 1), (2, 7, 3, 3), (1, 33, 5, 1), (3, 17, 7, 7),
    (2, 40, 8, 2), (1, 300, 12, 3), (2, 65, 24, 24), (1, 129, 33, 3), (2, 50, 64, 64),
    (1, 257, 96, 32), (3, 31, 130, 13), (1, 64, 128, 1), (2, 100, 320, 32), (1, 77, 321, 3),
    (5, 13, 512, 32), (1, 1030, 256, 32), (2, 19, 1001, 7), (1, 21, 1001, 1), (1, 40, 2048, 8),
    (1, 9, 2056, 8), (2, 11, 2560, 32), (1, 6, 4100, 4), (1, 12, 8192, 32), (1, 5, 8190, 90),
    (1, 3, 8192, 1), (300, 3, 32, 4),
]


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


def make(N, L, C, G, dtype, adt, seed):
    """Rows, parameters, a gradient, and the statistics in fp32."""
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(N, L, C, generator=gen) * torch.exp(0.3 * torch.randn(C, generator=gen))
         + 0.5 * torch.randn(C, generator=gen)).to(dtype)
    w = (1 + 0.3 * torch.randn(C, generator=gen)).to(adt)
    b = (0.3 * torch.randn(C, generator=gen)).to(adt)
    dy = torch.randn(N, L, C, generator=gen).to(dtype)
    xg = x.double().reshape(N, L, G, C // G)
    mean = xg.mean((1, 3))
    var = ((xg - mean[:, None, :, None]) ** 2).mean((1, 3))
    return x, w, b, dy, mean.float(), (1.0 / torch.sqrt(var + 1e-6)).float()


def cu(*ts):
    return [None if t is None else t.cuda() for t in ts]


def check_backward(gn, dy, x, mean, rstd, w, b, silu, what, saved=None):
    dyg, xg, mg, rg, wg, bg = cu(dy, x, mean, rstd, w, b)
    r = gn.group_norm_silu_rows_backward(dyg, xg if saved is None else saved, mg, rg, wg, bg, silu)
    p = w if w is not None else b
    wdt = torch.float32 if p is None else p.dtype
    assert r[0].dtype == dy.dtype and r[1].dtype == wdt and r[2].dtype == wdt
    # a channel's sum: at most 1024 rows of a lane in sequence, 8 tree steps
    N, L, C = dy.shape
    want = ref.group_norm_backward(dy, x, mean, rstd, w, b, silu, dy.dtype, wdt,
                                   min(L, 1024) + 10)
    for got, wv, bound, name in zip(r, want[:3], want[3:], ("dx", "dw", "db")):
        ref.check(got, wv, bound, "%s %s" % (what, name))
    return r


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(gn, shape, dtype, silu):
    N, L, C, G = shape
    adt = dtype if C % 3 else torch.float32
    print("case gn backward %s %s silu=%s affine=%s" % (shape, dtype, silu, adt), flush=True)
    x, w, b, dy, mean, rstd = make(N, L, C, G, dtype, adt, 13 * C + L)
    check_backward(gn, dy, x, mean, rstd, w, b, silu, (shape, dtype, silu))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(1, 20011, 40, 8), (2, 9000, 64, 32), (1, 5000, 321, 3),
                                   (1, 4096, 512, 32), (1, 2003, 2560, 32), (2, 5000, 64, 64),
                                   (1, 3001, 512, 1), (3, 1500, 2048, 4), (2, 4097, 8, 1),
                                   (130, 40, 64, 16), (1, 4096, 128, 32), (3, 4095, 32, 16)])
def test_many_rows(gn, shape, dtype):
    """Chunks of several rounds of rows, with remainders; samples on both sides
    of the single launch's limits."""
    N, L, C, G = shape
    print("case gn backward rows %s %s" % (shape, dtype), flush=True)
    x, w, b, dy, mean, rstd = make(N, L, C, G, dtype, torch.float32, L)
    check_backward(gn, dy, x, mean, rstd, w, b, True, (shape, dtype))


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [s for s in SHAPES if s[2] % 64 != 0] + [(2, 333, 256, 32)])
def test_apply_that_saves(gn, shape, dtype, silu):
    """y as the apply step's (where that takes the shape), bit for bit in
    bf16 and fp32, the checkpoint as checkpoint_rows, and the backward pass
    from it."""
    N, L, C, G = shape
    print("case gn save %s %s silu=%s" % (shape, dtype, silu), flush=True)
    x, w, b, dy, mean, rstd = make(N, L, C, G, dtype, torch.float32, 7 * C + L)
    xg, wg, bg, mg, rg = cu(x, w, b, mean, rstd)
    y, ck = gn.apply_rows(xg, mg, rg, wg, bg, silu, checkpoint=True)
    y0 = gn.apply_rows(xg, mg, rg, wg, bg, silu)
    if y0 is not None:
        if dtype != torch.float16:
            assert torch.equal(y, y0)
        else:
            # A value stored alone has its last product rounded straight to
            # fp16 (one instruction), a value stored in a wide access to fp32
            # first; the two kernels differ in which values they store alone.
            # The second rounding can go the other way only from an fp16
            # midpoint, by one step.
            step = torch.finfo(dtype).eps * y0.float().abs() + ref.tiny(dtype) * 2
            assert bool(((y.float() - y0.float()).abs() <= step).all())
    mu = mean.double().repeat_interleave(C // G, 1).unsqueeze(1)
    rs = rstd.double().repeat_interleave(C // G, 1).unsqueeze(1)
    wd, bd = w.double(), b.double()
    t = (x.double() - mu) * rs * wd + bd
    # t: the bound of the backward pass's; the output 8 roundings and |t| more
    # of the exponential's argument
    e = ref.U * (3 * (x.double() * wd * rs).abs() + 4 * (mu * wd * rs).abs() + bd.abs() + t.abs())
    want = t * torch.sigmoid(t) if silu else t
    if silu:
        e = 1.1 * e + ref.U * (8 + 2 * t.abs()) * want.abs()
    ref.check(y, want, 1.01 * e + ref.rounded(want, dtype), "y")
    codes, E, val = ref.checkpoint(x)
    assert torch.equal(ck.codes.cpu().to(torch.int64), codes)
    assert torch.equal(ck.scales.cpu().to(torch.int64), E)
    check_backward(gn, dy, val, mean, rstd, w, b, silu, (shape, dtype, silu, "saved"), saved=ck)
    # in place
    x2 = xg.clone()
    y2, ck2 = gn.apply_rows(x2, mg, rg, wg, bg, silu, out=x2, checkpoint=True)
    assert torch.equal(x2, y) and torch.equal(ck2.codes, ck.codes)
    assert torch.equal(ck2.scales, ck.scales)


@pytest.mark.parametrize("which", ["none", "weight", "bias"])
def test_absent_parameters(gn, which):
    x, w, b, dy, mean, rstd = make(2, 50, 96, 8, torch.bfloat16, torch.bfloat16, 3)
    w = w if which == "weight" else None
    b = b if which == "bias" else None
    r = check_backward(gn, dy, x, mean, rstd, w, b, True, which)
    dyg, xg, mg, rg, wg, bg = cu(dy, x, mean, rstd, w, b)
    alone = gn.group_norm_silu_rows_backward(dyg, xg, mg, rg, wg, bg, weight_grad=False)
    assert alone[1] is None and alone[2] is None and torch.equal(alone[0], r[0])


@pytest.mark.parametrize("dtype", DTYPES)
def test_unaligned_rows_in_place_and_surroundings(gn, dtype):
    """x, dy and dx at odd element offsets of larger buffers; dx in dy's place
    and in x's; what lies before and behind stays as it was."""
    for N, L, C, G in ((2, 37, 96, 8), (1, 50, 321, 3), (2, 9, 1001, 7), (1, 9000, 96, 8),
                       (2, 700, 4100, 4)):
        x, w, b, dy, mean, rstd = make(N, L, C, G, dtype, torch.float32, C)
        wg, bg, mg, rg = cu(w, b, mean, rstd)
        want = gn.group_norm_silu_rows_backward(dy.cuda(), x.cuda(), mg, rg, wg, bg)
        n = N * L * C
        for off in (1, 3):
            bufs = [torch.full((n + 16,), 3.0, dtype=dtype, device="cuda") for _ in range(3)]
            views = [t[off:off + n].view(N, L, C) for t in bufs]
            for target in (2, 0, 1):
                views[0].copy_(x.cuda())
                views[1].copy_(dy.cuda())
                print("case gn offset %d target %d %s" % (off, target, (N, L, C, G)), flush=True)
                r = gn.group_norm_silu_rows_backward(views[1], views[0], mg, rg, wg, bg,
                                                     out=views[target])
                for p, q in zip(r, want):
                    assert torch.equal(p, q)
            for t in bufs:
                assert bool((t[:off] == 3).all()) and bool((t[off + n:] == 3).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_extremes(gn, dtype):
    """Gradients of SiLU far out on both sides stay finite and right; one
    sample's NaN stays in its groups."""
    N, L, C, G = 2, 64, 64, 8
    x, w, b, dy, mean, rstd = make(N, L, C, G, dtype, torch.float32, 5)
    w, b = 30 * w, 100 * torch.sign(b)
    check_backward(gn, dy, x, mean, rstd, w, b, True, "far out")
    x[1, 5, 17] = float("nan")
    dyg, xg, mg, rg, wg, bg = cu(dy, x, mean, rstd, w, b)
    dx, dw, db = gn.group_norm_silu_rows_backward(dyg, xg, mg, rg, wg, bg)
    nan = torch.isnan(dx)
    assert bool(nan[1, :, 16:24].all()) and int(nan.sum()) == L * 8
    assert int(torch.isnan(dw).sum()) == 1 and int(torch.isnan(db).sum()) == 1


@pytest.mark.parametrize("shape", [(2, 3000, 320, 32), (2, 256, 320, 32), (3, 1000, 64, 16),
                                   (1, 700, 128, 32)])
def test_same_bits_on_every_call_stream_and_replay(gn, shape):
    """In the passes and in the single launch, of several samples and one."""
    x, w, b, dy, mean, rstd = make(*shape, torch.bfloat16, torch.float32, 1)
    x, w, b, dy, mean, rstd = cu(x, w, b, dy, mean, rstd)

    def call():
        return gn.group_norm_silu_rows_backward(dy, x, mean, rstd, w, b)

    first = call()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call()
        graphs.append((g, out))
    for turn in range(3):
        for _, out in graphs:
            for t in out:
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        graphs[0][0].replay()
        with torch.cuda.stream(other):
            graphs[1][0].replay()
            there = call()
        again = call()
        torch.cuda.synchronize()
        for got in (again, there, graphs[0][1], graphs[1][1]):
            for p, q in zip(first, got):
                assert torch.equal(p, q)


def test_gradient_against_differences(gn):
    """dx, dw and db against central differences of the forward definition in
    64 bits along random directions."""
    N, L, C, G = 2, 11, 24, 3
    x, w, b, v, mean, rstd = make(N, L, C, G, torch.float32, torch.float32, 21)
    grads = [t.cpu().double() for t in
             gn.group_norm_silu_rows_backward(*cu(v, x, mean, rstd, w, b))]
    theta = [x.double(), w.double(), b.double()]

    def f(t):
        z = t[0].reshape(N, L, G, C // G)
        d = z - z.mean((1, 3), keepdim=True)
        h = (d / torch.sqrt((d * d).mean((1, 3), keepdim=True) + 1e-6)).reshape(N, L, C)
        u = h * t[1] + t[2]
        return (v.double() * u * torch.sigmoid(u)).sum()

    gen = torch.Generator().manual_seed(2)
    for i in range(3):
        for _ in range(4):
            u = torch.randn(theta[i].shape, generator=gen, dtype=torch.float64)
            up, dn = list(theta), list(theta)
            up[i], dn[i] = theta[i] + 1e-5 * u, theta[i] - 1e-5 * u
            num = float((f(up) - f(dn)) / 2e-5)
            ana = float((grads[i] * u).sum())
            scale = float((grads[i].abs() * u.abs()).sum()) + float(v.abs().sum())
            assert abs(num - ana) <= (200 * ref.U + 1e-7) * scale


@pytest.mark.parametrize("adt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", [(1, 40, 64, 8), (2, 3000, 40, 8), (1, 50, 321, 3)])
def test_16bit_parameters_at_an_odd_element_offset(gn, shape, adt):
    """Parameters at addresses 2 mod 4, in the single launch and in the passes:
    dx as with fp32 copies of the same values, bit for bit, dw and db their
    fp32 gradients rounded once."""
    N, L, C, G = shape
    x, w, b, dy, mean, rstd = cu(*make(N, L, C, G, torch.bfloat16, adt, C))
    wb, bb = [torch.empty(C + 1, dtype=adt, device="cuda") for _ in range(2)]
    wb[1:], bb[1:] = w, b
    assert wb[1:].data_ptr() % 4 == 2
    got = gn.group_norm_silu_rows_backward(dy, x, mean, rstd, wb[1:], bb[1:])
    want = gn.group_norm_silu_rows_backward(dy, x, mean, rstd, w.float(), b.float())
    assert torch.equal(got[0], want[0])
    assert torch.equal(got[1], want[1].to(adt)) and torch.equal(got[2], want[2].to(adt))
    y1 = gn.apply_rows(x, mean, rstd, wb[1:], bb[1:], checkpoint=True)[0]
    assert torch.equal(y1, gn.apply_rows(x, mean, rstd, w.float(), b.float(), checkpoint=True)[0])


def test_offsets_beyond_32_bits(gn):
    """More than 2^31 values and 2^32 bytes: x and dy are zero but for the last
    rows, whose gradients are those of these rows alone, the group's means
    taken over all of it."""
    C, G, n = 8, 2, 24
    L = (1 << 28) + 1000
    x = torch.zeros(1, L, C, dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros_like(x)
    gen = torch.Generator().manual_seed(4)
    xe = torch.randn(n, C, generator=gen).to(torch.bfloat16)
    de = torch.randn(n, C, generator=gen).to(torch.bfloat16)
    x[0, L - n:], dy[0, L - n:] = xe.cuda(), de.cuda()
    w, b = torch.rand(C, generator=gen) + 0.5, torch.randn(C, generator=gen)
    mean, rstd = torch.tensor([[0.25, -0.5]]), torch.tensor([[2.0, 0.5]])
    dx, dw, db = gn.group_norm_silu_rows_backward(dy, x, *cu(mean, rstd, w, b))
    mu = mean.double().repeat_interleave(4, 1)
    rs = rstd.double().repeat_interleave(4, 1)
    h = (xe.double() - mu) * rs
    t = h * w.double() + b.double()
    s = torch.sigmoid(t)
    dt = de.double() * s * (1 + t * (1 - s))
    a = (w * dt).sum(0).reshape(G, 4).sum(1).repeat_interleave(4) / (L * 4)
    bb = (w * dt * h).sum(0).reshape(G, 4).sum(1).repeat_interleave(4) / (L * 4)
    want = rs * (w * dt - a - h * bb)
    # a few dozen fp32 roundings of the terms, and bf16's
    bound = 64 * ref.U * rs * (w * dt.abs() + 1) + ref.rounded(want, torch.bfloat16)
    ref.check(dx[0, L - n:], want, bound, "dx at the end")
    ref.check(dw, (dt * h).sum(0), 64 * ref.U * (dt * h).abs().sum(0) + 1e-7, "dw")
    ref.check(db, dt.sum(0), 64 * ref.U * dt.abs().sum(0) + 1e-7, "db")
    # elsewhere dy is zero: dx = -rstd*(a + h0*b), below 1e-6 here, the same in
    # every row
    assert torch.equal(dx[0, 5], dx[0, L // 2]) and float(dx[0, 7].abs().max()) < 1e-6
    del dy, dx
    ck = gn.checkpoint_rows(x)
    back = gn.restore_rows(ck)
    assert torch.equal(back[0, L - n:].cpu(), ref.checkpoint(xe)[2].to(torch.bfloat16))
    assert int(torch.count_nonzero(back[0, :L - n])) == 0


def test_calls_from_two_threads(gn):
    """Two host threads on streams of their own, interleaved: the bits of the
    calls made alone."""
    import threading
    sets = [cu(*make(2, 700 + 300 * i, 96, 8, torch.bfloat16, torch.float32, i)) for i in range(2)]
    alone = [gn.group_norm_silu_rows_backward(s[3], s[0], s[4], s[5], s[1], s[2]) for s in sets]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        x, w, b, dy, mean, rstd = sets[i]
        with torch.no_grad(), torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(30):
                r = gn.group_norm_silu_rows_backward(dy, x, mean, rstd, w, b)
                if not all(torch.equal(p, q) for p, q in zip(r, alone[i])):
                    bad.append(i)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not bad


def test_no_rows(gn):
    w = torch.ones(32, device="cuda")
    for N, L in ((0, 5), (2, 0)):
        x = torch.empty((N, L, 32), dtype=torch.bfloat16, device="cuda")
        st = torch.zeros((N, 4), device="cuda")
        dx, dw, db = gn.group_norm_silu_rows_backward(x, x, st, st, w, w)
        assert dx.shape == x.shape and bool((dw == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_apply_that_saves_no_rows(gn, dtype):
    """An empty batch goes through the saving apply step, and its checkpoint
    through the backward pass."""
    w = torch.ones(40, device="cuda")
    for N, L in ((0, 5), (2, 0), (0, 0)):
        x = torch.empty((N, L, 40), dtype=dtype, device="cuda")
        st = torch.zeros((N, 4), device="cuda")
        for out in (None, x):
            y, ck = gn.apply_rows(x, st, st, w, w, out=out, checkpoint=True)
            assert y.shape == x.shape and y.dtype == dtype and (out is None or y is out)
            assert ck.shape == x.shape and tuple(ck.scales.shape) == (N, L, 2)
            assert ck.dtype == dtype and gn.restore_rows(ck).shape == x.shape
        dx, dw, db = gn.group_norm_silu_rows_backward(x, ck, st, st, w, w)
        assert dx.shape == x.shape and bool((dw == 0).all()) and bool((db == 0).all())
        with pytest.raises(ValueError):     # the checks come first
            gn.apply_rows(x, st[:, :3], st, w, w, checkpoint=True)


class _GroupNormSilu(torch.autograd.Function):
    """How a training program uses the calls: statistics, the apply step that
    keeps x in 8 bits (or x itself), the backward pass."""

    @staticmethod
    def forward(ctx, gn, x, w, b, G, save):
        mean, rstd = gn.group_stats_rows(x, G)
        if save:
            y, kept = gn.apply_rows(x, mean, rstd, w, b, True, checkpoint=True)
        else:
            y, kept = gn.apply_rows(x, mean, rstd, w, b, True), x
        ctx.gn, ctx.kept = gn, kept
        ctx.save_for_backward(mean, rstd, w, b)
        return y

    @staticmethod
    def backward(ctx, dy):
        mean, rstd, w, b = ctx.saved_tensors
        dx, dw, db = ctx.gn.group_norm_silu_rows_backward(dy.contiguous(), ctx.kept, mean, rstd,
                                                          w, b)
        return None, dx, dw, db, None, None


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gn, x, w, b, save):
        r = gn.layer_norm_rows(x, w, b, 1e-6, stats=True, checkpoint=save)
        ctx.gn, ctx.kept = gn, r[3] if save else x
        ctx.save_for_backward(r[1], r[2], w)
        return r[0]

    @staticmethod
    def backward(ctx, dy):
        mean, rstd, w = ctx.saved_tensors
        dx, dw, db = ctx.gn.layer_norm_rows_backward(dy.contiguous(), ctx.kept, mean, rstd, w)
        return None, dx, dw, db, None


@pytest.mark.parametrize("save", [False, True])
def test_block_trained_through_both_norms(gn, save):
    """x + layer_norm(group_norm_silu(x)) in fp32 under autograd, against the
    same block differentiated in 64 bits -- with the saved inputs' values in
    the backward pass where they are kept in 8 bits.

    Bounds: without the checkpoint every gradient is a composition of the two
    operators; each one's error is a few dozen roundings of its terms' size
    (the tests above), so 1e-4 of the gradient's largest magnitude leaves two
    orders.  With it, each input is off by at most half a step of its block,
    2^-7 of the block's largest magnitude, which moves the gradients by about
    as much relative to their size (the normalised values times the second
    derivative, both of order one): 2^-7 * 8 of the largest magnitude."""
    N, L, C, G = 2, 48, 96, 8
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(N, L, C, generator=gen)
    ps = [1 + 0.2 * torch.randn(C, generator=gen), 0.2 * torch.randn(C, generator=gen),
          1 + 0.2 * torch.randn(C, generator=gen), 0.2 * torch.randn(C, generator=gen)]
    v = torch.randn(N, L, C, generator=gen)
    leaves = [t.cuda().requires_grad_() for t in [x] + ps]
    with torch.enable_grad():
        h = _GroupNormSilu.apply(gn, leaves[0], leaves[1], leaves[2], G, save)
        y = leaves[0] + _LayerNorm.apply(gn, h, leaves[3], leaves[4], save)
        (y * v.cuda()).sum().backward()
    exact = [t.double().requires_grad_() for t in [x] + ps]
    with torch.enable_grad():
        xg = exact[0].reshape(N, L, G, C // G)
        d = xg - xg.mean((1, 3), keepdim=True)
        t = (d / torch.sqrt((d * d).mean((1, 3), keepdim=True) + 1e-6)).reshape(N, L, C)
        t = t * exact[1] + exact[2]
        t = t * torch.sigmoid(t)
        d = t - t.mean(-1, keepdim=True)
        t = d / torch.sqrt((d * d).mean(-1, keepdim=True) + 1e-6) * exact[3] + exact[4]
        ((exact[0] + t) * v.double()).sum().backward()
    tol = 2.0 ** -4 if save else 1e-4
    for got, want in zip(leaves, exact):
        g = got.grad.cpu().double()
        assert float((g - want.grad).abs().max()) <= tol * float(want.grad.abs().max())
