"""The product of rows in 8 bits against the definition in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

import rows8_reference as ref  # noqa: E402
import rows_reference as rows  # noqa: E402

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


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


def make(gn, M, N, K, dtype, seed, pad=0):
    """Rows (K + pad apart) and weights in 8 bits on the GPU, any int8 value."""
    gen = torch.Generator().manual_seed(seed)
    a = torch.randint(-128, 128, (M, K + pad), generator=gen, dtype=torch.int8).cuda()[:, :K]
    b = torch.randint(-128, 128, (N, K), generator=gen, dtype=torch.int8).cuda()
    sa = (0.01 * (0.5 + torch.rand(M, generator=gen))).cuda()
    sb = (0.01 * (0.5 + torch.rand(N, generator=gen))).cuda()
    return gn.Rows8(a, sa, dtype), gn.Rows8(b, sb, dtype)


def extras(M, N, dtype, adt, seed):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(N, generator=gen).to(adt).cuda(),
            torch.randn(M, N, generator=gen).to(dtype).cuda())


def check(z, x, w, bias, res, dtype, what):
    want, e = ref.matmul(x.codes, x.scales, w.codes, w.scales, bias, res, dtype)
    assert z.dtype == dtype
    rows.check(z, want, e, str(what))


SIZES = [(1, 1, 1), (1, 16, 64), (1, 4096, 64), (1, 1000, 4096), (2, 33, 17), (7, 100, 129),
         (15, 257, 500), (16, 128, 1024), (17, 128, 128), (31, 65, 127), (33, 640, 2560),
         (48, 1024, 513), (63, 96, 65), (64, 256, 256), (65, 255, 300), (100, 1000, 1000),
         (127, 129, 640), (128, 128, 128), (129, 384, 191), (200, 2051, 333), (255, 257, 1025),
         (256, 256, 512), (257, 513, 129), (300, 4100, 96), (511, 700, 2003), (1001, 1537, 203),
         (1024, 1024, 1024), (2049, 520, 260), (4097, 256, 64), (1, 17, 16384), (5, 30000, 70),
         (3000, 17, 1), (700, 1, 40)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_sizes(gn, M, N, K, dtype):
    """Dense rows (off 16-byte boundaries where K is) and rows on them, with and
    without bias and residual."""
    adt = {torch.bfloat16: torch.float32, torch.float16: torch.float16,
           torch.float32: torch.bfloat16}[dtype]
    bias, res = extras(M, N, dtype, adt, M + N)
    for pad, with_b, with_r in ((0, True, True), (-K % 16, False, True), (-K % 16 + 16, True, False)):
        what = (M, N, K, dtype, pad)
        print("case int8_matmul %s" % (what,), flush=True)
        x, w = make(gn, M, N, K, dtype, M + 3 * N + K, pad)
        z = gn.int8_matmul(x, gn.pack_int8_weight(w), bias if with_b else None,
                           residual=res if with_r else None)
        check(z, x, w, bias if with_b else None, res if with_r else None, dtype, what)


# (rows, channels) of a tile, kernel; sizes that take it, ragged in both, at one and
# more steps of 128 input channels
KINDS = [
    (16, 16, 0, [(148, 1, 65), (5, 100, 1500)]), (16, 32, 0, [(3, 4499, 65), (2, 7001, 1300)]),
    (16, 64, 0, [(13, 10283, 67)]), (32, 16, 0, [(2124, 33, 72)]),
    (32, 32, 0, [(20, 4161, 69), (27, 4161, 1200)]), (32, 64, 0, [(56, 4124, 66), (59, 4133, 1100)]),
    (48, 32, 0, [(33, 5529, 71)]), (48, 64, 0, [(66, 5719, 67), (90, 5719, 513)]),
    (64, 32, 0, [(2800, 135, 71)]), (64, 64, 0, [(99, 6028, 65), (250, 4090, 600)]),
    (64, 128, 1, [(4378, 5520, 115), (1698, 7005, 228), (1163, 6533, 380), (718, 6808, 504),
                  (706, 6901, 550), (643, 5387, 736), (513, 6796, 867), (522, 6709, 922)]),
    (128, 128, 1, [(4482, 4174, 128), (1928, 5286, 230), (4672, 1548, 347), (4637, 1569, 403),
                   (4130, 713, 618), (4898, 589, 741), (390, 7010, 773), (387, 7026, 969)]),
    (128, 256, 1, [(3867, 3995, 123), (1090, 6390, 256), (842, 7012, 319), (4948, 1164, 454),
                   (4907, 1189, 613), (4882, 1168, 715), (4471, 1315, 845), (4875, 1186, 979)]),
]


@pytest.mark.parametrize("bm,bn,kernel,size,i", [(m, n, k, s, i) for m, n, k, sizes in KINDS
                                                 for i, s in enumerate(sizes)])
def test_every_tile(gn, bm, bn, kernel, size, i):
    M, N, K = size
    plan = gn.int8_matmul_plan(M, N, K)
    assert (plan["rows"], plan["channels"], plan["tiles_kernel"]) == (bm, bn, kernel)
    dtype = DTYPES[(i + bm // 16) % 3]
    print("case int8_matmul tile %s %s" % (size, dtype), flush=True)
    x, w = make(gn, M, N, K, dtype, M + K, (0, -K % 16, 3)[i % 3])
    bias, res = extras(M, N, dtype, (torch.float32, dtype)[i % 2], N)
    res = None if i % 4 == 3 else res
    z = gn.int8_matmul(x, gn.pack_int8_weight(w), bias, residual=res)
    check(z, x, w, bias, res, dtype, size)


@pytest.mark.parametrize("M", [1, 3, 16, 17, 40, 64, 65, 128, 200, 300])
def test_bits_do_not_depend_on_the_rows_beside(gn, M):
    """A row's result is the same in any batch: its sums are exact."""
    x, w = make(gn, 300, 500, 700, torch.bfloat16, 1)
    p = gn.pack_int8_weight(w)
    bias, res = extras(300, 500, torch.bfloat16, torch.bfloat16, 2)
    full = gn.int8_matmul(x, p, bias, residual=res)
    part = gn.int8_matmul(gn.Rows8(x.codes[:M], x.scales[:M], x.dtype), p, bias, residual=res[:M])
    assert torch.equal(part, full[:M])


def test_shapes_strides_and_what_lies_between_rows(gn):
    x, w = make(gn, 60, 130, 200, torch.float16, 4)
    p = gn.pack_int8_weight(w)
    assert p.shape == (130, 200)
    x3 = gn.Rows8(x.codes.reshape(3, 20, 200), x.scales.reshape(3, 20), torch.float16)
    bias, res = extras(60, 130, torch.float16, torch.float16, 5)
    want = gn.int8_matmul(x, p, bias, residual=res)
    z = gn.int8_matmul(x3, p, bias, residual=res.reshape(3, 20, 130))
    assert z.shape == (3, 20, 130) and torch.equal(z.reshape(60, 130), want)
    wide = torch.full((60, 141), 9.0, dtype=torch.float16, device="cuda")
    rwide = torch.full((60, 135), 9.0, dtype=torch.float16, device="cuda")
    rwide[:, 1:131] = res
    got = gn.int8_matmul(x, p, bias, residual=rwide[:, 1:131], out=wide[:, 3:133])
    assert torch.equal(got, want)
    assert bool((wide[:, :3] == 9).all()) and bool((wide[:, 133:] == 9).all())
    # the residual joined in place, and one residual row for all
    r = res.clone()
    assert gn.int8_matmul(x, p, bias, residual=r, out=r) is r and torch.equal(r, want)
    one = res[:1].expand(60, 130)
    assert torch.equal(gn.int8_matmul(x, p, residual=one),
                       gn.int8_matmul(x, p, residual=one.contiguous()))
    # one row for all rows of x; an unaligned start; a weight packed in the call
    e = gn.Rows8(x.codes[:1].expand(60, 200), x.scales, torch.float16)
    check(gn.int8_matmul(e, p), e, w, None, None, torch.float16, "expanded")
    u = gn.Rows8(x.codes[:, 5:], x.scales, torch.float16)
    wu = gn.Rows8(w.codes[:, 5:], w.scales, torch.float16)
    check(gn.int8_matmul(u, wu), u, wu, None, None, torch.float16, "unaligned")
    for dt in DTYPES:
        check(gn.int8_matmul(x, p, dtype=dt), x, w, None, None, dt, dt)


@pytest.mark.parametrize("M", [1, 20, 300])
def test_largest_sums(gn, M):
    """Every product at its largest magnitude, K at its limit: 2^30."""
    K, N = gn.INT8_MAX_K, 48
    a = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    b = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    b[1::2] = 127
    x = gn.Rows8(a, torch.full((M,), 2.0 ** -10, device="cuda"), torch.float32)
    w = gn.Rows8(b, torch.full((N,), 2.0 ** -10, device="cuda"), torch.float32)
    z = gn.int8_matmul(x, gn.pack_int8_weight(w))
    want = torch.tensor([2.0 ** 10, -127.0 * 8], device="cuda").repeat(N // 2).expand(M, N)
    assert torch.equal(z, want)


@pytest.mark.parametrize("M", [3, 40, 300])
def test_nan_scales_stay_in_their_row_or_channel(gn, M):
    x, w = make(gn, M, 70, 100, torch.bfloat16, 8)
    x.scales[1] = float("nan")
    w.scales[5] = float("inf")
    z = gn.int8_matmul(x, gn.pack_int8_weight(w))
    assert bool(torch.isnan(z[1]).all())
    keep = [i for i in range(70) if i != 5]
    assert not torch.isfinite(z[:, 5]).any()
    assert bool(torch.isfinite(z[[i for i in range(M) if i != 1]][:, keep]).all())


def test_declined_and_refused_on_the_gpu(gn):
    x, w = make(gn, 4, 32, 64, torch.bfloat16, 8)
    p = gn.pack_int8_weight(w)
    res = torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda")
    assert gn.int8_matmul(x, p, residual=res.half()) is None
    assert gn.int8_matmul(x, p, torch.zeros(32)) is None            # bias on the CPU
    with torch.enable_grad():
        assert gn.int8_matmul(x, p) is None
    for call in (lambda: gn.int8_matmul(x, p, torch.zeros(31, device="cuda")),
                 lambda: gn.int8_matmul(x, p, residual=res[:3]),
                 lambda: gn.int8_matmul(x, p, out=res[:3]),
                 lambda: gn.int8_matmul(x, p, out=res.half())):
        with pytest.raises(ValueError):
            call()
    e = gn.Rows8(torch.empty(0, 64, dtype=torch.int8, device="cuda"),
                 torch.empty(0, device="cuda"), torch.bfloat16)
    assert gn.int8_matmul(e, p).shape == (0, 32)


def layer(gn, x, res, w, p1, b1, p2):
    """Norm, product, norm of the sum with the stream, product back onto it."""
    q, h = gn.rms_norm_rows(x, w, 1e-6, residual=res, quantize=True)
    z = gn.int8_matmul(q, p1, b1)
    q2 = gn.quantize_rows(z)
    return h, z, gn.int8_matmul(q2, p2, residual=h)


def check_layer(gn, M, C, F, dtype):
    gen = torch.Generator().manual_seed(M + C)
    x, res = [torch.randn(M, C, generator=gen).to(dtype).cuda() for _ in range(2)]
    w = (1 + 0.2 * torch.randn(C, generator=gen)).to(dtype).cuda()
    w1, w2 = [gn.quantize_rows((torch.randn(n, k, generator=gen) * k ** -0.5).to(dtype).cuda())
              for n, k in ((F, C), (C, F))]
    b1 = torch.randn(F, generator=gen).to(dtype).cuda()
    p1, p2 = gn.pack_int8_weight(w1), gn.pack_int8_weight(w2)
    h, z, out = layer(gn, x, res, w, p1, b1, p2)
    wh, _, _, wq, ws, _, _, es = ref.rms_norm(x, w.cpu(), 1e-6, dtype, res)
    assert torch.equal(h.cpu(), wh)
    wz, ez = ref.matmul(wq, ws, w1.codes, w1.scales, b1, None, dtype)
    # the row scales' own bound, relative, on top of the product's
    rows.check(z, wz, ez + wz.abs() * 2 * (es / ws).unsqueeze(-1) + (es / ws).unsqueeze(-1)
               * b1.cpu().double().abs() * 2, "z")
    q2, s2, _ = ref.quantize(z)
    wo, eo = ref.matmul(q2, s2, w2.codes, w2.scales, None, h, dtype)
    rows.check(out, wo, eo + rows.U * (wo.abs() + h.cpu().double().abs()), "out")
    return x, res, w, p1, b1, p2


@pytest.mark.parametrize("M,C,F,dtype", [(1, 256, 1024, torch.bfloat16), (5, 333, 777, torch.float16),
                                         (150, 512, 1280, torch.bfloat16),
                                         (700, 129, 400, torch.float32)])
def test_norm_product_norm_product(gn, M, C, F, dtype):
    check_layer(gn, M, C, F, dtype)


def test_layer_captured_and_replayed(gn):
    args = check_layer(gn, 33, 333, 777, torch.bfloat16)
    x = args[0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = layer(gn, *args)
    for k in range(4):
        x.normal_(generator=torch.Generator(device="cuda").manual_seed(k))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, layer(gn, *args)):
            assert torch.equal(a, b)


def test_offsets_beyond_32_bits(gn):
    """z of more than 2^32 bytes and rows of x more than 2^32 bytes apart."""
    K, N = 64, 64
    x, w = make(gn, 3, N, K, torch.float32, 2)
    p = gn.pack_int8_weight(w)
    buf = torch.zeros(2 * (1 << 32) + 64, dtype=torch.int8, device="cuda")
    far = buf.as_strided((3, K), (1 << 32, 1))
    far.copy_(x.codes)
    assert torch.equal(gn.int8_matmul(gn.Rows8(far, x.scales, torch.float32), p),
                       gn.int8_matmul(x, p))
    del far, buf
    zs = (1 << 30) + 4
    zbuf = torch.empty(2 * zs + N, device="cuda")
    z = zbuf.as_strided((3, N), (zs, 1))
    assert torch.equal(gn.int8_matmul(x, p, out=z), gn.int8_matmul(x, p))


def test_one_row_without_a_batch(gn):
    x, w = make(gn, 5, 40, 70, torch.bfloat16, 3)
    p = gn.pack_int8_weight(w)
    one = gn.Rows8(x.codes[2].contiguous(), x.scales[2].clone(), torch.bfloat16)
    assert one.shape == (70,) and one.scales.shape == ()
    z = gn.int8_matmul(one, p)
    assert z.shape == (40,) and torch.equal(z, gn.int8_matmul(x, p)[2])
    v = torch.randn(70, device="cuda").bfloat16()
    q, h = gn.rms_norm_rows(v, residual=v, quantize=True)
    assert q.shape == (70,) and h.shape == (70,) and q.scales.shape == ()
    q2 = gn.rms_norm_rows(v[None], residual=v[None], quantize=True)[0]
    assert torch.equal(q.codes, q2.codes[0]) and torch.equal(gn.quantize_rows(v).codes,
                                                             gn.quantize_rows(v[None]).codes[0])
    assert gn.dequantize_rows(q).shape == (70,)


def test_streams_and_threads_at_once(gn):
    """Calls of every kernel at once share nothing."""
    import threading
    cases = []
    for M, N, K in ((1, 500, 700), (40, 5529, 300), (600, 700, 900), (1163, 6533, 380)):
        x, w = make(gn, M, N, K, torch.bfloat16, M)
        cases.append((x, gn.pack_int8_weight(w)))
    want = [gn.int8_matmul(x, p) for x, p in cases]
    torch.cuda.synchronize()
    got, errors = {}, []

    def work(t):
        try:
            with torch.no_grad(), torch.cuda.stream(torch.cuda.Stream()):
                r = [[gn.int8_matmul(x, p) for x, p in cases] for _ in range(5)]
                torch.cuda.current_stream().synchronize()
                got[t] = r
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(t,)) for t in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and len(got) == 3
    for r in got.values():
        for zs in r:
            for z, z0 in zip(zs, want):
                assert torch.equal(z, z0)


def test_two_captured_graphs_replayed_beside_eager_work(gn):
    x, w = make(gn, 700, 900, 500, torch.float16, 4)
    y, _ = make(gn, 9, 900, 500, torch.float16, 5)
    p = gn.pack_int8_weight(w)
    gn.int8_matmul(x, p), gn.int8_matmul(y, p)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for r in (x, y):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(gn.int8_matmul(r, p))
        graphs.append(g)
    for k in range(4):
        for r in (x, y):
            r.codes.random_(-128, 128, generator=torch.Generator(device="cuda").manual_seed(k))
        graphs[k % 2].replay()
        eager = [gn.int8_matmul(r, p) for r in (x, y)]
        graphs[1 - k % 2].replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, eager):
            assert torch.equal(a, b)
