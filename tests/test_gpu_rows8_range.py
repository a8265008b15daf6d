"""Rows in 8 bits, the root-mean-square norm and the product of 8-bit rows near the
ends of the ranges that their definitions promise."""
import pytest

torch = pytest.importorskip("torch")

import rows8_reference as ref  # noqa: E402
import rows_reference as rows  # noqa: E402

pytestmark = pytest.mark.gpu

WIDE = [torch.bfloat16, torch.float32]      # the types with fp32's exponents


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


def check_codes(q, codes, scales, es, what):
    assert torch.equal(q.codes.cpu().to(torch.int64), codes), "%s codes" % (what,)
    rows.check(q.scales, scales, es, "%s scales" % (what,))


def border_rows(C, dtype):
    """Values on the borders between two codes and one step of the type beside
    them, in both signs, their largest magnitude 127 * 2^k for every k that the
    type holds, and rows up to the type's largest number."""
    k = torch.arange(C) % 127
    t = (k + 0.5) * torch.where(torch.arange(C) % 2 == 0, 1.0, -1.0)
    t[0] = 127.0
    out = []
    for e in (-100, -101, -106, -107, -108, 93, 94, 95, 100, 118, 119, 120, 121):
        out.append((t.double() * 2.0 ** e).to(dtype))
        near = out[-1].float() * (1 + torch.finfo(dtype).eps * (torch.arange(C) % 3 - 1))
        near[0] = out[-1][0].float()
        out.append(near.to(dtype))
    top = torch.finfo(dtype).max
    g = torch.Generator().manual_seed(C)
    for largest in (top, top * 0.75, 2.0 ** 126, 2.0 ** 126 * (1 + 2.0 ** -7), 2.0 ** 127):
        r = (torch.rand(C, generator=g) * 2 - 1).double() * largest
        r[C // 2] = -largest
        out.append(r.to(dtype))
    return torch.stack(out)


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("C", [1, 3, 8, 127, 1280, 4097, 16384])
def test_codes_over_the_types_range(gn, C, dtype):
    x = border_rows(C, dtype)
    q = gn.quantize_rows(x.cuda())
    check_codes(q, *ref.quantize(x), "quantize %d %s" % (C, dtype))


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("C", [8, 127, 1280, 4097])
def test_norm_codes_of_large_products(gn, C, dtype):
    """Rows within the norm's range whose products with the weight go up to fp32's
    largest numbers."""
    t = border_rows(C, torch.float32)[-5:]
    w = torch.full((C,), 2.0 ** 100)
    w[1::3] = 2.0 ** 99
    # at most 2^128 / 2^100, and (h * w) finite
    h = (t.double() * 2.0 ** -100).to(dtype)
    h = torch.where((h.double() * w.double()).abs() < torch.finfo(torch.float32).max, h, h * 0.5)
    q = gn.rms_norm_rows(h.cuda(), w.cuda(), 1e-6, quantize=True)
    _, _, _, wq, ws, _, _, es = ref.rms_norm(h, w, 1e-6, dtype)
    check_codes(q, wq, ws, es, "rms_norm %d %s" % (C, dtype))


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("C", [1, 2, 8, 100, 341, 1024, 4096, 5000, 16384])
def test_norm_at_the_ends_of_its_range(gn, C, dtype):
    """Magnitudes just below 1e18, and just above 1e-18 without an eps: every
    output of both passes."""
    g = torch.Generator().manual_seed(C)
    for M in (7, 1100):     # backward from columns read again, and from partial rows
        sign = torch.where(torch.rand(M, C, generator=g) < 0.5, -1.0, 1.0)
        size = 0.1 + 0.9 * torch.rand(M, C, generator=g)
        size[0] = size[-1] = 1.0
        w = 1 + 0.3 * torch.randn(C, generator=g)
        dy = torch.randn(M, C, generator=g).to(dtype)
        for x, eps in ((sign * size * 9.9e17, 1e-6), (sign * (1.02e-18 / size), 0.0)):
            x = x.to(dtype)
            xg, wg = x.cuda(), w.cuda()
            what = "(%d, %d) %s eps %g" % (M, C, dtype, eps)
            _, wy, wr, wq, ws, ey, er, es = ref.rms_norm(x, w, eps, dtype)
            y, rstd = gn.rms_norm_rows(xg, wg, eps, stats=True)
            rows.check(rstd, wr, er, what + " rstd")
            rows.check(y, wy, ey, what + " y")
            check_codes(gn.rms_norm_rows(xg, wg, eps, quantize=True), wq, ws, es, what)
            dx, dw = gn.rms_norm_rows_backward(dy.cuda(), xg, rstd, wg)
            wx, ww, ex, ew = ref.rms_norm_backward(dy, x, rstd, w, None, dtype, torch.float32,
                                                   M + 16)
            rows.check(dx, wx, ex, what + " dx")
            rows.check(dw, ww, ew, what + " dw")


@pytest.mark.parametrize("dtype", WIDE)
def test_norm_scales_of_small_products(gn, dtype):
    """A row's scale is that of its norm however small its products with the
    weight are: their largest over 127 may be a subnormal number."""
    C = 1000
    g = torch.Generator().manual_seed(5)
    h = (torch.randn(40, C, generator=g) * 1e-16).to(dtype)
    w = torch.full((C,), 4e-23)
    q = gn.rms_norm_rows(h.cuda(), w.cuda(), 0.0, quantize=True)
    _, _, _, wq, ws, _, _, es = ref.rms_norm(h, w, 0.0, dtype)
    check_codes(q, wq, ws, es, "small products %s" % dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("M,N,K,tiles", [(3, 70, 100, 0), (27, 4161, 1200, 0), (643, 5387, 736, 1),
                                         (390, 7010, 773, 1), (842, 7012, 319, 1)])
def test_product_of_rows_with_large_scales(gn, M, N, K, tiles, dtype):
    """Rows whose sum times their own scale leaves fp32's range, which the
    channel's scale brings back, beside ordinary rows."""
    assert gn.int8_matmul_plan(M, N, K)["tiles_kernel"] == tiles
    gen = torch.Generator().manual_seed(M)
    a = torch.randint(-127, 128, (M, K), generator=gen, dtype=torch.int8)
    a[1] = 0
    b = torch.randint(-127, 128, (N, K), generator=gen, dtype=torch.int8)
    sa = torch.tensor([2.6e36, 1e36, 1e33, 1.6e29, 1e29, 1e32])[torch.arange(M) % 6]
    sb = (0.5 + torch.rand(N, generator=gen)) * (1e-38 if dtype == torch.float16 else 1e-33)
    bias = torch.randn(N, generator=gen).to(dtype)
    res = torch.randn(M, N, generator=gen).to(dtype)
    x = gn.Rows8(a.cuda(), sa.cuda(), dtype)
    p = gn.pack_int8_weight(gn.Rows8(b.cuda(), sb.cuda(), dtype))
    for bi, r in ((None, None), (bias, res)):
        z = gn.int8_matmul(x, p, None if bi is None else bi.cuda(),
                           residual=None if r is None else r.cuda())
        want, e = ref.matmul(a, sa, b, sb, bi, r, dtype)
        # a product below fp32's normal numbers is rounded to them first
        rows.check(z, want, e + 2.0 ** -149, "%s %s" % ((M, N, K), dtype))


@pytest.mark.parametrize("M", [1, 300])
@pytest.mark.parametrize("sa,sb", [(2.0 ** 97 * (1 - 2.0 ** -24), 2.0 ** -100), (2.0 ** 97, 2.0 ** -100),
                                   (2.0 ** 121, 2.0 ** -140)])
def test_largest_sums_with_large_scales(gn, M, sa, sb):
    K, N = gn.INT8_MAX_K, 48
    a = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    x = gn.Rows8(a, torch.full((M,), sa, device="cuda"), torch.float32)
    w = gn.Rows8(a[:1].expand(N, K).contiguous(), torch.full((N,), sb, device="cuda"),
                 torch.float32)
    z = gn.int8_matmul(x, gn.pack_int8_weight(w))
    assert torch.equal(z.cpu().double(), torch.full((M, N), 2.0 ** 30 * sa * sb, dtype=torch.float64))
