"""The GroupNorm(+SiLU) backward passes, the saving apply step and the 8-bit
checkpoints where a workgroup takes several batches of rows (a round of the
grid, 2048 workgroups of 256 lanes, holds 2 pieces a lane of 16 bytes, 4 in the
second pass from x itself), the last one partial; the single launch at its
widest and largest strips; a block trained from saved inputs.  Against 64 bits."""
import pytest

torch = pytest.importorskip("torch")

import rows_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


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


def make(N, L, C, G, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(N, L, C, generator=gen) * torch.exp(0.3 * torch.randn(C, generator=gen))
         + 0.5 * torch.randn(C, generator=gen)).to(dtype)
    w = 1 + 0.3 * torch.randn(C, generator=gen)
    b = 0.3 * torch.randn(C, generator=gen)
    dy = torch.randn(N, L, C, generator=gen).to(dtype)
    xg = x.double().reshape(N, L, G, C // G)
    mean = xg.mean((1, 3))
    var = ((xg - mean[:, None, :, None]) ** 2).mean((1, 3))
    return x, w, b, dy, mean.float(), (1.0 / torch.sqrt(var + 1e-6)).float()


def check_backward(gn, dy, x, given, mean, rstd, w, b, silu, what):
    got = gn.group_norm_silu_rows_backward(dy.cuda(), given, mean.cuda(), rstd.cuda(), w.cuda(),
                                           b.cuda(), silu)
    # a channel's sum: at most 1024 rows of a lane in sequence, 10 tree steps
    want = ref.group_norm_backward(dy, x, mean, rstd, w, b, silu, dy.dtype, FP32,
                                   min(dy.shape[1], 1024) + 10)
    for g, v, bound, name in zip(got, want[:3], want[3:], ("dx", "dw", "db")):
        ref.check(g, v, bound, "%s %s" % (what, name))


@pytest.mark.parametrize("shape,dtype", [
    ((1, 35011, 512, 32), BF16), ((3, 18001, 333, 3), BF16), ((1, 20011, 1001, 7), FP16),
    ((1, 17011, 512, 32), FP32), ((2, 14011, 333, 3), FP32), ((3, 300001, 5, 5), FP16)])
def test_backward(gn, shape, dtype):
    print("case gn batches %s %s" % (shape, dtype), flush=True)
    x, w, b, dy, mean, rstd = make(*shape, dtype, shape[1])
    check_backward(gn, dy, x, x.cuda(), mean, rstd, w, b, True, (shape, dtype))


# the first one's x is beyond 16 MiB: the first pass's wider workgroups
@pytest.mark.parametrize("shape,dtype,silu", [
    ((1, 19001, 512, 32), BF16, True), ((2, 15013, 333, 3), BF16, False),
    ((1, 9501, 1001, 7), FP16, True), ((1, 9001, 512, 32), FP32, True),
    ((2, 7011, 333, 3), FP32, True), ((3, 300001, 5, 1), BF16, True)])
def test_apply_that_saves_and_backward_from_it(gn, shape, dtype, silu):
    print("case gn batches saved %s %s silu=%s" % (shape, dtype, silu), flush=True)
    N, L, C, G = shape
    x, w, b, dy, mean, rstd = make(*shape, dtype, L)
    y, ck = gn.apply_rows(x.cuda(), mean.cuda(), rstd.cuda(), w.cuda(), b.cuda(), silu,
                          checkpoint=True)
    codes, E, val = ref.checkpoint(x)
    assert torch.equal(ck.codes.cpu().to(torch.int64), codes)
    assert torch.equal(ck.scales.cpu().to(torch.int64), E)
    mu = mean.double().repeat_interleave(C // G, 1).unsqueeze(1)
    rs = rstd.double().repeat_interleave(C // G, 1).unsqueeze(1)
    wd, bd = w.double(), b.double()
    t = (x.double() - mu) * rs * wd + bd
    # t: one fma on scale = w*rs and shift = b - mu*scale; the output 8
    # roundings and |t| more of the exponential's argument
    e = ref.U * (3 * (x.double() * wd * rs).abs() + 4 * (mu * wd * rs).abs() + bd.abs() + t.abs())
    want = t * torch.sigmoid(t) if silu else t
    if silu:
        e = 1.1 * e + ref.U * (8 + 2 * t.abs()) * want.abs()
    ref.check(y, want, 1.01 * e + ref.rounded(want, dtype), "y")
    back = gn.restore_rows(ck)
    assert torch.equal(back.cpu(), val.to(dtype))
    check_backward(gn, dy, val, ck, mean, rstd, w, b, silu, (shape, dtype, silu, "saved"))


@pytest.mark.parametrize("M,C,dtype", [(20011, 1001, FP16), (40003, 256, BF16),
                                       (20003, 256, FP32), (9003, 505, FP32), (200003, 7, BF16)])
def test_rows_saved_and_restored(gn, M, C, dtype):
    print("case checkpoint batches M=%d C=%d %s" % (M, C, dtype), flush=True)
    gen = torch.Generator().manual_seed(M)
    x = (torch.randn(M, C, generator=gen)
         * torch.exp(2.0 * torch.randn(M, 1, generator=gen))).to(dtype)
    ck = gn.checkpoint_rows(x.cuda())
    codes, E, val = ref.checkpoint(x)
    assert torch.equal(ck.codes.cpu().to(torch.int64), codes)
    assert torch.equal(ck.scales.cpu().to(torch.int64), E)
    assert torch.equal(gn.restore_rows(ck).cpu(), val.to(dtype))


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("shape,dtype", [
    ((2, 9, 24, 3), BF16), ((17, 3, 24, 3), FP32), ((128, 5, 64, 1), BF16), ((129, 5, 64, 1), FP16),
    ((255, 2, 32, 1), FP32), ((257, 3, 40, 8), BF16), ((1025, 9, 33, 3), FP32),
    ((3000, 16, 64, 8), BF16), ((1100, 3, 7, 7), FP16), ((600, 2, 200, 2), BF16),
    # a wave's tile of a few partials: groups of 1 to 64 channels, and beyond
    ((30, 3, 96, 96), BF16), ((200, 3, 2048, 1), BF16), ((64, 1, 2048, 32), FP16),
    ((70, 4, 640, 32), BF16), ((40, 5, 1000, 25), FP32), ((30, 70, 330, 10), BF16),
    ((60, 2, 4092, 66), FP32), ((50, 700, 252, 4), BF16), ((9, 999, 1001, 7), FP16)])
def test_weight_gradients_of_many_samples(gn, shape, dtype, saved):
    """Samples on both sides of a round of the sum over samples (128), in the
    single launch (up to 256) and behind the passes."""
    print("case gn samples %s %s saved=%s" % (shape, dtype, saved), flush=True)
    N, L, C, G = shape
    x, w, b, dy, mean, rstd = make(*shape, dtype, N)
    given = gn.checkpoint_rows(x.cuda()) if saved else x.cuda()
    if saved:
        x = ref.checkpoint(x)[2]
    check_backward(gn, dy, x, given, mean, rstd, w, b, True, (shape, dtype, saved))


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("shape,dtype", [
    ((1, 30, 2048, 2), BF16), ((3, 32, 1024, 1), FP16), ((2, 25, 1024, 2), FP32),   # 128 pieces
    ((2, 33, 1016, 1), BF16),                                                       # 127
    ((1, 61, 1024, 2), BF16), ((1, 31, 2048, 4), FP16),                             # 64
    ((6, 2048, 512, 32), BF16), ((5, 2047, 384, 24), FP32)])                        # 2, 4
def test_widest_and_largest_strips_of_the_single_launch(gn, shape, dtype, silu, saved):
    print("case gn strips %s %s silu=%s saved=%s" % (shape, dtype, silu, saved), flush=True)
    x, w, b, dy, mean, rstd = make(*shape, dtype, shape[1])
    given = gn.checkpoint_rows(x.cuda()) if saved else x.cuda()
    if saved:
        x = ref.checkpoint(x)[2]
    check_backward(gn, dy, x, given, mean, rstd, w, b, silu, (shape, dtype, silu, saved))


def test_block_trained_from_saved_inputs(gn):
    """x + layer_norm(group_norm_silu(x)) in fp32, both inputs kept in 8 bits:
    the gradients of the formulas in 64 bits at the restored values, with the
    statistics of the forward pass."""
    N, L, C, G = 2, 48, 96, 8
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(N, L, C, generator=gen)
    w1, w2 = [1 + 0.2 * torch.randn(C, generator=gen) for _ in range(2)]
    b1, b2 = [0.2 * torch.randn(C, generator=gen) for _ in range(2)]
    v = torch.randn(N, L, C, generator=gen)
    xg, w1g, b1g, w2g, b2g, vg = [t.cuda() for t in (x, w1, b1, w2, b2, v)]
    m1, r1 = gn.group_stats_rows(xg, G)
    h, ck1 = gn.apply_rows(xg, m1, r1, w1g, b1g, True, checkpoint=True)
    _, m2, r2, ck2 = gn.layer_norm_rows(h, w2g, b2g, 1e-6, checkpoint=True)
    dh, dw2, db2 = gn.layer_norm_rows_backward(vg, ck2, m2, r2, w2g)
    dx, dw1, db1 = gn.group_norm_silu_rows_backward(dh, ck1, m1, r1, w1g, b1g)
    dx = dx + vg

    xv, hv = ref.checkpoint(x)[2], ref.checkpoint(h)[2]
    edh = ref.layer_norm_backward(v, hv, m2, r2, w2, FP32, FP32, N * L + 16)
    for g, value, bound, name in zip((dh, dw2, db2), edh[:3], edh[3:], ("dh", "dw2", "db2")):
        ref.check(g, value, bound, name)
    # GroupNorm's pass on the exact dh; what the fp32 dh is off by goes through
    # it linearly: dt by at most 1.1 (SiLU's largest slope) of it
    want = ref.group_norm_backward(edh[0], xv, m1, r1, w1, b1, True, FP32, FP32, L + 10)
    e = 1.1 * edh[3]
    mu = m1.cpu().double().repeat_interleave(C // G, 1).unsqueeze(1)
    rs = r1.cpu().double().repeat_interleave(C // G, 1).unsqueeze(1)
    hh = ((xv - mu) * rs).abs()

    def over_group(t):
        return (t.sum(1).reshape(N, G, C // G).mean(2) / L).repeat_interleave(C // G, 1).unsqueeze(1)

    wa = w1.double().abs()
    ex = rs * (wa * e + over_group(wa * e) + hh * over_group(wa * e * hh))
    ref.check(dx, want[0] + v.double(),
              1.01 * (want[3] + ex) + ref.U * (want[0].abs() + v.double().abs()), "dx")
    ref.check(dw1, want[1], 1.01 * (want[4] + (e * hh).sum((0, 1))), "dw1")
    ref.check(db1, want[2], 1.01 * (want[5] + e.sum((0, 1))), "db1")
