"""8-bit checkpoints of rows: the codes and scales by their definition, the
values they stand for, at every width around the pieces and blocks."""
import pytest

torch = pytest.importorskip("torch")

import rows_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
WIDTHS = [1, 2, 3, 4, 5, 7, 8, 9, 12, 15, 16, 31, 32, 33, 40, 63, 64, 65, 96, 100, 127, 129, 255,
          256, 320, 511, 1001, 2047, 2048, 2056, 4100, 8192, 16384]


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


def rows(M, C, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(M, C, generator=gen) * torch.exp(2.0 * torch.randn(M, 1, generator=gen))
    x[torch.rand(M, C, generator=gen) < 0.05] = 0.0
    return x.to(dtype)


def compare(gn, x, ck, what):
    codes, E, val = ref.checkpoint(x)
    assert torch.equal(ck.codes.cpu().to(torch.int64), codes), what
    assert torch.equal(ck.scales.cpu().to(torch.int64), E), what
    for dt in DTYPES:
        back = gn.restore_rows(ck, dt)
        want = val.to(dt)
        assert back.dtype == dt and back.shape == x.shape
        got = back.cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(want)), what
        keep = ~torch.isnan(want)
        assert torch.equal(got[keep], want[keep]), what


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("C", WIDTHS)
def test_codes_scales_and_values(gn, C, dtype):
    for M in (1, 3, 70):
        print("case checkpoint M=%d C=%d %s" % (M, C, dtype), flush=True)
        x = rows(M, C, dtype, C + M)
        compare(gn, x, gn.checkpoint_rows(x.cuda()), (M, C, dtype))


@pytest.mark.parametrize("dtype", DTYPES)
def test_ties_clamps_and_extremes(gn, dtype):
    """Halves of the step (to even), the clamp at the top of a block's range,
    the type's largest and smallest numbers, signed zeros."""
    C = 96
    x = torch.zeros(10, C)
    k = torch.arange(C) - 48.0
    x[0] = (k + 0.5) / 64.0                                # ties under a top of 1.0 ...
    x[0, ::32] = 1.0
    x[1] = -(k + 0.5) / 64.0
    x[1, 5::32] = -1.5
    x[2] = 1.9921875                                       # 127.5 steps: the clamp
    x[3] = -0.0
    fi = torch.finfo(dtype)
    x[4] = fi.max
    x[5] = float(fi.smallest_normal)
    x[6] = float(fi.smallest_normal) * fi.eps              # the smallest subnormal
    x[7] = torch.where(torch.arange(C) % 2 == 0, 3.0, -3.0)
    x[8, 40] = 1e-3                                        # one value in its block
    x[9] = fi.min
    x = x.to(dtype)
    print("case checkpoint extremes %s" % dtype, flush=True)
    compare(gn, x, gn.checkpoint_rows(x.cuda()), dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_infinity_and_nan_take_their_block_only(gn, dtype):
    x = rows(6, 131, dtype, 5)
    x[0, 0] = float("inf")
    x[1, 40] = float("nan")
    x[2, 130] = float("-inf")
    x[4, 64] = float("nan")
    x[4, 65] = float("inf")
    print("case checkpoint inf/nan %s" % dtype, flush=True)
    ck = gn.checkpoint_rows(x.cuda())
    compare(gn, x, ck, dtype)
    assert int((ck.scales == 255).sum()) == 4


@pytest.mark.parametrize("dtype", DTYPES)
def test_strided_unaligned_and_broadcast_rows(gn, dtype):
    big = rows(40, 211, dtype, 9).cuda()
    for view in (big[:, 3:100], big[::2, 1:210], big.reshape(5, 8, 211)[:, :, 7:180],
                 big[7].expand(12, 211), big[:1, 5:6], big[3]):
        print("case checkpoint view %s %s" % (tuple(view.shape), view.stride()), flush=True)
        compare(gn, view.cpu(), gn.checkpoint_rows(view), tuple(view.stride()))
    # rows that are not evenly spaced, or not dense: declined
    assert gn.checkpoint_rows(big.reshape(4, 10, 211)[:, ::3, :]) is None
    assert gn.checkpoint_rows(big[:, ::2]) is None
    # an output of wider rows: what lies between the rows stays as it was
    ck = gn.checkpoint_rows(big[:, 3:100])
    wide = torch.full((40, 130), 7.0, dtype=dtype, device="cuda")
    assert gn.restore_rows(ck, out=wide[:, 9:106]) is not None
    assert torch.equal(wide[:, 9:106].cpu(), gn.restore_rows(ck).cpu())
    assert bool((wide[:, :9] == 7).all()) and bool((wide[:, 106:] == 7).all())


def test_empty_rows(gn):
    for shape in ((0, 64), (3, 0, 64)):
        x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        ck = gn.checkpoint_rows(x)
        assert ck.shape == x.shape and tuple(ck.scales.shape) == shape[:-1] + (2,)
        assert gn.restore_rows(ck).shape == x.shape


def test_nothing_is_written_beyond_the_checkpoint(gn):
    """Codes and scales inside a larger buffer: the bytes around them stay."""
    import ctypes
    M, C = 13, 77
    x = rows(M, C, torch.bfloat16, 3).cuda()
    nb = -(-C // 32)
    buf = torch.full((M * C + 64 + M * nb + 64,), 0x55, dtype=torch.int8, device="cuda")
    at, st = 17, 17 + M * C + 13
    code = gn.gn_checkpoint_rows(ctypes.c_void_p(x.data_ptr()), C,
                                 ctypes.c_void_p(buf.data_ptr() + at),
                                 ctypes.c_void_p(buf.data_ptr() + st), M, C, 0,
                                 ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert code == 0
    codes, E, _ = ref.checkpoint(x)
    got = buf.cpu().to(torch.int64)
    assert torch.equal(got[at:at + M * C], codes.reshape(-1))
    assert torch.equal(got[st:st + M * nb] & 255, E.reshape(-1))
    for part in (got[:at], got[at + M * C:st], got[st + M * nb:]):
        assert bool((part == 0x55).all())
