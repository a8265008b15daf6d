"""The backward passes where the input's spread is so small, or so large, that
rstd*rstd leaves fp32's normal range although every gradient lies within it."""
import pytest

torch = pytest.importorskip("torch")

import rows_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

SPREADS = [1e-20, 1e21]             # rstd = 1e20 (its square: infinity), 1e-21 (1e-42)
DTYPES = [torch.bfloat16, torch.float32]


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


def make(shape, dtype, spread, seed):
    gen = torch.Generator().manual_seed(seed)
    C = shape[-1]
    x = (spread * torch.randn(*shape, generator=gen)).to(dtype)
    dy = torch.randn(*shape, generator=gen).to(dtype)
    w = 1 + 0.3 * torch.randn(C, generator=gen)
    b = 0.3 * torch.randn(C, generator=gen)
    return x, dy, w, b


def compare(got, want, what):
    for g, v, bound, name in zip(got, want[:3], want[3:], ("dx", "dw", "db")):
        assert bool(torch.isfinite(v.to(g.dtype)).all())
        ref.check(g, v, bound, "%s %s" % (what, name))


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("spread", SPREADS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,C", [(5, 5), (37, 321), (1500, 64), (1100, 2560)])
def test_layer_norm(gn, M, C, dtype, spread, saved):
    print("case layer norm M=%d C=%d %s %g" % (M, C, dtype, spread), flush=True)
    x, dy, w, _ = make((M, C), dtype, spread, C)
    mean = x.double().mean(-1).float()
    rstd = (1.0 / x.double().std(-1, unbiased=False)).float()
    given = gn.checkpoint_rows(x.cuda()) if saved else x.cuda()
    if saved:
        x = ref.checkpoint(x)[2]
    got = gn.layer_norm_rows_backward(dy.cuda(), given, mean.cuda(), rstd.cuda(), w.cuda())
    compare(got, ref.layer_norm_backward(dy, x, mean, rstd, w, dtype, torch.float32, M + 16),
            (M, C, dtype, spread))


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("spread", SPREADS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(2, 70, 96, 8),          # the single launch
                                   (1, 60, 33, 3), (2, 5000, 64, 8), (1, 40, 2048, 8)])
def test_group_norm(gn, shape, dtype, spread, saved):
    N, L, C, G = shape
    print("case group norm %s %s %g" % (shape, dtype, spread), flush=True)
    x, dy, w, b = make((N, L, C), dtype, spread, L)
    xg = x.double().reshape(N, L, G, C // G)
    mean = xg.mean((1, 3))
    rstd = (1.0 / ((xg - mean[:, None, :, None]) ** 2).mean((1, 3)).sqrt()).float()
    mean = mean.float()
    given = gn.checkpoint_rows(x.cuda()) if saved else x.cuda()
    if saved:
        x = ref.checkpoint(x)[2]
    for silu in (False, True):
        got = gn.group_norm_silu_rows_backward(dy.cuda(), given, mean.cuda(), rstd.cuda(),
                                               w.cuda(), b.cuda(), silu)
        compare(got, ref.group_norm_backward(dy, x, mean, rstd, w, b, silu, dtype, torch.float32,
                                             min(L, 1024) + 10), (shape, dtype, spread, silu))
