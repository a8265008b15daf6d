"""Layer norm where a row slot takes several rows: the backward pass beyond
1024 rows (partial rows and their column sums) at every width class, from x and
from the checkpoint, and the forward pass beyond one round of workgroups, all
against the definition in 64 bits."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import rows_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
EPS = 1e-6
# every count of lanes and pieces a row, on both sides; single values to the limit
WIDTHS = [1, 2, 3, 4, 5, 7, 8, 9, 16, 17, 24, 33, 64, 65, 129, 257, 513, 1001, 1030, 2049, 2560,
          4097, 5000, 8192, 8193, 12288, 16383, 16384]


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


def workspace(gn, M, C, dtype=0):
    out = ctypes.c_int64(-1)
    assert gn.gn_layer_norm_rows_backward_workspace(M, C, dtype, ctypes.byref(out)) == 0
    return out.value


def moments(x):
    """Statistics as a forward pass returns them: rounded to fp32."""
    x = x.double()
    mean = x.mean(-1, keepdim=True)
    var = ((x - mean) ** 2).mean(-1)
    return mean.squeeze(-1).float(), (1.0 / torch.sqrt(var + EPS)).float()


def check(got, want, bound, what):
    """ref.check, where a value beyond the type's largest number by half a step
    or more is rounded to infinity (a restored single value per row lies
    rstd = 1000 steps of its checkpoint from its mean)."""
    fi = torch.finfo(got.dtype)
    half = fi.max * fi.eps / 4              # just below half a step there
    got = got.cpu()
    out = want.abs() - bound >= fi.max + half       # surely rounded to infinity
    assert torch.equal(got[out].double(), torch.sign(want[out]) * float("inf")), what
    near = ~out & (want.abs() + bound >= fi.max) & torch.isinf(got)
    keep = ~(out | near)
    assert torch.equal(torch.sign(got[near]).double(), torch.sign(want[near])), what
    ref.check(got[keep], want[keep], bound.expand_as(want)[keep], what)


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("C", WIDTHS)
def test_backward_of_many_rows(gn, C, dtype, saved):
    M = 2500 if C <= 1030 else 1037     # an uneven last round of 256 workgroups
    print("case layer_norm backward M=%d C=%d %s saved=%s" % (M, C, dtype, saved), flush=True)
    assert workspace(gn, M, C, gn.dtype_code(dtype)) > 0
    adt = torch.float32 if saved else dtype
    x, w, _, dy = make(M, C, dtype, adt, 3 * C + M)
    mean, rstd = moments(x)
    given = gn.checkpoint_rows(x.cuda()) if saved else x.cuda()
    if saved:
        x = ref.checkpoint(x)[2]
    got = gn.layer_norm_rows_backward(dy.cuda(), given, mean.cuda(), rstd.cuda(), w.cuda())
    want = ref.layer_norm_backward(dy, x, mean, rstd, w, dtype, adt, M + 16)
    for g, v, bound, name in zip(got, want[:3], want[3:], ("dx", "dw", "db")):
        check(g, v, bound, "%s %s" % ((M, C, dtype, saved), name))


# More rows than 2048 workgroups of 256 lanes (or their like) take in one round.
@pytest.mark.parametrize("save", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,C", [(270003, 5), (140001, 24), (40001, 130), (20001, 257),
                                 (9001, 1001), (4200, 2560), (2101, 4097), (1301, 8200),
                                 (1031, 16384)])
def test_forward_of_several_rounds(gn, M, C, dtype, save):
    print("case layer_norm rounds M=%d C=%d %s save=%s" % (M, C, dtype, save), flush=True)
    x, w, b, _ = make(M, C, dtype, torch.float32, M + C)
    r = gn.layer_norm_rows(x.cuda(), w.cuda(), b.cuda(), EPS, stats=True, checkpoint=save)
    want = ref.layer_norm(x, w, b, EPS, dtype)
    for g, v, bound, name in zip(r, want[:3], want[3:], ("y", "mean", "rstd")):
        ref.check(g, v, bound, "%s %s" % ((M, C, dtype, save), name))
    if save:
        codes, E, _ = ref.checkpoint(x)
        assert torch.equal(r[3].codes.cpu().to(torch.int64), codes)
        assert torch.equal(r[3].scales.cpu().to(torch.int64), E)


@pytest.mark.parametrize("saved", [False, True])
def test_captured_graphs_with_a_workspace_each(gn, saved):
    """Two captured backward passes that need a workspace, replayed at once on
    two streams beside eager calls, give the eager bits."""
    sets, eager, graphs, outs = [], [], [], []
    for C in (777, 2304):
        M = 1537
        assert workspace(gn, M, C) > 0
        x, w, b, dy = [t.cuda() for t in make(M, C, torch.bfloat16, torch.float32, C)]
        r = gn.layer_norm_rows(x, w, b, EPS, checkpoint=True)
        sets.append((dy, r[3] if saved else x, r[1], r[2], w))
        eager.append(gn.layer_norm_rows_backward(*sets[-1]))
    torch.cuda.synchronize()
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(gn.layer_norm_rows_backward(*s))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(4):
        for o in outs:
            for t in o:
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        mine = gn.layer_norm_rows_backward(*sets[turn % 2])
        torch.cuda.synchronize()
        for p, q in zip(mine, eager[turn % 2]):
            assert torch.equal(p, q)
        for o, e in zip(outs, eager):
            for p, q in zip(o, e):
                assert torch.equal(p, q)
