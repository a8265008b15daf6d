"""The README's autograd function, taken from its text: it runs, its gradients
are those of the formulas, its saved tensors go through autograd's hooks, and a
second derivative is refused in words."""
import os
import re

import pytest

torch = pytest.importorskip("torch")

import rows_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def gn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import groupnorm_silu_normalization_amd as gn
    return gn


@pytest.fixture(scope="module")
def function(gn):
    """GroupNormSilu, after the whole block that holds it has run."""
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    block, = [b for b in blocks if "class GroupNormSilu" in b]
    names = {"torch": torch, "gn": gn}
    exec(compile(block, "README.md", "exec"), names)
    assert names["back"].shape == names["r"].shape
    return names["GroupNormSilu"]


def leaves(N, L, C, seed):
    gen = torch.Generator().manual_seed(seed)
    ts = [torch.randn(N, L, C, generator=gen), 1 + 0.2 * torch.randn(C, generator=gen),
          0.2 * torch.randn(C, generator=gen)]
    return [t.cuda().requires_grad_() for t in ts], torch.randn(N, L, C, generator=gen).cuda()


def test_gradients(gn, function):
    G = 8
    (x, w, b), v = leaves(2, 48, 96, 3)
    kept = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: kept.append(t) or t, lambda t: t):
        y = function.apply(x, w, b, G)
    assert {t.dtype for t in kept} == {torch.int8, torch.uint8, torch.float32}
    assert not any(t.shape == x.shape and t.dtype == x.dtype for t in kept)    # x itself is not kept
    grads = torch.autograd.grad(y, (x, w, b), v)
    with torch.no_grad():
        mean, rstd = gn.group_stats_rows(x, G)
    want = ref.group_norm_backward(v.cpu(), ref.checkpoint(x.detach())[2], mean, rstd, w.detach(),
                                   b.detach(), True, torch.float32, torch.float32, 58)
    for g, value, bound, name in zip(grads, want[:3], want[3:], ("dx", "dw", "db")):
        ref.check(g, value, bound, name)


def test_second_derivative_is_refused(function):
    (x, w, b), v = leaves(1, 20, 32, 4)
    y = function.apply(x, w, b, 4)
    dx, = torch.autograd.grad(y, x, v.requires_grad_(), create_graph=True)
    assert bool(torch.isfinite(dx).all())
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dx.sum().backward()


def test_a_width_without_a_layout_is_declined_by_the_statistics(gn):
    """... and taken by the other calls with the caller's mean and rstd."""
    x = torch.randn(2, 9, 1001, device="cuda")
    with torch.no_grad():
        assert gn.plan_rows(2, 9, 1001, 7) is None and gn.group_stats_rows(x, 7) is None
        g = x.double().reshape(2, 9, 7, 143)
        mean = g.mean((1, 3))
        var = ((g - mean[:, None, :, None]) ** 2).mean((1, 3))
        mean, rstd = mean.float(), (1 / torch.sqrt(var + 1e-6)).float()
        y, kept = gn.apply_rows(x, mean, rstd, None, None, True, checkpoint=True)
        dx, dw, db = gn.group_norm_silu_rows_backward(torch.ones_like(y), kept, mean, rstd)
        assert dx.shape == x.shape and dw.shape == (1001,) and db.shape == (1001,)
