"""The README's layer of 8-bit products, taken from its text, runs and gives what
its definitions give."""
import os
import re

import pytest

torch = pytest.importorskip("torch")

import rows8_reference as ref  # noqa: E402
import rows_reference as rows  # noqa: E402

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_layer_of_8_bit_products():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import groupnorm_silu_normalization_amd as gn

    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    block, = [b for b in blocks if "int8_matmul" in b]
    n = {"torch": torch, "gn": gn}
    exec(compile(block, "README.md", "exec"), n)
    assert n["stream"].shape == n["x"].shape and n["h"].shape == (48, n["F"])
    bf16 = torch.bfloat16
    want = n["q"].codes.cpu().double() * n["q"].scales.cpu().double().unsqueeze(-1)
    rows.check(n["back"], want, rows.U * want.abs() + rows.rounded(want, bf16), "back")
    x, g = n["x"], n["g"]
    _, y, rstd, _, _, ey, er, _ = ref.rms_norm(x, g, 1e-6, bf16)
    rows.check(n["y"], y, ey, "y")
    rows.check(n["rstd"], rstd, er, "rstd")
    dx, dg, ex, eg = ref.rms_norm_backward(torch.ones_like(x), x, n["rstd"], g, x, bf16,
                                           torch.float32, 48 + 16)
    rows.check(n["dx"], dx, ex, "dx")
    rows.check(n["dg"], dg, eg, "dg")
