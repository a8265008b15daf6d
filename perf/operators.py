"""Workloads of the normalisations' training operators, with plain forms.

Layer norm's forward and backward pass, the backward pass of GroupNorm(+SiLU)
and the 8-bit checkpoints that both backward passes can read in the place of
their input.  ``listed()`` names the cases, ``prepare`` makes a case's inputs,
``run`` is one pass through an operator -- its plain form, or the library's
(``own``) -- ``exact`` the same in 64 bits and ``work`` the bytes and
operations that a pass cannot do without.
"""
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = 32      # channels that share one scale of an 8-bit checkpoint
EPS = 1e-6


# ---- the cases ---------------------------------------------------------------
# op: layer_norm       y (and mean, rstd where stats; and the checkpoint's values where save)
#     layer_norm_grad  dx, dweight, dbias (saved: x comes as an 8-bit checkpoint)
#     group_norm_grad  dx, dweight, dbias of GroupNorm(+SiLU) (saved: as above)
#     group_norm_save  GroupNorm's apply step that saves its input, and the saved values
#     checkpoint       rows saved in 8 bits, and the saved values
# n, l, c: (N, L, C) rows; affine: the type of weight and bias
def _case(name, op, n, l, c, dtype, affine, **more):
    d = {"name": name, "op": op, "n": n, "l": l, "c": c, "dtype": dtype, "affine": affine}
    d.update(more)
    return d


def listed():
    return [
        # one new token of a serving loop: latency alone
        _case("ln_token", "layer_norm", 1, 1, 1024, "bf16", "bf16", stats=False, save=False),
        # a long training batch of a wide model
        _case("ln_long", "layer_norm", 4, 4096, 4096, "bf16", "fp32", stats=True, save=False),
        # a ragged batch: odd rows and an odd width
        _case("ln_odd", "layer_norm", 1, 4099, 1003, "fp16", "fp32", stats=True, save=False),
        # the forward pass of a training step that keeps its input in 8 bits
        _case("ln_save", "layer_norm", 2, 4096, 2560, "bf16", "bf16", stats=True, save=True),
        # the gradient of a short text batch in full precision
        _case("ln_grad_short", "layer_norm_grad", 1, 77, 768, "fp32", "fp32", saved=False),
        # the gradient of the long batch
        _case("ln_grad_long", "layer_norm_grad", 4, 4096, 4096, "bf16", "fp32", saved=False),
        # a ragged batch's gradient from its 8-bit checkpoint
        _case("ln_grad_saved", "layer_norm_grad", 3, 1667, 1537, "bf16", "bf16", saved=True),
        # the decoder's smallest GroupNorm (1, 128, 64, 64)
        _case("gn_grad_small", "group_norm_grad", 1, 4096, 128, "bf16", "fp32", g=32, silu=True,
              saved=False),
        # the decoder's (1, 256, 1024, 1024)
        _case("gn_grad_large", "group_norm_grad", 1, 1048576, 256, "bf16", "fp32", g=32,
              silu=True, saved=False),
        # the decoder's (1, 512, 256, 256), its input kept in 8 bits
        _case("gn_grad_saved", "group_norm_grad", 1, 65536, 512, "bf16", "fp32", g=32, silu=True,
              saved=True),
        # the forward pass that keeps it, (1, 512, 512, 512)
        _case("gn_save", "group_norm_save", 1, 262144, 512, "bf16", "fp32", g=32, silu=True),
        # rows of an odd width kept in 8 bits
        _case("rows_save", "checkpoint", 1, 20011, 1001, "fp16", "fp32"),
    ]


def draw(rng):
    """A case of the ranges above: widths to 8192, one row to millions, at most
    2^25 values, at least eight values to each set of statistics (with fewer,
    a gradient is a difference of nearly equal numbers)."""
    def spread(lo, hi):
        return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))

    op = rng.choice(["layer_norm", "layer_norm", "layer_norm_grad", "layer_norm_grad",
                     "group_norm_grad", "group_norm_grad", "group_norm_save", "checkpoint"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    affine = rng.choice(["fp32", dtype])
    n = rng.choice([1, 1, 2, 3, 5])
    if op.startswith("group_norm"):
        g = rng.choice([1, 2, 8, 16, 24, 32, 32])
        c = g * spread(1, 8192 // g if g < 8 else 128)
        least = -(-8 * g // c)
        l = spread(least, max(least, (1 << 25) // (c * n)))
        d = {"op": op, "n": n, "l": l, "c": c, "dtype": dtype, "affine": affine, "g": g,
             "silu": rng.random() < 0.7}
        if op == "group_norm_grad":
            d["saved"] = rng.random() < 0.4
        return d
    c = spread(1, 1024) * 8 if rng.random() < 0.6 else spread(8, 8192)
    l = spread(1, max(1, (1 << 25) // (c * n)))
    d = {"op": op, "n": n, "l": l, "c": c, "dtype": dtype, "affine": affine}
    if op == "layer_norm":
        d["save"] = rng.random() < 0.4
        d["stats"] = d["save"] or rng.random() < 0.6
    elif op == "layer_norm_grad":
        d["saved"] = rng.random() < 0.4
    return d


# ---- the inputs --------------------------------------------------------------
def prepare(case, seed):
    """Activations as residual streams and decoders hold them: a mean and a
    spread of its own for each channel, a few channels far wider than the
    rest; gradients of unit spread; weights around one.  The statistics and
    checkpoints that a backward pass reads are those of its forward pass."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    n, l, c = case["n"], case["l"], case["c"]
    dt, at = DTYPES[case["dtype"]], DTYPES[case["affine"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    centre = 0.3 * randn(c)
    width = torch.exp(0.3 * randn(c))
    wide = torch.rand(c, generator=gen, device=dev) < 0.01
    width = torch.where(wide, 8.0 * width, width)
    x = randn(n, l, c).mul_(width).add_(centre).to(dt)
    st = {"case": case, "x": x,
          "weight": (1.0 + 0.2 * randn(c)).to(at), "bias": (0.2 * randn(c)).to(at)}
    op = case["op"]
    if op.endswith("_grad"):
        st["dy"] = randn(n, l, c).to(dt)
    if op == "layer_norm_grad":
        st["mean"], st["rstd"] = (s.float().reshape(n, l) for s in _row_moments(x.double()))
    if op.startswith("group_norm"):
        g = case["g"]
        xg = x.reshape(n, l, g, c // g)
        mean = torch.zeros(n, g, device=dev, dtype=torch.float64)
        for i in range(n):          # a group's plane at a time, for the largest cases
            for j in range(g):
                v = xg[i, :, j].double()
                m = v.mean()
                mean[i, j] = m
                st.setdefault("var", torch.zeros_like(mean))[i, j] = ((v - m) ** 2).mean()
        st["mean"] = mean.float()
        st["rstd"] = (1.0 / torch.sqrt(st.pop("var") + EPS)).float()
    if case.get("saved"):
        st["codes"], st["scales"] = _encode(x)
        del st["x"]
    return st


def _row_moments(x):
    mean = x.sum(-1, keepdim=True) / x.shape[-1]
    d = x - mean
    return mean, 1.0 / torch.sqrt((d * d).sum(-1, keepdim=True) / x.shape[-1] + EPS)


# ---- the 8-bit checkpoint in its plain form ----------------------------------
def _blocks(x):
    """(..., C) as (..., ceil(C/32), 32), the last block filled up with zeros."""
    c = x.shape[-1]
    nb = (c + BLOCK - 1) // BLOCK
    if nb * BLOCK != c:
        x = torch.nn.functional.pad(x, (0, nb * BLOCK - c))
    return x.reshape(*x.shape[:-1], nb, BLOCK)


def _exponents(x):
    """The exponent field of each block's largest magnitude, biased by 127."""
    top = _blocks(x).float().abs().amax(-1)
    _, e = torch.frexp(top)
    return torch.where(top > 0, (e + 126).clamp(min=0), torch.zeros_like(e))


def _encode(x):
    """Codes and scales; the products by powers of two are exact in fp32."""
    e = _exponents(x)
    f = torch.exp2((133 - e).double()).unsqueeze(-1)
    codes = (_blocks(x).double() * f).round_().clamp_(-127, 127).to(torch.int8)
    return (codes.reshape(*x.shape[:-1], -1)[..., :x.shape[-1]].contiguous(),
            e.to(torch.uint8))


def _decode(codes, scales):
    f = torch.exp2(scales.to(torch.float64) - 133).unsqueeze(-1)
    v = _blocks(codes).double() * f
    return v.reshape(*codes.shape[:-1], -1)[..., :codes.shape[-1]].float()


# ---- one pass ----------------------------------------------------------------
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_plain(st):
    case = st["case"]
    op, dt, c = case["op"], DTYPES[case["dtype"]], case["c"]
    if op == "checkpoint":
        return [_decode(*_encode(st["x"])).to(dt)]
    w, b = st["weight"].float(), st["bias"].float()
    if op == "layer_norm":
        x = st["x"].float()
        mean, rstd = _row_moments(x)
        y = ((x - mean) * rstd * w + b).to(dt)
        out = [y]
        if case["stats"]:
            out += [mean.squeeze(-1), rstd.squeeze(-1)]
        if case["save"]:
            out.append(_decode(*_encode(st["x"])).to(dt))
        return out
    if op == "layer_norm_grad":
        x = _decode(st["codes"], st["scales"]) if case["saved"] else st["x"].float()
        dy = st["dy"].float()
        rstd = st["rstd"].unsqueeze(-1)
        h = (x - st["mean"].unsqueeze(-1)) * rstd
        g = dy * w
        dx = rstd * (g - g.sum(-1, keepdim=True) / c - h * ((g * h).sum(-1, keepdim=True) / c))
        at = DTYPES[case["affine"]]
        return [dx.to(dt), (dy * h).sum((0, 1)).to(at), dy.sum((0, 1)).to(at)]
    n, l, g = case["n"], case["l"], case["g"]
    mean = st["mean"].reshape(n, 1, g, 1)
    rstd = st["rstd"].reshape(n, 1, g, 1)
    wg, bg = w.reshape(g, c // g), b.reshape(g, c // g)
    if op == "group_norm_save":
        x = st["x"].float().reshape(n, l, g, c // g)
        t = (x - mean) * rstd * wg + bg
        y = t / (1.0 + torch.exp(-t)) if case["silu"] else t
        return [y.reshape(n, l, c).to(dt), _decode(*_encode(st["x"])).to(dt)]
    x = _decode(st["codes"], st["scales"]) if case["saved"] else st["x"].float()
    x = x.reshape(n, l, g, c // g)
    dt_ = st["dy"].float().reshape(n, l, g, c // g)
    h = (x - mean) * rstd
    if case["silu"]:
        t = h * wg + bg
        s = 1.0 / (1.0 + torch.exp(-t))
        dt_ = dt_ * (s * (1.0 + t * (1.0 - s)))
    m = l * (c // g)
    dth = dt_ * h
    dg = dt_ * wg
    a = dg.sum((1, 3), keepdim=True) / m
    bb = (dg * h).sum((1, 3), keepdim=True) / m
    dx = rstd * (dg - a - h * bb)
    at = DTYPES[case["affine"]]
    return [dx.reshape(n, l, c).to(dt), dth.sum((0, 1)).reshape(c).to(at),
            dt_.sum((0, 1)).reshape(c).to(at)]


def _run_own(st):
    import groupnorm_silu_normalization_amd as gn

    case = st["case"]
    op, dt = case["op"], DTYPES[case["dtype"]]
    with torch.no_grad():
        if op == "checkpoint":
            return [gn.restore_rows(gn.checkpoint_rows(st["x"]))]
        if op == "layer_norm":
            r = gn.layer_norm_rows(st["x"], st["weight"], st["bias"], EPS, stats=case["stats"],
                                   checkpoint=case["save"])
            if not case["stats"]:
                return [r]
            if case["save"]:
                return [r[0], r[1], r[2], gn.restore_rows(r[3])]
            return list(r)
        if op == "group_norm_save":
            y, kept = gn.apply_rows(st["x"], st["mean"], st["rstd"], st["weight"], st["bias"],
                                    case["silu"], checkpoint=True)
            return [y, gn.restore_rows(kept)]
        x = gn.Checkpoint8(st["codes"], st["scales"], dt) if case["saved"] else st["x"]
        if op == "layer_norm_grad":
            return list(gn.layer_norm_rows_backward(st["dy"], x, st["mean"], st["rstd"],
                                                    st["weight"]))
        return list(gn.group_norm_silu_rows_backward(st["dy"], x, st["mean"], st["rstd"],
                                                     st["weight"], st["bias"], case["silu"]))


# ---- what a pass cannot do without ---------------------------------------------
def work(case):
    e = case["n"] * case["l"] * case["c"]
    size = 4 if case["dtype"] == "fp32" else 2
    par = case["c"] * (4 if case["affine"] == "fp32" else 2)
    rows = case["n"] * case["l"]
    kept = e + rows * ((case["c"] + BLOCK - 1) // BLOCK)   # codes and scales
    op = case["op"]
    if op == "checkpoint":         # x in; the checkpoint out and in again; its values out
        return {"bytes": 2 * e * size + 2 * kept, "flops": 5 * e}
    if op == "layer_norm":
        by = 2 * e * size + 2 * par + (8 * rows if case["stats"] else 0)
        if case["save"]:
            by += 2 * kept + e * size
        return {"bytes": by, "flops": (8 + (5 if case["save"] else 0)) * e}
    if op == "layer_norm_grad":
        return {"bytes": (kept if case["saved"] else e * size) + 2 * e * size + 8 * rows + 3 * par,
                "flops": 16 * e}
    stats = 8 * case["n"] * case["g"]
    if op == "group_norm_save":
        return {"bytes": 3 * e * size + 2 * kept + 2 * par + stats, "flops": 15 * e}
    return {"bytes": (kept if case["saved"] else e * size) + 2 * e * size + 4 * par + stats,
            "flops": 24 * e}


# ---- the definition in 64 bits -------------------------------------------------
def exact(case, seed):
    """The outputs of ``run`` from the definitions, in 64 bits, a sample and
    a slab of its rows at a time."""
    st = prepare(case, seed)
    op, n, l, c = case["op"], case["n"], case["l"], case["c"]
    f64 = torch.float64
    dev = st["weight"].device
    w, b = st["weight"].to(f64), st["bias"].to(f64)
    channel = torch.arange(c, device=dev)
    slab = max(1, (1 << 25) // c)
    spans = [(i, r, min(l, r + slab)) for i in range(n) for r in range(0, l, slab)]

    def kept(x):
        """What an 8-bit checkpoint stands for, by its definition: each value
        to the nearest multiple of 2^(k-6), at most 127 of them, 2^k the
        power of two at or below the block's largest magnitude."""
        v = x.to(f64)
        nb = (c + BLOCK - 1) // BLOCK
        top = torch.zeros(v.shape[0], nb, dtype=f64, device=dev)
        top.scatter_reduce_(1, (channel // BLOCK).expand(v.shape[0], c), v.abs(), "amax")
        k = torch.floor(torch.log2(top.clamp(min=2.0 ** -127)))
        k = torch.where(torch.exp2(k) > top, k - 1, k)
        k = torch.where(torch.exp2(k + 1) <= top, k + 1, k).clamp(min=-127)
        step = torch.exp2(k - 6)[:, channel // BLOCK]
        return torch.minimum(torch.maximum(torch.round(v / step), -127 + 0 * v),
                             127 + 0 * v) * step

    def rows(i, r0, r1):
        if case.get("saved"):
            e = st["scales"][i, r0:r1].to(f64)[:, channel // BLOCK]
            return st["codes"][i, r0:r1].to(f64) * 2.0 ** (e - 133)
        return st["x"][i, r0:r1].to(f64)

    def empty(*shape):
        return torch.empty(*shape, dtype=f64, device=dev)

    if op == "checkpoint":
        out = empty(n, l, c)
        for i, r0, r1 in spans:
            out[i, r0:r1] = kept(st["x"][i, r0:r1])
        return [out]
    if op == "layer_norm":
        y, mean, rstd = empty(n, l, c), empty(n, l), empty(n, l)
        sv = empty(n, l, c) if case["save"] else None
        for i, r0, r1 in spans:
            x = rows(i, r0, r1)
            mu = x.mean(1)
            rs = (x.var(1, unbiased=False) + EPS) ** -0.5
            y[i, r0:r1] = w * ((x - mu[:, None]) * rs[:, None]) + b
            mean[i, r0:r1], rstd[i, r0:r1] = mu, rs
            if sv is not None:
                sv[i, r0:r1] = kept(st["x"][i, r0:r1])
        return [y] + ([mean, rstd] if case["stats"] else []) + ([sv] if case["save"] else [])
    if op == "layer_norm_grad":
        dx, dw, db = empty(n, l, c), torch.zeros_like(w), torch.zeros_like(w)
        for i, r0, r1 in spans:
            dy = st["dy"][i, r0:r1].to(f64)
            rs = st["rstd"][i, r0:r1, None].to(f64)
            h = (rows(i, r0, r1) - st["mean"][i, r0:r1, None].to(f64)) * rs
            gr = dy * w
            dx[i, r0:r1] = rs * (gr - gr.mean(1, keepdim=True)
                                 - h * (gr * h).mean(1, keepdim=True))
            dw += (dy * h).sum(0)
            db += dy.sum(0)
        return [dx, dw, db]
    group = channel // (c // case["g"])
    mu, rs = st["mean"].to(f64)[:, group], st["rstd"].to(f64)[:, group]     # (n, c)
    if op == "group_norm_save":
        y, sv = empty(n, l, c), empty(n, l, c)
        for i, r0, r1 in spans:
            t = w * (rows(i, r0, r1) - mu[i]) * rs[i] + b
            y[i, r0:r1] = t * torch.sigmoid(t) if case["silu"] else t
            sv[i, r0:r1] = kept(st["x"][i, r0:r1])
        return [y, sv]

    def grads(i, r0, r1):
        h = (rows(i, r0, r1) - mu[i]) * rs[i]
        d = st["dy"][i, r0:r1].to(f64)
        if case["silu"]:
            t = w * h + b
            s = torch.sigmoid(t)
            d = d * (s + t * s * (1 - s))
        return h, d

    s1 = torch.zeros(n, c, dtype=f64, device=dev)
    s2 = torch.zeros(n, c, dtype=f64, device=dev)
    for i, r0, r1 in spans:
        h, d = grads(i, r0, r1)
        s1[i] += d.sum(0)
        s2[i] += (d * h).sum(0)
    m = l * (c // case["g"])
    a = torch.zeros(n, case["g"], dtype=f64, device=dev).index_add_(1, group, s1 * w) / m
    bb = torch.zeros(n, case["g"], dtype=f64, device=dev).index_add_(1, group, s2 * w) / m
    dx = empty(n, l, c)
    for i, r0, r1 in spans:
        h, d = grads(i, r0, r1)
        dx[i, r0:r1] = rs[i] * (d * w - a[i, group] - h * bb[i, group])
    return [dx, s2.sum(0), s1.sum(0)]
