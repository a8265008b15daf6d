"""Workloads of the operators around 8-bit matrix products, with plain forms.

The root-mean-square norm with the residual's addition and an output in the
rows' type or in 8 bits, its backward pass, rows kept in 8 bits with a scale
each, and the matrix product of such rows.  ``listed()`` names the cases,
``prepare`` makes a case's inputs, ``run`` is one pass through an operator --
its plain form, or the library's (``own``) -- ``exact`` the same in 64 bits and
``work`` the bytes and operations that a pass cannot do without.
"""
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
BLOCK = 32      # channels that share one scale of an 8-bit checkpoint
EPS = 1e-6


# ---- the cases ---------------------------------------------------------------
# op: rms_norm       y, or the values its 8 bits stand for (quantize); and h = x + residual
#                    where residual; and rstd where stats
#     rms_norm_grad  dx, dweight (saved: h comes as an 8-bit checkpoint; stream: with the
#                    gradient that reaches h past the norm)
#     quantize       the values that the 8-bit rows stand for
#     int8_matmul    z of 8-bit rows (m, k) and weights (n, k)
# n, l, c: (N, L, C) rows; affine: the type of weight (bias)
def _case(name, op, **more):
    d = {"name": name, "op": op}
    d.update(more)
    return d


def listed():
    return [
        # one new token of a serving loop, its residual stream updated: latency alone
        _case("rms_token", "rms_norm", n=1, l=1, c=1024, dtype="bf16", affine="bf16",
              residual=True, quantize=True, stats=False),
        # the forward pass of a long training batch
        _case("rms_long", "rms_norm", n=4, l=4096, c=4096, dtype="bf16", affine="fp32",
              residual=True, quantize=False, stats=True),
        # a ragged batch of an odd width on its way to an 8-bit product
        _case("rms_odd", "rms_norm", n=1, l=4099, c=1003, dtype="fp16", affine="fp16",
              residual=True, quantize=True, stats=False),
        # the gradient of a short text batch in full precision
        _case("rms_grad_short", "rms_norm_grad", n=1, l=77, c=768, dtype="fp32", affine="fp32",
              saved=False, stream=False),
        # the gradient of the long batch, joined by the residual stream's
        _case("rms_grad_long", "rms_norm_grad", n=4, l=4096, c=4096, dtype="bf16", affine="fp32",
              saved=False, stream=True),
        # a ragged batch's gradient from its 8-bit checkpoint
        _case("rms_grad_saved", "rms_norm_grad", n=3, l=1667, c=1537, dtype="bf16", affine="bf16",
              saved=True, stream=False),
        # a prompt's activations before a product that no norm precedes
        _case("quant_rows", "quantize", n=2, l=4096, c=2560, dtype="bf16"),
        # rows of an odd width
        _case("quant_odd", "quantize", n=1, l=5003, c=1001, dtype="fp32"),
        # one token through a square layer
        _case("mm_token", "int8_matmul", m=1, n=4096, k=4096, dtype="bf16", affine="bf16",
              bias=False, residual=False),
        # a decoding batch through a widening layer
        _case("mm_decode", "int8_matmul", m=48, n=10240, k=2560, dtype="bf16", affine="bf16",
              bias=True, residual=False),
        # a short prompt, odd sizes throughout
        _case("mm_odd", "int8_matmul", m=1001, n=1537, k=2003, dtype="fp16", affine="fp32",
              bias=True, residual=True),
        # a long prompt through a square layer that joins the residual stream
        _case("mm_long", "int8_matmul", m=16384, n=4096, k=4096, dtype="bf16", affine="bf16",
              bias=False, residual=True),
    ]


def draw(rng):
    """A case of the ranges above: rows of up to 8192 values, at most 2^25 of
    them, at least eight to a norm; products of up to 2^38 multiplications."""
    def spread(lo, hi):
        return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))

    op = rng.choice(["rms_norm", "rms_norm", "rms_norm_grad", "quantize", "int8_matmul",
                     "int8_matmul", "int8_matmul"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    affine = rng.choice(["fp32", dtype])
    if op == "int8_matmul":
        n = spread(2, 1024) * 16 if rng.random() < 0.6 else spread(17, 16384)
        k = spread(1, 256) * 64 if rng.random() < 0.6 else spread(17, 16384)
        m = spread(1, max(1, min(16384, (1 << 38) // (n * k))))
        return {"op": op, "m": m, "n": n, "k": k, "dtype": dtype, "affine": affine,
                "bias": rng.random() < 0.5, "residual": rng.random() < 0.5}
    n = rng.choice([1, 1, 2, 3, 5])
    c = spread(1, 1024) * 8 if rng.random() < 0.6 else spread(8, 8192)
    l = spread(1, max(1, (1 << 25) // (c * n)))
    d = {"op": op, "n": n, "l": l, "c": c, "dtype": dtype}
    if op == "quantize":
        return d
    d["affine"] = affine
    if op == "rms_norm":
        d.update(residual=rng.random() < 0.6, quantize=rng.random() < 0.5,
                 stats=rng.random() < 0.4)
    else:
        d.update(saved=rng.random() < 0.4, stream=rng.random() < 0.5)
    return d


# ---- the inputs --------------------------------------------------------------
def prepare(case, seed):
    """Activations as residual streams hold them: a spread of its own for each
    channel, a few channels far wider than the rest; gradients of unit spread;
    norm weights around one.  A product's rows are such activations in 8 bits,
    its weights those of an initialised layer, laid out once."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    at = DTYPES[case["affine"]] if "affine" in case else None

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def rows(*shape):
        width = torch.exp(0.3 * randn(shape[-1]))
        wide = torch.rand(shape[-1], generator=gen, device=dev) < 0.01
        width = torch.where(wide, 8.0 * width, width)
        return randn(*shape).mul_(width).to(dt)

    st = {"case": case}
    op = case["op"]
    if op == "int8_matmul":
        m, n, k = case["m"], case["n"], case["k"]
        st["a"], st["sa"] = _encode(rows(m, k).float())
        st["b"], st["sb"] = _encode(randn(n, k) * k ** -0.5)
        if case["bias"]:
            st["bias"] = (0.2 * randn(n)).to(at)
        if case["residual"]:
            st["residual"] = rows(m, n)
        if own:
            import groupnorm_silu_normalization_amd as gn
            with torch.no_grad():
                st["packed"] = gn.pack_int8_weight(gn.Rows8(st["b"], st["sb"], dt))
        return st
    shape = (case["n"], case["l"], case["c"])
    st["x"] = rows(*shape)
    if op == "quantize":
        return st
    st["weight"] = (1.0 + 0.2 * randn(shape[-1])).to(at)
    if op == "rms_norm":
        if case["residual"]:
            st["residual"] = rows(*shape)
        return st
    st["dy"] = randn(*shape).to(dt)
    if case["stream"]:
        st["dh"] = randn(*shape).to(dt)
    h = st["x"].double()
    st["rstd"] = (1.0 / torch.sqrt((h * h).mean(-1) + EPS)).float()
    if case["saved"]:
        st["codes"], st["scales"] = _keep(st.pop("x"))
    return st


# ---- rows in 8 bits, in their plain form -------------------------------------
def _encode(t, rstd=None):
    """Codes and scales of fp32 rows t: the codes are t's share of the row's
    largest magnitude in 127ths (in 64 bits, for the values next to a border),
    the scale a 127th of that magnitude (times rstd)."""
    t = t.double()
    top = t.abs().amax(-1, keepdim=True)
    codes = torch.where(top > 0, t * 127.0 / top, torch.zeros_like(t)).round_().to(torch.int8)
    scales = top.squeeze(-1) / 127.0
    if rstd is not None:
        scales = scales * rstd
    return codes, scales.float()


# the 8-bit checkpoint of a norm's input: blocks of 32 channels
def _blocks(x):
    c = x.shape[-1]
    nb = (c + BLOCK - 1) // BLOCK
    if nb * BLOCK != c:
        x = torch.nn.functional.pad(x, (0, nb * BLOCK - c))
    return x.reshape(*x.shape[:-1], nb, BLOCK)


def _keep(x):
    """Codes and scales; the products by powers of two are exact."""
    v = _blocks(x).double()
    top = v.abs().amax(-1)
    _, e = torch.frexp(top)
    e = torch.where(top > 0, (e + 126).clamp(min=0), torch.zeros_like(e))
    codes = (v * torch.exp2((133 - e).double()).unsqueeze(-1)).round_().clamp_(-127, 127)
    return (codes.to(torch.int8).reshape(*x.shape[:-1], -1)[..., :x.shape[-1]].contiguous(),
            e.to(torch.uint8))


def _kept(codes, scales):
    v = _blocks(codes).double() * torch.exp2(scales.double() - 133).unsqueeze(-1)
    return v.reshape(*codes.shape[:-1], -1)[..., :codes.shape[-1]]


# ---- one pass ----------------------------------------------------------------
def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


def _run_plain(st):
    case = st["case"]
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op == "int8_matmul":
        z = torch.matmul(st["a"].float(), st["b"].float().t())
        z = z * st["sa"].unsqueeze(-1) * st["sb"]
        if case["bias"]:
            z = z + st["bias"].float()
        if case["residual"]:
            z = z + st["residual"].float()
        return [z.to(dt)]
    if op == "quantize":
        codes, scales = _encode(st["x"].float())
        return [(codes.float() * scales.unsqueeze(-1)).to(dt)]
    w = st["weight"].float()
    if op == "rms_norm":
        h = st["x"]
        if case["residual"]:
            h = (h.float() + st["residual"].float()).to(dt)
        hf = h.float()
        rstd = 1.0 / torch.sqrt((hf * hf).sum(-1) / case["c"] + EPS)
        if case["quantize"]:
            codes, scales = _encode(hf * w, rstd)
            out = [(codes.float() * scales.unsqueeze(-1)).to(dt)]
        else:
            out = [(hf * rstd.unsqueeze(-1) * w).to(dt)]
        return out + ([h] if case["residual"] else []) + ([rstd] if case["stats"] else [])
    h = _kept(st["codes"], st["scales"]).float() if case["saved"] else st["x"].float()
    rstd = st["rstd"].unsqueeze(-1)
    dy = st["dy"].float()
    nh = h * rstd
    g = dy * w
    dx = rstd * (g - nh * ((g * nh).sum(-1, keepdim=True) / case["c"]))
    if case["stream"]:
        dx = dx + st["dh"].float()
    return [dx.to(dt), (dy * nh).sum((0, 1)).to(DTYPES[case["affine"]])]


def _run_own(st):
    import groupnorm_silu_normalization_amd as gn

    case = st["case"]
    op, dt = case["op"], DTYPES[case["dtype"]]
    with torch.no_grad():
        if op == "int8_matmul":
            return [gn.int8_matmul(gn.Rows8(st["a"], st["sa"], dt), st["packed"], st.get("bias"),
                                   residual=st.get("residual"))]
        if op == "quantize":
            return [gn.dequantize_rows(gn.quantize_rows(st["x"]))]
        if op == "rms_norm":
            r = gn.rms_norm_rows(st["x"], st["weight"], EPS, residual=st.get("residual"),
                                 quantize=case["quantize"], stats=case["stats"])
            r = list(r) if isinstance(r, tuple) else [r]
            if case["quantize"]:
                r[0] = gn.dequantize_rows(r[0])
            return r
        x = gn.Checkpoint8(st["codes"], st["scales"], dt) if case["saved"] else st["x"]
        return list(gn.rms_norm_rows_backward(st["dy"], x, st["rstd"], st["weight"],
                                              residual_grad=st.get("dh")))


# ---- what a pass cannot do without -------------------------------------------
def work(case):
    op, size = case["op"], BYTES[case["dtype"]]
    asize = BYTES[case["affine"]] if "affine" in case else 0
    if op == "int8_matmul":
        m, n, k = case["m"], case["n"], case["k"]
        b = m * k + n * k + 4 * (m + n) + size * m * n
        b += asize * n * case["bias"] + size * m * n * case["residual"]
        return {"bytes": b, "flops": 2 * m * n * k}
    rows, c = case["n"] * case["l"], case["c"]
    v = rows * c
    eight = v + 4 * rows            # 8-bit rows, written and read again by whoever widens them
    if op == "quantize":
        return {"bytes": 2 * size * v + 2 * eight, "flops": 4 * v}
    if op == "rms_norm":
        b = size * v + asize * c + 4 * rows * case["stats"] + 2 * size * v * case["residual"]
        b += size * v + (2 * eight if case["quantize"] else 0)
        return {"bytes": b, "flops": (8 if case["quantize"] else 5) * v}
    b = 2 * size * v + 4 * rows + 2 * asize * c + size * v * case["stream"]
    b += v + rows * ((c + BLOCK - 1) // BLOCK) if case["saved"] else size * v
    return {"bytes": b, "flops": 10 * v}


# ---- the definition in 64 bits -----------------------------------------------
def exact(case, seed):
    """What ``run`` returns, from the operators' definitions, a few rows at a
    time.  The 8-bit codes are of products rounded to 32 bits, by definition."""
    st = prepare(case, seed)
    op, dt, f64 = case["op"], DTYPES[case["dtype"]], torch.float64

    if op == "int8_matmul":
        m, n = case["m"], case["n"]
        z = torch.zeros(m, n, dtype=f64, device="cuda")
        b = st["b"].to(f64).t().contiguous() * st["sb"].to(f64)
        for i in range(0, m, 2048):
            z[i:i + 2048] = (st["a"][i:i + 2048].to(f64)
                             * st["sa"][i:i + 2048].to(f64)[:, None]) @ b
        if case["bias"]:
            z += st["bias"].to(f64)
        if case["residual"]:
            z += st["residual"].to(f64)
        return [z]

    def by_127(t, r):
        """The values that rows t (times r each) stand for in 8 bits."""
        top = t.abs().max(1).values[:, None]
        step = torch.where(top == 0, torch.ones_like(top), top) / 127
        q = torch.round(t / torch.where(top == 0, torch.ones_like(top), top) * 127)
        # t / top was rounded: a product next to a border is settled by whole numbers
        off = t * 127 - q * top
        q = q + (off > top / 2).to(f64) - (off < -top / 2).to(f64)
        tie = (t * 127 - q * top).abs() == top / 2
        q = torch.where(tie & (q % 2 != 0), q + torch.sign(t * 127 - q * top), q)
        return q * step * (top > 0) * r

    n, l, c = case["n"], case["l"], case["c"]
    flat = {key: v.reshape(n * l, c) for key, v in st.items()
            if key in ("x", "residual", "dy", "dh", "codes")}
    span = max(1, (1 << 24) // c)
    parts = [(i, min(i + span, n * l)) for i in range(0, n * l, span)]

    def whole(pieces):
        return torch.cat(pieces).reshape(n, l, c)

    if op == "quantize":
        return [whole([by_127(flat["x"][i:j].to(f64), 1.0) for i, j in parts])]
    w = st["weight"].to(f64)
    if op == "rms_norm":
        ys, hs, rs = [], [], []
        for i, j in parts:
            h = flat["x"][i:j].to(f64)
            if case["residual"]:
                h = (h + flat["residual"][i:j].to(f64)).to(dt).to(f64)
            r = (h.pow(2).mean(1) + EPS) ** -0.5
            if case["quantize"]:
                ys.append(by_127((h * w).to(torch.float32).to(f64), r[:, None]))
            else:
                ys.append(w * (h * r[:, None]))
            hs.append(h)
            rs.append(r)
        return ([whole(ys)] + ([whole(hs)] if case["residual"] else [])
                + ([torch.cat(rs).reshape(n, l)] if case["stats"] else []))
    rstd = st["rstd"].reshape(n * l, 1).to(f64)
    scales = st["scales"].reshape(n * l, -1) if case["saved"] else None
    dxs, dw = [], torch.zeros(c, dtype=f64, device="cuda")
    for i, j in parts:
        if case["saved"]:
            step = torch.pow(2.0, scales[i:j].to(f64) - 133)
            h = flat["codes"][i:j].to(f64) * step.repeat_interleave(BLOCK, 1)[:, :c]
        else:
            h = flat["x"][i:j].to(f64)
        r, dy = rstd[i:j], flat["dy"][i:j].to(f64)
        g = w * dy
        dx = r * g - r ** 3 * h * (g * h).mean(1, keepdim=True)
        if case["stream"]:
            dx = dx + flat["dh"][i:j].to(f64)
        dxs.append(dx)
        dw += (dy * h * r).sum(0)
    return [whole(dxs), dw]
