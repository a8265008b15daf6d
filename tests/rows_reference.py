"""Layer norm, GroupNorm(+SiLU) gradients and 8-bit checkpoints in 64 bits,
with bounds on how far a 32-bit computation may be from them.

Every bound counts roundings: u = 2^-24 for an fp32 operation, eps/2 of the
output's type for the final one.  A sum of n terms added in any fixed order of
at most `depth` sequential additions per term is off by at most
depth * u * sum|terms|.
"""
import torch

U = 2.0 ** -24
F64 = torch.float64
BLOCK = 32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half the spacing of the type's subnormal numbers."""
    return float(torch.finfo(dtype).smallest_normal) * torch.finfo(dtype).eps / 2


def rounded(v, dtype):
    """The error of rounding v to dtype."""
    return v.abs() * half_step(dtype) + tiny(dtype)


def check(got, want, bound, what):
    got = got.detach().cpu().to(F64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what + ": NaN elsewhere"
    fine = ~torch.isnan(want)
    d = (got - want).abs()[fine]
    b = bound.expand_as(want)[fine]
    bad = ~(d <= b)
    if bad.any():
        i = int(torch.argmax(torch.where(bad, d - b, torch.zeros_like(d))))
        raise AssertionError("%s: %d of %d beyond the bound, worst off by %.3e (bound %.3e, value "
                             "%.6e)" % (what, int(bad.sum()), d.numel(), float(d[i]), float(b[i]),
                                        float(want[fine][i])))


# Sequential additions of a layer norm row's sums: at most 32 values per lane,
# 6 lane steps, 8 waves, and the division and product that follow.
ROW_DEPTH = 48


def layer_norm(x, w, b, eps, dtype):
    """y, mean, rstd and their bounds; x (..., C) as held by the kernel."""
    x = x.cpu().to(F64)
    C = x.shape[-1]
    w = torch.ones(C, dtype=F64) if w is None else w.cpu().to(F64)
    b = torch.zeros(C, dtype=F64) if b is None else b.cpu().to(F64)
    mean = x.sum(-1, keepdim=True) / C
    d = x - mean
    var = (d * d).sum(-1, keepdim=True) / C
    rstd = 1.0 / torch.sqrt(var + eps)
    h = d * rstd
    y = h * w + b
    dm = (ROW_DEPTH * x.abs().mean(-1, keepdim=True) + mean.abs()) * U
    # var: the differences carry dm and a rounding each (dm's first-order part
    # cancels in the sum, its square does not), the sum its depth
    dv = (ROW_DEPTH + 4) * U * var + dm * dm + 2 * dm * U * d.abs().mean(-1, keepdim=True)
    dr = rstd * (0.5 * dv / (var + eps) + 3 * U)
    ey = (w.abs() * (rstd * (dm + U * d.abs()) + d.abs() * dr + 2 * U * h.abs())
          + U * (y.abs() + b.abs()))
    return (y, mean.squeeze(-1), rstd.squeeze(-1),
            1.01 * ey + rounded(y, dtype), 1.01 * dm.squeeze(-1), 1.01 * dr.squeeze(-1))


def layer_norm_backward(dy, x, mean, rstd, w, dtype, wdtype, rows_depth):
    """dx, dw, db and their bounds, of the given fp32 mean and rstd."""
    C = x.shape[-1]
    dy, x = dy.cpu().to(F64), x.cpu().to(F64)
    mean, rstd = mean.cpu().to(F64).unsqueeze(-1), rstd.cpu().to(F64).unsqueeze(-1)
    w = torch.ones(C, dtype=F64) if w is None else w.cpu().to(F64)
    h = (x - mean) * rstd
    g = dy * w
    a = g.sum(-1, keepdim=True) / C
    b = (g * h).sum(-1, keepdim=True) / C
    dx = rstd * (g - a - h * b)
    da = (ROW_DEPTH + 3) * U * g.abs().mean(-1, keepdim=True)
    db_ = (ROW_DEPTH + 6) * U * (g * h).abs().mean(-1, keepdim=True)
    ex = rstd * (4 * U * (g.abs() + a.abs() + (h * b).abs()) + da + h.abs() * db_
                 + 2 * U * (h * b).abs())
    flat = tuple(range(dy.dim() - 1))
    dw, db = (dy * h).sum(flat), dy.sum(flat)
    ew = (rows_depth + 4) * U * (dy * h).abs().sum(flat)
    eb = (rows_depth + 2) * U * dy.abs().sum(flat)
    return (dx, dw, db, 1.01 * ex + rounded(dx, dtype), 1.01 * ew + rounded(dw, wdtype),
            1.01 * eb + rounded(db, wdtype))


def group_norm_backward(dy, x, mean, rstd, w, b, silu, dtype, wdtype, rows_depth):
    """dx, dw, db and their bounds for (N, L, C) rows, of the given (N, G)
    statistics."""
    N, L, C = dy.shape
    G = mean.shape[1]
    Cg = C // G
    dy, x = dy.cpu().to(F64), x.cpu().to(F64)
    w = torch.ones(C, dtype=F64) if w is None else w.cpu().to(F64)
    b = torch.zeros(C, dtype=F64) if b is None else b.cpu().to(F64)
    mu = mean.cpu().to(F64).repeat_interleave(Cg, 1).unsqueeze(1)
    rs = rstd.cpu().to(F64).repeat_interleave(Cg, 1).unsqueeze(1)
    h = (x - mu) * rs
    dt = dy
    e_dt = torch.zeros_like(dy)
    if silu:
        t = h * w + b
        s = torch.sigmoid(t)
        dt = dy * s * (1 + t * (1 - s))
        # t is one fma on x with scale = w*rs and shift = b - mu*scale: each
        # factor rounded once; SiLU's second derivative is at most 1/2.  The
        # exponential's argument is rounded (relative error of s up to |t|u),
        # the exponential, reciprocal and the three operations after them are
        # off by at most 8u together, and s*(1+t*(1-s)) by |t| more of each.
        e_t = U * (3 * (x * w * rs).abs() + 4 * (mu * w * rs).abs() + b.abs() + t.abs())
        e_dt = dy.abs() * (0.5 * e_t + 2 * U * (8 + 2 * t.abs()) * s * (1 + t.abs() * (1 - s)))
    s1, s2 = dt.sum(1), (dt * h).sum(1)
    e_h = 2 * U * h.abs()
    e1 = (e_dt + (rows_depth + 2) * U * dt.abs()).sum(1)
    e2 = (e_dt * h.abs() + dt.abs() * e_h + (rows_depth + 4) * U * (dt * h).abs()).sum(1)
    M = L * Cg

    def over_group(v):
        return (v.reshape(N, G, Cg).sum(2) / M).repeat_interleave(Cg, 1).unsqueeze(1)

    a, bb = over_group(w * s1), over_group(w * s2)
    ea, eb = over_group(w.abs() * (e1 + 2 * U * s1.abs())), over_group(w.abs() * (e2 + 2 * U * s2.abs()))
    dx = rs * (w * dt - a - h * bb)
    ex = rs * (w.abs() * (e_dt + 3 * U * dt.abs()) + ea + 2 * U * a.abs()
               + h.abs() * (eb + 5 * U * bb.abs()) + 3 * U * (a.abs() + (h * bb).abs()))
    dw, db = s2.sum(0), s1.sum(0)
    return (dx, dw, db, 1.01 * ex + rounded(dx, dtype),
            1.01 * (e2.sum(0) + U * dw.abs()) + rounded(dw, wdtype),
            1.01 * (e1.sum(0) + U * db.abs()) + rounded(db, wdtype))


def checkpoint(x):
    """Codes (int64), scale bytes and the values they stand for, of rows
    (..., C): the definition, value by value, in 64 bits."""
    x = x.cpu().to(F64)
    C = x.shape[-1]
    nb = -(-C // BLOCK)
    pad = torch.zeros(*x.shape[:-1], nb * BLOCK - C, dtype=F64)
    v = torch.cat([x, pad], -1).reshape(*x.shape[:-1], nb, BLOCK)
    top = v.abs().amax(-1)
    bad = ~torch.isfinite(v).all(-1)
    top = torch.where(bad, torch.ones_like(top), top)
    _, e = torch.frexp(top)                     # top = m * 2^e, 1/2 <= m < 1
    E = torch.where(top > 0, (e.to(torch.int64) + 126).clamp(min=0), torch.zeros_like(e, dtype=torch.int64))
    step = torch.exp2(E.to(F64) - 133).unsqueeze(-1)
    codes = torch.round(v / step).clamp(-127, 127)
    codes = torch.where(bad.unsqueeze(-1), torch.zeros_like(codes), codes)
    E = torch.where(bad, torch.full_like(E, 255), E)
    val = torch.where(bad.unsqueeze(-1), torch.full_like(v, float("nan")), codes * step)

    def rows(t):
        return t.reshape(*x.shape[:-1], nb * BLOCK)[..., :C]

    return rows(codes).to(torch.int64), E, rows(val)
