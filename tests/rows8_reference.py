"""Root-mean-square norm, rows in 8 bits and their matrix product in 64 bits,
with bounds on how far a 32-bit computation may be from them (roundings counted
as in rows_reference)."""
import torch

from rows_reference import F64, ROW_DEPTH, U, rounded


def codes_of(t):
    """Codes (int64) and largest magnitudes of rows t of fp32 values, by whole
    multiples of the magnitudes: |127 t - q top| <= top / 2, ties to even."""
    t = t.to(F64)
    bad = ~torch.isfinite(t).all(-1, keepdim=True)
    t = torch.where(bad, torch.zeros_like(t), t)
    top = t.abs().amax(-1, keepdim=True)
    safe = torch.where(top > 0, top, torch.ones_like(top))
    # the quotient of 31-bit by 24-bit numbers, rounded to 53 bits, is a half
    # only where it is exactly one: it is 2^-26 away from it otherwise
    q = torch.round(t * 127 / safe)
    top = torch.where(bad, torch.full_like(top, float("nan")), top)
    return q.to(torch.int64), top.squeeze(-1)


def quantize(x):
    """Codes, scales and the scales' bounds."""
    q, top = codes_of(x.cpu().float())
    s = top / 127
    return q, s, s.abs() * U + 2.0 ** -150


def rms_norm(x, w, eps, dtype, residual=None):
    """h, y, rstd, codes, scales and the bounds of y, rstd and scales."""
    h = x.cpu()
    if residual is not None:
        h = (h.float() + residual.cpu().float()).to(dtype)
    hd = h.to(F64)
    C = hd.shape[-1]
    w = torch.ones(C, dtype=F64) if w is None else w.cpu().to(F64)
    ms = (hd * hd).sum(-1, keepdim=True) / C
    rstd = 1.0 / torch.sqrt(ms + eps)
    y = hd * rstd * w
    # squares and their sum, the division, eps, root and reciprocal
    dr = rstd * (0.5 * ((ROW_DEPTH + 2) * U * ms / (ms + eps) + U) + 3 * U)
    ey = w.abs() * hd.abs() * dr + 3 * U * y.abs()
    q, top = codes_of((hd * w).float())
    s = top.unsqueeze(-1) / 127 * rstd
    es = top.unsqueeze(-1) / 127 * dr + 3 * U * s.abs() + 2.0 ** -149
    return (h, y, rstd.squeeze(-1), q, s.squeeze(-1), 1.01 * ey + rounded(y, dtype),
            1.01 * dr.squeeze(-1), 1.01 * es.squeeze(-1))


def rms_norm_backward(dy, h, rstd, w, dh, dtype, wdtype, rows_depth):
    """dx, dw and their bounds, of the given fp32 rstd."""
    C = dy.shape[-1]
    dy, h, r = dy.cpu().to(F64), h.cpu().to(F64), rstd.cpu().to(F64).unsqueeze(-1)
    w = torch.ones(C, dtype=F64) if w is None else w.cpu().to(F64)
    n = h * r
    g = dy * w
    b = (g * n).sum(-1, keepdim=True) / C
    dx = r * (g - n * b)
    db = (ROW_DEPTH + 6) * U * (g * n).abs().mean(-1, keepdim=True)
    ex = r * (4 * U * (g.abs() + (n * b).abs()) + n.abs() * db)
    if dh is not None:
        dx = dx + dh.cpu().to(F64)
        ex = ex + U * dx.abs()
    flat = tuple(range(dy.dim() - 1))
    dw = (dy * n).sum(flat)
    ew = (rows_depth + 4) * U * (dy * n).abs().sum(flat)
    return dx, dw, 1.01 * ex + rounded(dx, dtype), 1.01 * ew + rounded(dw, wdtype)


def matmul(a, sa, b, sb, bias, residual, dtype):
    """z and its bound: the sum is exact, its conversion, two scales and the
    additions of bias and residual round."""
    # sums of at most 2^30 are exact in 64 bits
    acc = a.cpu().to(F64) @ b.cpu().to(F64).t()
    p = acc * sa.cpu().to(F64).unsqueeze(-1) * sb.cpu().to(F64)
    z = p
    e = 4 * U * p.abs()
    if bias is not None:
        z = z + bias.cpu().to(F64)
        e = e + U * z.abs()
    if residual is not None:
        z = z + residual.cpu().to(F64)
        e = e + U * z.abs()
    return z, 1.01 * e + rounded(z, dtype)
