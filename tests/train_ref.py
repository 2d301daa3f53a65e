"""Plain float64 forms of the training-step operators, and error bounds.

Every bound counts roundings. U = 2^-24 is half an fp32 step; a sum of terms
added along a chain of at most D additions is off by at most about
D U sum|terms|; an output in type t adds half a step of t, eps(t) / 2
relative to the value (fp32: U)."""
import torch

U = 2.0 ** -24
F8 = torch.float64


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def close(got, want, tol, what=""):
    """|got - want| <= tol element by element; infinities and NaN in the same places."""
    got, want = got.to(F8), want.to(F8)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fin = torch.isfinite(want)
    assert torch.equal(fin, torch.isfinite(got)), what
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    err = (got - want).abs()[fin]
    tol = (tol + torch.zeros_like(want))[fin]
    bad = err > tol
    assert not bool(bad.any()), (what, float(err[bad].max()), float(tol[bad].min()), int(bad.sum()))


# Chains of a row's sums: at most 64 elements per thread, 5 shuffle steps, 16 warps.
D_ROW = 64 + 5 + 16


def layernorm(x, w, bias, eps):
    """(y, mean, rstd) and their bounds, before y's own rounding."""
    x8 = x.to(F8)
    w8 = torch.ones(x.shape[1], dtype=F8, device=x.device) if w is None else w.to(F8)
    b8 = torch.zeros(x.shape[1], dtype=F8, device=x.device) if bias is None else bias.to(F8)
    mean = x8.mean(1, keepdim=True)
    c = x8 - mean
    var = c.square().mean(1, keepdim=True)
    rstd = 1.0 / torch.sqrt(var + eps)
    y = c * rstd * w8 + b8
    e_mean = (D_ROW + 2) * U * x8.abs().mean(1, keepdim=True)
    # the squares are of values that are all off by e_mean and each by one rounding
    e_var = (D_ROW + 4) * U * var + 2 * e_mean * c.abs().mean(1, keepdim=True) * 2 * U + (1.001 * e_mean) ** 2
    rel = 0.5 * e_var / (var + eps) + 4 * U
    rel = 1.01 * rel + rel ** 2
    e_y = w8.abs() * rstd * (1 + rel) * (e_mean + U * c.abs() + c.abs() * rel) + 4 * U * (y.abs() + 2 * b8.abs())
    return (y, mean[:, 0], rstd[:, 0]), (e_y, e_mean[:, 0], (rel * rstd)[:, 0])


def layernorm_grad(dy, x, w, mean, rstd):
    """(dx, dw, dbias) for the mean and rstd given, and their bounds, before dx's own rounding."""
    x8, dy8 = x.to(F8), dy.to(F8)
    w8 = torch.ones(x.shape[1], dtype=F8, device=x.device) if w is None else w.to(F8)
    r = rstd.to(F8)[:, None]
    xh = (x8 - mean.to(F8)[:, None]) * r
    g = dy8 * w8
    s1, s2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = r * (g - s1 - xh * s2)
    e1 = (D_ROW + 4) * U * g.abs().mean(1, keepdim=True)
    e2 = (D_ROW + 8) * U * (g * xh).abs().mean(1, keepdim=True)
    e_dx = r * (e1 + xh.abs() * e2 + 6 * U * (g.abs() + s1.abs() + (xh * s2).abs()))
    # columns: at most n / 256 rows per thread beyond the first, then 8 warps, 5
    # shuffle steps, 60 partial rows per thread and 8 threads
    chain = x.shape[0] / 256 + 100
    e_dw = (chain + 4) * U * (dy8 * xh).abs().sum(0)
    e_db = chain * U * dy8.abs().sum(0)
    return (dx, (dy8 * xh).sum(0), dy8.sum(0)), (e_dx, e_dw, e_db)


def normalize(x):
    x8 = x.to(F8)
    return x8 / x8.square().sum(1, keepdim=True).clamp(min=1e-12).sqrt()


def normalize_grad(dy, x):
    """dx and its bound, before dx's own rounding."""
    x8, g = x.to(F8), dy.to(F8)
    sq = x8.square().sum(1, keepdim=True)
    clamped = sq < 1e-12
    norm = sq.clamp(min=1e-12).sqrt()
    inner = torch.where(clamped, torch.zeros_like(sq), (x8 * g).sum(1, keepdim=True))
    dx = (g - x8 * inner / norm ** 2) / norm
    mag = (x8 * g).abs().sum(1, keepdim=True) / norm ** 2
    e = ((D_ROW + 4) * U * x8.abs() * mag * 2 + 4 * U * (g.abs() + (x8 * inner).abs() / norm ** 2)
         + (D_ROW + 4) * U * (g.abs() + x8.abs() * mag)) / norm
    return dx, e
