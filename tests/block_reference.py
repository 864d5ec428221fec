"""Definitions in 64 bits of the operators around the projections, and what their outputs may be off.

U is half a step of fp32 at 1, half_step(t) that of an output type: a kernel rounds its output once
(half_step, relative) after fp32 arithmetic, whose bounds the callers count in U.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
FLOATS = (torch.bfloat16, torch.float16, torch.float32)
EPS = 1e-6


def half_step(t) -> float:
    return torch.finfo(t).eps / 2


def allowed(ref, dtype, fp32_error):
    """Bound of |output - ref|: the one rounding to dtype (of the value and of its error; absolute below
    the smallest normal number) on top of the error of the fp32 arithmetic."""
    f = torch.finfo(dtype)
    h = 0.0 if dtype == torch.float32 else f.eps / 2
    return (ref.abs() + fp32_error) * h + fp32_error + (f.smallest_normal * f.eps if h else 2.0 ** -149)


def assert_within(got, ref, bound):
    assert got.shape == ref.shape
    off = (got.double() - ref).abs()
    bad = ~(off <= bound)
    assert not bool(bad.any()), (
        f"{int(bad.sum())} of {bad.numel()} values outside: worst {float((off / bound).nan_to_num(float('inf')).max()):.3g} "
        f"times the bound")


def group_rows(p, rows, M):
    """Row m of the result is row m // rows of p (double)."""
    return p.double().reshape(-1, p.shape[-1])[torch.arange(M, device=p.device) // rows]


def layer_norm(X, weight, bias, rows, offset, eps=EPS):
    """(y, xhat, mean, rstd, bound of y's fp32 error).

    A sum of K <= 16384 values in any tree whose longest chain of additions is 128 is within
    128 U sum|v|; the mean's error then counts in x - mean, the variance's half in rstd, and the
    last operations a few U each."""
    x = X.double()
    M, K = x.shape
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + eps)
    xhat = d * rstd
    w = torch.ones_like(x) if weight is None else offset + group_rows(weight, rows, M)
    b = torch.zeros_like(x) if bias is None else group_rows(bias, rows, M)
    shift = 130 * U * x.abs().mean(1, keepdim=True) * rstd
    # offset + weight rounds once, relative to their sum of magnitudes
    wa = w.abs() if weight is None else abs(offset) + group_rows(weight, rows, M).abs()
    xerr = shift * (1 + xhat.abs()) + 140 * U * xhat.abs()
    y = xhat * w + b
    return y, xhat, mean[:, 0], rstd[:, 0], xerr * wa + 4 * U * (xhat.abs() * wa + b.abs())


def layer_norm_backward(dY, X, mean, rstd, weight, rows, groups, offset):
    """dX, dweight, dbias from the fp32 statistics, and the bounds of their fp32 errors: row sums as
    above, column sums of n rows within n U sum|v| in whatever order."""
    x, dy = X.double(), dY.double()
    M, K = x.shape
    r = rstd.double()[:, None]
    xhat = (x - mean.double()[:, None]) * r
    w = torch.ones_like(x) if weight is None else offset + group_rows(weight, rows, M)
    wa = w.abs() if weight is None else abs(offset) + group_rows(weight, rows, M).abs()
    g, ga = dy * w, dy.abs() * wa
    m0, m1 = g.mean(1, keepdim=True), (g * xhat).mean(1, keepdim=True)
    dx = r * (g - m0 - xhat * m1)
    dxe = 140 * U * r * (ga + ga.mean(1, keepdim=True) + xhat.abs() * (ga * xhat.abs()).mean(1, keepdim=True))
    pad = groups * rows - M
    grouped = lambda v: torch.nn.functional.pad(v, (0, 0, 0, max(0, pad))).reshape(groups, -1, K)  # noqa: E731
    dw, db = grouped(dy * xhat).sum(1), grouped(dy).sum(1)
    n = min(rows, M) + 8
    # xhat itself is within 2 U of what the statistics say, plus the rounding of x - mean
    xa = xhat.abs() + 0 * r
    return (dx, dw, db), (dxe, (n + 4) * U * grouped(dy.abs() * xa).sum(1), n * U * grouped(dy.abs()).sum(1))


def quantize_rows(X, col_scale=None):
    """int8 rows and fp32 scales, exactly: xhat rounded to fp32, the quotient's rounding decided in 64 bits."""
    x = X.double()
    if col_scale is not None:
        x = (x * col_scale.double()).float().double()
    top = x.abs().amax(1)
    bad = ~torch.isfinite(top)
    safe = torch.where((top == 0) | bad, torch.ones_like(top), top)
    q = torch.round(127 * x / safe[:, None])
    q = torch.where(bad[:, None] | (top == 0)[:, None], torch.zeros_like(q), q)
    scale = (top / 127).float()  # in 64 bits first: torch divides fp32 by a number through its reciprocal on a GPU
    return q.to(torch.int8), torch.where(bad, torch.full_like(scale, float("nan")), scale)


def i8_product(xq, x_scale, wq, w_scale, bias):
    """Y and the bound of its fp32 error: the sum's conversion, two scalings and the bias round once each."""
    p = (xq.double() @ wq.double().t()) * x_scale.double()[:, None] * w_scale.double()
    b = torch.zeros_like(p) if bias is None else bias.double().expand_as(p)
    return p + b, 4 * U * (p.abs() + b.abs())


def cos_sin(pos, pairs, theta, shared):
    """cos, sin and angle of every token and pair, in 64 bits."""
    P = sum(pairs)
    cols = []
    for a, n in enumerate(pairs):
        for i in range(n):
            power = len(cols) / P if shared else i / n
            cols.append(pos[:, a].double() * theta ** -power)
    angle = torch.stack(cols, 1)
    return angle.cos(), angle.sin(), angle


def turn_error(angle):
    """Bound of the error of cos and sin: the reduced angle (at most pi) rounds to fp32 (2^-23), the fp32
    sine and cosine are within 2^-23, and the fp64 frequency within 2^-50 of its value."""
    return 2.0 ** -22 + 2.0 ** -50 * angle.abs()


def rope(x, cos, sin, angle, halves, inverse):
    """Rotated heads and the bound of their fp32 error."""
    P = cos.shape[1]
    s = -sin if inverse else sin
    v = x.double()
    out, err = v.clone(), torch.zeros_like(v)
    a, b = (slice(0, P), slice(P, 2 * P)) if halves else (slice(0, 2 * P, 2), slice(1, 2 * P, 2))
    u, w = v[..., a], v[..., b]
    c, s, e = cos[:, None], s[:, None], turn_error(angle)[:, None]
    out[..., a], out[..., b] = u * c - w * s, w * c + u * s
    err[..., a] = err[..., b] = (u.abs() + w.abs()) * (e + 3 * U)
    return out, err
