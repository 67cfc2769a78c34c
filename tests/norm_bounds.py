"""Group norm, activations and their gradients in float64, each with a bound of
the error that float32 arithmetic and the rounding of the result may leave.

The bounds count roundings.  E = 2^-24 is float32's half step; a thread sums at
most about 32 values before float64 takes over, so a sum of float32 terms is
within 32 E of the sum of their magnitudes, and the statistics, joined about a
pivot a few deviations off, within 64 E relative.  Activations are within 2^-20
of their argument's size.  Everything is then propagated to first order.
"""

import numpy as np
import torch

E = 2.0 ** -24
HALF = {torch.float32: E, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -126}


def act_and_slope(u, act):
    if act == "relu":
        return torch.where(u > 0, u, 0 * u), (u > 0).to(u.dtype)
    if act == "silu":
        s = torch.sigmoid(u)
        return u * s, s * (1 + u * (1 - s))
    if act == "gelu":
        c = torch.special.ndtr(u)
        return u * c, c + u * torch.exp(-0.5 * u * u) / np.sqrt(2 * np.pi)
    return u, torch.ones_like(u)


def _vec(t, n, fill):
    return torch.full((n,), fill, dtype=torch.float64) if t is None else t.detach().double().cpu()


def rounded(value, bound, dtype):
    """The bound of `value` once it is rounded to `dtype`."""
    return bound + HALF[dtype] * (value.abs() + bound) + TINY[dtype]


def norm(x, groups, weight, bias, act, eps, grad=None, readout=None, offset=None, pdtype=torch.float32,
         dtype=None):
    """{name: (value, bound)} of the outputs and, with `grad`, of every gradient; tensors on the CPU in float64."""
    B, C = x.shape[0], x.shape[-1]
    dtype = dtype or x.dtype
    D, G = C // groups, groups
    xd = x.detach().double().cpu().reshape(B, -1, G, D)
    S = xd.shape[1]
    N = S * D
    w, b = _vec(weight, C, 1.0).reshape(G, D), _vec(bias, C, 0.0).reshape(G, D)
    mean = xd.mean(dim=(1, 3), keepdim=True)
    d = xd - mean
    rstd = 1 / torch.sqrt((d * d).mean(dim=(1, 3), keepdim=True) + eps)
    a = rstd * w
    u = d * a + b
    du_ = 64 * E * ((d.abs() + mean.abs()) * a.abs() + b.abs())
    y, sl = act_and_slope(u, act)
    dy_ = 1.2 * du_ + 2.0 ** -20 * u.abs()
    out = {}
    shape = x.shape
    if readout is None:
        out["y"] = (y.reshape(shape), rounded(y, dy_, dtype).reshape(shape))
    else:
        r = _vec(readout, C, 0.0).reshape(G, D)
        off = _vec(offset, 1, 0.0)
        f = (y * r).sum(dim=(2, 3)) + off
        fb = ((dy_ + C * E * y.abs()) * r.abs()).sum(dim=(2, 3)) + E * off.abs()
        out["field"] = (f.reshape(shape[:-1]), rounded(f, fb, torch.float32).reshape(shape[:-1]))
    if grad is None:
        return out
    g = grad.detach().double().cpu()
    if readout is None:
        dy = g.reshape(B, S, G, D)
    else:
        df = g.reshape(B, S, 1, 1)
        dy = df * r
        t = (df * y).sum(dim=(0, 1))
        tb = (df.abs() * (dy_ + 32 * E * y.abs())).sum(dim=(0, 1))
        out["readout"] = (t.reshape(C), rounded(t, tb, pdtype).reshape(C))
        out["offset"] = (df.sum().reshape(1), rounded(df.sum(), 32 * E * df.abs().sum(), pdtype).reshape(1))
    q = dy * sl
    if act == "relu":   # on either side of the jump where u is within its error of 0
        qb = dy.abs() * (u.abs() <= du_)
    else:               # slopes of the slopes are below 1
        qb = dy.abs() * (du_ + 2.0 ** -20 * (1 + u.abs()))
    qb = qb + 4 * E * q.abs()
    xhat = d * rstd
    xb = 64 * E * (d.abs() + mean.abs()) * rstd
    A1, A1b = q.sum(dim=1, keepdim=True), (qb + 32 * E * q.abs()).sum(dim=1, keepdim=True)
    A2 = (q * xhat).sum(dim=1, keepdim=True)
    A2b = (qb * xhat.abs() + q.abs() * xb + 32 * E * (q * xhat).abs()).sum(dim=1, keepdim=True)
    for name, v, vb in (("bias", A1, A1b), ("weight", A2, A2b)):
        v, vb = v.sum(dim=(0, 1)).reshape(C), vb.sum(dim=(0, 1)).reshape(C)
        out[name] = (v, rounded(v, vb, pdtype))
    m1, m1b = (A1 * w).sum(dim=3, keepdim=True) / N, (A1b * w.abs()).sum(dim=3, keepdim=True) / N
    m2, m2b = (A2 * w).sum(dim=3, keepdim=True) / N, (A2b * w.abs()).sum(dim=3, keepdim=True) / N
    dx = rstd * (q * w - m1 - xhat * m2)
    parts = (q * w).abs() + m1.abs() + (xhat * m2).abs()
    dxb = rstd * (qb * w.abs() + m1b + xhat.abs() * m2b + xb * m2.abs() + 64 * E * parts)
    out["x"] = (dx.reshape(shape), rounded(dx, dxb, dtype).reshape(shape))
    return out


def worst(got, want):
    """Largest error over its bound; NaN or infinities must agree in place and kind."""
    value, bound = want
    got = got.detach().double().cpu()
    assert got.shape == value.shape
    fin = torch.isfinite(value)
    assert torch.equal(torch.isnan(got), torch.isnan(value))
    assert torch.equal(got[~fin & ~torch.isnan(value)], value[~fin & ~torch.isnan(value)])
    if not fin.any():
        return 0.0
    return float(((got - value).abs() / bound)[fin].max())
