"""The operators of a residual block in float64, each with a bound of the error that the kernels' float32 arithmetic and
the rounding of the result may leave.

The bounds count roundings to first order; E = 2^-24 is float32's half step.
"""

import torch

from tests.norm_bounds import E, _vec
from tests.norm_bounds import rounded as _rounded


def rounded(value, bound, dtype):
    """Reference inputs in float64 stand for float32 ones moved by a step."""
    return _rounded(value, bound, torch.float32 if dtype == torch.float64 else dtype)


def residual(x, branch, gate=None, weight=None, branch_weight=None, norm_branch=True, scale=1.0, eps=1e-6, gy=None, gz=None,
             pdtype=torch.float32, ztype=None):
    """{name: (value, bound)} of residual_norm (rms_norm where branch is None) and, with gy or gz, of every gradient.

    Squares are summed in float64, so a factor 1 / rms has one rounding of its own.  Sums along a row: 16 elements a lane
    and a tree over at most 512 lanes, 25 roundings; sums over rows: 16 and 16 of a thread and a tree over at most 256
    rows, 40 roundings, before float64 takes over."""
    B, C = x.shape[0], x.shape[-1]
    ztype = ztype or (x if branch is None else branch).dtype
    xd = x.detach().double().cpu().reshape(B, -1, C)
    w, wb = _vec(weight, C, 1.0), _vec(branch_weight, C, 1.0)
    g = _vec(gate, C, 1.0)
    per_sample = gate is not None and gate.dim() == 2
    if per_sample:
        g = g[:, None]

    def rms(v):
        return 1 / torch.sqrt((v * v).mean(dim=-1, keepdim=True) + eps)

    if branch is None:
        y, y_ = xd, torch.zeros_like(xd)
        rb, hb, n = torch.ones(1, dtype=torch.float64), torch.zeros_like(xd), torch.zeros_like(xd)
        scale = 1.0
    else:
        bd = branch.detach().double().cpu().reshape(xd.shape)
        rb = rms(bd) if norm_branch else torch.ones_like(xd[..., :1])
        hb = bd * rb
        n = hb * wb
        t = g * n
        y = scale * xd + t
        # the factor, its product with the branch, the weight, the gate; the scale's own rounding; the sum
        y_ = 4 * E * t.abs() + E * (scale * xd).abs() + E * y.abs()
    ry = rms(y)
    rel = (y.abs() * y_).sum(dim=-1, keepdim=True) / ((y * y).sum(dim=-1, keepdim=True) + C * eps).clamp_min(1e-300) + 2 * E
    z = y * ry * w
    z_ = z.abs() * (rel + 3 * E) + y_ * ry * w.abs()
    shape = x.shape
    out = {}
    if branch is not None:
        out["y"] = (y.reshape(shape), rounded(y, y_, x.dtype).reshape(shape))
    out["z"] = (z.reshape(shape), rounded(z, z_, ztype).reshape(shape))
    if gy is None and gz is None:
        return out
    zero = torch.zeros_like(xd)
    dy = zero if gy is None else gy.detach().double().cpu().reshape(xd.shape)
    dz = zero if gz is None else gz.detach().double().cpu().reshape(xd.shape)
    hy = y * ry
    hy_ = y_ * ry + hy.abs() * (rel + E)
    rows = (0, 1)

    def summed(name, term, term_, dims, dtype):
        v, b = term.sum(dim=dims), (term_ + 41 * E * term.abs()).sum(dim=dims)
        out[name] = (v, rounded(v, b, dtype))

    summed("weight", dz * hy, dz.abs() * hy_, rows, pdtype)
    q = dz * w
    m = (q * hy).mean(dim=-1, keepdim=True)
    m_ = (q.abs() * hy_ + 30 * E * (q * hy).abs()).mean(dim=-1, keepdim=True)
    inner = q - hy * m
    inner_ = 3 * E * (q.abs() + (hy * m).abs()) + hy_ * m.abs() + hy.abs() * m_
    dY = dy + ry * inner
    dY_ = ry * (inner_ + (rel + 2 * E) * inner.abs()) + E * dY.abs()
    dx = scale * dY
    out["x"] = (dx.reshape(shape), rounded(dx, abs(scale) * dY_ + 2 * E * dx.abs(), x.dtype).reshape(shape))
    if branch is None:
        return out
    summed("gate", dY * n, dY_ * n.abs() + 4 * E * (dY * n).abs(), 1 if per_sample else rows, pdtype)
    dn = dY * g
    dn_ = dY_ * g.abs() + E * dn.abs()
    summed("branch_weight", dn * hb, dn_ * hb.abs() + 3 * E * (dn * hb).abs(), rows, pdtype)
    p = dn * wb
    p_ = dn_ * wb.abs() + E * p.abs()
    db, db_ = p, p_
    if norm_branch:
        m = (p * hb).mean(dim=-1, keepdim=True)
        m_ = (p_ * hb.abs() + 32 * E * (p * hb).abs()).mean(dim=-1, keepdim=True)
        inner = p - hb * m
        inner_ = p_ + E * p.abs() + hb.abs() * m_ + 5 * E * (hb * m).abs()
        db = rb * inner
        db_ = rb * inner_ + 3 * E * db.abs()
    out["branch"] = (db.reshape(shape), rounded(db, db_, branch.dtype).reshape(shape))
    return out
