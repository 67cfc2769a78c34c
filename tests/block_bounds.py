"""The operators of a residual block in float64, each with a bound of the error that the kernels' float32 arithmetic and
the rounding of the result may leave.

The bounds count roundings to first order; E = 2^-24 is float32's half step.
"""

import torch

from tests.norm_bounds import HALF, TINY, E, _vec, act_and_slope
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


def recurrence(x, gate, state=None, lengths=None, gh=None, glast=None):
    """{name: (value, bound)} of gated_recurrence and, with gh or glast, of every gradient.

    m, the smaller of k and 1 - k, is off by (3 |gate| + 8) E relative: half a step of the exponent's two factors, |gate| E
    each and doubled by the sum 1 + e at most half, and a step or half of one for the exponential, the sum, the reciprocal
    and the product.  A step adds that share of what m multiplies, |x| + |h| at most, and roundings of the state: its own,
    those of the run that it is part of and of the joins, 8 E together.  Errors pass on as states do, by k; magnitudes H
    of states are those of the sums of absolute values."""
    xd, f = x.detach().double().cpu(), gate.detach().double().cpu()
    B, T, C = xd.shape
    n = torch.full((B,), T) if lengths is None else lengths.cpu().clamp(0, T)
    inside = (torch.arange(T)[None] < n[:, None])[..., None]
    xd, f = torch.where(inside, xd, 0.0), torch.where(inside, f, 0.0)
    k, blend = torch.where(inside, torch.sigmoid(f), 1.0), torch.where(inside, torch.sigmoid(-f), 0.0)
    m = torch.minimum(k, blend)
    rel = (3 * f.abs() + 8) * E
    h = torch.zeros(B, C, dtype=torch.float64) if state is None else state.detach().double().cpu()
    H, err = h.abs(), torch.zeros_like(h)
    before, before_, out, out_ = (torch.empty_like(xd) for _ in range(4))
    for t in range(T):
        before[:, t], before_[:, t] = h, err
        local = (rel[:, t] + 2 * E) * m[:, t] * (xd[:, t].abs() + H)
        h = k[:, t] * h + blend[:, t] * xd[:, t]
        H = k[:, t] * H + blend[:, t] * xd[:, t].abs()
        err = k[:, t] * err + local + 8 * E * H + 2.0 ** -126
        out[:, t], out_[:, t] = h, err
    res = {"h": (torch.where(inside, out, 0.0), torch.where(inside, rounded(out, out_, x.dtype), 0.0) + 1e-300),
           "last": (h, err + 1e-300)}
    if gh is None and glast is None:
        return res
    d = torch.zeros_like(xd) if gh is None else torch.where(inside, gh.detach().double().cpu(), 0.0)
    e = torch.zeros(B, C, dtype=torch.float64) if glast is None else glast.detach().double().cpu()
    G, e_ = e.abs(), torch.zeros_like(e)
    D, D_ = torch.empty_like(xd), torch.empty_like(xd)
    for t in range(T - 1, -1, -1):
        G = d[:, t].abs() + G
        D[:, t] = d[:, t] + e
        D_[:, t] = e_ + 2 * E * G
        local = (rel[:, t] + 2 * E) * m[:, t] * G + 8 * E * k[:, t] * G
        e, G = k[:, t] * D[:, t], k[:, t] * G
        e_ = k[:, t] * D_[:, t] + local + 2.0 ** -126
    dx = blend * D
    dx_ = blend * D_ + (rel + 2 * E) * m * D.abs() + 2 * E * dx.abs()
    diff, kb = before - xd, k * blend
    df = D * diff * kb
    df_ = kb * diff.abs() * D_ + kb * D.abs() * (before_ + E * diff.abs()) + df.abs() * (2 * rel + 6 * E)
    for name, v, b in (("x", dx, dx_), ("gate", df, df_)):
        res[name] = (torch.where(inside, v, 0.0), torch.where(inside, rounded(v, b, x.dtype), 0.0) + 1e-300)
    if state is not None:
        res["state"] = (e, e_ + 1e-300)
    return res


def gated_linear(x, w_gate, w_up, b_gate=None, b_up=None, act="silu", gh=None):
    """{name: (value, bound)} of gated_linear and, with gh, of every gradient.

    A sum of n products in float32 has at most n roundings of partial sums and, from float32 elements, one of every
    product: n + 1 roundings of the sum of magnitudes.  The gradients of the projections are rounded to the element type
    before they are multiplied (up to 512 rows in two parts); the biases' are not, and are summed over at most 64 rows a lane, two waves and the tiles
    in float64: 68 roundings."""
    dt = x.dtype if x.dtype != torch.float64 else torch.float32
    xd = x.detach().double().cpu().reshape(-1, x.shape[-1])
    wg, wu = w_gate.detach().double().cpu(), w_up.detach().double().cpu()
    (n, C), F = xd.shape, wg.shape[0]
    bg, bu = _vec(b_gate, F, 0.0), _vec(b_up, F, 0.0)

    def project(w, b):
        return xd @ w.T + b, (C + 1) * E * (xd.abs() @ w.abs().T + b.abs())

    (a, a_), (b, b_) = project(wg, bg), project(wu, bu)
    y, sl = act_and_slope(a, act)
    y_ = 1.2 * a_ + 2.0 ** -20 * a.abs()
    h = y * b
    h_ = y.abs() * b_ + b.abs() * y_ + y_ * b_ + E * h.abs()
    shape = (*x.shape[:-1], F)
    out = {"h": (h.reshape(shape), rounded(h, h_, dt).reshape(shape))}
    if gh is None:
        return out
    g = gh.detach().double().cpu().reshape(n, F)
    sl_ = (a.abs() <= a_).double() if act == "relu" else a_ + 2.0 ** -20 * (1 + a.abs())
    da, db = g * b * sl, g * y
    da_ = g.abs() * (b.abs() * sl_ + sl.abs() * b_ + b_ * sl_) + 3 * E * da.abs()
    db_ = g.abs() * y_ + 2 * E * db.abs()
    for name, v, b in (("b_gate", da, da_), ("b_up", db, db_)):
        s, s_ = v.sum(0), (b + 68 * E * v.abs()).sum(0)
        out[name] = (s, rounded(s, s_, dt))
    if dt != torch.float32 and n <= 512:  # in two parts: the second one's rounding is a half step of a half step
        ra, rb = (v_ + HALF[dt] ** 2 * v.abs() + TINY[dt] for v, v_ in ((da, da_), (db, db_)))
    else:
        ra, rb = rounded(da, da_, dt), rounded(db, db_, dt)
    dx = da @ wg + db @ wu
    dx_ = ra @ wg.abs() + rb @ wu.abs() + (2 * F + 1) * E * (da.abs() @ wg.abs() + db.abs() @ wu.abs())
    out["x"] = (dx.reshape(x.shape), rounded(dx, dx_, dt).reshape(x.shape))
    for name, v, r in (("w_gate", da, ra), ("w_up", db, rb)):
        s, s_ = v.T @ xd, r.T @ xd.abs() + (n + 1) * E * (v.abs().T @ xd.abs())
        out[name] = (s, rounded(s, s_, dt))
    return out
