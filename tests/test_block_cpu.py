"""A residual block's operators on the CPU: bad arguments are refused before a GPU is touched, by the library and by the
binding; workspaces grow as they should; the float64 references' gradients agree with differences."""

import ctypes

import pytest
import torch

import euler_characteristic_curves_amd as E
from tests.block_bounds import gated_linear, recurrence, residual

FAKE = ctypes.c_void_p(0x1000)   # never dereferenced: validation fails first
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    from euler_characteristic_curves_amd import _lib
    return _lib


def res_fwd(L, x=FAKE, xd=0, b=FAKE, d=0, B=2, S=9, C=8, gate=FAKE, per=0, w=FAKE, bw=FAKE, pd=0, nb=1, scale=1.0, eps=1e-6,
            y=FAKE, z=FAKE, ws=None, wsb=None):
    return L.lib.ecc_residual_norm_fwd(x, xd, b, d, B, S, C, gate, per, w, bw, pd, nb, scale, eps, y, z, None, None)


def res_bwd(L, x=FAKE, xd=0, b=FAKE, d=0, B=2, S=9, C=8, gate=FAKE, per=0, w=FAKE, bw=FAKE, pd=0, nb=1, scale=1.0,
            stats=FAKE, gy=FAKE, gz=FAKE, g=(FAKE,) * 5, ws=FAKE, wsb=1 << 40):
    return L.lib.ecc_residual_norm_bwd(x, xd, b, d, B, S, C, gate, per, w, bw, pd, nb, scale, stats, gy, gz, *g, ws, wsb, None)


@pytest.mark.parametrize("call", [res_fwd, res_bwd], ids=["fwd", "bwd"])
def test_residual_argument_errors(L, call):
    assert call(L, x=None) == L.ECC_E_NULL and b"x is NULL" in L.lib.ecc_last_error()
    for bad in (dict(d=3), dict(d=-1), dict(xd=1), dict(xd=2, d=1), dict(pd=1), dict(xd=1, d=1, pd=2)):
        assert call(L, **bad) == L.ECC_E_DTYPE, bad
    for bad in (dict(B=0), dict(S=0), dict(C=0), dict(C=8193), dict(S=1 << 38), dict(B=32769, per=1)):
        assert call(L, **bad) == L.ECC_E_SHAPE, bad
    # a norm alone has no gate and no norm of a branch
    for bad in (dict(b=None), dict(b=None, gate=None), dict(b=None, gate=None, bw=None)):
        assert call(L, **bad) == L.ECC_E_NULL, bad
    assert call(L, nb=0) == L.ECC_E_VALUE
    for scale in (NAN, INF):
        assert call(L, scale=scale) == L.ECC_E_VALUE
    if call is res_fwd:
        assert call(L, z=None) == L.ECC_E_NULL and call(L, y=None) == L.ECC_E_NULL
        for eps in (-1.0, NAN, INF):
            assert call(L, eps=eps) == L.ECC_E_VALUE
        return
    assert call(L, stats=None) == L.ECC_E_NULL and call(L, gy=None, gz=None) == L.ECC_E_NULL
    assert call(L, g=(None,) * 5) == L.ECC_E_NULL
    assert call(L, gate=None) == L.ECC_E_NULL and call(L, w=None) == L.ECC_E_NULL and call(L, bw=None) == L.ECC_E_NULL
    assert call(L, ws=None) == L.ECC_E_WORKSPACE and call(L, ws=ctypes.c_void_p(0x1010)) == L.ECC_E_WORKSPACE
    need = L.lib.ecc_residual_norm_workspace_bytes(2, 9, 8, 0)
    assert need and call(L, wsb=need - 1) == L.ECC_E_WORKSPACE


def test_residual_workspace(L):
    f = L.lib.ecc_residual_norm_workspace_bytes
    assert f(0, 1, 8, 0) == f(1, 0, 8, 0) == f(1, 1, 0, 0) == f(1, 1, 8193, 0) == f(32769, 1, 8, 1) == 0
    assert f(32769, 1, 8, 0) > 0
    # partial rows: bounded by the launch, and by a 256th of the rows where these are many
    assert f(1, 1 << 18, 1024, 0) <= 1024 * 3 * 1024 * 4 + 256
    assert f(1, 1 << 28, 1024, 0) <= (1 << 28) // 256 * 3 * 1024 * 4 + 256


def glu_fwd(L, x=FAKE, d=0, R=90, C=9, H=10, wg=FAKE, wu=FAKE, act=2, h=FAKE, ws=FAKE, wsb=1 << 40):
    return L.lib.ecc_gated_linear_fwd(x, d, R, C, H, wg, wu, None, None, act, h, ws, wsb, None)


def glu_bwd(L, x=FAKE, d=0, R=90, C=9, H=10, wg=FAKE, wu=FAKE, act=2, h=FAKE, g=(FAKE, FAKE, FAKE, None, None), ws=FAKE,
            wsb=1 << 40):
    return L.lib.ecc_gated_linear_bwd(x, d, R, C, H, wg, wu, None, None, act, h, *g, ws, wsb, None)


@pytest.mark.parametrize("call", [glu_fwd, glu_bwd], ids=["fwd", "bwd"])
def test_gated_linear_argument_errors(L, call):
    for bad in (dict(x=None), dict(wg=None), dict(wu=None), dict(h=None)):
        assert call(L, **bad) == L.ECC_E_NULL, bad
    assert call(L, d=3) == L.ECC_E_DTYPE and call(L, act=4) == L.ECC_E_ACT and call(L, act=-1) == L.ECC_E_ACT
    for bad in (dict(R=0), dict(C=0), dict(H=-1), dict(C=32769), dict(H=32769), dict(R=1 << 38), dict(R=1 << 37, C=1, H=1)):
        assert call(L, **bad) == L.ECC_E_SHAPE, bad
    if call is glu_bwd:
        assert call(L, g=(None,) * 5) == L.ECC_E_NULL
        assert call(L, g=(FAKE,) * 4 + (None,)) == L.ECC_E_NULL  # of a bias that is not there
    assert call(L, ws=None) == L.ECC_E_WORKSPACE
    need = L.lib.ecc_gated_linear_workspace_bytes(90, 9, 10, 0, int(call is glu_bwd))
    assert call(L, wsb=need - 1) == L.ECC_E_WORKSPACE


def test_gated_linear_workspace(L):
    def f(*a):
        return L.lib.ecc_gated_linear_workspace_bytes(*a, 1)

    assert f(0, 8, 8, 0) == f(1, 0, 8, 0) == f(1, 8, 0, 0) == f(1, 8, 8, 3) == 0
    # both projections' gradients, and at most as much again and some shares
    for rows, c, h, e in ((1 << 16, 64, 160, 2), (1 << 14, 1024, 2816, 2), (4000, 333, 877, 0)):
        size = rows * 2 * (h + 63) * (2 if e else 4)
        assert rows * 2 * h * (2 if e else 4) <= f(rows, c, h, e) <= 2 * size + 512 * 256 * 128 * 4
    # forward: nothing, or copies of the operands
    for R, C, want in ((64, 9, 256), (1 << 20, 1024, 256), (65, 9, (65 + 20) * 16 * 4 + 3 * 256)):
        assert L.lib.ecc_gated_linear_workspace_bytes(R, C, 10, 0, 0) <= want


def rec_fwd(L, x=FAKE, f=FAKE, d=0, B=2, T=9, C=8, n=None, h=FAKE, last=FAKE, ws=FAKE, wsb=1 << 40):
    return L.lib.ecc_gated_recurrence_fwd(x, f, d, B, T, C, None, n, h, last, None, ws, wsb, None)


def rec_bwd(L, x=FAKE, f=FAKE, d=0, B=2, T=9, C=8, n=None, saved=FAKE, gh=FAKE, gl=FAKE, g=(FAKE,) * 3, ws=FAKE, wsb=1 << 40):
    return L.lib.ecc_gated_recurrence_bwd(x, f, d, B, T, C, n, saved, gh, gl, *g, ws, wsb, None)


@pytest.mark.parametrize("call", [rec_fwd, rec_bwd], ids=["fwd", "bwd"])
def test_recurrence_argument_errors(L, call):
    assert call(L, x=None) == L.ECC_E_NULL and call(L, f=None) == L.ECC_E_NULL
    assert call(L, d=3) == L.ECC_E_DTYPE
    for bad in (dict(B=0), dict(T=0), dict(C=0), dict(T=1 << 40), dict(C=(1 << 20) + 1), dict(B=1 << 32, T=1, C=1), dict(B=1 << 62)):
        assert call(L, **bad) == L.ECC_E_SHAPE, bad
    assert call(L, ws=None) == L.ECC_E_WORKSPACE
    need = L.lib.ecc_gated_recurrence_workspace_bytes(1, 100000, 8, 0)
    assert need > 256 and call(L, B=1, T=100000, wsb=need - 1) == L.ECC_E_WORKSPACE
    if call is rec_fwd:
        assert call(L, h=None) == L.ECC_E_NULL and call(L, last=None) == L.ECC_E_NULL
    else:
        assert call(L, saved=None) == L.ECC_E_NULL and call(L, gh=None, gl=None) == L.ECC_E_NULL
        assert call(L, g=(None,) * 3) == L.ECC_E_NULL


def test_recurrence_sizes(L):
    ws, saved = L.lib.ecc_gated_recurrence_workspace_bytes, L.lib.ecc_gated_recurrence_saved_bytes
    assert ws(0, 1, 1, 0) == saved(1, 0, 1, 0) == saved(1, 1, 1, 3) == 0
    for B, T, C, d in ((64, 256, 1024, 2), (1, 65536, 96, 0), (12, 8192, 201, 1), (64, 1, 1024, 2), (3, 7, 1, 0)):
        assert saved(B, T, C, d) % (B * C * 4) == 0 and saved(B, T, C, d) >= B * C * 4
        # small beside the features: a state for 32 steps or more, four numbers for every part
        if T >= 64:
            assert saved(B, T, C, d) <= B * C * 4 * (T // 32 + 1) and ws(B, T, C, d) <= 4 * saved(B, T, C, d) + 256


def test_binding_refusals():
    x = torch.zeros(2, 3, 8)
    for fn in (lambda: E.residual_norm(x, x), lambda: E.rms_norm(x), lambda: E.gated_recurrence(x, x),
               lambda: E.gated_linear(x, x[0], x[0])):
        with pytest.raises(ValueError, match="ROCm device"):
            fn()
    with pytest.raises(ValueError, match="act must be"):
        E.gated_linear(x, x[0], x[0], act="tanh")


def along_differences(run, args, grads, outs, got):
    h = 1e-5
    gen = torch.Generator().manual_seed(2)
    for name, t in args.items():
        d = torch.randn(t.shape, generator=gen, dtype=torch.float64)
        side = [run(**{**args, name: t + s * h * d}) for s in (1, -1)]
        slope = sum(float(((side[0][o][0] - side[1][o][0]) * g).sum()) for o, g in zip(outs, grads)) / (2 * h)
        along = float((got[name][0] * d).sum())
        assert abs(slope - along) <= 1e-7 * (1 + float((got[name][0] * d).abs().sum())), name


@pytest.mark.parametrize("per_sample", [False, True])
@pytest.mark.parametrize("norm_branch", [False, True])
def test_residual_reference(per_sample, norm_branch):
    gen = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    args = {"x": rnd(2, 3, 6), "branch": rnd(2, 3, 6), "gate": rnd(2, 6) if per_sample else rnd(6), "weight": rnd(6)}
    if norm_branch:
        args["branch_weight"] = rnd(6)
    kw = dict(norm_branch=norm_branch, scale=0.7, eps=1e-3)
    gy, gz = rnd(2, 3, 6), rnd(2, 3, 6)
    along_differences(lambda **a: residual(**a, **kw), args, (gy, gz), ("y", "z"), residual(**args, **kw, gy=gy, gz=gz))
    alone = residual(args["x"], None, weight=args["weight"], gz=gz)
    along_differences(lambda x, weight: residual(x, None, weight=weight), {"x": args["x"], "weight": args["weight"]}, (gz,),
                      ("z",), alone)


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_gated_linear_reference(act):
    gen = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    args = {"x": rnd(2, 3, 6), "w_gate": rnd(5, 6), "w_up": rnd(5, 6), "b_gate": rnd(5), "b_up": rnd(5)}
    g = rnd(2, 3, 5)
    along_differences(lambda **a: gated_linear(**a, act=act), args, (g,), ("h",), gated_linear(**args, act=act, gh=g))


@pytest.mark.parametrize("ragged", [False, True])
def test_recurrence_reference(ragged):
    gen = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    args = {"x": rnd(3, 7, 4), "gate": 2 * rnd(3, 7, 4), "state": rnd(3, 4)}
    n = torch.tensor([7, 0, 3]) if ragged else None
    g, gl = rnd(3, 7, 4), rnd(3, 4)
    along_differences(lambda **a: recurrence(**a, lengths=n), args, (g, gl), ("h", "last"),
                      recurrence(**args, lengths=n, gh=g, glast=gl))
