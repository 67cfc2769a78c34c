"""The training operators on the CPU: the library exports what
include/ecc_train.h declares, the binding mirrors its constants, bad arguments
are refused before a GPU is touched, and the float64 reference's gradients
agree with differences."""

import ctypes
import os
import re

import pytest
import torch

import euler_characteristic_curves_amd as E
from tests.norm_bounds import norm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ecc_train.h")
FAKE = ctypes.c_void_p(0x1000)   # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def L():
    from euler_characteristic_curves_amd import _lib
    return _lib


def declared_functions():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return set(re.findall(r"\b(ecc_\w+)\s*\(", text))


def test_exports_match_the_header(L):
    assert declared_functions() == set(L.TRAIN_EXPORTS)
    lib = ctypes.CDLL(L.LIB_PATH)
    for name in L.TRAIN_EXPORTS:
        assert hasattr(lib, name), name


def test_constants_match_the_binding(L):
    text = open(HEADER).read()
    consts = dict(re.findall(r"#define\s+(ECC_\w+)\s+(\d+)\b", text))
    assert len(consts) >= 13
    for name, val in consts.items():
        assert getattr(L, name) == int(val), name
    for code in (L.ECC_E_GROUPS, L.ECC_E_ACT, L.ECC_E_VALUE):
        assert L.lib.ecc_status_string(code) != b"unknown status"


def fwd(L, x=FAKE, dtype=0, B=2, S=9, C=8, G=2, pdtype=0, act=2, eps=1e-5, y=FAKE, stats=FAKE, ws=FAKE, wsb=1 << 40,
        readout=None):
    if readout is not None:
        r = None if readout == "null" else FAKE
        return L.lib.ecc_norm_readout_fwd(x, dtype, B, S, C, G, None, None, r, None, pdtype, act, eps, y, stats, ws, wsb,
                                          None)
    return L.lib.ecc_norm_fwd(x, dtype, B, S, C, G, None, None, pdtype, act, eps, y, stats, ws, wsb, None)


def bwd(L, x=FAKE, dtype=0, B=2, S=9, C=8, G=2, pdtype=0, act=2, stats=FAKE, g=FAKE, gx=FAKE, gw=None, ws=FAKE,
        wsb=1 << 40, readout=None):
    if readout is not None:
        r = None if readout == "null" else FAKE
        return L.lib.ecc_norm_readout_bwd(x, dtype, B, S, C, G, None, None, r, pdtype, act, stats, g, gx, gw, None, None,
                                          None, ws, wsb, None)
    return L.lib.ecc_norm_bwd(x, dtype, B, S, C, G, None, None, pdtype, act, stats, g, gx, gw, None, ws, wsb, None)


@pytest.mark.parametrize("readout", [None, "yes"], ids=["norm", "readout"])
@pytest.mark.parametrize("call", [fwd, bwd], ids=["fwd", "bwd"])
def test_norm_argument_errors(L, call, readout):
    def st(**kw):
        return call(L, readout=readout, **kw)
    assert st(x=None) == L.ECC_E_NULL
    assert b"x is NULL" in L.lib.ecc_last_error()
    assert st(stats=None) == L.ECC_E_NULL
    assert st(dtype=3) == L.ECC_E_DTYPE and st(dtype=-1) == L.ECC_E_DTYPE
    assert st(dtype=0, pdtype=1) == L.ECC_E_DTYPE and st(dtype=2, pdtype=1) == L.ECC_E_DTYPE
    assert st(act=4) == L.ECC_E_ACT and st(act=-1) == L.ECC_E_ACT
    for bad in (dict(B=0), dict(S=0), dict(C=0), dict(B=32769), dict(C=8193, G=1), dict(S=1 << 38)):
        assert st(**bad) == L.ECC_E_SHAPE, bad
    assert st(G=0) == L.ECC_E_GROUPS and st(G=3) == L.ECC_E_GROUPS and st(G=16) == L.ECC_E_GROUPS
    assert st(ws=None) == L.ECC_E_WORKSPACE
    assert st(ws=ctypes.c_void_p(0x1010)) == L.ECC_E_WORKSPACE
    need = L.lib.ecc_norm_workspace_bytes(2, 9, 8, 2)
    assert need > 0 and st(wsb=need - 1) == L.ECC_E_WORKSPACE
    assert b"needs" in L.lib.ecc_last_error()
    if call is fwd:
        assert st(y=None) == L.ECC_E_NULL
        for eps in (-1.0, float("nan"), float("inf")):
            assert st(eps=eps) == L.ECC_E_VALUE
    else:
        assert st(g=None) == L.ECC_E_NULL
        assert st(gx=None) == L.ECC_E_NULL   # no gradient is wanted at all
    if readout:
        assert call(L, readout="null") == L.ECC_E_NULL
        assert st(C=1032, G=2) == L.ECC_E_SHAPE


def test_norm_workspace_bytes(L):
    f = L.lib.ecc_norm_workspace_bytes
    assert f(0, 9, 8, 2) == 0 and f(2, 0, 8, 2) == 0 and f(2, 9, 8, 3) == 0 and f(2, 9, 0, 1) == 0
    assert f(2, 9, 8, 2) < f(2, 1 << 20, 8, 2)
    # the launch, and with it the workspace, stops growing with the features
    assert f(1, 1 << 26, 64, 8) == f(1, 1 << 24, 64, 8)


def test_binding_refusals():
    x = torch.zeros(2, 3, 4, 8)
    for fn in (lambda: E.group_norm_act(x, 2), lambda: E.group_norm_readout(x, 2, None, None, torch.zeros(8))):
        with pytest.raises(ValueError, match="ROCm device"):
            fn()


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("readout", [False, True])
def test_reference_gradients_agree_with_differences(act, readout):
    gen = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    v = {"x": rnd(2, 3, 4, 6), "weight": 1 + 0.2 * rnd(6), "bias": 0.2 * rnd(6)}
    if readout:
        v.update(readout=rnd(6), offset=rnd(1))
    grad = rnd(2, 3, 4) if readout else rnd(2, 3, 4, 6)

    def outs(v, g=None):
        return norm(v["x"], 3, v["weight"], v["bias"], act, 1e-3, g, v.get("readout"), v.get("offset"),
                    dtype=torch.float32)

    got = outs(v, grad)
    h = 1e-5
    for name, t in v.items():
        d = rnd(*t.shape)
        side = [outs({**v, name: t + s * h * d})["field" if readout else "y"][0] for s in (1, -1)]
        slope = float(((side[0] - side[1]) * grad).sum()) / (2 * h)
        along = float((got[name][0] * d).sum())
        # float64 rounding over the step (1e-16 / 1e-5 a term, some hundred terms) and the step's square
        assert abs(slope - along) <= 1e-7 * (1 + float((got[name][0] * d).abs().sum())), name


def orth(L, g=FAKE, dtype=0, B=2, rows=30, cols=40, steps=5, eps=1e-7, co=(3.4445, -4.775, 2.0315), out=FAKE, ws=FAKE,
         wsb=1 << 40):
    return L.lib.ecc_orthogonalize(g, dtype, B, rows, cols, steps, eps, *co, out, ws, wsb, None)


def muon(L, g=FAKE, dtype=0, B=2, rows=30, cols=40, steps=5, eps=1e-7, co=(3.4445, -4.775, 2.0315), out=FAKE, ws=FAKE,
         wsb=1 << 40, buffer=FAKE, lr=0.1, momentum=0.9, decay=0.0, scale=1.0):
    return L.lib.ecc_muon_step(out, 0, g, dtype, buffer, B, rows, cols, lr, momentum, 1, decay, scale, steps, eps, *co,
                               ws, wsb, None)


@pytest.mark.parametrize("call", [orth, muon], ids=["orth", "muon"])
def test_matrix_argument_errors(L, call):
    assert call(L, g=None) == L.ECC_E_NULL and call(L, out=None) == L.ECC_E_NULL
    assert call(L, dtype=3) == L.ECC_E_DTYPE
    for bad in (dict(B=0), dict(rows=0), dict(cols=-1), dict(rows=32769), dict(cols=32769), dict(B=32769),
                dict(B=32768, rows=32768, cols=32768)):
        assert call(L, **bad) == L.ECC_E_SHAPE, bad
    nan, inf = float("nan"), float("inf")
    for bad in (dict(steps=0), dict(steps=65), dict(eps=-1.0), dict(eps=nan), dict(co=(nan, 0, 0)), dict(co=(1, inf, 0)),
                dict(co=(20.0, 0.0, 0.0)), dict(co=(3.0, 0.0, 0.0))):
        assert call(L, **bad) == L.ECC_E_VALUE, bad
        assert L.lib.ecc_last_error()
    assert call(L, ws=None) == L.ECC_E_WORKSPACE
    assert call(L, wsb=L.lib.ecc_orth_workspace_bytes(2, 30, 40) - 1) == L.ECC_E_WORKSPACE
    assert L.lib.ecc_orth_workspace_bytes(0, 30, 40) == 0 and L.lib.ecc_orth_workspace_bytes(1, 0, 40) == 0
    if call is muon:
        assert call(L, buffer=None) == L.ECC_E_NULL
        for bad in (dict(lr=nan), dict(momentum=inf), dict(decay=nan), dict(scale=inf)):
            assert call(L, **bad) == L.ECC_E_VALUE, bad
