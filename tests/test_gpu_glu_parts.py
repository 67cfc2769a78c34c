"""The gradients of the projections between gated_linear's products, in 16 bits: what dx and dW lose by them is far below
the results' own rounding at every size, and float16's range does not end where the results' does not."""

import pytest
import torch

import euler_characteristic_curves_amd as E
from tests.block_bounds import gated_linear
from tests.gpu_util import banner, need_gpu
from tests.norm_bounds import HALF, _vec, act_and_slope, rounded, worst
from tests.norm_bounds import E as STEP
from tests.test_gpu_glu import check_all
from tests.test_gpu_glu import make as make_all

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
NAMES = ("x", "w_gate", "w_up", "b_gate", "b_up")


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def make(rows, C, F, dtype, scale=1.0, bias=True, seed=0):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    t = {"x": rnd(rows, C), "w_gate": rnd(F, C) / C ** 0.5, "w_up": rnd(F, C) / C ** 0.5}
    if bias:
        t.update(b_gate=0.3 * rnd(F), b_up=0.3 * rnd(F))
    # of one sign mostly, so that sums over rows are of the size of their terms
    gh = (scale * (0.25 + torch.rand(rows, F, generator=gen))).to(dtype)
    return {k: v.to(dtype) for k, v in t.items()}, gh


def gradients(t, gh, act):
    d = {k: v.cuda().requires_grad_() for k, v in t.items()}
    out = E.gated_linear(*(d.get(k) for k in NAMES), act=act)
    return dict(zip(d, torch.autograd.grad(out, list(d.values()), gh.cuda())))


def bounds(t, gh, act):
    """{name: (value, bound)} of dx and both dW: da and db in two parts, the second one's rounding a half step of a half
    step, and below float16's range 2^-32 (the second part is kept 2^7 times as large).  The rest is as in
    block_bounds.gated_linear."""
    dt = gh.dtype
    xd, wg, wu = (t[k].double() for k in ("x", "w_gate", "w_up"))
    (n, C), F = xd.shape, wg.shape[0]
    bg, bu = _vec(t.get("b_gate"), F, 0.0), _vec(t.get("b_up"), F, 0.0)
    a, b = xd @ wg.T + bg, xd @ wu.T + bu
    a_, b_ = ((C + 1) * STEP * (xd.abs() @ w.abs().T + v.abs()) for w, v in ((wg, bg), (wu, bu)))
    y, sl = act_and_slope(a, act)
    y_ = 1.2 * a_ + 2.0 ** -20 * a.abs()
    sl_ = a_ + 2.0 ** -20 * (1 + a.abs())
    g = gh.double()
    da, db = g * b * sl, g * y
    da_ = g.abs() * (b.abs() * sl_ + sl.abs() * b_ + b_ * sl_) + 3 * STEP * da.abs()
    db_ = g.abs() * y_ + 2 * STEP * db.abs()
    tiny = 2.0 ** -32 if dt == F16 else 2.0 ** -126
    ra, rb = (v_ + HALF[dt] ** 2 * v.abs() + tiny for v, v_ in ((da, da_), (db, db_)))
    # parts are products of their own: twice as many terms
    dx = da @ wg + db @ wu
    dx_ = ra @ wg.abs() + rb @ wu.abs() + (4 * F + 1) * STEP * (da.abs() @ wg.abs() + db.abs() @ wu.abs())
    out = {"x": (dx, rounded(dx, dx_, dt))}
    for name, v, r in (("w_gate", da, ra), ("w_up", db, rb)):
        s, s_ = v.T @ xd, r.T @ xd.abs() + (2 * n + 1) * STEP * (v.abs().T @ xd.abs())
        out[name] = (s, rounded(s, s_, dt))
    return out


# up to 512 rows and beyond, in small tiles and large, narrow sums, sums in shares
SHAPES = [(512, 48, 24), (513, 48, 24), (600, 33, 17), (2050, 136, 24), (5000, 64, 40), (4100, 40, 9), (3000, 72, 1610)]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_two_parts_at_every_size(shape, act, dtype):
    banner("glu parts", shape, act, dtype)
    t, gh = make(*shape, dtype, bias=act == "silu", seed=sum(shape))
    want, got = bounds(t, gh, act), gradients(t, gh, act)
    for name in want:
        ratio = worst(got[name], want[name])
        assert ratio <= 1, (name, ratio)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("shape", [(700, 64, 96), (4500, 64, 160), (2048, 512, 1408)], ids=lambda s: "x".join(map(str, s)))
def test_error_is_the_results_own_rounding(shape, dtype):
    """Root mean squares: the second part leaves HALF of a rounding, the float32 sums some sqrt(n) 2^-24 of the terms,
    2e-5 of HALF / sqrt 3 = 2.8e-4 at most; both in quadrature are below a hundredth of the rounding."""
    banner("glu rounding", shape, dtype)
    t, gh = make(*shape, dtype, seed=1)
    gh = (gh - 0.75).to(dtype)
    want, got = gated_linear(**t, gh=gh), gradients(t, gh, "silu")
    for name in ("x", "w_gate", "w_up"):
        exact = want[name][0]
        own = (exact.to(dtype).double() - exact).norm()
        err = (got[name].double().cpu() - exact).norm()
        assert err <= 1.02 * own, (name, float(err / own))


@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("shape", [(1, 64, 160), (300, 64, 160), (5000, 64, 160), (2100, 520, 160)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("scale", [2.0 ** -22, 2.0 ** -16, 2.0 ** 14], ids=["tiny", "small", "large"])
def test_range_of_float16(scale, shape, act):
    """Gradients as a scaled loss has them and as one without scaling has: da and db pass float16's largest number, or
    are a few of its smallest steps, where dx and dW are numbers of their own."""
    banner("glu range", scale, shape, act)
    t, gh = make(*shape, F16, scale, bias=False, seed=2)
    want, got = bounds(t, gh, act), gradients(t, gh, act)
    for name in want:
        v, b = want[name]
        there = v.abs() < 65000  # (the others round to infinity, or may)
        assert there.any()
        ratio = worst(got[name].cpu()[there], (v[there], b[there]))
        assert ratio <= 1, (name, ratio)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("rows", [40, 700])
def test_infinite_gradient(rows, dtype):
    """An infinite gradient is infinite in both parts of nothing: where weights have one sign, so has the result."""
    banner("glu infinite gradient", rows, dtype)
    t, gh = make(rows, 24, 16, dtype, bias=False, seed=3)
    t["x"], t["w_gate"], t["w_up"] = (v.abs() + 0.1 for v in (t["x"], t["w_gate"], t["w_up"]))
    gh[7, 5] = float("inf")
    got = {k: v.cpu() for k, v in gradients(t, gh, "none").items()}
    assert (got["x"][7] == float("inf")).all()
    for k in ("w_gate", "w_up"):
        assert (got[k][5] == float("inf")).all()
        rest = [i for i in range(16) if i != 5]
        assert torch.isfinite(got[k][rest]).all()
    rest = [i for i in range(rows) if i != 7]
    assert torch.isfinite(got["x"][rest]).all()


@pytest.mark.parametrize("dtype", [torch.float32, F16, BF16], ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("act", ["none", "relu", "silu"])
@pytest.mark.parametrize("bias", [True, False], ids=["bias", "plain"])
def test_every_activation_in_large_tiles(bias, act, dtype):
    banner("glu large", act, bias, dtype)
    for C in (72, 70):   # whole chunks, and rows that are packed
        check_all(*make_all((2050, C), 1610, dtype, bias, seed=7), act)
