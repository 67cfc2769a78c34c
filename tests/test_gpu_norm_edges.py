"""Group norm with an activation and its read-out where values, lengths or
layouts are at an edge: groups that are constant or nearly so, sums over many
rows, arguments that float32 does not hold, strided inputs."""

import pytest
import torch

import euler_characteristic_curves_amd as E
from euler_characteristic_curves_amd._lib import lib
from tests.gpu_util import banner, need_gpu
from tests.norm_bounds import act_and_slope
from tests.test_gpu_norm import call, check_all, make

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
EPS = 1e-5
HALF32 = 2.0 ** -24


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("value", [3.25, 100.0, -1000.0])
@pytest.mark.parametrize("readout", [False, True], ids=["norm", "readout"])
@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=["f32", "f16", "bf16"])
def test_constant_group_gives_the_bias(dtype, readout, value):
    """x - mean is exactly 0, so u is the bias, whatever the mean is against 1 / sqrt(eps)."""
    banner("norm constant", dtype, readout, value)
    gen = torch.Generator().manual_seed(1)
    C = 16
    x = torch.full((2, 40, 9, C), value).to(dtype)
    w, b, r, o = (torch.randn(n, generator=gen) for n in (C, C, C, 1))
    if not readout:
        y = E.group_norm_act(x.cuda(), 4, w.cuda(), b.cuda())
        assert torch.equal(y.cpu(), b.to(dtype).expand(x.shape))
        return
    for act in ("none", "silu"):
        f = E.group_norm_readout(x.cuda(), 4, w.cuda(), b.cuda(), r.cuda(), o.cuda(), act=act).double().cpu()
        terms = act_and_slope(b.double(), act)[0] * r.double()
        # C fused additions in float32, and 2^-20 of an activation's argument
        tol = C * HALF32 * (terms.abs().sum() + o.abs()) + 2.0 ** -20 * (b * r).abs().sum()
        assert ((f - (terms.sum() + o.double())).abs() <= tol).all(), act


def near_constant(level, spread, shape=(2, 40, 37, 16), seed=2):
    """Float32 values about `level` with a deviation of `spread`; channels of a group alike."""
    gen = torch.Generator().manual_seed(seed)
    return (level + spread * torch.randn(*shape, generator=gen, dtype=torch.float64)).float()


@pytest.mark.parametrize("level,spread", [(1000.0, 1e-3), (1e4, 1e-3), (-3e5, 0.05), (7.7, 1e-5)])
@pytest.mark.parametrize("shape", [(2, 40, 37, 16), (1, 60, 50, 520)], ids=["joined-here", "joined-apart"])
def test_mean_that_float32_does_not_hold(level, spread, shape):
    """A group about its mean by less than the mean's own rounding is normalised to float32's digits of x - mean, and
    the gradients see the same mean."""
    banner("norm near constant", level, spread, shape)
    x = near_constant(level, spread, shape)
    gen = torch.Generator().manual_seed(3)
    B, C, G = shape[0], shape[-1], 4
    w, b = 1 + 0.2 * torch.randn(C, generator=gen), 0.2 * torch.randn(C, generator=gen)
    grad = torch.randn(*shape, generator=gen)
    # about the level: 10^5 values of 10^4 cost even float64 the digits that are looked at
    v = x.double().reshape(B, -1, G, C // G) - level
    mean = v.mean(dim=(1, 3), keepdim=True)
    var = (v - mean).square().mean(dim=(1, 3), keepdim=True)
    rstd = 1 / torch.sqrt(var + EPS)
    xhat = ((v - mean) * rstd).reshape(shape)
    u = xhat * w.double() + b.double()
    leaves = [t.cuda().requires_grad_() for t in (x, w, b)]
    y = E.group_norm_act(leaves[0], G, leaves[1], leaves[2], eps=EPS)
    # xhat: roundings of numbers of its size and, through the mean, of its deviation's; and half a step, twice, of what
    # float32 leaves of the mean, which no later step can give back
    rest = (mean - ((mean + level).float().double() - level)).abs() * rstd
    wd, rms = w.double().abs(), torch.sqrt(var) * rstd
    xb = (64 * HALF32 * (xhat.abs().reshape(v.shape) + rms) + 2 * HALF32 * rest).reshape(shape)
    assert ((y.detach().double().cpu() - u).abs() / (xb * wd + 4 * HALF32 * (b.double().abs() + u.abs()))).max() <= 1
    gx, gw, gb = torch.autograd.grad(y, leaves, grad.cuda())
    q, dims, group = grad.double(), tuple(range(len(shape) - 1)), (1, 3)
    gwb = q.abs() * xb + 32 * HALF32 * (q * xhat).abs()
    assert ((gw.double().cpu() - (q * xhat).sum(dim=dims)).abs() / gwb.sum(dim=dims)).max() <= 1
    t, tb = (q * w.double()).reshape(v.shape), (gwb * wd).reshape(v.shape).mean(dim=group, keepdim=True)
    h, hb = xhat.reshape(v.shape), xb.reshape(v.shape)
    m1, m2 = t.mean(dim=group, keepdim=True), (t * h).mean(dim=group, keepdim=True)
    dx = rstd * (t - m1 - h * m2)
    dxb = rstd * (32 * HALF32 * t.abs().mean(dim=group, keepdim=True) + h.abs() * tb + hb * m2.abs()
                  + 64 * HALF32 * (t.abs() + m1.abs() + (h * m2).abs()))
    assert ((gx.double().cpu().reshape(v.shape) - dx).abs() / dxb).max() <= 1


def test_sums_over_many_rows():
    """A thousand rows a thread: sums of float32 leave it for float64 on the way, so that neither a constant gradient,
    whose roundings all go one way, nor an empty border slice, which the first rows of every thread lie in, costs digits."""
    banner("norm long sums")
    n, border = 1 << 28, 1 << 20
    x = torch.randn(1, n, 1, device="cuda", generator=torch.Generator("cuda").manual_seed(4)).add_(1000.0)
    x[:, :border] = 0.0
    # float64 moments, chunk by chunk
    s = torch.zeros(2, dtype=torch.float64)
    for c in x.view(16, -1):
        d = c.double() - 1000.0
        s += torch.stack([d.sum(), (d * d).sum()]).cpu()
    mean = float(s[0]) / n
    var = float(s[1]) / n - mean ** 2
    b, r, o = (torch.full((1,), v, device="cuda", requires_grad=True) for v in (0.0, 1.0, 0.0))
    f = E.group_norm_readout(x, 1, None, b, r, o)
    # a thread's first run, an eighth of its rows at most, lies 1000 off its pivot: 40 roundings of that much
    share = 128 * 2 ** 18 / n
    tol = 40 * HALF32 * (1 + share * 1e6 / var)
    at = torch.arange(border, n, 99991, device="cuda")
    want = (x[0, at, 0].double() - 1000.0 - mean) / (var + EPS) ** 0.5
    got = f.detach()[0, at].double()
    assert ((got - want).abs() <= tol * (want.abs() + 1e-2) + 64 * HALF32 * want.abs()).all()
    step = 0.1
    grads = torch.autograd.grad(f, [b, r, o], torch.full((), step, device="cuda").expand(f.shape))
    total = float(torch.tensor(step).double()) * n
    for name, g in (("bias", grads[0]), ("offset", grads[2])):
        assert abs(float(g.double()) - total) <= 40 * HALF32 * total, name


@pytest.mark.parametrize("readout", [False, True], ids=["norm", "readout"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_arguments_beyond_float32(act, readout):
    """weight * xhat overflows to an infinity: its activation is infinity or 0 and its slope 1 or 0, as for the value
    that float32 does not hold."""
    banner("norm overflow", act, readout)
    x = torch.zeros(1, 2, 25, 1)
    x[0, 0, 0], x[0, 0, 1] = 5.0, -5.0        # xhat: 5 and -5, the rest 0
    up, down = torch.tensor([3e38]), torch.tensor([1.0])
    leaves = [t.cuda().requires_grad_() for t in (x, up, torch.zeros(1))]
    grad = torch.zeros(1, 2, 25) if readout else torch.zeros(x.shape)
    grad[0, 0, 0], grad[0, 0, 1] = 1.0, 2.0
    if readout:
        out = E.group_norm_readout(*leaves[:1], 1, leaves[1], leaves[2], down.cuda(), act=act)
    else:
        out = E.group_norm_act(leaves[0], 1, leaves[1], leaves[2], act=act)
    flat = out.detach().reshape(50).cpu()
    assert flat[0] == float("inf") and flat[1] == 0.0 and torch.equal(flat[2:], torch.zeros(48))
    (gb,) = torch.autograd.grad(out, [leaves[2]], grad.cuda())
    assert float(gb) == 1.0


@pytest.mark.parametrize("readout", [False, True], ids=["norm", "readout"])
def test_a_strided_input_is_copied_once(readout):
    """Channels-first features in memory: what a forward call allocates is the copy that the kernels read, the result
    and less than a megabyte of scratch."""
    banner("norm copies", readout)
    x = torch.randn(2, 64, 256, 256, device="cuda").permute(0, 2, 3, 1)
    r = torch.ones(64, device="cuda")

    def call():
        return E.group_norm_readout(x, 8, None, None, r) if readout else E.group_norm_act(x, 8)

    call()
    before = torch.cuda.memory_stats()["allocated_bytes.all.allocated"]
    out = call()
    spent = torch.cuda.memory_stats()["allocated_bytes.all.allocated"] - before
    scratch = lib.ecc_norm_workspace_bytes(2, 256 * 256, 64, 8)
    assert spent <= x.numel() * 4 + out.numel() * 4 + scratch + (1 << 20)


@pytest.mark.parametrize("readout", [False, True], ids=["norm", "readout"])
@pytest.mark.parametrize("shape,groups", [((300, 3, 3, 48), 6), ((33, 9000, 16), 4), ((2000, 1, 8), 8), ((64, 40, 520), 20)],
                         ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else None)
def test_large_batches(shape, groups, readout):
    """Workspaces without folded rows, one workgroup a sample and several."""
    banner("norm batches", shape, groups, readout)
    x, p, grad = make(shape, BF16, seed=21, readout=readout)
    check_all(x, groups, p, grad, "silu")


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("C", [384, 640, 1000, 1024, 1025, 1280, 2047])
def test_wide_rows_of_16_bits(C, dtype):
    """Two vectors a lane at most; beyond 1024 channels, chunks of columns."""
    banner("norm 16-bit rows", C, dtype)
    for readout in (False, True):
        if readout and C > 1024:
            continue
        x, p, grad = make((2, 41, C), dtype, seed=C, readout=readout)
        check_all(x, 1 if C % 2 else 4, p, grad, "silu")


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=["f32", "f16", "bf16"])
def test_nan_passes_every_activation(dtype, act):
    """One NaN makes its group's values, field and gradients NaN, and no others; the clamps of the activations do not
    swallow it."""
    banner("norm nan", dtype, act)
    x, p, grad = make((3, 5, 7, 16), dtype, seed=6, readout=True)
    x[1, 2, 3, 5] = float("nan")          # sample 1, group 1 of 4
    hit = torch.zeros(3, 35, 4, 4, dtype=torch.bool)
    hit[1, :, 1] = True
    leaves = [x.cuda().requires_grad_(), *(v.cuda().requires_grad_() for v in p.values())]
    y = E.group_norm_act(leaves[0], 4, leaves[1], leaves[2], act=act)
    (gx,) = torch.autograd.grad(y, leaves[:1], torch.ones_like(y))
    for t in (y.detach(), gx):
        assert torch.equal(torch.isnan(t).reshape(hit.shape).cpu(), hit)
    f = E.group_norm_readout(leaves[0], 4, *leaves[1:], act=act)
    assert torch.equal(torch.isnan(f).reshape(3, 35).cpu(), hit.any(dim=3).any(dim=2))
    grads = torch.autograd.grad(f, leaves, grad.cuda())
    assert torch.equal(torch.isnan(grads[0]).reshape(hit.shape).cpu(), hit)
    channels = hit.any(dim=1).any(dim=0).reshape(16)
    for name, g in zip(p, grads[1:4]):
        # the bias's gradient has no x in it where there is no activation
        want = torch.zeros(16, dtype=torch.bool) if act == "none" and name == "bias" else channels
        assert torch.equal(torch.isnan(g).cpu(), want), name
    assert torch.isfinite(grads[4]).all()


@pytest.mark.parametrize("readout", [False, True], ids=["norm", "readout"])
@pytest.mark.parametrize("dtype", [F32, F16], ids=["f32", "f16"])
def test_infinite_gradient(dtype, readout):
    """An infinite upstream gradient, as a scaled loss that overflows gives, makes its channels' gradients infinite with
    the sign of their factors, and not NaN; others stay finite."""
    banner("norm infinite gradient", dtype, readout)
    x, p, grad = make((2, 9, 11, 16), dtype, seed=14, readout=readout)
    where = (1, 4, 5) if readout else (1, 4, 5, 6)
    grad[where] = float("inf")
    leaves = [x.cuda().requires_grad_(), *(v.cuda().requires_grad_() for v in p.values())]
    out = call(leaves[0], 4, dict(zip(p, leaves[1:])), "none")
    gw, gb = torch.autograd.grad(out, leaves[1:3], grad.cuda())
    v = x.double().reshape(2, 99, 4, 4)
    xhat = (v - v.mean(dim=(1, 3), keepdim=True)).reshape(x.shape)[1, 4, 5]
    factor = p["readout"].double() if readout else torch.ones(16, dtype=torch.float64)
    hit = torch.ones(16, dtype=torch.bool) if readout else torch.arange(16) == 6
    for g, f in ((gw, factor * xhat), (gb, factor)):
        g = g.double().cpu()
        assert torch.equal(g[hit], torch.sign(f[hit]) * float("inf"))
        assert torch.isfinite(g[~hit]).all()
