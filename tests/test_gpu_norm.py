"""Group norm with an activation and its read-out on the GPU against float64
(tests/norm_bounds.py): outputs and every gradient, over types, channel counts
that fill a vector, straddle it or exceed a wave, odd sizes, offsets, strides,
streams and graphs."""

import pytest
import torch

import euler_characteristic_curves_amd as E
from tests.gpu_util import banner, need_gpu
from tests.norm_bounds import norm, worst

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
EPS = 1e-5


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def make(shape, dtype, pdtype=None, seed=0, readout=False, offset_scale=0.7):
    gen = torch.Generator().manual_seed(seed)
    C = shape[-1]
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = (rnd(*shape) * (0.5 + rnd(C).abs()) + offset_scale * rnd(C)).to(dtype)
    pdtype = pdtype or F32
    p = {"weight": (1 + 0.2 * rnd(C)).to(pdtype), "bias": (0.2 * rnd(C)).to(pdtype)}
    if readout:
        p["readout"] = (rnd(C) / C ** 0.5).to(pdtype)
        p["offset"] = (0.1 * rnd(1)).to(pdtype)
        grad = rnd(*shape[:-1])
    else:
        grad = rnd(*shape).to(dtype)
    return x, p, grad


def call(x, groups, p, act, eps=EPS):
    if "readout" in p:
        return E.group_norm_readout(x, groups, p["weight"], p["bias"], p["readout"], p["offset"], act=act, eps=eps)
    return E.group_norm_act(x, groups, p["weight"], p["bias"], act=act, eps=eps)


def check_all(x, groups, p, grad, act, pdtype=F32, eps=EPS, dev_x=None):
    """Forward without and with gradients, and the backward pass, against the bounds."""
    want = norm(x, groups, p["weight"], p["bias"], act, eps, grad, p.get("readout"), p.get("offset"), pdtype)
    dx = (x.cuda() if dev_x is None else dev_x).requires_grad_()
    dp = {k: v.cuda().requires_grad_() for k, v in p.items()}
    with torch.no_grad():
        plain = call(dx, groups, dp, act, eps)
    out = call(dx, groups, dp, act, eps)
    torch.cuda.synchronize()
    assert torch.equal(plain, out) or torch.isnan(plain).any()
    names = ["x", *dp]
    grads = torch.autograd.grad(out, [dx, *dp.values()], grad.cuda())
    torch.cuda.synchronize()
    got = {"field" if "readout" in p else "y": out, **dict(zip(names, grads))}
    for name, t in got.items():
        ratio = worst(t, want[name])
        assert ratio <= 1.0, (name, ratio)
        ref = x if name in ("x", "y") else None
        assert t.dtype == (ref.dtype if ref is not None else F32 if name == "field" else p[name].dtype)


SHAPES = [  # (shape, groups)
    ((1, 1, 1, 8), 8), ((1, 1, 1, 8), 1), ((2, 3, 5, 7, 24), 4), ((3, 17, 9, 51), 3), ((1, 33, 31, 32), 8),
    ((2, 29, 12), 4), ((1, 5, 5, 1), 1), ((4, 6, 5, 3), 3), ((2, 7, 11, 64), 16), ((1, 9, 7, 96), 12),
    ((2, 65, 100), 10), ((2, 13, 320), 32), ((1, 40, 384), 1), ((1, 21, 520), 520), ((1, 3, 1024), 16),
    ((1, 300, 300, 16), 2), ((5, 64, 40), 8),
]


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("readout", [False, True], ids=["norm", "readout"])
@pytest.mark.parametrize("shape,groups", SHAPES, ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else None)
def test_shapes(shape, groups, readout, dtype):
    banner("norm", shape, groups, readout, dtype)
    x, p, grad = make(shape, dtype, seed=sum(shape), readout=readout)
    check_all(x, groups, p, grad, "silu")


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("readout", [False, True], ids=["norm", "readout"])
@pytest.mark.parametrize("dtype,pdtype", [(F32, F32), (BF16, BF16), (F16, F16), (F16, F32)],
                         ids=["f32", "bf16", "f16", "f16-f32"])
def test_activations_and_parameter_types(act, readout, dtype, pdtype):
    banner("norm act", act, readout, dtype, pdtype)
    x, p, grad = make((2, 11, 13, 48), dtype, pdtype, seed=5, readout=readout)
    check_all(x, 6, p, grad, act, pdtype)


@pytest.mark.parametrize("dtype,C", [(F32, 1028), (F32, 1030), (BF16, 2056), (F16, 2061), (F32, 8192)])
def test_rows_wider_than_four_waves(dtype, C):
    banner("norm wide", dtype, C)
    x, p, grad = make((2, 9, C), dtype, seed=C)
    check_all(x, 1 if C % 2 else 2, p, grad, "gelu")


@pytest.mark.parametrize("readout", [False, True], ids=["norm", "readout"])
def test_far_offset_and_far_first_value(readout):
    """The mean a thousand deviations off, and a first voxel far outside the rest."""
    banner("norm offsets", readout)
    x, p, grad = make((2, 40, 37, 16), F32, seed=3, readout=readout)
    check_all(x + 1000.0, 4, p, grad, "silu")
    x[:, 0, 0] = -300.0
    check_all(x, 4, p, grad, "silu")


def test_constant_input_and_zero_eps_variance():
    banner("norm constant")
    x, p, grad = make((2, 5, 6, 16), F32, seed=4)
    check_all(torch.full_like(x, 3.25), 4, p, grad, "silu")


def test_nan_and_inf_stay_in_their_sample_and_group():
    banner("norm nan")
    for bad in (float("nan"), float("inf")):
        x, p, grad = make((3, 6, 7, 16), F32, seed=6)
        x[1, 2, 3, 5] = bad          # sample 1, group 1 of 4
        out = call(x.cuda(), 4, {k: v.cuda() for k, v in p.items()}, "gelu").cpu()
        broken = torch.isnan(out).reshape(3, 42, 4, 4).all(dim=3).all(dim=1)
        clean = ~torch.isnan(out).reshape(3, 42, 4, 4).any(dim=3).any(dim=1)
        assert broken[1, 1] and clean.sum() == 11


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("readout", [False, True], ids=["norm", "readout"])
def test_unaligned_base_and_strides(dtype, readout):
    """Storage that starts one element in, and tensors that are not contiguous."""
    banner("norm strides", dtype, readout)
    shape = (2, 9, 10, 24)
    x, p, grad = make(shape, dtype, seed=7, readout=readout)
    flat = torch.zeros(x.numel() + 1, dtype=dtype, device="cuda")
    flat[1:] = x.cuda().reshape(-1)
    check_all(x, 4, p, grad, "silu", dev_x=flat[1:].view(shape).detach())
    first = x.permute(0, 3, 1, 2).contiguous().cuda().permute(0, 2, 3, 1)  # channels first in memory
    assert not first.is_contiguous()
    check_all(x, 4, p, grad, "silu", dev_x=first.detach())
    expanded = grad[:1, :1].expand(grad.shape)
    check_all(x, 4, p, expanded, "silu")


def test_parameters_left_out():
    banner("norm none")
    x, p, grad = make((2, 8, 9, 24), F32, seed=8)
    want = norm(x, 4, None, None, "silu", EPS, grad)
    dx = x.cuda().requires_grad_()
    out = E.group_norm_act(dx, 4, act="silu")
    (gx,) = torch.autograd.grad(out, [dx], grad.cuda())
    assert worst(out, want["y"]) <= 1 and worst(gx, want["x"]) <= 1
    # only the parameters, and only one of them
    want = norm(x, 4, p["weight"], p["bias"], "silu", EPS, grad)
    w = p["weight"].cuda().requires_grad_()
    out = E.group_norm_act(x.cuda(), 4, w, p["bias"].cuda(), act="silu")
    (gw,) = torch.autograd.grad(out, [w], grad.cuda())
    assert worst(gw, want["weight"]) <= 1
    r = torch.ones(24, device="cuda", requires_grad=True)
    out = E.group_norm_readout(x.cuda(), 4, None, None, r)
    want = norm(x, 4, None, None, "none", EPS, torch.ones(2, 8, 9), torch.ones(24))
    (gr,) = torch.autograd.grad(out.sum(), [r])
    assert worst(out, want["field"]) <= 1 and worst(gr, want["readout"]) <= 1


def test_empty():
    banner("norm empty")
    for shape in ((0, 4, 4, 8), (2, 0, 4, 8)):
        x = torch.zeros(shape, device="cuda", requires_grad=True)
        w = torch.ones(8, device="cuda", requires_grad=True)
        y = E.group_norm_act(x, 2, w, act="relu")
        assert y.shape == x.shape
        gx, gw = torch.autograd.grad(y.sum(), [x, w])
        assert gx.shape == x.shape and torch.equal(gw.cpu(), torch.zeros(8))
        f = E.group_norm_readout(x, 2, w, None, w)
        assert f.shape == x.shape[:-1]


def test_differences():
    """The gradients against central differences of the forward pass: the forward pass's own error over the step
    bounds how far the two may be apart beyond what float64 gives for the same step."""
    banner("norm differences")
    h = 2.0 ** -6
    for act in ("silu", "gelu"):
        x, p, grad = make((1, 6, 7, 16), F32, seed=9)
        dx = x.cuda().requires_grad_()
        dp = {k: v.cuda() for k, v in p.items()}
        (gx,) = torch.autograd.grad(call(dx, 4, dp, act), [dx], grad.cuda())
        v = torch.sign(gx.cpu())
        sides = [norm(x + s * h * v, 4, p["weight"], p["bias"], act, EPS)["y"] for s in (1, -1)]
        outs = [call((x + s * h * v).cuda(), 4, dp, act).double().cpu() for s in (1, -1)]
        g = grad.double()
        mine = float(((outs[0] - outs[1]) * g).sum()) / (2 * h)
        ref = float(((sides[0][0] - sides[1][0]) * g).sum()) / (2 * h)
        slack = float(((sides[0][1] + sides[1][1]) * g.abs()).sum()) / (2 * h)
        assert abs(mine - ref) <= slack
        along = float((gx.double().cpu() * v.double()).sum())
        # the term of third order, from float64 differences at this step and at half of it (a quarter of it is left)
        half = [norm(x.double() + s * (h / 2) * v, 4, p["weight"], p["bias"], act, EPS, dtype=F32)["y"][0] for s in (1, -1)]
        cubic = 4 / 3 * abs(ref - float(((half[0] - half[1]) * g).sum()) / h)
        assert abs(mine - along) <= slack + 2 * cubic + 1e-5 * float(gx.abs().sum())


def test_another_stream_and_repeatability():
    banner("norm stream")
    x, p, grad = make((2, 33, 35, 48), BF16, seed=10, readout=True)
    dx, dp, g = x.cuda(), {k: v.cuda() for k, v in p.items()}, grad.cuda()
    leaves = [dx.requires_grad_(), *(v.requires_grad_() for v in dp.values())]

    def step():
        out = call(dx, 6, dp, "gelu")
        return [out.detach(), *torch.autograd.grad(out, leaves, g)]

    first = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for a, b in zip(first, second):
        assert torch.equal(a, b)


@pytest.mark.parametrize("readout", [False, True], ids=["norm", "readout"])
def test_graph_replays(readout):
    """Forward and backward in one graph, replayed with eager work in between.  The captured pass has leaves of its
    own: a backward pass must not be captured while an eager graph of the same leaves is alive."""
    banner("norm graph", readout)
    x, p, grad = make((2, 19, 21, 24), F32, seed=11, readout=readout)
    leaves = [t.cuda().requires_grad_() for t in (x, *p.values())]
    g = grad.cuda()

    def step(ts):
        out = call(ts[0], 4, dict(zip(p, ts[1:])), "silu")
        return [out.detach(), *torch.autograd.grad(out, ts, g)]

    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        step(leaves)
    torch.cuda.current_stream().wait_stream(warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(leaves)
    for i in range(3):
        fresh, _, _ = make((2, 19, 21, 24), F32, seed=20 + i, readout=readout)
        with torch.no_grad():
            leaves[0].copy_(fresh.cuda())
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in outs]
        eager = step([t.detach().clone().requires_grad_() for t in leaves])
        torch.cuda.synchronize()
        for a, b in zip(kept, eager):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("readout", [False, True], ids=["norm", "readout"])
@pytest.mark.parametrize("groups", [1, 4, 64])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_many_partial_rows(dtype, groups, readout):
    """Wide groups over many workgroups: partial rows are folded before they are joined."""
    banner("norm fold", dtype, groups, readout)
    x, p, grad = make((1, 41, 50, 512), dtype, seed=12, readout=readout)
    check_all(x, groups, p, grad, "silu")


def test_any_subset_of_gradients():
    """Parameters left out and inputs that need no gradient, in every combination, against the full set."""
    banner("norm subsets")
    x, p, grad = make((2, 6, 7, 24), F32, seed=13, readout=True)
    names = ["x", "weight", "bias", "readout", "offset"]
    for absent in ((), ("weight",), ("bias",), ("weight", "bias", "offset")):
        full = {k: v for k, v in {"x": x, **p}.items()}
        want = norm(x, 4, None if "weight" in absent else p["weight"], None if "bias" in absent else p["bias"], "silu", EPS,
                    grad, p["readout"], None if "offset" in absent else p["offset"])
        here = [n for n in names if n not in absent]
        for mask in range(1, 1 << len(here)):
            ts = {n: (full[n].cuda() if n in here else None) for n in names}
            leaves = [n for i, n in enumerate(here) if mask >> i & 1]
            for n in leaves:
                ts[n].requires_grad_()
            out = E.group_norm_readout(ts["x"], 4, ts["weight"], ts["bias"], ts["readout"], ts["offset"], act="silu")
            grads = torch.autograd.grad(out, [ts[n] for n in leaves], grad.cuda())
            for n, g in zip(leaves, grads):
                assert worst(g, want[n]) <= 1, (absent, leaves, n)


def test_backward_is_differentiable_once():
    banner("norm twice")
    x = torch.randn(2, 5, 6, 8, device="cuda", requires_grad=True)
    y = E.group_norm_act(x, 2, act="silu")
    (g,) = torch.autograd.grad(y.sum(), [x], create_graph=True)
    with pytest.raises(RuntimeError, match="once"):
        g.sum().backward()


def test_changed_input_is_noticed():
    banner("norm changed")
    x = torch.randn(2, 5, 6, 8, device="cuda")
    w = torch.ones(8, device="cuda", requires_grad=True)
    y = E.group_norm_act(x, 2, w)
    x.add_(1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_refusals():
    banner("norm refusals")
    x = torch.zeros(2, 3, 4, 8, device="cuda")
    one = torch.ones(8, device="cuda")
    for kw, exc in ((dict(groups=3), ValueError), (dict(groups=0), ValueError), (dict(groups=2.0), TypeError),
                    (dict(act="tanh"), ValueError), (dict(weight=one[:4]), ValueError), (dict(weight=one.half()), TypeError),
                    (dict(weight=one[None]), ValueError), (dict(bias=one.cpu()), ValueError), (dict(eps=-1.0), E.EccError),
                    (dict(eps=float("nan")), E.EccError), (dict(x=x.double()), TypeError), (dict(x=x[0, 0]), ValueError)):
        args = {"x": x, "groups": 2, "weight": one, "bias": one, **kw}
        for grad in (False, True):
            with pytest.raises(exc):
                E.group_norm_act(args["x"].detach().clone().requires_grad_(grad), args["groups"], args["weight"], args["bias"],
                                 act=args.get("act", "none"), eps=args.get("eps", EPS))
    with pytest.raises(TypeError):
        E.group_norm_readout(x, 2, None, None, None)
    with pytest.raises(ValueError):
        E.group_norm_readout(x, 2, one, None, one, one)
    half = x.half()
    with pytest.raises(TypeError):
        E.group_norm_act(half, 2, one, one.half())
    wide = torch.zeros(1, 2, 8193, device="cuda")
    with pytest.raises(E.EccError):
        E.group_norm_act(wide, 1)
    with pytest.raises(E.EccError):
        E.group_norm_readout(wide[..., :1030].contiguous(), 1, None, None, torch.zeros(1030, device="cuda"))
