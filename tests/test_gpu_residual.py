"""Norms around a block with gate and residual scale on the GPU against float64 (tests/block_bounds.py): outputs and
every gradient, over types, row widths that fill a vector, straddle it or exceed a wave, gates, strides, streams and
graphs."""

import pytest
import torch
import torch.autograd.forward_ad as fa

import euler_characteristic_curves_amd as E
from tests.block_bounds import residual
from tests.gpu_util import banner, need_gpu
from tests.norm_bounds import worst

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [(F32, F32), (F16, F16), (BF16, BF16), (F32, F16), (F32, BF16)]
IDS = ["f32", "f16", "bf16", "f32-f16", "f32-bf16"]


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def make(shape, xt, bt, pt=None, gate="channel", norm=True, seed=0):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    C, pt = shape[-1], pt or F32
    t = {"x": (rnd(*shape) * (1 + 2 * rnd(C).abs())).to(xt), "branch": (rnd(*shape) * (0.3 + rnd(C).abs())).to(bt)}
    if gate:
        t["gate"] = (0.5 + 0.5 * rnd(*((C,) if gate == "channel" else (shape[0], C)))).to(pt)
    t["weight"] = (1 + 0.2 * rnd(C)).to(pt)
    if norm:
        t["branch_weight"] = (1 + 0.2 * rnd(C)).to(pt)
    return t, rnd(*shape).to(xt), rnd(*shape).to(bt)


def call(t, **kw):
    return E.residual_norm(t["x"], t["branch"], t.get("gate"), t.get("weight"), t.get("branch_weight"), **kw)


def check_all(t, gy, gz, pt=F32, dev=None, **kw):
    want = residual(**t, **kw, gy=gy, gz=gz, pdtype=pt)
    d = {k: v.cuda() for k, v in t.items()} if dev is None else dev
    d = {k: v.requires_grad_() for k, v in d.items()}
    with torch.no_grad():
        plain = call(d, **kw)
    outs = call(d, **kw)
    torch.cuda.synchronize()
    for a, b in zip(plain, outs):
        assert torch.equal(a, b)
    pairs = [(o, g) for o, g in zip(outs, (gy, gz)) if g is not None]
    grads = torch.autograd.grad([o for o, _ in pairs], list(d.values()), [g.cuda() for _, g in pairs])
    torch.cuda.synchronize()
    got = {"y": outs[0], "z": outs[1], **dict(zip(d, grads))}
    for name, v in got.items():
        assert v.dtype == {"y": t["x"], "z": t["branch"]}.get(name, t.get(name)).dtype
        ratio = worst(v, want[name])
        assert ratio <= 1.0, (name, ratio)


SHAPES = [(1, 1, 1), (1, 3), (2, 1, 7), (3, 5, 8), (2, 70, 9), (1, 129, 17), (2, 3, 5, 7, 24), (4, 33, 64), (1, 40, 129),
          (3, 37, 411), (2, 9, 512), (1, 5, 1000), (2, 6, 1024), (1, 3, 2051), (1, 2, 4096), (2, 2, 8192), (1, 700, 3)]


@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_shapes(shape, types):
    banner("residual", shape, types)
    check_all(*make(shape, *types, seed=sum(shape)))


@pytest.mark.parametrize("gate", [None, "channel", "sample"])
@pytest.mark.parametrize("norm", [True, False], ids=["norm", "plain"])
@pytest.mark.parametrize("types,pt", [((F32, F32), F32), ((BF16, BF16), BF16), ((F32, F16), F16), ((F16, F16), F32)])
def test_forms(gate, norm, types, pt):
    banner("residual forms", gate, norm, types, pt)
    t, gy, gz = make((3, 11, 13, 72), *types, pt, gate, norm, seed=5)
    check_all(t, gy, gz, pt, norm_branch=norm, scale=0.7, eps=1e-3)


@pytest.mark.parametrize("which", ["y", "z"])
def test_one_gradient_alone(which):
    banner("residual one", which)
    t, gy, gz = make((2, 9, 40), F32, BF16, gate="sample", seed=6)
    check_all_some(t, gy if which == "y" else None, gz if which == "z" else None)


def check_all_some(t, gy, gz):
    want = residual(**t, gy=gy, gz=gz)
    d = {k: v.cuda().requires_grad_() for k, v in t.items()}
    out = call(d)[0 if gz is None else 1]
    names = [k for k in d if not (gz is None and k == "weight")]
    grads = torch.autograd.grad(out, [d[k] for k in names], (gy if gz is None else gz).cuda())
    for name, v in zip(names, grads):
        assert worst(v, want[name]) <= 1, name


def test_many_rows_and_samples():
    """More rows than a launch has slots for, and more samples than the join has workgroups."""
    banner("residual many")
    check_all(*make((1, 40000, 24), BF16, BF16, seed=7))
    check_all(*make((1500, 3, 16), F32, F32, gate="sample", seed=8))


def test_rows_of_one_thread_are_summed_in_runs():
    """2^24 rows alike, 64 of them a thread: sums are n times one row's, and so are their bounds."""
    banner("residual alike")
    C, n = 4, 1 << 24
    t = {"x": torch.ones(1, 1, C), "branch": torch.tensor([1.0, 2.0, 3.0, 4.0])[None, None], "gate": torch.full((C,), 0.3),
         "weight": torch.full((C,), 1.1), "branch_weight": torch.full((C,), 0.7)}
    gy, gz = torch.full((1, 1, C), 0.1), torch.full((1, 1, C), 0.1).mul(torch.tensor([1.0, -2.0, 3.0, 0.3]))
    want = residual(**t, gy=gy, gz=gz)
    d = {k: v.cuda() for k, v in t.items()}
    for k in ("x", "branch"):
        d[k] = d[k].expand(1, n, C).contiguous()
    names = ["gate", "weight", "branch_weight"]
    for k in names:
        d[k].requires_grad_()
    grads = torch.autograd.grad(call(d), [d[k] for k in names], [g.cuda().expand(1, n, C).contiguous() for g in (gy, gz)])
    for k, v in zip(names, grads):
        assert worst(v, (n * want[k][0], n * want[k][1])) <= 1, k


def test_extremes():
    """Rows whose squares overflow or vanish in float32, rows of zeros, infinities that stay in their row."""
    banner("residual extremes")
    t, gy, gz = make((1, 6, 40), F32, F32, seed=9)
    t["x"][0, 0] *= 1e25
    t["branch"][0, 0] *= 1e30
    t["branch"][0, 1] *= 1e-30
    t["x"][0, 2] = 0
    t["branch"][0, 2] = 0
    want = residual(**t, eps=1e-20)
    y, z = call({k: v.cuda() for k, v in t.items()}, eps=1e-20)
    assert worst(y, want["y"]) <= 1 and worst(z, want["z"]) <= 1
    for bad in (float("inf"), float("nan")):
        t2 = {**t, "branch": t["branch"].clone()}
        t2["branch"][0, 4, 7] = bad
        d = {k: v.cuda().requires_grad_() for k, v in t2.items()}
        outs = call(d, eps=1e-20)
        gx, gb = torch.autograd.grad(outs, [d["x"], d["branch"]], [gy.cuda(), gz.cuda()])
        for v in (*outs, gx, gb):
            clean = torch.isfinite(v).all(dim=-1).cpu()[0]
            assert clean[[1, 2, 3, 5]].all(), bad
        assert torch.isnan(outs[1][0, 4]).any()


@pytest.mark.parametrize("gate", ["channel", "sample"])
def test_infinite_parameters_stay_in_their_channel(gate):
    """A gate that is infinite in one channel does not reach sums through rows or lanes that are not there."""
    banner("residual infinite gate", gate)
    t, gy, gz = make((2, 3, 11), F32, F32, gate=gate, seed=10)
    t["weight"][5] = float("inf")
    t["branch_weight"][5] = float("inf")
    d = {k: v.cuda().requires_grad_() for k, v in t.items()}
    y, z = call(d)
    ok = [c for c in range(11) if c != 5]
    assert torch.isfinite(y[..., ok]).all()
    (gw,) = torch.autograd.grad(y, [d["gate"]], gy.cuda())
    assert torch.isfinite(gw[..., ok]).all()


def test_unaligned_and_strided():
    banner("residual strides")
    for types in ((F32, BF16), (F16, F16)):
        t, gy, gz = make((3, 14, 40), *types, seed=11)
        dev = {}
        for k, v in t.items():
            flat = torch.zeros(v.numel() + 1, dtype=v.dtype, device="cuda")
            flat[1:] = v.cuda().reshape(-1)
            dev[k] = flat[1:].view(v.shape).detach()
        check_all(t, gy, gz, dev=dev)
        dev = {k: v.cuda() for k, v in t.items()}
        dev["x"] = dev["x"].transpose(1, 2).contiguous().transpose(1, 2).detach()
        dev["branch"] = torch.cat([dev["branch"], dev["branch"]], dim=2)[..., :40].detach()
        dev["weight"] = torch.stack([dev["weight"]] * 2, dim=1)[:, 0].detach()
        assert not dev["branch"].is_contiguous()
        check_all(t, gy, gz, dev=dev)
        check_all(t, gy[:1, :1].expand(gy.shape), gz[:, :, :1].expand(gz.shape))


@pytest.mark.parametrize("types", TYPES, ids=IDS)
def test_norm_alone(types):
    banner("rms norm", types)
    t, _, gz = make((2, 21, 100), *types, seed=12)
    want = residual(t["x"], None, weight=t["weight"], gz=gz, ztype=types[1])
    x, w = t["x"].cuda().requires_grad_(), t["weight"].cuda().requires_grad_()
    z = E.rms_norm(x, w, dtype=types[1])
    gx, gw = torch.autograd.grad(z, [x, w], gz.cuda())
    assert z.dtype == types[1]
    for name, v in (("z", z), ("x", gx), ("weight", gw)):
        assert worst(v, want[name]) <= 1, name
    assert worst(E.rms_norm(x.detach()), residual(t["x"], None)["z"]) <= 1


def test_subsets_of_gradients():
    banner("residual subsets")
    t, gy, gz = make((2, 7, 24), F32, F32, gate="sample", seed=13)
    want = residual(**t, gy=gy, gz=gz)
    for mask in range(1, 32):
        d = {k: v.cuda() for k, v in t.items()}
        names = [k for i, k in enumerate(d) if mask >> i & 1]
        for k in names:
            d[k].requires_grad_()
        outs = call(d)
        need = [(o, g.cuda()) for o, g in zip(outs, (gy, gz))]
        grads = torch.autograd.grad([o for o, _ in need], [d[k] for k in names], [g for _, g in need])
        for k, v in zip(names, grads):
            assert worst(v, want[k]) <= 1, (names, k)


def test_empty():
    banner("residual empty")
    for shape in ((0, 4, 8), (2, 0, 8)):
        x = torch.zeros(shape, device="cuda", requires_grad=True)
        w = torch.ones(8, device="cuda", requires_grad=True)
        y, z = E.residual_norm(x, x, w, w, w)
        gx, gw = torch.autograd.grad([y.sum() + z.sum()], [x, w])
        assert y.shape == z.shape == gx.shape == shape and torch.equal(gw.cpu(), torch.zeros(8))


def test_differences():
    """Along one direction, the step's terms of third order taken from float64."""
    banner("residual differences")
    t, gy, gz = make((2, 5, 16), F32, F32, gate="sample", seed=14)
    h = 2.0 ** -7
    d = {k: v.cuda().requires_grad_() for k, v in t.items()}
    grads = dict(zip(d, torch.autograd.grad(call(d), list(d.values()), [gy.cuda(), gz.cuda()])))
    for name in t:
        gen = torch.Generator().manual_seed(1)
        v = torch.sign(torch.randn(t[name].shape, generator=gen))
        refs = []
        for step in (h, h / 2):
            side = [residual(**{k: (u.double() if k != name else u.double() + s * step * v) for k, u in t.items()})
                    for s in (1, -1)]
            refs.append(sum(float(((side[0][o][0] - side[1][o][0]) * g.double()).sum())
                            for o, g in (("y", gy), ("z", gz))) / (2 * step))
        sides = [call({k: (u if k != name else u + s * h * v).cuda() for k, u in t.items()}) for s in (1, -1)]
        mine = sum(float(((a.double() - b.double()).cpu() * g.double()).sum()) for a, b, g in zip(*sides, (gy, gz))) / (2 * h)
        bounds = residual(**t)
        slack = 2 * sum(float((bounds[o][1] * 1.2 * g.double().abs()).sum()) for o, g in (("y", gy), ("z", gz))) / (2 * h)
        along = float((grads[name].double().cpu() * v.double()).sum())
        cubic = 4 / 3 * abs(refs[0] - refs[1])
        assert abs(mine - along) <= slack + 2 * cubic + 1e-5 * float(grads[name].abs().sum()), name


def test_stream_and_graph():
    banner("residual graph")
    t, gy, gz = make((2, 65, 96), F32, BF16, gate="sample", seed=15)
    gy, gz = gy.cuda(), gz.cuda()

    def step(ts):
        outs = call(ts)
        return [*(o.detach() for o in outs), *torch.autograd.grad(outs, list(ts.values()), [gy, gz])]

    def leaves():
        return {k: v.cuda().requires_grad_() for k, v in t.items()}

    first = step(leaves())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = step(leaves())
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for a, b in zip(first, second):
        assert torch.equal(a, b)
    mine = leaves()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(mine)
    for i in range(3):
        fresh, _, _ = make((2, 65, 96), F32, BF16, gate="sample", seed=20 + i)
        with torch.no_grad():
            for k in mine:
                mine[k].copy_(fresh[k].cuda())
        graph.replay()
        torch.cuda.synchronize()
        kept = [o.clone() for o in outs]
        eager = step({k: v.detach().clone().requires_grad_() for k, v in mine.items()})
        torch.cuda.synchronize()
        for a, b in zip(kept, eager):
            assert torch.equal(a, b), i


def test_refusals():
    banner("residual refusals")
    x = torch.zeros(2, 3, 8, device="cuda")
    one = torch.ones(8, device="cuda")
    for kw, exc in ((dict(branch=x[..., :4]), ValueError), (dict(branch=x.double()), TypeError), (dict(branch=x.cpu()), ValueError),
                    (dict(gate=one[:4]), ValueError), (dict(gate=torch.ones(3, 8, device="cuda")), ValueError),
                    (dict(gate=one.half()), TypeError), (dict(weight=one[None]), ValueError), (dict(weight=one.cpu()), ValueError),
                    (dict(norm_branch=False, branch_weight=one), ValueError), (dict(eps=-1.0), E.EccError),
                    (dict(scale=float("inf")), E.EccError), (dict(x=x[0, 0], branch=x[0, 0]), ValueError),
                    (dict(x=x.half()), TypeError), (dict(x=x.half(), branch=x.bfloat16()), TypeError)):
        for grad in (False, True):
            a = {"x": x, "branch": x, **kw}
            a["x"] = a["x"].detach().clone().requires_grad_(grad)
            with pytest.raises(exc):
                E.residual_norm(**a)
    with pytest.raises(TypeError):
        E.residual_norm(x, None)
    with pytest.raises(TypeError):
        E.rms_norm(x.half(), dtype=F32)
    wide = torch.zeros(1, 2, 8193, device="cuda")
    with pytest.raises(E.EccError):
        E.rms_norm(wide)
    y, z = E.residual_norm(x.requires_grad_(), x)
    (g,) = torch.autograd.grad(z.sum(), [x], create_graph=True)
    with pytest.raises(RuntimeError, match="once"):
        g.sum().backward()


def test_duals_and_changed_inputs():
    """Tangents are refused, not dropped, and an input written after the call is noticed by its backward pass."""
    banner("residual duals")
    x = torch.zeros(2, 3, 8, device="cuda")
    w = torch.ones(8, device="cuda", requires_grad=True)
    args = [x, torch.zeros_like(x), w, w, w]
    for i in range(len(args)):
        with fa.dual_level(), pytest.raises(NotImplementedError, match="forward-mode"):
            kept = args[i]
            args[i] = fa.make_dual(kept.detach(), torch.ones_like(kept))
            try:
                E.residual_norm(*args)
            finally:
                args[i] = kept
    out = E.residual_norm(*args)
    x.add_(1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        (out[0] if isinstance(out, tuple) else out).sum().backward()
