"""The gated pair of projections on the GPU against float64 (tests/block_bounds.py): outputs and every gradient, over
types, sizes that fill tiles, straddle them and end within a step, activations, strides, streams and graphs."""

import pytest
import torch
import torch.autograd.forward_ad as fa

import euler_characteristic_curves_amd as E
from tests.block_bounds import gated_linear
from tests.gpu_util import banner, need_gpu
from tests.norm_bounds import worst

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
NAMES = ("x", "w_gate", "w_up", "b_gate", "b_up")


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def make(shape, hidden, dtype, bias=True, seed=0):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    C = shape[-1]
    t = {"x": rnd(*shape), "w_gate": rnd(hidden, C) / C ** 0.5, "w_up": rnd(hidden, C) / C ** 0.5}
    if bias:
        t.update(b_gate=0.3 * rnd(hidden), b_up=0.3 * rnd(hidden))
    return {k: v.to(dtype) for k, v in t.items()}, rnd(*shape[:-1], hidden).to(dtype)


def call(d, act):
    return E.gated_linear(*(d.get(k) for k in NAMES), act=act)


def check_all(t, gh, act="silu", dev=None):
    want = gated_linear(**t, act=act, gh=gh)
    d = {k: v.cuda() for k, v in t.items()} if dev is None else dev
    d = {k: v.requires_grad_() for k, v in d.items()}
    with torch.no_grad():
        plain = call(d, act)
    out = call(d, act)
    torch.cuda.synchronize()
    assert torch.equal(plain, out)
    grads = torch.autograd.grad(out, list(d.values()), gh.cuda())
    torch.cuda.synchronize()
    for name, v in {"h": out, **dict(zip(d, grads))}.items():
        assert v.dtype == t["x"].dtype
        ratio = worst(v, want[name])
        assert ratio <= 1.0, (name, ratio)


SHAPES = [((1, 1), 1), ((2, 3), 5), ((1, 40), 33), ((3, 5, 8), 16), ((64, 32), 64), ((65, 33), 66), ((16, 200), 130),
          ((17, 71), 129), ((2, 64, 64), 100), ((300, 130), 257), ((7, 1000), 40), ((1000, 24), 72), ((4, 33, 96), 512),
          ((31, 513), 7), ((515, 16), 1)]


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape,hidden", SHAPES, ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else str(v))
def test_shapes(shape, hidden, dtype):
    banner("glu", shape, hidden, dtype)
    check_all(*make(shape, hidden, dtype, seed=sum(shape)))


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_activations(act, bias, dtype):
    banner("glu act", act, bias, dtype)
    check_all(*make((130, 48), 72, dtype, bias, seed=5), act)


# large tiles, sums in shares, ends of tiles and steps inside
LARGE = [((2050, 72), 1610), ((2048, 64), 1664), ((25001, 130), 200), ((24576, 128), 256), ((300, 1033), 900), ((520, 1024), 704)]


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape,hidden", LARGE, ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else str(v))
def test_large(shape, hidden, dtype):
    banner("glu large", shape, hidden, dtype)
    check_all(*make(shape, hidden, dtype, seed=6), "gelu")


# sums of up to four steps over many rows: rows that end within a step or a chunk, units within a tile, several turns of a
# workgroup
NARROW = [((4097, 8), 70), ((5000, 40), 33), ((4200, 64), 64), ((4133, 100), 130), ((9000, 17), 5), ((4300, 128), 16),
          ((4160, 16), 6400), ((64, 65, 48), 1)]


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("shape,hidden", NARROW, ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else str(v))
def test_narrow(shape, hidden, act, dtype):
    banner("glu narrow", shape, hidden, act, dtype)
    check_all(*make(shape, hidden, dtype, act == "silu", seed=13), act)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_narrow_keeps_nan_in_its_row(dtype):
    """What lies behind a row's end belongs to the next row."""
    banner("glu narrow nan", dtype)
    t, gh = make((4200, 40), 24, dtype, seed=14)
    t["x"][7, 0] = float("nan")
    t["x"][4199, 39] = float("inf")
    d = {k: v.cuda().requires_grad_() for k, v in t.items()}
    h = call(d, "silu")
    ok = torch.ones(4200, dtype=torch.bool)
    ok[[7, 4199]] = False
    assert torch.equal(torch.isfinite(h).all(dim=1).cpu(), ok)
    (gx,) = torch.autograd.grad(h, [d["x"]], gh.cuda())
    assert torch.isfinite(gx.cpu()[ok]).all()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 8, 9, 16, 17, 32, 33])
def test_few_rows(rows, dtype):
    """What a serving program calls: few rows, weights of any alignment."""
    banner("glu few", rows, dtype)
    for C, F in ((256, 352), (1000, 77), (131, 300), (2048, 16)):
        t, _ = make((rows, C), F, dtype, bias=C != 256, seed=rows + C)
        want = gated_linear(**t)["h"]
        with torch.no_grad():
            ratio = worst(call({k: v.cuda() for k, v in t.items()}, "silu"), want)
        assert ratio <= 1, (C, F, ratio)


def test_weights_as_they_lie():
    """Weights that are identities and permutations: results are exact, and every element is where it belongs."""
    banner("glu exact")
    gen = torch.Generator().manual_seed(3)
    for dtype in (F32, F16, BF16):
        for rows, C in ((70, 96), (200, 130), (5, 300)):
            x = torch.randint(-8, 9, (rows, C), generator=gen).to(dtype)
            p, q = torch.randperm(C, generator=gen), torch.randperm(C, generator=gen)
            eye = torch.eye(C, dtype=dtype)
            h = call({"x": x.cuda(), "w_gate": eye[p].cuda(), "w_up": eye[q].cuda()}, "none")
            assert torch.equal(h.cpu(), x[:, p] * x[:, q]), (dtype, rows, C)


@pytest.mark.parametrize("dtype", [F32, F16], ids=["f32", "f16"])
def test_unaligned_and_strided(dtype):
    banner("glu strides", dtype)
    t, gh = make((90, 64), 96, dtype, seed=7)
    dev = {}
    for k, v in t.items():
        flat = torch.zeros(v.numel() + 1, dtype=v.dtype, device="cuda")
        flat[1:] = v.cuda().reshape(-1)
        dev[k] = flat[1:].view(v.shape).detach()
    check_all(t, gh, dev=dev)
    dev = {k: v.cuda() for k, v in t.items()}
    dev["x"] = dev["x"].t().contiguous().t().detach()
    dev["w_gate"] = torch.cat([dev["w_gate"]] * 2, dim=1)[:, :64].detach()
    dev["w_up"] = dev["w_up"].t().contiguous().t().detach()
    dev["b_up"] = torch.stack([dev["b_up"]] * 2, dim=1)[:, 0].detach()
    check_all(t, gh, dev=dev)
    check_all(t, gh[:1].expand(gh.shape))


def test_shared_weight_sums_its_gradient():
    """One matrix as both weights: autograd adds the two gradients."""
    banner("glu shared")
    t, gh = make((50, 40), 24, F32, bias=False, seed=8)
    w = t["w_gate"].cuda().requires_grad_()
    (g,) = torch.autograd.grad(E.gated_linear(t["x"].cuda(), w, w), [w], gh.cuda())
    want = gated_linear(t["x"], t["w_gate"], t["w_gate"], gh=gh)
    v, b = (want["w_gate"][i] + want["w_up"][i] for i in (0, 1))
    assert worst(g, (v, b + 2.0 ** -24 * v.abs())) <= 1


def test_nan_and_infinity_stay_in_their_row_and_unit():
    banner("glu nan")
    for dtype in (F32, BF16):
        for rows, C, F in ((70, 40, 100), (3, 40, 100)):
            for bad in (float("nan"), float("inf")):
                t, gh = make((rows, C), F, dtype, seed=9)
                t["x"][1, C - 1] = bad
                d = {k: v.cuda().requires_grad_() for k, v in t.items()}
                h = call(d, "silu")
                assert torch.isfinite(h[[0, 2]]).all() and not torch.isfinite(h[1]).all()
                (gx,) = torch.autograd.grad(h, [d["x"]], gh.cuda())
                assert torch.isfinite(gx[[0, 2]]).all()
                t, gh = make((rows, C), F, dtype, seed=9)
                t["w_up"][F - 1, 0] = bad
                h = call({k: v.cuda() for k, v in t.items()}, "silu")
                assert torch.isfinite(h[:, :F - 1]).all() and not torch.isfinite(h[:, F - 1]).any()


def test_subsets_of_gradients():
    banner("glu subsets")
    t, gh = make((70, 24), 40, F32, seed=10)
    want = gated_linear(**t, gh=gh)
    for absent in ((), ("b_gate",), ("b_up",)):
        here = [k for k in NAMES if k not in absent]
        ref = want if not absent else gated_linear(**{k: t[k] for k in here}, gh=gh)
        for mask in range(1, 1 << len(here)):
            d = {k: t[k].cuda() for k in here}
            names = [k for i, k in enumerate(here) if mask >> i & 1]
            for k in names:
                d[k].requires_grad_()
            grads = torch.autograd.grad(call(d, "silu"), [d[k] for k in names], gh.cuda())
            for k, v in zip(names, grads):
                assert worst(v, ref[k]) <= 1, (absent, names, k)


def test_empty():
    banner("glu empty")
    x = torch.zeros(0, 4, 8, device="cuda", requires_grad=True)
    w = torch.ones(6, 8, device="cuda", requires_grad=True)
    h = E.gated_linear(x, w, w)
    assert h.shape == (0, 4, 6)
    gx, gw = torch.autograd.grad(h.sum(), [x, w])
    assert gx.shape == x.shape and torch.equal(gw, torch.zeros_like(w))


def test_differences():
    """Along one direction, the step's terms of third order taken from float64."""
    banner("glu differences")
    t, gh = make((9, 24), 12, F32, seed=11)
    h = 2.0 ** -6
    d = {k: v.cuda().requires_grad_() for k, v in t.items()}
    grads = dict(zip(d, torch.autograd.grad(call(d, "gelu"), list(d.values()), gh.cuda())))
    bound = gated_linear(**t, act="gelu")["h"][1]
    for name in t:
        v = torch.sign(torch.randn(t[name].shape, generator=torch.Generator().manual_seed(1)))
        refs = []
        for step in (h, h / 2):
            side = [gated_linear(**{k: (u.double() if k != name else u.double() + s * step * v) for k, u in t.items()},
                                 act="gelu")["h"][0] for s in (1, -1)]
            refs.append(float(((side[0] - side[1]) * gh.double()).sum()) / (2 * step))
        sides = [call({k: (u if k != name else u + s * h * v).cuda() for k, u in t.items()}, "gelu") for s in (1, -1)]
        mine = float(((sides[0].double() - sides[1].double()).cpu() * gh.double()).sum()) / (2 * h)
        slack = 2.4 * float((bound * gh.double().abs()).sum()) / (2 * h)
        along = float((grads[name].double().cpu() * v.double()).sum())
        cubic = 4 / 3 * abs(refs[0] - refs[1])
        assert abs(mine - along) <= slack + 2 * cubic + 1e-5 * float(grads[name].abs().sum()), name


@pytest.mark.parametrize("shape,hidden", [((130, 72), 100), ((8200, 64), 70)])
def test_streams_and_graph(shape, hidden):
    """Two streams at once, and a graph replayed with eager work between."""
    banner("glu graph", shape, hidden)
    t, gh = make(shape, hidden, BF16, seed=12)
    gh = gh.cuda()

    def step(d):
        out = call(d, "silu")
        return [out.detach(), *torch.autograd.grad(out, list(d.values()), gh)]

    def leaves():
        return {k: v.cuda().requires_grad_() for k, v in t.items()}

    first = step(leaves())
    streams, results = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                results.append(step(leaves()))
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for r in results:
        for a, b in zip(first, r):
            assert torch.equal(a, b)
    del results
    mine = leaves()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(mine)
    for i in range(3):
        fresh, _ = make(shape, hidden, BF16, seed=20 + i)
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
    banner("glu refusals")
    x, w, b = (torch.zeros(*s, device="cuda") for s in ((3, 8), (5, 8), (5,)))
    for kw, exc in ((dict(w_gate=w[:, :4]), ValueError), (dict(w_up=w[:4]), ValueError), (dict(w_gate=w[0]), ValueError),
                    (dict(w_gate=w.half()), TypeError), (dict(w_up=w.cpu()), ValueError), (dict(b_gate=b[:3]), ValueError),
                    (dict(b_up=b.half()), TypeError), (dict(b_gate=w), ValueError), (dict(x=x.double()), TypeError),
                    (dict(act="tanh"), ValueError), (dict(w_up=None), TypeError), (dict(x=x[..., :0]), ValueError),
                    (dict(w_gate=w[:0], w_up=w[:0]), ValueError)):
        with pytest.raises(exc):
            E.gated_linear(**{"x": x, "w_gate": w, "w_up": w, **kw})
    wide = torch.zeros(32769, 2, device="cuda")
    with pytest.raises(E.EccError):
        E.gated_linear(x[:, :2], wide, wide)
    h = E.gated_linear(x.requires_grad_(), w, w)
    (g,) = torch.autograd.grad(h.sum(), [x], create_graph=True)
    with pytest.raises(RuntimeError, match="once"):
        g.sum().backward()


def test_duals_and_changed_inputs():
    """Tangents are refused, not dropped, and an input written after the call is noticed by its backward pass."""
    banner("glu duals")
    x = torch.zeros(3, 8, device="cuda")
    w, b = (torch.zeros(*s, device="cuda", requires_grad=True) for s in ((5, 8), (5,)))
    args = [x, w, w, b, b]
    for i in range(len(args)):
        with fa.dual_level(), pytest.raises(NotImplementedError, match="forward-mode"):
            kept = args[i]
            args[i] = fa.make_dual(kept.detach(), torch.ones_like(kept))
            try:
                E.gated_linear(*args)
            finally:
                args[i] = kept
    out = E.gated_linear(*args)
    x.add_(1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        (out[0] if isinstance(out, tuple) else out).sum().backward()
