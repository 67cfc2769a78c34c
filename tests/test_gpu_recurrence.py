"""The gated recurrence on the GPU against float64 (tests/block_bounds.py): states, outputs and every gradient, over
types, lengths from one step to many tiles and parts, odd channel counts, ragged batches, gates at their ends."""

import pytest
import torch
import torch.autograd.forward_ad as fa

import euler_characteristic_curves_amd as E
from tests.block_bounds import recurrence
from tests.gpu_util import banner, need_gpu
from tests.norm_bounds import worst

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def make(B, T, C, dtype, state=True, lengths=None, seed=0):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    t = {"x": rnd(B, T, C).to(dtype), "gate": (rnd(B, T, C) + 7 * torch.rand(C, generator=gen) - 1).to(dtype)}
    if state:
        t["state"] = rnd(B, C)
    n = None
    if lengths:
        n = torch.randint(0, T + 1, (B,), generator=gen)
        n[0], n[-1] = T, 0
    return t, n, rnd(B, T, C).to(dtype), rnd(B, C)


def check_all(t, n, gh, gl, dev=None):
    want = recurrence(**t, lengths=n, gh=gh, glast=gl)
    d = {k: v.cuda() for k, v in t.items()} if dev is None else dev
    d = {k: v.requires_grad_() for k, v in d.items()}
    dn = None if n is None else n.cuda()
    with torch.no_grad():
        plain = E.gated_recurrence(**d, lengths=dn)
    outs = E.gated_recurrence(**d, lengths=dn)
    torch.cuda.synchronize()
    for a, b in zip(plain, outs):
        assert torch.equal(a, b)
    pairs = [(o, g) for o, g in zip(outs, (gh, gl)) if g is not None]
    grads = torch.autograd.grad([o for o, _ in pairs], list(d.values()), [g.cuda() for _, g in pairs])
    torch.cuda.synchronize()
    got = {"h": outs[0], "last": outs[1], **dict(zip(d, grads))}
    for name, v in got.items():
        assert v.dtype == (F32 if name in ("last", "state") else t["x"].dtype)
        ratio = worst(v, want[name])
        assert ratio <= 1.0, (name, ratio)


SHAPES = [(1, 1, 1), (3, 1, 2), (2, 2, 3), (1, 4, 130), (2, 5, 8), (1, 9, 17), (3, 64, 64), (2, 65, 129), (1, 257, 33),
          (2, 1000, 7), (1, 3001, 96), (4, 130, 513), (300, 70, 5)]


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_shapes(shape, dtype):
    banner("recurrence", shape, dtype)
    check_all(*make(*shape, dtype, seed=sum(shape)))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(5, 3, 9), (6, 70, 40), (4, 1500, 11)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("state", [True, False])
def test_ragged(shape, dtype, state):
    """What lies behind a sequence's length holds NaN and infinities, which reach nothing."""
    banner("recurrence ragged", shape, dtype, state)
    t, n, gh, gl = make(*shape, dtype, state, True, seed=7)
    behind = torch.arange(shape[1])[None] >= n[:, None]
    for v, bad in ((t["x"], float("nan")), (t["gate"], float("inf")), (gh, float("nan"))):
        v[behind] = bad
    t["gate"][behind.nonzero()[-1][0], -1] = float("nan")
    check_all(t, n, gh, gl)


def test_lengths_out_of_range_are_cut():
    banner("recurrence lengths")
    t, _, gh, gl = make(3, 20, 6, F32, seed=8)
    check_all(t, torch.tensor([-5, 1 << 40, 7]), gh, gl)


@pytest.mark.parametrize("which", ["h", "last"])
def test_one_gradient_alone(which):
    banner("recurrence one", which)
    t, n, gh, gl = make(3, 150, 20, F32, lengths=True, seed=9)
    check_all(t, n, gh if which == "h" else None, gl if which == "last" else None)


@pytest.mark.parametrize("value", [0.0, 7.0, 12.0, -12.0])
def test_gates_alike(value):
    """The same gate at every step: errors of k would add up, over as many steps as a state lasts."""
    banner("recurrence alike", value)
    t, n, gh, gl = make(1, 6000, 4, F32, seed=10)
    t["gate"] = torch.full_like(t["gate"], value)
    t["x"] = 1 + 0.1 * t["x"]
    check_all(t, n, gh, gl)
    # a constant input is the steady state, whatever the gates: within half a step of every step's own scale
    ones = torch.ones(1, 6000, 4, device="cuda")
    h, last = E.gated_recurrence(ones, t["gate"].cuda(), torch.ones(1, 4, device="cuda"))
    assert torch.equal(h, ones) and torch.equal(last, torch.ones_like(last))


def test_gates_at_their_ends():
    """Infinite gates keep or replace the state exactly; a state far larger than what replaces it leaves nothing."""
    banner("recurrence ends")
    inf = float("inf")
    x = torch.arange(1.0, 9.0).reshape(1, 8, 1).repeat(1, 1, 2)
    gate = torch.tensor([inf, -inf, inf, inf, -inf, -200.0, 200.0, -inf]).reshape(1, 8, 1).repeat(1, 1, 2)
    h, last = E.gated_recurrence(x.cuda(), gate.cuda(), torch.full((1, 2), 1e30, device="cuda"))
    want = torch.tensor([1e30, 2, 2, 2, 5, 6, 6, 8])
    assert torch.equal(h[0, :, 0].cpu(), want) and torch.equal(last.cpu(), torch.full((1, 2), 8.0))
    t, n, gh, gl = make(1, 300, 3, F32, seed=11)
    t["state"] = t["state"] * 1e20
    t["gate"][:, 150] = -60.0
    check_all(t, n, gh, gl)


def test_nan_stays_in_its_channel_and_behind():
    banner("recurrence nan")
    for bad in (float("nan"), float("inf")):
        t, _, gh, gl = make(2, 200, 6, F32, seed=12)
        t["x"][1, 90, 3] = bad
        d = {k: v.cuda().requires_grad_() for k, v in t.items()}
        h, last = E.gated_recurrence(**d)
        ok = torch.ones(2, 200, 6, dtype=torch.bool)
        ok[1, 90:, 3] = False
        assert torch.equal(torch.isfinite(h).cpu(), ok)
        gx, gg = torch.autograd.grad([h, last], [d["x"], d["gate"]], [gh.cuda(), gl.cuda()])
        assert torch.isfinite(gx).all()  # the gradient of x does not see x
        assert torch.isfinite(gg[0]).all() and torch.isfinite(gg[1][:, [0, 1, 2, 4, 5]]).all()
        assert torch.isfinite(gg[1, :90, 3]).all()


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=["f32", "f16", "bf16"])
def test_steps_in_turn_are_the_sequence(dtype):
    """A sequence in pieces, one step at a time among them, states carried: the same states to their roundings."""
    banner("recurrence pieces", dtype)
    t, _, _, _ = make(3, 150, 37, dtype, seed=13)
    d = {k: v.cuda() for k, v in t.items()}
    want = recurrence(**t)
    state, parts, at = d["state"], [], 0
    for size in (1, 1, 1, 64, 3, 70, 1, 9):
        h, state = E.gated_recurrence(d["x"][:, at:at + size], d["gate"][:, at:at + size], state)
        parts.append(h)
        at += size
    assert at == 150
    assert worst(torch.cat(parts, dim=1), want["h"]) <= 1 and worst(state, want["last"]) <= 1


def test_unaligned_and_strided():
    banner("recurrence strides")
    for dtype in (F32, F16):
        t, n, gh, gl = make(3, 75, 22, dtype, lengths=True, seed=14)
        dev = {}
        for k, v in t.items():
            flat = torch.zeros(v.numel() + 1, dtype=v.dtype, device="cuda")
            flat[1:] = v.cuda().reshape(-1)
            dev[k] = flat[1:].view(v.shape).detach()
        check_all(t, n, gh, gl, dev=dev)
        dev = {k: v.cuda() for k, v in t.items()}
        dev["x"] = dev["x"].transpose(1, 2).contiguous().transpose(1, 2).detach()
        dev["gate"] = torch.cat([dev["gate"], dev["gate"]], dim=1)[:, :75].detach()
        dev["state"] = dev["state"].t().contiguous().t().detach()
        check_all(t, n, gh, gl, dev=dev)
        check_all(t, n, gh[:1, :1].expand(gh.shape), gl[:1].expand(gl.shape))


def test_shared_state_sums_its_gradient():
    """One initial state for the whole batch: its gradient is the sum over the batch."""
    banner("recurrence shared state")
    t, _, gh, gl = make(5, 40, 6, F32, seed=15)
    one = t["state"][:1].cuda().requires_grad_()
    h, last = E.gated_recurrence(t["x"].cuda(), t["gate"].cuda(), one.expand(5, 6))
    (g,) = torch.autograd.grad([h, last], [one], [gh.cuda(), gl.cuda()])
    v, b = recurrence(t["x"], t["gate"], t["state"][:1].expand(5, 6), gh=gh, glast=gl)["state"]
    assert worst(g, (v.sum(0, keepdim=True), b.sum(0, keepdim=True) + 5 * 2.0 ** -24 * v.abs().sum(0, keepdim=True))) <= 1


def test_empty():
    banner("recurrence empty")
    for B, T in ((0, 5), (3, 0)):
        x = torch.zeros(B, T, 4, device="cuda", requires_grad=True)
        s = torch.randn(B, 4, device="cuda", requires_grad=True)
        h, last = E.gated_recurrence(x, x, s)
        assert h.shape == x.shape and torch.equal(last, s)
        gx, gs = torch.autograd.grad(last.sum() + h.sum(), [x, s])
        assert gx.shape == x.shape and torch.equal(gs, torch.ones_like(s))
        assert torch.equal(E.gated_recurrence(x, x)[1], torch.zeros_like(s))


def test_differences():
    """Along one direction, the step's terms of third order taken from float64."""
    banner("recurrence differences")
    t, n, gh, gl = make(2, 30, 5, F32, lengths=False, seed=16)
    h = 2.0 ** -6
    d = {k: v.cuda().requires_grad_() for k, v in t.items()}
    grads = dict(zip(d, torch.autograd.grad(E.gated_recurrence(**d), list(d.values()), [gh.cuda(), gl.cuda()])))
    both = (("h", gh), ("last", gl))
    bounds = recurrence(**t)
    for name in t:
        v = torch.sign(torch.randn(t[name].shape, generator=torch.Generator().manual_seed(1)))
        refs = []
        for step in (h, h / 2):
            side = [recurrence(**{k: (u.double() if k != name else u.double() + s * step * v) for k, u in t.items()})
                    for s in (1, -1)]
            refs.append(sum(float(((side[0][o][0] - side[1][o][0]) * g.double()).sum()) for o, g in both) / (2 * step))
        sides = [E.gated_recurrence(**{k: (u if k != name else u + s * h * v).cuda() for k, u in t.items()}) for s in (1, -1)]
        mine = sum(float(((a.double() - b.double()).cpu() * g.double()).sum()) for a, b, g in zip(*sides, (gh, gl))) / (2 * h)
        slack = 2.4 * sum(float((bounds[o][1] * g.double().abs()).sum()) for o, g in both) / (2 * h)
        along = float((grads[name].double().cpu() * v.double()).sum())
        cubic = 4 / 3 * abs(refs[0] - refs[1])
        assert abs(mine - along) <= slack + 2 * cubic + 1e-5 * float(grads[name].abs().sum()), name


def test_streams_and_graph():
    """Two streams at once, and a graph replayed with eager work between."""
    banner("recurrence graph")
    shape = (3, 700, 48)
    t, n, gh, gl = make(*shape, BF16, lengths=True, seed=17)
    gh, gl, n = gh.cuda(), gl.cuda(), n.cuda()

    def step(ts):
        outs = E.gated_recurrence(**ts, lengths=n)
        return [*(o.detach() for o in outs), *torch.autograd.grad(outs, list(ts.values()), [gh, gl])]

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
        fresh = make(*shape, BF16, lengths=True, seed=20 + i)[0]
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
    banner("recurrence refusals")
    x = torch.zeros(2, 3, 4, device="cuda")
    s, n = torch.zeros(2, 4, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")
    for kw, exc in ((dict(x=x[0]), ValueError), (dict(gate=x[:, :2]), ValueError), (dict(gate=x.half()), TypeError),
                    (dict(x=x.double(), gate=x.double()), TypeError), (dict(gate=x.cpu()), ValueError),
                    (dict(state=s.half()), TypeError), (dict(state=s[:1]), ValueError), (dict(state=s.cpu()), ValueError),
                    (dict(lengths=n.int()), TypeError), (dict(lengths=n[:1]), ValueError), (dict(lengths=n.cpu()), ValueError),
                    (dict(lengths=[1, 2]), TypeError), (dict(x=x[..., :0], gate=x[..., :0]), ValueError)):
        with pytest.raises(exc):
            E.gated_recurrence(**{"x": x, "gate": x, **kw})
    h, _ = E.gated_recurrence(x.requires_grad_(), x.detach())
    (g,) = torch.autograd.grad(h.sum(), [x], create_graph=True)
    with pytest.raises(RuntimeError, match="once"):
        g.sum().backward()


def test_duals_and_changed_inputs():
    """Tangents are refused, not dropped, and an input written after the call is noticed by its backward pass."""
    banner("recurrence duals")
    x = torch.zeros(2, 3, 4, device="cuda")
    args = [x, torch.zeros_like(x), torch.zeros(2, 4, device="cuda", requires_grad=True)]
    for i in range(len(args)):
        with fa.dual_level(), pytest.raises(NotImplementedError, match="forward-mode"):
            kept = args[i]
            args[i] = fa.make_dual(kept.detach(), torch.ones_like(kept))
            try:
                E.gated_recurrence(*args)
            finally:
                args[i] = kept
    out = E.gated_recurrence(*args)
    x.add_(1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        (out[0] if isinstance(out, tuple) else out).sum().backward()
