"""The operators of a residual block as they are used: together, over soft curves read as sequences, trained, replayed from
a graph, carried on step by step; and over tensors whose offsets pass 32 bits."""

import pytest
import torch

import euler_characteristic_curves_amd as E
from tests.gpu_util import banner, need_gpu

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
C, HIDDEN, T, B = 48, 80, 40, 6


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def weights(gen, dtype):
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    w = {"embed": rnd(1, C), "n0": 1 + 0.1 * rnd(C), "value": rnd(C, C) / C ** 0.5, "forget": rnd(C, C) / C ** 0.5,
         "g1": 1 + 0.1 * rnd(C), "n1": 1 + 0.1 * rnd(C), "a1": 1 + 0.1 * rnd(C), "up": rnd(HIDDEN, C) / C ** 0.5,
         "gate": rnd(HIDDEN, C) / C ** 0.5, "down": rnd(HIDDEN, C) / HIDDEN ** 0.5, "g2": 1 + 0.1 * rnd(C),
         "n2": 1 + 0.1 * rnd(C)}
    vectors = ("n0", "g1", "n1", "a1", "g2", "n2")
    return {k: v.to(F32 if k in vectors else dtype) for k, v in w.items()}


def block(w, curve, lengths, state, dtype):
    """Curves [batch, thresholds] to features and the recurrence's last state: norm, recurrence, gate and norms, gated
    pair and its way back, gate and norm.  The residual stream is float32."""
    stream = curve[:, :, None] * w["embed"].float()
    z = E.rms_norm(stream, w["n0"], dtype=dtype)
    h, last = E.gated_recurrence(z @ w["value"], z @ w["forget"], state, lengths)
    stream, z = E.residual_norm(stream, h, w["g1"], w["n1"], w["a1"])
    u = E.gated_linear(z, w["gate"], w["up"]) @ w["down"]
    stream, z = E.residual_norm(stream, u, w["g2"], w["n2"], norm_branch=False)
    return z, last


def plain(w, curve, lengths, state):
    def rms(v):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6)

    stream = curve[:, :, None] * w["embed"]
    z = rms(stream) * w["n0"]
    x, f = z @ w["value"], z @ w["forget"]
    k, s, hs = torch.sigmoid(f), state, []
    for t in range(x.shape[1]):
        on = (t < lengths)[:, None]
        s = torch.where(on, k[:, t] * s + (1 - k[:, t]) * x[:, t], s)
        hs.append(torch.where(on, s, 0.0))
    stream = stream + w["g1"] * rms(torch.stack(hs, 1)) * w["a1"]
    z = rms(stream) * w["n1"]
    a = z @ w["gate"].T
    stream = stream + w["g2"] * ((a * torch.sigmoid(a) * (z @ w["up"].T)) @ w["down"])
    return rms(stream) * w["n2"], s


def curves(gen):
    fields = torch.randn(B, 12, 13, 14, generator=gen).cuda()
    tau = torch.linspace(-2.0, 2.0, T, device="cuda")
    return E.soft_ecc_batched(fields, tau, 5.0) / 100


@pytest.mark.parametrize("dtype,tol", [(F32, 2e-5), (F16, 8e-3), (BF16, 6e-2)], ids=["f32", "f16", "bf16"])
def test_together(dtype, tol):
    """Against float64 autograd.  Tolerance, relative to each result's norm: some 16 roundings to the element type lie
    between input and gradient, 16 half steps where all point one way."""
    banner("block", dtype)
    gen = torch.Generator().manual_seed(0)
    curve = curves(gen)
    w = weights(gen, dtype)
    lengths = torch.tensor([T, 7, 0, 1, T - 1, 20])
    state = torch.randn(B, C, generator=gen)
    g, gl = torch.randn(B, T, C, generator=gen), torch.randn(B, C, generator=gen)
    d = {k: v.cuda().requires_grad_() for k, v in w.items()}
    ds = state.cuda().requires_grad_()
    z, last = block(d, curve, lengths.cuda(), ds, dtype)
    got = torch.autograd.grad([z, last], [*d.values(), ds], [g.to(dtype).cuda(), gl.cuda()])
    r = {k: v.double().requires_grad_() for k, v in w.items()}
    rs = state.double().requires_grad_()
    rz, rlast = plain(r, curve.double().cpu(), lengths, rs)
    want = torch.autograd.grad([rz, rlast], [*r.values(), rs], [g.to(dtype).double(), gl.double()])
    for name, a, b in zip(("z", "last", *w, "state"), (z, last, *got), (rz, rlast, *want)):
        err = float((a.detach().double().cpu() - b.detach()).norm() / b.detach().norm())
        assert err <= tol, (name, err)


def test_step_by_step():
    """A stream carried on one threshold at a time, as a serving program calls it, is the whole sequence's."""
    banner("block steps")
    gen = torch.Generator().manual_seed(1)
    curve, w = curves(gen), {k: v.cuda() for k, v in weights(gen, BF16).items()}
    full = torch.full((B,), T, device="cuda")
    state = torch.zeros(B, C, device="cuda")
    with torch.no_grad():
        z, last = block(w, curve, full, state, BF16)
        parts = []
        for t in range(T):
            p, state = block(w, curve[:, t:t + 1], None, state, BF16)
            parts.append(p)
    err = float((torch.cat(parts, 1).float() - z.float()).norm() / z.float().norm())
    # products of one row and of many are summed in different orders: some of 8 roundings to bfloat16 fall differently
    assert err <= 8 * 2.0 ** -8, err
    assert float((state - last).norm() / last.norm()) <= 8 * 2.0 ** -8


def test_training_step_from_a_graph():
    """Forward, backward and update captured once, replayed with eager work between, and two such graphs in turn."""
    banner("block graph")
    gen = torch.Generator().manual_seed(2)
    curve = curves(gen).detach()
    lengths = torch.tensor([T, 7, 0, 1, T - 1, 20], device="cuda")
    state = torch.zeros(B, C, device="cuda")
    start = {k: v.cuda() for k, v in weights(gen, BF16).items()}

    def step(w):
        z, _ = block(w, curve, lengths, state, BF16)
        grads = torch.autograd.grad((z.float() ** 2).mean(), list(w.values()))
        with torch.no_grad():
            for t, g in zip(w.values(), grads):
                t.sub_(0.1 * g)
        return z.detach()

    def leaves():
        return {k: v.clone().requires_grad_() for k, v in start.items()}

    eager = leaves()
    want = [step(eager).clone() for _ in range(6)]
    graphs = []
    for _ in range(2):
        mine = leaves()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(mine)
        graphs.append((graph, out, mine))   # (the leaves live as long as the graph that updates them)
    for i in range(6):
        for graph, *_ in graphs:
            graph.replay()
        step(leaves())
        torch.cuda.synchronize()
        for _, out, _ in graphs:
            assert torch.equal(out, want[i]), i


def test_recurrence_beyond_32_bits():
    banner("recurrence far")
    steps, c, tail = (1 << 21) + 5, 1030, 300
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty(1, steps, c, dtype=BF16, device="cuda").normal_(generator=gen).requires_grad_()
    gate = torch.empty(1, steps, c, dtype=BF16, device="cuda").normal_(generator=gen)
    gate[:, steps - tail] = float("-inf")   # what was before leaves nothing
    gate[:, tail] = float("-inf")
    gate.requires_grad_()
    assert x.numel() > 1 << 31
    h, last = E.gated_recurrence(x, gate)
    g = torch.randn(1, tail, c, device="cuda", generator=gen).to(BF16)
    gh = torch.zeros_like(h)
    gh[:, -tail:] = g
    gx, gg = torch.autograd.grad(h, [x, gate], gh)
    xs, gs = (t.detach()[:, -tail:].clone().requires_grad_() for t in (x, gate))
    hs, ls = E.gated_recurrence(xs, gs)
    gxs, ggs = torch.autograd.grad(hs, [xs, gs], g)
    # runs are joined elsewhere in a tile: the results' own rounding may fall differently
    for a, b in ((h[:, -tail:], hs), (last, ls), (gx[:, -tail:], gxs)):
        assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -7, atol=1e-5)
    # (at the first of them the gate's gradient has the state before, which the slice does not)
    assert torch.allclose(gg[:, 1 - tail:].float(), ggs[:, 1:].float(), rtol=2.0 ** -7, atol=1e-4)
    assert not gx[:, :-tail].any()


def test_norms_beyond_32_bits():
    banner("residual far")
    rows, c = (1 << 21) + 3, 1100
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.empty(1, rows, c, dtype=F16, device="cuda").normal_(generator=gen)
    b = torch.empty(1, rows, c, dtype=F16, device="cuda").normal_(generator=gen)
    assert x.numel() > 1 << 31
    w = torch.randn(c, device="cuda", generator=gen)
    last = [t[:, -50:].clone().requires_grad_() for t in (x, b)]
    x.requires_grad_(), b.requires_grad_()
    y, z = E.residual_norm(x, b, w, w, w)
    ys, zs = E.residual_norm(*last, w, w, w)
    assert torch.equal(y[:, -50:], ys) and torch.equal(z[:, -50:], zs)
    got = torch.autograd.grad(z, [x, b], z.detach())
    want = torch.autograd.grad(zs, last, zs.detach())
    for a, s in zip(got, want):
        assert torch.equal(a[:, -50:], s)


@pytest.mark.parametrize("rows,c,hidden", [((1 << 25) + 7, 72, 40), ((1 << 22) + 9, 520, 24)])
def test_projections_beyond_32_bits(rows, c, hidden):
    banner("glu far", rows, c, hidden)
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty(rows, c, dtype=BF16, device="cuda").normal_(generator=gen)
    assert x.numel() > 1 << 31
    wg, wu = (torch.randn(hidden, c, device="cuda", generator=gen).to(BF16) / c ** 0.5 for _ in range(2))
    n = 8192
    last = x[-n:].clone().requires_grad_()
    x.requires_grad_()
    h = E.gated_linear(x, wg, wu)
    hs = E.gated_linear(last, wg, wu)
    assert torch.equal(h[-n:], hs)
    (gx,) = torch.autograd.grad(h, [x], h.detach())
    (gs,) = torch.autograd.grad(hs, [last], hs.detach())
    # (sums may be shared out differently)
    assert torch.allclose(gx[-n:].float(), gs.float(), rtol=2.0 ** -6, atol=1e-3)


def conjugate_part(t):
    """t as the imaginary part of a conjugate: in memory it lies negated."""
    out = torch.complex(torch.zeros_like(t), -t).conj().imag
    assert out.is_neg()
    return out


def test_lazily_negated():
    banner("block negated")
    gen = torch.Generator().manual_seed(6)
    t = {k: torch.randn(*s, generator=gen).cuda() for k, s in (
        ("x", (2, 7, 12)), ("b", (2, 7, 12)), ("w", (12,)), ("wg", (9, 12)), ("wu", (9, 12)), ("s", (2, 12)))}
    gy, gh = torch.randn(2, 7, 12, generator=gen).cuda(), torch.randn(2, 7, 9, generator=gen).cuda()

    def run(t, gy, gh):
        t = {k: v.detach().requires_grad_() for k, v in t.items()}
        out = [*E.residual_norm(t["x"], t["b"], t["w"], t["w"]), *E.gated_recurrence(t["x"], t["b"], t["s"]),
               E.gated_linear(t["x"], t["wg"], t["wu"]), E.rms_norm(t["x"], t["w"]),
               E.group_norm_act(t["x"], 3, t["w"], t["w"])]
        leaves = list(t.values())
        grads = [*torch.autograd.grad(out[:2], [leaves[0], leaves[1], leaves[2]], [gy, gy]),
                 *torch.autograd.grad(out[2], [leaves[0], leaves[1], leaves[5]], gy),
                 *torch.autograd.grad(out[4], [leaves[0], leaves[3], leaves[4]], gh)]
        return [o.detach() for o in out] + grads

    want = run(t, gy, gh)
    got = run({k: conjugate_part(v) for k, v in t.items()}, conjugate_part(gy), conjugate_part(gh))
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), i


@pytest.mark.parametrize("which", ["norm", "recurrence", "linear"])
def test_capture_beside_an_eager_graph_is_refused(which):
    """A captured backward pass of leaves that an eager graph holds would have the leaves' stream wait for the capturing
    one.  It is refused before, and the leaves can be captured once that graph is gone."""
    banner("block capture", which)
    gen = torch.Generator().manual_seed(7)
    x, w = torch.randn(2, 7, 12, generator=gen).cuda().requires_grad_(), torch.randn(12, 12, generator=gen).cuda()
    call = {"norm": lambda: E.rms_norm(x, w[0]), "recurrence": lambda: E.gated_recurrence(x, x)[0],
            "linear": lambda: E.gated_linear(x, w, w)}[which]
    g = torch.ones(2, 7, 12, device="cuda")
    held = call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
        with pytest.raises(RuntimeError, match="free that graph first"):
            torch.autograd.grad(out, [x], g)
    (want,) = torch.autograd.grad(held, [x], g)
    want = want.clone()
    del held, out
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (got,) = torch.autograd.grad(call(), [x], g)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("steps", [9, 700])
def test_infinite_input_of_the_recurrence(steps):
    banner("recurrence infinite", steps)
    gen = torch.Generator().manual_seed(8)
    x, gate = (torch.randn(2, steps, 5, generator=gen).cuda() for _ in range(2))
    want, _ = E.gated_recurrence(x, gate)
    x[1, 4, 3] = float("inf")
    h, last = E.gated_recurrence(x, gate)
    # x - h is infinite: infinity or, where the gate takes x and gives back a part of the difference, NaN
    assert not torch.isfinite(h[1, 4:, 3]).any() and not torch.isfinite(last[1, 3])
    keep = torch.ones_like(h, dtype=torch.bool)
    keep[1, 4:, 3] = False
    assert torch.equal(h[keep], want[keep])
