"""Newton-Schulz orthogonalisation and the momentum step on the GPU against
float64 (tests/orth_bounds.py)."""

import pytest
import torch

import euler_characteristic_curves_amd as E
from tests.gpu_util import banner, need_gpu
from tests.orth_bounds import HALF, check, orthogonal

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def gradient(shape, dtype=F32, seed=0, scale=1e-3):
    """A few strong directions over a weak background."""
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    *lead, m, n = shape
    r = max(1, min(m, n) // 8)
    strong = (rnd(*lead, m, r) * torch.linspace(1, 0.05, r)) @ rnd(*lead, r, n)
    return ((strong / r ** 0.5 + 0.3 * rnd(*shape)) * scale).to(dtype)


SIZES = [(1, 1), (1, 7), (7, 1), (3, 5), (27, 64), (64, 27), (33, 31), (64, 64), (65, 64), (64, 200), (100, 300),
         (129, 128), (127, 400), (400, 127), (513, 260), (300, 1000), (16, 4000), (4000, 5), (640, 640)]


@pytest.mark.parametrize("m,n", SIZES, ids=lambda v: str(v))
def test_sizes(m, n):
    banner("orth", m, n)
    g = gradient((m, n), seed=m + n)
    check(E.orthogonalize(g.cuda()), g, F32)


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(3, 40, 70), (5, 200, 90), (2, 150, 151), (24, 64, 216), (1, 256, 2100), (40, 8, 9)],
                         ids=lambda s: "x".join(map(str, s)))
def test_stacks_and_types(shape, dtype):
    banner("orth stack", shape, dtype)
    g = gradient(shape, dtype, seed=sum(shape))
    out = E.orthogonalize(g.cuda())
    assert out.dtype == dtype and out.shape == g.shape
    for i in range(shape[0]):
        check(out[i], g[i], dtype)


@pytest.mark.parametrize("m,n", [(20, 30), (192, 256)], ids=str)
def test_steps_and_coefficients(m, n):
    banner("orth coefficients", m, n)
    g = gradient((m, n), seed=2)
    for kw in (dict(steps=1), dict(steps=2), dict(steps=9), dict(steps=8, coefficients=(1.5, -0.5, 0.0)),
               dict(steps=6, coefficients=(15 / 8, -10 / 8, 3 / 8)), dict(steps=3, coefficients=(0.5, 0.0, 0.0)),
               dict(eps=0.5)):
        check(E.orthogonalize(g.cuda(), **kw), g, F32, **kw)


@pytest.mark.parametrize("m,n", [(20, 30), (150, 260)], ids=str)
def test_scales(m, n):
    """Gradients far below eps keep float32's relative precision, and ones whose squares overflow float32 too."""
    banner("orth scales", m, n)
    for scale in (1e-15, 1e-9, 1e-3, 1e15, 1e30):
        g = gradient((m, n), seed=3, scale=scale)
        check(E.orthogonalize(g.cuda()), g, F32)
    assert torch.equal(E.orthogonalize(torch.zeros(m, n, device="cuda")).cpu(), torch.zeros(m, n))


@pytest.mark.parametrize("m,n", [(20, 30), (150, 260)], ids=str)
def test_low_rank_and_diagonal(m, n):
    banner("orth rank", m, n)
    gen = torch.Generator().manual_seed(4)
    one = torch.randn(m, 1, generator=gen) @ torch.randn(1, n, generator=gen)
    check(E.orthogonalize(one.cuda()), one, F32)
    eye = torch.eye(m, n) * torch.linspace(1, 1e-3, m)[:, None]
    check(E.orthogonalize(eye.cuda()), eye, F32)


@pytest.mark.parametrize("m,n", [(20, 30), (130, 200)], ids=str)
def test_nan_stays_in_its_matrix(m, n):
    banner("orth nan", m, n)
    for bad in (float("nan"), float("inf")):
        g = gradient((3, m, n), seed=5)
        g[1, 2, 3] = bad
        out = E.orthogonalize(g.cuda())
        assert torch.isnan(out[1]).all()
        check(out[0], g[0], F32)
        check(out[2], g[2], F32)


def test_layouts():
    banner("orth layouts")
    g = gradient((90, 140), seed=6)
    t = g.T.contiguous().cuda().T
    assert not t.is_contiguous()
    check(E.orthogonalize(t), g, F32)
    flat = torch.zeros(g.numel() + 1, device="cuda")
    flat[1:] = g.cuda().reshape(-1)
    check(E.orthogonalize(flat[1:].view(90, 140)), g, F32)
    d = g.cuda()
    assert E.orthogonalize(d, out=d) is d
    check(d, g, F32)
    assert E.orthogonalize(torch.zeros(0, 5, 6, device="cuda")).shape == (0, 5, 6)
    assert E.orthogonalize(torch.zeros(5, 0, device="cuda")).shape == (5, 0)


def reference_step(p, g, buf, lr, momentum, nesterov, decay, scale, **kw):
    """(param, its bound, buffer, its bound) in float64 for one matrix."""
    dt = p.dtype
    p, g, buf = p.double(), g.double(), buf.double()
    new = momentum * buf + (1 - momentum) * g
    nb = 4 * 2.0 ** -24 * ((momentum * buf).abs() + ((1 - momentum) * g).abs())
    u = (1 - momentum) * g + momentum * new if nesterov else new
    want, bound = orthogonal(u, **kw)
    # the update's own rounding enters the iteration as a relative error of its input
    a = 3.9 ** kw.get("steps", 5)
    bound = bound + a * 8 * 2.0 ** -24
    out = (1 - lr * decay) * p - lr * scale * want
    pb = HALF[dt] * out.abs() + 4 * 2.0 ** -24 * (p.abs() + lr * scale * want.abs())
    return out, (float(torch.linalg.matrix_norm(pb)) + lr * scale * bound), new, nb


@pytest.mark.parametrize("pdtype,gdtype", [(F32, F32), (F32, BF16), (BF16, BF16), (F16, F16), (F32, F16)],
                         ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("shape", [(3, 64, 216), (130, 90), (2, 140, 300)], ids=lambda s: "x".join(map(str, s)))
def test_muon(shape, nesterov, pdtype, gdtype):
    banner("muon", shape, nesterov, pdtype, gdtype)
    gen = torch.Generator().manual_seed(7)
    p = (torch.randn(*shape, generator=gen) / shape[-1] ** 0.5).to(pdtype)
    g, buf = gradient(shape, gdtype, seed=8), gradient(shape, seed=9)
    dp, dg, db = p.cuda(), g.cuda(), buf.cuda()
    kw = dict(lr=0.02, momentum=0.95, nesterov=nesterov)
    scale = max(1.0, shape[-2] / shape[-1]) ** 0.5
    before = dp._version
    E.muon_step([dp], [dg], [db], weight_decay=0.1, **kw)
    assert dp._version > before
    assert torch.equal(dg.cpu(), g)
    sel = [()] if len(shape) == 2 else list(range(shape[0]))
    for i in sel:
        out, ob, new, nb = reference_step(p[i], g[i], buf[i], decay=0.1, scale=scale, **kw)
        assert ((db[i].double().cpu() - new).abs() <= nb).all()
        assert float(torch.linalg.matrix_norm(dp[i].double().cpu() - out)) <= ob


def test_muon_list_and_repeat():
    """Two parameters in one call give what two calls give, bit for bit, on any stream."""
    banner("muon list")
    gen = torch.Generator().manual_seed(10)
    ps = [torch.randn(*s, generator=gen) for s in ((3, 30, 50), (200, 170))]
    gs, bs = [gradient(p.shape, seed=11) for p in ps], [gradient(p.shape, seed=12) for p in ps]
    cu = lambda ts: [t.cuda() for t in ts]  # noqa: E731
    a, b = (cu(ps), cu(gs), cu(bs)), (cu(ps), cu(gs), cu(bs))
    E.muon_step(*a, lr=0.1, scale=0.5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for i in range(2):
            E.muon_step([b[0][i]], [b[1][i]], [b[2][i]], lr=0.1, scale=0.5)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for x, y in zip(a, b):
        for t, u in zip(x, y):
            assert torch.equal(t, u)


@pytest.mark.parametrize("shape", [(4, 27, 64), (2, 140, 300)], ids=lambda s: "x".join(map(str, s)))
def test_graph_replays(shape):
    banner("muon graph", shape)
    gen = torch.Generator().manual_seed(13)
    p0 = torch.randn(*shape, generator=gen)
    p, g, b = p0.cuda(), gradient(shape, seed=14).cuda(), torch.zeros(shape, device="cuda")
    ep, eg, eb = p.clone(), g.clone(), b.clone()
    E.muon_step([ep.clone()], [eg], [eb.clone()], lr=0.05)  # loads the kernels
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        E.muon_step([p], [g], [b], lr=0.05)
    for i in range(3):
        fresh = gradient(shape, seed=20 + i).cuda()
        g.copy_(fresh)
        graph.replay()
        torch.cuda.synchronize()
        E.muon_step([ep], [fresh], [eb], lr=0.05)
        torch.cuda.synchronize()
        assert torch.equal(p, ep) and torch.equal(b, eb), i


def test_refusals():
    banner("orth refusals")
    g = torch.ones(4, 6, device="cuda")
    for bad, exc in ((dict(steps=0), E.EccError), (dict(steps=65), E.EccError), (dict(eps=-1.0), E.EccError),
                     (dict(coefficients=(float("nan"), 0, 0)), E.EccError),
                     (dict(coefficients=(40.0, 0.0, 0.0)), E.EccError), (dict(coefficients=(1.0, 2.0)), ValueError),
                     (dict(out=torch.ones(6, 4, device="cuda")), ValueError),
                     (dict(out=torch.ones(4, 6, device="cuda", dtype=F16)), TypeError)):
        with pytest.raises(exc):
            E.orthogonalize(g, **bad)
    with pytest.raises(TypeError):
        E.orthogonalize(g.double())
    with pytest.raises(ValueError):
        E.orthogonalize(g[0])
    p, b = g.clone(), g.clone()
    for args in (([p], [g], []), ([p], [g.half()[:2]], [b]), ([p, g[0]], [g, g[0]], [b, b[0]])):
        with pytest.raises(ValueError):
            E.muon_step(*args, lr=0.1)
    with pytest.raises(TypeError):
        E.muon_step([p], [g], [b.half()], lr=0.1)
    with pytest.raises(E.EccError):
        E.muon_step([p], [g], [b], lr=float("inf"))
    torch.cuda.synchronize()
    assert torch.equal(p, g) and torch.equal(b, g)


# short sides of one to four tiles of 16, and longer ones; one workgroup a matrix, and several; both orientations
CARRIED = [(2, 16, 300), (3, 45, 47), (2, 777, 37), (2, 37, 777), (1, 48, 3001), (1, 3000, 61), (1, 64, 2500), (2, 1500, 64),
           (1, 5, 9000), (300, 20, 70), (70, 170), (170, 70), (2, 100, 900), (900, 130), (3, 129, 260), (1, 300, 2500)]


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", CARRIED, ids=lambda s: "x".join(map(str, s)))
def test_short_side_carried_through_the_steps(shape, dtype):
    banner("orth carried", shape, dtype)
    g = gradient(shape, dtype, seed=sum(shape))
    d = g.cuda()
    out = E.orthogonalize(d)
    assert E.orthogonalize(d, out=d) is d and torch.equal(d, out)
    stack, outs = (g, out) if g.dim() == 3 else (g[None], out[None])
    for i in sorted({0, len(stack) // 2, len(stack) - 1}):
        check(outs[i], stack[i], dtype)


@pytest.mark.parametrize("m,n", [(20, 60), (40, 900), (900, 40), (100, 700)], ids=str)
def test_short_side_steps_scales_and_broken_values(m, n):
    """Few and many steps (which turn to the direct iteration), both ends of the range, NaN, zero and rank one."""
    banner("orth carried steps", m, n)
    for kw in (dict(steps=1), dict(steps=2), dict(steps=8), dict(steps=9), dict(steps=12, coefficients=(1.5, -0.5, 0.0)),
               dict(steps=3, coefficients=(0.5, 0.0, 0.0)), dict(eps=0.5)):
        g = gradient((m, n), seed=2)
        check(E.orthogonalize(g.cuda(), **kw), g, F32, **kw)
    for scale in (1e-15, 1e-9, 1e15, 1e30):
        g = gradient((m, n), seed=3, scale=scale)
        check(E.orthogonalize(g.cuda()), g, F32)
    assert torch.equal(E.orthogonalize(torch.zeros(m, n, device="cuda")).cpu(), torch.zeros(m, n))
    gen = torch.Generator().manual_seed(4)
    one = torch.randn(m, 1, generator=gen) @ torch.randn(1, n, generator=gen)
    check(E.orthogonalize(one.cuda()), one, F32)
    for bad in (float("nan"), float("inf")):
        g = gradient((3, m, n), seed=5)
        g[1, 2, 3] = bad
        out = E.orthogonalize(g.cuda())
        assert torch.isnan(out[1]).all()
        check(out[0], g[0], F32)
        check(out[2], g[2], F32)


def test_unaligned_carried():
    banner("orth carried unaligned")
    for m, n in ((33, 131), (131, 33), (40, 901), (901, 40)):
        g = gradient((m, n), BF16, seed=6)
        flat = torch.zeros(g.numel() + 1, dtype=BF16, device="cuda")
        flat[1:] = g.cuda().reshape(-1)
        check(E.orthogonalize(flat[1:].view(m, n)), g, BF16)


def test_tiles_beyond_whole_rounds():
    """More tiles than the card holds at a time: the last ones are shared out."""
    banner("orth rounds")
    g = gradient((40, 640, 800), seed=8)
    out = E.orthogonalize(g.cuda())
    for i in (0, 20, 38, 39):
        check(out[i], g[i], F32)


@pytest.mark.parametrize("pdtype,gdtype", [(F32, F32), (F32, BF16), (BF16, BF16), (F16, F16)], ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("shape", [(2, 27, 64), (2, 50, 901), (900, 33), (100, 700)], ids=lambda s: "x".join(map(str, s)))
def test_muon_carried(shape, nesterov, pdtype, gdtype):
    test_muon(shape, nesterov, pdtype, gdtype)


@pytest.mark.parametrize("shape", [(2, 50, 900), (700, 100)], ids=lambda s: "x".join(map(str, s)))
def test_graph_replays_carried(shape):
    test_graph_replays(shape)


@pytest.mark.parametrize("shape", [(2, 140, 300), (2, 45, 700), (1000, 1000), (9, 130, 140)],
                         ids=lambda s: "x".join(map(str, s)))
def test_repeats_bit_for_bit(shape):
    """No value depends on which workgroup wrote last."""
    banner("orth repeats", shape)
    g = gradient(shape, seed=15).cuda()
    first = E.orthogonalize(g)
    for _ in range(20):
        assert torch.equal(E.orthogonalize(g), first)
