"""The gated recurrence behind a sequence's end: steps that are not there leave the state, and the gradient that comes to
it, as they are, infinite ones too, in one part and in several."""

import pytest
import torch

import euler_characteristic_curves_amd as E
from tests.gpu_util import banner, need_gpu

pytestmark = pytest.mark.gpu
INF = float("inf")
# one tile, tiles in turn, parts; channels alone and in pairs
SHAPES = [(3, 3, 5), (3, 40, 1), (2, 700, 6), (2, 5000, 7), (300, 900, 33)]


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def make(B, T, C, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    x, gate = (torch.randn(B, T, C, generator=gen).to(dtype) for _ in range(2))
    return x, gate, torch.randn(B, C, generator=gen), torch.zeros(B, dtype=torch.int64)


def run(x, gate, state, n, gh=None, gl=None):
    t = [v.cuda().requires_grad_() for v in (x, gate, state)]
    h, last = E.gated_recurrence(*t, n.cuda())
    out = [h.detach().cpu(), last.detach().cpu()]
    if gl is not None:
        outs, grads = ([last], [gl.cuda()]) if gh is None else ([h, last], [gh.cuda(), gl.cuda()])
        out += [g.cpu() for g in torch.autograd.grad(outs, t, grads)]
    return out


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16], ids=["f32", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_no_steps(shape, dtype):
    banner("recurrence no steps", shape, dtype)
    x, gate, state, n = make(*shape, dtype, 1)
    state[0, 0], state[1, -1], state[1, 0] = INF, -INF, float("nan")
    gl = torch.randn(state.shape, generator=torch.Generator().manual_seed(2))
    gl[0, -1], gl[-1, 0] = -INF, INF
    h, last, gx, gg, gs = run(x, gate, state, n, gl=gl)
    assert torch.equal(last.nan_to_num(nan=7.0), state.nan_to_num(nan=7.0)) and torch.equal(gs, gl)
    assert not h.any() and not gx.any() and not gg.any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16], ids=["f32", "f16"])
@pytest.mark.parametrize("shape", SHAPES[1:], ids=lambda s: "x".join(map(str, s)))
def test_infinite_last_step(shape, dtype):
    """An infinite input that a step takes in part is an infinite state, and stays one."""
    banner("recurrence infinite end", shape, dtype)
    B, T, C = shape
    x, gate, state, n = make(*shape, dtype, 3)
    n += torch.arange(B) * 37 % T
    n[0], n[1] = T, max(T - 5, 1)
    plain = run(x, gate, state, n)
    for b in range(B):
        if n[b] > 0:
            x[b, n[b] - 1, 0], gate[b, n[b] - 1, 0] = INF, 2.0
    h, last = run(x, gate, state, n)
    some = n > 0
    assert (h[some, n[some] - 1, 0] == INF).all() and (last[some, 0] == INF).all()
    assert torch.equal(last[:, 1:], plain[1][:, 1:]) and torch.equal(last[~some], state[~some])


@pytest.mark.parametrize("shape", SHAPES[1:], ids=lambda s: "x".join(map(str, s)))
def test_infinite_gradient_of_the_last_state(shape):
    """It reaches the last step there is, where what a step takes in part is infinite."""
    banner("recurrence infinite gradient", shape)
    B, T, C = shape
    x, gate, state, n = make(*shape, torch.float32, 4)
    n += 1 + torch.arange(B) * 37 % (T - 1)
    gl, every = torch.ones(B, C), torch.arange(B)
    gate[every, n - 1, 0] = 2.0
    plain = run(x, gate, state, n, gl=gl)
    gl[:, 0] = INF
    got = run(x, gate, state, n, gl=gl)
    assert (got[2][every, n - 1, 0] == INF).all()
    for a, b in zip(got[2:], plain[2:]):
        assert torch.equal(a[..., 1:], b[..., 1:])
