"""Backward passes of a residual block's operators captured beside graphs of the same leaves that are alive: those that
the capture can join are taken, the others leave the rest alone."""

import pytest
import torch

import euler_characteristic_curves_amd as E
from tests.gpu_util import banner, need_gpu

pytestmark = pytest.mark.gpu
CALLS = {"norm": lambda x, w: E.rms_norm(x, w[0]), "recurrence": lambda x, w: E.gated_recurrence(x, x * 0.5)[0],
         "residual": lambda x, w: E.residual_norm(x, x * 0.5)[1], "linear": lambda x, w: E.gated_linear(x, w, w)}


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def leaves(seed):
    gen = torch.Generator().manual_seed(seed)
    return [torch.randn(*s, generator=gen).cuda().requires_grad_() for s in ((2, 7, 12), (12, 12))]


def replays(graph, got, want):
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        torch.ones(1000, device="cuda").sum()   # the program's own work between
        torch.cuda.synchronize()


@pytest.mark.parametrize("which", CALLS)
def test_warmed_up_on_a_side_stream(which):
    """The usual recipe: some steps on a side stream, of which the last one's loss is still held, then a capture."""
    banner("block warm-up", which)
    x, w = leaves(1)
    g = torch.ones(2, 7, 12, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            held = CALLS[which](x, w)
            want = torch.autograd.grad(held, [x], g, retain_graph=True)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(CALLS[which](x, w), [x], g)
    replays(graph, got, want)
    assert held.grad_fn is not None


@pytest.mark.parametrize("which", ["linear", "norm"])
def test_gradients_that_are_not_wanted(which):
    """An eager graph holds the weights; the captured pass is of the features alone."""
    banner("block not wanted", which)
    x, w = leaves(2)
    call = CALLS["linear"]
    if which == "norm":
        w = w.detach()[0].clone().requires_grad_()
        call = E.rms_norm
    g = torch.ones(2, 7, 12, device="cuda")
    held = call(torch.ones(2, 7, 12, device="cuda"), w)
    want = torch.autograd.grad(call(x, w), [x], g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(call(x, w), [x], g)
    replays(graph, got, want)
    assert held.grad_fn is not None
