"""Orthogonalisation and the momentum step at the edges of their arguments:
what autograd sees of tensors written in place, tensors that share memory,
step counts, graded matrices, and shapes for every way a product is shared
out."""

import pytest
import torch

import euler_characteristic_curves_amd as E
from tests.gpu_util import banner, need_gpu
from tests.orth_bounds import HALF
from tests.orth_products import STACKS, orthogonal_on_device
from tests.test_gpu_orth import gradient

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def test_out_is_seen_by_autograd():
    """A tensor that was saved for a backward pass and is then written through `out` is noticed there."""
    banner("orth version")
    for shape in ((20, 30), (100, 120)):
        g = gradient(shape, seed=1).cuda()
        kept, w = torch.randn(shape, device="cuda"), torch.ones(shape, device="cuda", requires_grad=True)
        loss = (w * kept).sum()
        E.orthogonalize(g, out=kept)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
        loss = (w * g).sum()
        E.orthogonalize(g, out=g)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()


def test_shared_memory_is_refused():
    """Before anything is launched, and only where memory is shared in part."""
    banner("orth overlap")
    flat = torch.randn(30 * 40 + 40, device="cuda")
    g, later = flat[:1200].view(30, 40), flat[40:].view(30, 40)
    before = flat.clone()
    for a, b in ((g, later), (later, g)):
        with pytest.raises(ValueError, match="memory"):
            E.orthogonalize(a, out=b)
    p, m = torch.randn(30, 40, device="cuda"), torch.zeros(30, 40, device="cuda")
    for args in ((g, later, m), (p, g, later), (g, p, later), (p, g, g), (p, p, m)):
        with pytest.raises(ValueError, match="share memory"):
            E.muon_step(*([t] for t in args), lr=0.1)
    torch.cuda.synchronize()
    assert torch.equal(flat, before) and not m.any()
    want = E.orthogonalize(g.clone())
    one, two = torch.stack([g, g]).unbind()       # neighbours in memory
    assert torch.equal(E.orthogonalize(one, out=two), want)
    assert torch.equal(E.orthogonalize(g, out=g), want)


def test_steps_are_a_whole_number():
    """A fraction is refused, and so is a number that a 32-bit argument would cut."""
    banner("orth steps")
    g, b = gradient((20, 30), seed=1).cuda(), torch.zeros(20, 30, device="cuda")
    p = g.clone()
    for steps, exc in ((5.7, TypeError), (True, TypeError), ("5", TypeError), (None, TypeError), (2 ** 32 + 5, E.EccError),
                       (-2 ** 32 + 5, E.EccError)):
        with pytest.raises(exc):
            E.orthogonalize(g, steps=steps)
        with pytest.raises(exc):
            E.muon_step([p], [g], [b], lr=0.1, steps=steps)
    torch.cuda.synchronize()
    assert torch.equal(p, g) and not b.any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", STACKS, ids=lambda s: "x".join(map(str, s)))
def test_every_way_products_are_shared_out(shape, dtype):
    """Accuracy of the first, a middle and the last matrix, and the same bits when run again."""
    banner("orth products", shape, dtype)
    g = gradient(shape, dtype, seed=sum(shape)).cuda()
    out = E.orthogonalize(g)
    for _ in range(4):
        assert torch.equal(E.orthogonalize(g), out)
    for i in sorted({0, shape[0] // 2, shape[0] - 1}):
        want, bound = orthogonal_on_device(g[i])
        size = float(want.square().sum().sqrt())
        total = bound + HALF[dtype] * size + 1e-7 * HALF[dtype] * want.numel() ** 0.5
        err = float((out[i].double() - want).square().sum().sqrt())
        assert err <= total, (i, err, total)


@pytest.mark.parametrize("shape", [(1, 1409, 1411), (4, 1411, 1000), (32, 260, 257), (6, 1537, 769)],
                         ids=lambda s: "x".join(map(str, s)))
def test_muon_step_on_shared_products(shape):
    """The update of the parameter in the last product of every kind of workgroup."""
    banner("muon products", shape)
    g = gradient(shape, seed=5).cuda()
    p = torch.randn(shape, generator=torch.Generator().manual_seed(6)).cuda()
    new, buf = p.clone(), torch.zeros_like(p)
    E.muon_step([new], [g], [buf], lr=0.5, momentum=0.0, nesterov=False, weight_decay=0.125, scale=1.0)
    assert torch.equal(buf, g)
    # one fused multiply-add from the product that orthogonalize rounds to float32
    want = p.double() * (1 - 0.5 * 0.125) - 0.5 * E.orthogonalize(g).double()
    assert ((new.double() - want).abs() <= 2.0 ** -23 * (p.double().abs() + want.abs() + 1)).all()


GRADED = [(130, 200), (200, 130), (512, 700), (1409, 1411), (100, 700), (512, 6000), (6000, 130), (40, 900), (64, 66)]


def iterate(g, steps=5):
    """The iteration in g's own type."""
    if g.shape[0] > g.shape[1]:
        return iterate(g.T.contiguous(), steps).T
    a, b, c = 3.4445, -4.7750, 2.0315
    x = (g / (g.double().square().sum().sqrt() + 1e-7)).to(g.dtype)
    for _ in range(steps):
        gram = x @ x.T.contiguous()
        x = a * x + (b * gram + c * gram @ gram) @ x
    return x


@pytest.mark.parametrize("shape", GRADED, ids=lambda s: "x".join(map(str, s)))
def test_graded_rows_and_columns(shape):
    """Rows and columns far below the others have the error of float32 arithmetic, down to the floor that a pair's lowest
    bit sets.

    Operands of 22 bits for 24 are 4 times as coarse; 8 allows for a row's error being one draw of many.  A pair ends at
    2^-50 of its matrix's bound (half a step of float16's smallest number, 2^-25, after the factor 2^11, over 2^14):
    sqrt(n) such errors in a row, which the five steps multiply by 3.4445 each and add to, 525 in all, and twice that for
    those of A and P.
    """
    banner("orth graded", shape)
    g = torch.randn(shape, generator=torch.Generator().manual_seed(8))
    for i, s in {3: 1e-3, 11: 1e-5, 17: 1e-7, 23: 1e-9}.items():
        g[i] *= s
        g[:, i + 1] *= s
    g = g.cuda()
    out, plain, want = E.orthogonalize(g).double(), iterate(g).double(), iterate(g.double())
    floor = 3 * 525 * max(shape) ** 0.5 * 2.0 ** -50
    for dim in (0, 1):
        err, yard = ((t - want).square().sum(dim=dim).sqrt() for t in (out, plain))
        worst = (err / (8 * yard + floor)).max()
        assert worst <= 1, (dim, float(worst))
