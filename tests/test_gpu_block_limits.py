"""A residual block's operators at sizes where a launch, a sum or a workspace reaches its limit."""

import pytest
import torch

import euler_characteristic_curves_amd as E
from tests.gpu_util import banner, need_gpu

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_more_sequences_than_one_launch_has_threads_for(dtype):
    """2^24 - 1 workgroups of 256 threads are a launch's most.  What lies before, at and behind that border is what
    the same sequences give by themselves, bit for bit."""
    banner("recurrence batch", dtype)
    n, T, C = (1 << 24) + 300, 3, 2
    gen = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    x, gate, state = rnd(n, T, C).to(dtype), rnd(n, T, C).to(dtype), rnd(n, C)
    lengths = torch.randint(0, T + 1, (n,), device="cuda", generator=gen)
    gh, gl = rnd(n, T, C).to(dtype), rnd(n, C)

    def step(at):
        t = [v[at].detach().requires_grad_() for v in (x, gate, state)]
        outs = E.gated_recurrence(*t, lengths[at])
        return [*(o.detach() for o in outs), *torch.autograd.grad(outs, t, [gh[at], gl[at]])]

    every = step(slice(None))
    border = (1 << 24) - 1
    for at in (slice(0, 1000), slice(border - 500, border + 300), slice(n - 200, n)):
        for a, b in zip(every, step(at)):
            assert torch.equal(a[at], b), at
    # and all of it is the formula's, within some roundings of float32 and the result's own
    k, v, s = torch.sigmoid(gate.float()), x.float(), state
    for t in range(T):
        on = (t < lengths)[:, None]
        s = torch.where(on, k[:, t] * s + (1 - k[:, t]) * v[:, t], s)
        want = torch.where(on, s, 0.0)
        assert torch.allclose(every[0][:, t].float(), want, rtol=torch.finfo(dtype).eps, atol=1e-5)
    assert torch.allclose(every[1], s, rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=["f32", "f16", "bf16"])
def test_sums_over_many_units(dtype):
    """dx of more than 8192 hidden units, in tiles enough for the card: sums that are not shared.  In 16 bits the error
    is the result's own rounding, in float32 within a rounding for each of the 2 F terms of a sum and the (C + 4) of a
    projection."""
    banner("glu units", dtype)
    rows, C, F = 16500, 1030, 8300
    gen = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    x, wg, wu = rnd(rows, C).to(dtype), (rnd(F, C) / C ** 0.5).to(dtype), (rnd(F, C) / C ** 0.5).to(dtype)
    gh = rnd(rows, F).to(dtype)
    x.requires_grad_()
    (got,) = torch.autograd.grad(E.gated_linear(x, wg, wu, act="none"), [x], gh)
    x, g, v, u = (t.detach().double() for t in (x, gh, wg, wu))
    da, db = g * (x @ u.T), g * (x @ v.T)
    want = da @ v + db @ u
    err = (got.double() - want).abs()
    if dtype == F32:
        size = da.abs() @ v.abs() + db.abs() @ u.abs()
        reach = g.abs() * (x.abs() @ u.abs().T), g.abs() * (x.abs() @ v.abs().T)   # of the projections' roundings
        bound = 2.0 ** -24 * ((2 * F + 4) * size + (C + 4) * (reach[0] @ v.abs() + reach[1] @ u.abs()))
        assert (err <= bound).all()
    else:
        own = (want.to(dtype).double() - want).norm()
        assert err.norm() <= 1.02 * own, float(err.norm() / own)
