"""Group norm with an activation and its read-out where values, lengths or
layouts are at an edge: groups that are constant or nearly so, sums over many
rows, arguments that float32 does not hold, strided inputs."""

import pytest
import torch

import euler_characteristic_curves_amd as E
from tests.gpu_util import banner, need_gpu
from tests.norm_bounds import act_and_slope

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
EPS = 1e-5
HALF32 = 2.0 ** -24


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("value", [3.25, 100.0, -1000.0])
@pytest.mark.parametrize("readout", [False, True], ids=["norm", "readout"])
@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=["f32", "f16", "bf16"])
def test_constant_group_gives_the_bias(dtype, readout, value):
    """x - mean is exactly 0, so u is the bias, whatever the mean is against 1 / sqrt(eps)."""
    banner("norm constant", dtype, readout, value)
    gen = torch.Generator().manual_seed(1)
    C = 16
    x = torch.full((2, 40, 9, C), value).to(dtype)
    w, b, r, o = (torch.randn(n, generator=gen) for n in (C, C, C, 1))
    if not readout:
        y = E.group_norm_act(x.cuda(), 4, w.cuda(), b.cuda())
        assert torch.equal(y.cpu(), b.to(dtype).expand(x.shape))
        return
    for act in ("none", "silu"):
        f = E.group_norm_readout(x.cuda(), 4, w.cuda(), b.cuda(), r.cuda(), o.cuda(), act=act).double().cpu()
        terms = act_and_slope(b.double(), act)[0] * r.double()
        # C fused additions in float32, and 2^-20 of an activation's argument
        tol = C * HALF32 * (terms.abs().sum() + o.abs()) + 2.0 ** -20 * (b * r).abs().sum()
        assert ((f - (terms.sum() + o.double())).abs() <= tol).all(), act
