"""The torch binding of the training operators on the CPU: what it refuses, and
what it asks of its arguments, before a GPU is touched."""

import pytest
import torch
import torch.autograd.forward_ad as fa

import euler_characteristic_curves_amd as E  # noqa: F401  (loads the library that the binding needs)
from euler_characteristic_curves_amd import _torch


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("dual", range(5), ids=["x", "weight", "bias", "readout", "offset"])
def test_forward_mode_is_refused(dual, grad):
    """A tangent is not dropped: no voxels, so that nothing is launched."""
    args = [torch.zeros(0, 3, 4), *(torch.zeros(n) for n in (4, 4, 4, 1))]
    plan = ([0, 3, 4, 2], 0, 0, 0, 0, 1e-5, True)
    assert _torch.norm(*args, *plan).shape == (0, 3)
    with fa.dual_level():
        args[dual] = fa.make_dual(args[dual].requires_grad_(grad), torch.ones_like(args[dual]))
        for enabled in (True, False):
            with torch.set_grad_enabled(enabled), pytest.raises(NotImplementedError, match="forward-mode"):
                _torch.norm(*args, *plan)
