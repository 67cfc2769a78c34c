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


def test_overlap():
    """Byte ranges that meet, over types and views that start inside each other."""
    from euler_characteristic_curves_amd.train import _overlap
    t = torch.zeros(100)
    half = torch.zeros(100, dtype=torch.float16)
    for a, b, want in ((t, t, True), (t[:50], t[50:], False), (t[:51], t[50:], True), (t[50:], t[:51], True),
                       (t[10:20], t, True), (t, t[99:], True), (t, half, False), (t[:0], t, False),
                       (half[:10], half.view(torch.float32)[4:], True), (half[:10], half.view(torch.float32)[5:], False)):
        assert _overlap(a, b) is want


def test_whole_steps():
    from euler_characteristic_curves_amd.train import _whole
    assert _whole(5) == 5 and _whole(5.0) == 5
    for big in (2 ** 31, 2 ** 32 + 5, 10 ** 30):
        assert _whole(big) == 2 ** 31 - 1 and _whole(-big) == -1
    for bad in (5.7, True, "5", None):
        with pytest.raises(TypeError):
            _whole(bad)


def test_norm_workspace_of_large_batches():
    """Rows for folded partial sums are there only where a sample has more partial rows than it is folded to: a batch
    of small samples takes a fraction of its features, not several times them."""
    from euler_characteristic_curves_amd._lib import lib
    for batch, voxels, channels, groups in ((1024, 64, 512, 32), (32768, 1, 64, 8), (64, 64 * 64, 320, 32), (256, 1024, 64, 8)):
        need = lib.ecc_norm_workspace_bytes(batch, voxels, channels, groups)
        # two rows a sample where one workgroup sums it, and no more than 1024 + batch where several do
        rows = batch + max(batch, 1024 + batch)
        assert need <= rows * (3 * channels + 1) * 8 + batch * groups * 8 + 256
    # 40 workgroups a sample: folded to 32
    assert lib.ecc_norm_workspace_bytes(1, 40 * 8192, 1, 1) >= (40 + 1 + 32) * 4 * 8


def test_factors_of_the_momentum_step_beyond_float32():
    """Finite arguments whose products the kernels could only have as infinity are refused, not applied."""
    from euler_characteristic_curves_amd import _lib
    from tests.test_train_cpu import muon
    for bad in (dict(momentum=1e39), dict(momentum=-1e300), dict(lr=1e20, scale=1e20), dict(lr=1e20, decay=-1e20),
                dict(lr=-1e39)):
        assert muon(_lib, **bad) == _lib.ECC_E_VALUE, bad
        assert b"float32" in _lib.lib.ecc_last_error()
    # in range, and refused for the workspace only
    assert muon(_lib, lr=1e30, scale=1e-30, decay=1e-30, ws=None) == _lib.ECC_E_WORKSPACE
