"""Sizes of a residual block's operators at the limits of a launch, a sum or a workspace, without a GPU."""

import ctypes

import pytest

FAKE = ctypes.c_void_p(0x1000)   # never dereferenced


@pytest.fixture(scope="module")
def L():
    from euler_characteristic_curves_amd import _lib
    return _lib


def test_batches_of_the_recurrence(L):
    """Any batch below 2^31 is taken, in launches of at most 2^24 - 1 workgroups of 256 threads."""
    for f in (L.lib.ecc_gated_recurrence_workspace_bytes, L.lib.ecc_gated_recurrence_saved_bytes):
        for B, T, C in (((1 << 24) - 1, 4, 8), (1 << 24, 4, 8), ((1 << 31) - 1, 1, 1), (1 << 20, 1, 1 << 20)):
            assert f(B, T, C, 2) > 0, (B, T, C)
        assert f(1 << 31, 1, 1, 2) == 0
    call = L.lib.ecc_gated_recurrence_fwd
    assert call(FAKE, FAKE, 2, 1 << 31, 1, 1, None, None, FAKE, FAKE, None, FAKE, 1 << 40, None) == L.ECC_E_SHAPE
