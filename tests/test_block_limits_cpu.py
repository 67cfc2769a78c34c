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


def test_rows_of_the_projections(L):
    """Rows that one launch has threads for, 2^24 - 1 workgroups of 256, are taken, others refused: the forward pass of
    narrow sums, 64 turns of 64 rows a workgroup, the gradients, tiles of 256 rows."""
    f = L.lib.ecc_gated_linear_workspace_bytes
    for rows, C, F, d, backward, ok in ((1 << 34, 8, 8, 2, 0, True), ((1 << 36) - (1 << 16), 8, 8, 2, 0, True),
                                        (1 << 36, 8, 8, 2, 0, False), ((1 << 32) - 512, 8, 8, 2, 1, True),
                                        ((1 << 32) + 1, 8, 8, 2, 1, False), (1 << 23, 1024, 16384, 2, 0, True),
                                        (1 << 25, 256, 32768, 2, 0, False), (1 << 23, 1024, 2816, 2, 1, True)):
        assert (f(rows, C, F, d, backward) > 0) == ok, (rows, C, F, d, backward)
    args = (FAKE, 2, 1 << 36, 8, 8, FAKE, FAKE, None, None, 2)
    assert L.lib.ecc_gated_linear_fwd(*args, FAKE, FAKE, 1 << 62, None) == L.ECC_E_SHAPE
    # beside an operand that is not aligned, tiles of 256 rows
    odd = ctypes.c_void_p(0x1002)
    assert L.lib.ecc_gated_linear_fwd(FAKE, 2, 1 << 34, 8, 8, odd, FAKE, None, None, 2, FAKE, FAKE, 1 << 62, None) == L.ECC_E_SHAPE
    assert L.lib.ecc_gated_linear_bwd(*args, FAKE, *([FAKE] * 3), None, None, FAKE, 1 << 62, None) == L.ECC_E_SHAPE


def test_workspace_of_wide_gradients(L):
    """dx's sums are not shared out where there are tiles enough, however many units they run over: the workspace holds
    the projections' gradients (8 bytes a unit and row in 16 bits, 8 in float32) and little beside."""
    f = L.lib.ecc_gated_linear_workspace_bytes
    for d in (0, 2):
        for hidden in (8192, 8193, 12000, 28672):
            rows, C = 131072, 4096
            room = rows * 8 * (hidden + 63)
            assert f(rows, C, hidden, d, 1) <= room + 2 * hidden * C * 4 * 9 + (1 << 24), (d, hidden)


def test_tiles_of_the_recurrence(L):
    """The sizes of tests/test_gpu_recurrence_tiles.py have several tiles a part, or parts for more than 64 groups."""
    from tests.test_gpu_recurrence_tiles import SHAPES

    for B, T, C in SHAPES:
        for d in (0, 1):
            tiles = L.lib.ecc_gated_recurrence_saved_bytes(B, T, C, d) // (B * C * 4)
            parts = max((L.lib.ecc_gated_recurrence_workspace_bytes(B, T, C, d) - 256) // (B * C * 16), 1)
            if B == 1:
                assert parts > 64, (B, T, C, d, tiles, parts)
            else:
                assert tiles > parts and (parts > 1) == (T == 4000), (B, T, C, d, tiles, parts)
