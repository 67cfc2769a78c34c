"""What the built library's metadata says of its kernels: none of a residual block's keeps registers in memory."""

import os
import struct

import pytest

import euler_characteristic_curves_amd

msgpack = pytest.importorskip("msgpack")
LIB = os.path.join(os.path.dirname(euler_characteristic_curves_amd.__file__), "libecc_mi355.so")


def kernels():
    """{name: metadata} of every kernel, from the notes of the code objects in the library."""
    with open(LIB, "rb") as f:
        data = f.read()
    found, at = {}, data.find(b"AMDGPU\0\0")
    while at >= 0:
        size, desc, kind = struct.unpack("<III", data[at - 12:at])
        if (size, kind) == (7, 32):
            for k in msgpack.unpackb(data[at + 8:at + 8 + desc], strict_map_key=False)["amdhsa.kernels"]:
                found[k[".name"]] = k
        at = data.find(b"AMDGPU\0\0", at + 8)
    return found


@pytest.mark.parametrize("part", ["glu_", "recurrence_", "residual_"])
def test_no_kernel_keeps_registers_in_memory(part):
    mine = {n: k for n, k in kernels().items() if part in n}
    assert mine
    # (scalar registers are kept in a vector register's lanes, never in memory)
    bad = {n: (k[".vgpr_spill_count"], k[".private_segment_fixed_size"]) for n, k in mine.items()}
    bad = {n: v for n, v in bad.items() if any(v)}
    assert not bad, bad
