"""The shapes of tests/orth_products.py take every way in which
orth_share (csrc/ecc_train_internal.hpp) hands a product out, so that the GPU
tests run every product kernel: compiled for the host and asked."""

import os
import shutil
import subprocess

import pytest

from tests.orth_products import STACKS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "euler_characteristic_curves_amd", "csrc")


@pytest.fixture(scope="module")
def classes(tmp_path_factory):
    """Function from stacks to the set of (way, product, tile, pair, deep, shared, has whole workgroups)."""
    cxx = shutil.which("g++")
    if cxx is None or not os.path.exists("/opt/rocm/include/hip/hip_runtime.h"):
        pytest.skip("g++ or the HIP headers are not available")
    exe = str(tmp_path_factory.mktemp("orth") / "orth_products")
    r = subprocess.run([cxx, "-O1", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", f"-I{CSRC}",
                        os.path.join(ROOT, "tests", "host", "orth_products.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def ask(stacks):
        out = subprocess.run([exe] + ["%d,%d,%d" % s for s in stacks], capture_output=True, text=True, check=True).stdout
        found = set()
        for line in out.splitlines():
            _, way, *products = line.split()
            for p in products:
                name, numbers = p.split(":")
                tile, pair, deep, splits, whole, _ = map(int, numbers.split(","))
                found.add((way, name, tile, pair, deep, splits > 1, whole > 0))
        return found
    return ask


def test_every_way_is_tested(classes):
    scan = [(b, m, n) for b in (1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 40) for m in range(65, 1800, 64)
            for n in (m, m + 30, 3 * m // 2, 2 * m - 1, 3 * m, 5 * m) if b * m * n <= 9e6 or (b == 40 and m == 641)]
    want, got = classes(scan), classes(STACKS)
    assert len(want) >= 30
    assert want <= got, sorted(want - got)
    # the four product kernels, each with and without shares
    for tile, pair, deep in ((64, 1, 0), (128, 1, 0), (128, 2, 0), (128, 1, 1)):
        for name in ("gram", "poly", "update", "last"):
            assert any(c[1:5] == (name, tile, pair, deep) for c in got), (name, tile, pair, deep)
