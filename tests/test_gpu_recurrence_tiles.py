"""The gated recurrence where a workgroup takes several tiles in turn, and where there are more parts than groups that
join them (tests/test_block_limits_cpu.py asserts that these sizes are such), against float64: states and gradients that
are carried from tile to tile, lengths that end inside a part, NaN behind them."""

import pytest
import torch

from tests.gpu_util import banner, need_gpu
from tests.test_gpu_recurrence import check_all, make

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
# whole sequences, parts of several tiles, parts beyond 64
SHAPES = [(260, 1100, 5), (260, 1100, 1), (70, 700, 300), (20, 4000, 201), (1, 45000, 2)]


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_tiles_in_turn(shape, dtype):
    banner("recurrence tiles", shape, dtype)
    t, n, gh, gl = make(*shape, dtype, True, shape[0] > 1, seed=sum(shape))
    if n is not None:
        behind = torch.arange(shape[1])[None] >= n[:, None]
        for v, bad in ((t["x"], float("nan")), (t["gate"], float("inf")), (gh, float("nan"))):
            v[behind] = bad
    check_all(t, n, gh, gl)


@pytest.mark.parametrize("which", ["h", "last"])
def test_one_gradient_through_tiles(which):
    banner("recurrence tiles one", which)
    t, n, gh, gl = make(70, 700, 300, BF16, True, True, seed=3)
    check_all(t, n, gh if which == "h" else None, gl if which == "last" else None)
