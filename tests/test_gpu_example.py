"""The example that trains through the curves runs, and learns."""

import importlib.util
import os

import pytest

from tests.gpu_util import banner, need_gpu

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_through_curves.py")


def test_training_through_the_curves():
    need_gpu()
    banner("train through curves")
    spec = importlib.util.spec_from_file_location("train_through_curves", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses = example.train(40)
    assert all(x == x for x in losses)
    # smooth and rough volumes have very different curves: chance is log 2 = 0.69
    assert sum(losses[-5:]) / 5 < 0.35 < sum(losses[:5]) / 5
