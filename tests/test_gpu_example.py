"""The training example runs, its loss falls far below chance (log 512 = 6.2),
and its first steps repeat."""
import math
import os
import sys

import pytest

from gpu_util import log

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def example():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import train_experts
    return train_experts


def test_training_example_learns(example):
    losses = example.train(steps=60, log=log)
    assert all(math.isfinite(x) for x in losses)
    assert abs(losses[0] - math.log(512)) < 2.0
    assert losses[-1] < 1.0


def test_training_example_repeats(example):
    """No atomics in the operators' sums: the first steps repeat closely (the
    embedding's gradient is added by torch in any order)."""
    a, b = example.train(steps=3, log=log), example.train(steps=3, log=log)
    assert a[0] == b[0]
    assert all(abs(x - y) < 1e-2 for x, y in zip(a, b))
