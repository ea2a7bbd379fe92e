"""The example that runs the operators and the sparse exchange together as one training step."""
import os
import runpy

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "train_step.py")


def test_the_training_step_learns_and_repeats():
    """The loss of a linear teacher falls by far more than half, and the same run gives the
    same losses: every sum of the path has a fixed order."""
    train = runpy.run_path(PATH)["train"]
    first = train(steps=40)
    assert first[-1] < 0.5 * first[0]
    assert train(steps=40) == first


def test_odd_sizes():
    train = runpy.run_path(PATH)["train"]
    losses = train(steps=25, nodes=3, examples=77, dim=101, out=63)
    assert losses[-1] < 0.7 * losses[0]
