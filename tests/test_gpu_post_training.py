"""The post-training example end to end: the operators, the accumulation and
the step together learn the task, and twice the same way."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import post_training
    post_training.nsg.build()
    return post_training


def test_policy_and_preference_tuning_learn(example):
    model = example.Model()
    rewards = example.policy_tuning(model)
    assert rewards[0] < 0.1 and rewards[-1] > 0.8
    losses = example.preference_tuning(model)
    assert abs(losses[0] - 0.693) < 0.01 and losses[-1] < 0.5 * losses[0]
    assert example.nsg.device_error() == 0


def test_steps_are_reproducible(example):
    import torch
    masters = []
    for _ in range(2):
        model = example.Model(3)
        example.policy_tuning(model, steps=3)
        example.preference_tuning(model, steps=2)
        masters.append(model.master.clone())
    assert torch.equal(masters[0], masters[1])
