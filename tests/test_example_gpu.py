"""The example's training steps: routing, grouped product, its gradients, allreduce and AdamW together."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_moe_steps_learn_and_repeat():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("moe_step", os.path.join(ROOT, "examples", "moe_step.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses = example.train(steps=30)
    print(losses, flush=True)
    assert all(v == v for v in losses) and losses[-1] < losses[0] / 2
    assert example.train(steps=3)[0] == losses[0]
