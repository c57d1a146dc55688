"""The example that trains an expert layer in bf16 and serves it in 4 bits: that it runs, and its gradients."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("expert_weights", os.path.join(ROOT, "examples", "expert_weights.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_runs_and_repeats(example):
    losses, served = example.train(steps=4)
    assert len(losses) == 4 and all(math.isfinite(v) for v in losses + [served])
    assert example.train(steps=4) == (losses, served)


def test_gradients(example):
    dev = torch.device("cuda:0")
    torch.manual_seed(1)
    layer, splits = example.Layer(dev), [300, 0, 17, 83]
    x, target = torch.randn(400, example.HIDDEN, device=dev).to(torch.bfloat16), torch.randn(400, example.OUT, device=dev)
    counts = torch.tensor(splits, dtype=torch.int32, device=dev)
    out, dx = layer.forward_backward(x, counts, target)
    w, xd = layer.copy.double(), x.double()
    at = 0
    for e, c in enumerate(splits):
        rows = slice(at, at + c)
        want = xd[rows] @ w[e].t()
        size = xd[rows].abs() @ w[e].abs().t()
        assert ((out[rows].double() - want).abs() <= size * 2 * example.HIDDEN * 2.0 ** -24 + want.abs() * 2.0 ** -24).all()
        d = (out[rows] - target[rows]).to(torch.bfloat16).double()  # what the gradients are of
        for got, value, size, terms in ((dx[rows], d @ w[e], d.abs() @ w[e].abs(), example.OUT),
                                        (layer.grad[e], d.t() @ xd[rows], d.abs().t() @ xd[rows].abs(), c + 1)):
            assert ((got.double() - value).abs() <= size * 2 * terms * 2.0 ** -24 + value.abs() * 2.0 ** -24).all()
        at += c
