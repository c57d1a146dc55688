"""Shapes that Muon refuses; no GPU needed."""
import pytest
import torch

from fp8_precision_allreduce_amd import lpc
from test_ops_abi_cpu import L  # noqa: F401


@pytest.mark.parametrize("what", ["grads", "m", "copies"])
def test_a_matrix_that_lies_the_other_way_round(L, what):  # noqa: F811
    """It has as many elements, and would be read as another matrix."""
    param = torch.zeros(4, 6)
    lists = {"grads": [param], "m": [param], "copies": [param.to(torch.bfloat16)]}
    lists[what] = [lists[what][0].t().contiguous()]
    with pytest.raises(ValueError, match=r"%s\[0\] has shape \(6, 4\), params\[0\] \(4, 6\)" % what):
        lpc.Muon([param], **lists)


@pytest.mark.parametrize("shape", [(4, 6), (1, 4, 6), (24,)])
def test_views_of_the_same_layout_pass(L, shape):  # noqa: F811
    """Up to the check that comes next: these are no GPU tensors."""
    param = torch.zeros(4, 6)
    with pytest.raises(ValueError, match="params\\[0\\] must be a GPU tensor"):
        lpc.Muon([param], [param.view(shape)], [param.view(shape)])
