"""Muon's symmetric products where a whole tile of 256 x 256 lies below the diagonal: its sums are stored on both sides of it."""
import pytest
import torch

from fp8_precision_allreduce_amd import lpc
from test_matrix_ops_gpu import BF16, check_muon, dev, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(56, 450, 460), (56, 460, 450), (56, 512, 576), (56, 385, 385)], ids=str)
def test_whole_tiles_below_the_diagonal(dev, shape):  # noqa: F811
    """A shorter side of 385 to 512 has three square tiles, the one below the diagonal with more than 128 rows; 56 such matrices have 21 of them
    for each XCD, too many for the last round to be split."""
    check_muon(dev, [shape], BF16)


@pytest.mark.parametrize("shape", [(450, 460), (460, 450)], ids=str)
def test_split_and_whole_tiles_agree(dev, shape):  # noqa: F811
    """One matrix by itself, whose tiles are split, and the same one 56 times: FP32 sums in another order, so that roundings to fp16 differ here and
    there; both are off by 4e-3 of the update at most."""
    g = randn(*shape, seed=5).to(dev)
    moved = []
    for batch in (1, 56):
        p = torch.zeros(batch, *shape, device=dev)
        lpc.Muon([p], [g.expand(batch, *shape).contiguous()], [torch.zeros_like(p)], scales=[1.0]).step(lr=1.0)
        assert all(torch.equal(p[0], p[i]) for i in range(batch))
        moved.append(p[0].double())
    assert float((moved[0] - moved[1]).norm() / moved[0].norm()) <= 8e-3
