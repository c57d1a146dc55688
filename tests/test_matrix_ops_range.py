"""The bf16 and 4-bit products at the ends of their types' ranges (include/lpc_ops.h): subnormal bf16 operands, sums below FP32's
normal numbers, every exponent byte.

Tolerance, the header's: 2 k u of the sum of the terms' magnitudes, u = 2^-24, and 2 k 2^-149 where these are below FP32's normal
numbers: each of the k additions there is off by at most a step of 2^-149, as matrix cores' additions are counted with twice the
half step of rounding to nearest; a term that vanishes because it is less than half of that step is one of them."""
import numpy as np
import pytest
import torch

from fp8_precision_allreduce_amd import lpc

pytestmark = pytest.mark.gpu
STEP, U = 2.0 ** -149, 2.0 ** -24
GRID = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
SIZES = [(3, 256, 40), (70, 640, 520), (300, 520, 512), (2100, 384, 1288)]  # narrow tiles of each kind, small and large ones


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lpc.lib()
    return torch.device("cuda:0")


def near(got, x, w, k):
    want, size = x @ w.t(), x.abs() @ w.abs().t()
    tol = 2 * k * torch.maximum(size * U, torch.tensor(STEP, dtype=torch.float64))
    bad = ~((got.cpu().double() - want).abs() <= tol)
    assert not bad.any(), "%d of %d" % (int(bad.sum()), bad.numel())


def scaled(rows, k, exponent, seed):
    """Normal data times 2^exponent, in bf16."""
    v = torch.from_numpy(np.random.RandomState(seed).standard_normal((rows, k)))
    return (v * 2.0 ** exponent).float().to(torch.bfloat16)


@pytest.mark.parametrize("rows,k,n", SIZES)
@pytest.mark.parametrize("ex,ew", [(-130, 100), (-128, 0), (-70, -70), (-70, -60), (60, 55), (120, -120)])
def test_bf16_products(dev, rows, k, n, ex, ew):
    print("[case] bf16", rows, k, n, ex, ew, flush=True)
    x, w = scaled(rows, k, ex, 1), scaled(n, k, ew, 2)
    out = torch.empty(rows, n, device=dev)
    lpc.lpc_gemm_bf16(x.to(dev), w.to(dev), out)
    near(out, x.double(), w.double(), k)
    y = torch.empty(rows, k, device=dev)
    dy = scaled(rows, n, ex, 3)
    lpc.lpc_gemm_bf16_dgrad(dy.to(dev), w.to(dev), y)
    near(y, dy.double(), w.double().t(), n)


@pytest.mark.parametrize("rows,k,n", [(r, -(-k // 128) * 128, n) for r, k, n in SIZES])
@pytest.mark.parametrize("ex,ew", [(0, 252), (2, 127), (2, 118), (60, 60), (55, 55), (2, 2), (180, 180), (250, 5), (None, 120)])
def test_mxfp4_products(dev, rows, k, n, ex, ew):
    """ex, ew: mean exponent bytes; None: any, block by block, that leaves sums finite."""
    print("[case] mxfp4", rows, k, n, ex, ew, flush=True)
    rng = np.random.RandomState(4)

    def operand(rows, byte):
        codes = torch.from_numpy(rng.randint(0, 16, (rows, k)))
        low, high = (0, 241) if byte is None else (max(byte - 2, 0), min(byte + 3, 253))
        scales = torch.from_numpy(rng.randint(low, high, (rows, k // 32)))
        values = GRID[codes] * torch.pow(2.0, (scales - 127).double()).repeat_interleave(32, 1)
        return (codes[:, ::2] | codes[:, 1::2] << 4).to(torch.uint8).to(dev), scales.to(torch.uint8).to(dev), values

    xc, xs, x = operand(rows, ex)
    wc, ws, w = operand(n, ew)
    out = torch.empty(rows, n, device=dev)
    lpc.lpc_gemm_mxfp4(xc, xs, wc, ws, out)
    near(out, x, w, k)
