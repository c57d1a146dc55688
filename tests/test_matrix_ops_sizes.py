"""The matrix operators at the ends of their sizes: the most groups, operands and results whose offsets pass 32 bits, the longest
sides of Muon's matrices; and a NaN that stays in its matrix."""
import numpy as np
import pytest
import torch

from fp8_precision_allreduce_amd import lpc
from test_matrix_ops_gpu import (BF16, F32, MX, U, Guarded, check_dgrad, check_mxfp4, check_product, check_wgrad, dev,  # noqa: F401
                                 mx_oracle, near, off_by, orthogonal64, randn, say)

pytestmark = pytest.mark.gpu


def many_groups(rows):
    """Up to four rows for some of 1024 groups, at most `rows` together."""
    rng = np.random.RandomState(rows)
    counts = rng.randint(0, 5, 1024)
    for g in rng.permutation(1024):
        if counts.sum() > rows:
            counts[g] = 0
    return counts.tolist()


@pytest.mark.parametrize("rows,k,n", [(5, 128, 72), (700, 128, 72), (2500, 256, 40)])
@pytest.mark.parametrize("check", [check_product, check_dgrad, check_wgrad, check_mxfp4])
def test_the_most_groups(dev, check, rows, k, n):  # noqa: F811
    check(dev, rows, k, n, many_groups(rows), F32)


WIDE, ROWS = 65544, 70000  # 2^32 elements and more


def some_rows(out, x, w, terms, what):
    """Rows of out = x w^T by 64-bit sums: those at both ends and at a stride."""
    for r in [0, 1, 4097, ROWS // 2, ROWS - 2, ROWS - 1]:
        near(out[r].cpu(), x[r].double().cpu() @ w.double().cpu().t(), x[r].double().abs().cpu() @ w.double().abs().cpu().t(), terms, out.dtype, "%s, row %d" % (what, r))


def test_bf16_results_past_32_bits(dev):  # noqa: F811
    x, w = randn(ROWS, 8, seed=1).to(BF16).to(dev), randn(WIDE, 8, seed=2).to(BF16).to(dev)
    out = Guarded((ROWS, WIDE), BF16, dev)
    say("product", ROWS, WIDE)
    lpc.lpc_gemm_bf16(x, w, out.t)
    some_rows(out.check(), x, w, 8, "product")
    say("row gradient", ROWS, WIDE)
    lpc.lpc_gemm_bf16_dgrad(x, w.t().contiguous(), out.t)
    some_rows(out.check(), x, w, 8, "row gradient")


def test_bf16_weight_gradient_past_32_bits(dev):  # noqa: F811
    dy, x = randn(16, ROWS, seed=3).to(BF16).to(dev), randn(16, WIDE, seed=4).to(BF16).to(dev)
    dw = Guarded((ROWS, WIDE), BF16, dev)
    say("weight gradient", ROWS, WIDE)
    lpc.lpc_gemm_bf16_wgrad(dy, x, dw.t)
    some_rows(dw.check(), dy.t(), x.t(), 16, "weight gradient")


def test_bf16_weights_past_32_bits(dev):  # noqa: F811
    groups, n, k = 9, 32768, 16384
    w = torch.zeros(groups, n, k, dtype=BF16, device=dev)
    w[-1, :, :64] = randn(n, 64, seed=5).to(BF16).to(dev)
    x = randn(groups, k, seed=6).to(BF16)
    counts = torch.ones(groups, dtype=torch.int32, device=dev)
    out = Guarded((groups, n), F32, dev)
    say("weights", groups, n, k)
    lpc.lpc_gemm_bf16(x.to(dev), w, out.t, counts=counts)
    got = out.check().cpu()
    xd, wd = x[-1:, :64].double(), w[-1, :, :64].cpu().double()
    near(got[-1:], xd @ wd.t(), xd.abs() @ wd.abs().t(), 64, F32, "last group")
    assert (got[:-1] == 0).all()


def test_mxfp4_results_past_32_bits(dev):  # noqa: F811
    k = 128
    (xc, xs, x), (wc, ws, w) = mx_oracle(randn(ROWS, k, seed=7)), mx_oracle(randn(WIDE + 1, k, seed=8))
    out = Guarded((ROWS, WIDE + 1), BF16, dev)
    say("4-bit product", ROWS, WIDE + 1)
    lpc.lpc_gemm_mxfp4(xc.to(dev), xs.to(dev), wc.to(dev), ws.to(dev), out.t)
    some_rows(out.check(), x, w, k, "4-bit product")


def test_mxfp4_weights_past_32_bits(dev):  # noqa: F811
    groups, n, k = 9, 65536, 16384
    wc = torch.zeros(groups, n, k // 2, dtype=torch.uint8, device=dev)
    ws = torch.zeros(groups, n, k // MX, dtype=torch.uint8, device=dev)
    (xc, xs, x), (c, s, w) = mx_oracle(randn(groups, k, seed=9)), mx_oracle(randn(n, k // 64, seed=10))
    wc[-1, :, :k // 128], ws[-1, :, :k // 64 // MX] = c.to(dev), s.to(dev)
    out = Guarded((groups, n), F32, dev)
    say("4-bit weights", groups, n, k)
    lpc.lpc_gemm_mxfp4(xc.to(dev), xs.to(dev), wc, ws, out.t, counts=torch.ones(groups, dtype=torch.int32, device=dev))
    got = out.check().cpu()
    near(got[-1:], x[-1:, :k // 64] @ w.t(), x[-1:, :k // 64].abs() @ w.abs().t(), k, F32, "last group")
    assert (got[:-1] == 0).all()


def test_mxfp4_codec_past_32_bits(dev):  # noqa: F811
    n = (1 << 32) + 96
    x = torch.zeros(n, dtype=BF16, device=dev)
    ends = randn(2, 96, seed=11).to(BF16)
    x[:96], x[-96:] = ends[0].to(dev), ends[1].to(dev)
    codes, scales = Guarded((n // 2,), torch.uint8, dev), Guarded((n // MX,), torch.uint8, dev)
    say("codec", n)
    lpc.lpc_quantize_mxfp4(x, codes.t, scales.t)
    c, s, v = mx_oracle(ends.float())
    for i, where in enumerate((slice(None, 96), slice(-96, None))):
        part = (slice(None, 48), slice(None, 3)) if i == 0 else (slice(-48, None), slice(-3, None))
        assert torch.equal(codes.check()[part[0]].cpu(), c[i]) and torch.equal(scales.check()[part[1]].cpu(), s[i])
    assert not codes.t[48:-48].any() and not scales.t[3:-3].any()
    x.fill_(1)
    lpc.lpc_dequantize_mxfp4(codes.t, scales.t, x)
    assert torch.equal(x[:96].cpu(), v[0].to(BF16)) and torch.equal(x[-96:].cpu(), v[1].to(BF16)) and not x[96:-96].any()


@pytest.mark.parametrize("shape", [(1 << 20, 33), (33, 1 << 20), (1 << 20, 16), (3, 1 << 20)], ids=str)
def test_muon_longest_sides(dev, shape):  # noqa: F811
    """Sums of 2^20 squares in steps of 32, each off by 2^-23 of the sum at most, leave X X^T off by d = 2^15 2^-23 of itself if all
    are off the same way.  At a singular value of 1 that is (b + 2 c) d / 0.7 = 1.0 d of x', and over five iterations (1 + 1.3 + ... +
    1.3^4) d = 9 d.  With a shorter side of 32 and less the sums are held in 64 bits."""
    say("muon", shape)
    d = max(shape) / 32 * 2.0 ** -23 if min(shape) > 32 else 0.0
    g = randn(*shape, seed=12)
    p, m = Guarded(shape, F32, dev), Guarded(shape, F32, dev)
    p.t.zero_()
    m.t.zero_()
    lpc.Muon([p.t], [g.to(dev)], [m.t], scales=[1.0]).step(lr=1.0)
    want = -orthogonal64(g.double(), 5)
    m.check()
    off = float((p.check().cpu().double() - want).norm() / want.norm())
    assert off <= off_by(min(shape), 5) + 9 * d + 4 * U, off


def test_muon_nan_stays_in_its_matrix(dev):  # noqa: F811
    """Two matrices with tiles and two without, one of each with a NaN in its gradient; then the same object after new momenta."""
    shapes = [(70, 90), (70, 90), (16, 40), (16, 40)]
    clean = [randn(*s, seed=13 + i).to(dev) for i, s in enumerate(shapes)]
    state = [[torch.zeros(s, device=dev) for s in shapes] for _ in range(4)]
    (p, m), (p2, m2) = state[:2], state[2:]
    g = [t.clone() for t in clean]
    opt, other = lpc.Muon(p, g, m), lpc.Muon(p2, clean, m2)
    for i in (0, 2):
        g[i][3, 5] = float("nan")
    opt.step(lr=1.0)
    other.step(lr=1.0)
    for i in range(4):
        if i % 2 == 0:
            assert torch.isnan(p[i]).any()
        else:
            assert torch.equal(p[i], p2[i]) and torch.equal(m[i], m2[i])
    for i in (0, 2):
        p[i].zero_()
        m[i].zero_()
        g[i].copy_(clean[i])
    for i in (1, 3):
        p[i].zero_()
        m[i].zero_()
    opt.step(lr=1.0)
    for i in range(4):
        assert torch.equal(p[i], p2[i]) and torch.equal(m[i], m2[i])
