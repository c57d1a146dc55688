"""The bf16 products, the 4-bit microscaled operators and Muon (include/lpc_ops.h) on the GPU against plain implementations in
64 bits, through the public binding.

Tolerances.  u = 2^-24 is half a step of fp32 (2^-8: of bf16).  A sum of n fp32 terms is off by at most (n - 1) u of the sum of
their magnitudes where each addition is rounded to nearest; the matrix cores' additions are counted with twice that.  Codes,
exponent bytes and the values they stand for have exactly one right value."""
import numpy as np
import pytest
import torch

from fp8_precision_allreduce_amd import lpc

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
F32, BF16 = torch.float32, torch.bfloat16
MX = 32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lpc.lib()
    return torch.device("cuda:0")


def say(*a):
    print("[case]", *a, flush=True)


def spans(counts, rows):
    """First and last row of each group: negative counts are none, and groups end at `rows`."""
    at, out = 0, []
    for c in [rows] if counts is None else counts:
        c = max(0, min(c, rows - at))
        out.append((at, at + c))
        at += c
    return out


class Guarded:
    """A result buffer with a page before and after it that has to stay as it was."""

    def __init__(self, shape, dtype, dev):
        n = int(np.prod(shape))
        self.all = torch.full((n + 8192,), 77, dtype=dtype, device=dev)
        self.t = self.all[4096:4096 + n].view(shape)
        self.t.fill_(float("nan") if dtype.is_floating_point else 99)

    def check(self):
        n = self.t.numel()
        assert (self.all[:4096] == 77).all() and (self.all[4096 + n:] == 77).all(), "written outside of the result"
        return self.t


def group_counts(counts, dev):
    return None if counts is None else torch.tensor(counts, dtype=torch.int32, device=dev)


def randn(*shape, seed=0):
    return torch.from_numpy(np.random.RandomState(seed).standard_normal(shape).astype(np.float32))


def near(got, want, size, terms, dtype, what):
    """size: the sum of the terms' magnitudes."""
    got = got.cpu().double()
    tol = size * (2 * terms * U) + want.abs() * HALF[dtype] * (1 + 2.0 ** -7)
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), "%s: %d of %d, worst %g" % (what, int(bad.sum()), bad.numel(), float(((got - want).abs() - tol).max()))


# ---------------------------------------------------------------------------
# bf16 products
# ---------------------------------------------------------------------------

def check_product(dev, rows, k, n, counts, dtype, poison=False):
    say("bf16 product rows=%d k=%d n=%d counts=%s %s" % (rows, k, n, counts, dtype))
    groups = 1 if counts is None else len(counts)
    x, w = randn(rows, k, seed=1).to(BF16), randn(groups, n, k, seed=2).to(BF16)
    x[:, ::3] *= 16
    where = spans(counts, rows)
    if poison:  # rows that belong to no group are not read for any other
        x[where[-1][1]:] = float("nan")
    out = Guarded((rows, n), dtype, dev)
    lpc.lpc_gemm_bf16(x.to(dev), w.to(dev), out.t, counts=group_counts(counts, dev))
    got = out.check().cpu()
    for g, (a, b) in enumerate(where):
        xd, wd = x[a:b].double(), w[g].double()
        near(got[a:b], xd @ wd.t(), xd.abs() @ wd.abs().t(), k, dtype, "group %d" % g)
    assert (got[where[-1][1]:] == 0).all()


def check_dgrad(dev, rows, k, n, counts, dtype):
    say("bf16 dgrad rows=%d k=%d n=%d counts=%s %s" % (rows, k, n, counts, dtype))
    groups = 1 if counts is None else len(counts)
    dy, w = randn(rows, n, seed=3).to(BF16), randn(groups, n, k, seed=4).to(BF16)
    where = spans(counts, rows)
    out = Guarded((rows, k), dtype, dev)
    lpc.lpc_gemm_bf16_dgrad(dy.to(dev), w.to(dev), out.t, counts=group_counts(counts, dev))
    got = out.check().cpu()
    for g, (a, b) in enumerate(where):
        d, wd = dy[a:b].double(), w[g].double()
        near(got[a:b], d @ wd, d.abs() @ wd.abs(), n, dtype, "group %d" % g)
    assert (got[where[-1][1]:] == 0).all()


def check_wgrad(dev, rows, k, n, counts, dtype):
    say("bf16 wgrad rows=%d k=%d n=%d counts=%s %s" % (rows, k, n, counts, dtype))
    groups = 1 if counts is None else len(counts)
    dy, x = randn(rows, n, seed=5).to(BF16), randn(rows, k, seed=6).to(BF16)
    where = spans(counts, rows)
    dy[where[-1][1]:] = float("inf")  # rows of no group count nowhere
    x[where[-1][1]:] = float("nan")
    out = Guarded((groups, n, k), dtype, dev)
    lpc.lpc_gemm_bf16_wgrad(dy.to(dev), x.to(dev), out.t, counts=group_counts(counts, dev))
    got = out.check().cpu()
    for g, (a, b) in enumerate(where):
        d, xd = dy[a:b].double(), x[a:b].double()
        near(got[g], d.t() @ xd, d.abs().t() @ xd.abs(), max(b - a, 1), dtype, "group %d" % g)


DENSE = [(1, 8, 1), (1, 64, 16), (1, 4096, 1000), (2, 72, 5), (15, 136, 127), (16, 128, 128), (17, 640, 1000), (33, 1000, 257),
         (64, 1032, 384), (127, 56, 129), (128, 64, 128), (129, 200, 255), (300, 1152, 1001), (777, 520, 513), (1030, 328, 768)]
GROUPED = [(1, 256, 96, [0, 1, 0]), (40, 392, 136, [0, 17, 0, 20]), (300, 640, 264, [128, 0, 172]), (300, 72, 128, [0, 0, 0]),
           (513, 896, 304, [256, 1, 255, 1]), (500, 384, 256, [-3, 200, 1000, 5]), (200, 128, 64, [50]),
           (700, 1160, 640, [3, 0, 500, 7, 40]), (90, 64, 72, [1] * 70 + [3]),
           (300, 200, 208, [4] * 70)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,k,n", DENSE)
def test_bf16_product(dev, rows, k, n, dtype):
    check_product(dev, rows, k, n, None, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,k,n,counts", GROUPED)
def test_bf16_product_groups(dev, rows, k, n, counts, dtype):
    check_product(dev, rows, k, n - 3, counts, dtype, poison=True)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,k,n", [(r, k, -(-n // 8) * 8) for r, k, n in DENSE])
def test_bf16_dgrad(dev, rows, k, n, dtype):
    check_dgrad(dev, rows, k, n, None, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,k,n,counts", GROUPED)
def test_bf16_dgrad_groups(dev, rows, k, n, counts, dtype):
    check_dgrad(dev, rows, k, n, counts, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,k,n", [(r, k, -(-n // 8) * 8) for r, k, n in DENSE])
def test_bf16_wgrad(dev, rows, k, n, dtype):
    check_wgrad(dev, rows, k, n, None, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,k,n,counts", GROUPED)
def test_bf16_wgrad_groups(dev, rows, k, n, counts, dtype):
    check_wgrad(dev, rows, k, n, counts, dtype)


@pytest.mark.parametrize("rows,k,n,counts", [(2100, 1152, 1160, None), (3001, 648, 1304, [5, 1500, 0, 900]), (4500, 520, 2048, None),
                                             (3000, 264, 3016, None), (3500, 264, 3016, [1100, 300, 1700]), (300, 3848, 2056, None)])
def test_bf16_large(dev, rows, k, n, counts):
    """More tiles than one round of the chip's CUs in some of them; every form."""
    check_product(dev, rows, k, n - 1, counts, BF16)
    check_product(dev, rows, k, n, counts, BF16)
    check_dgrad(dev, rows, k, n, counts, F32)
    check_wgrad(dev, rows, k, n, counts, F32)


def test_bf16_no_rows(dev):
    w = torch.ones(2, 64, 32, dtype=BF16, device=dev)
    none = torch.zeros(0, 32, dtype=BF16, device=dev)
    counts = torch.zeros(2, dtype=torch.int32, device=dev)
    lpc.lpc_gemm_bf16(none, w, torch.empty(0, 64, device=dev), counts=counts)
    dw = torch.full((2, 64, 32), 5.0, device=dev)
    lpc.lpc_gemm_bf16_wgrad(torch.zeros(0, 64, dtype=BF16, device=dev), none, dw, counts=counts)
    assert (dw == 0).all()


def test_bf16_gradients_against_differences(dev):
    """The loss sum(c * out) is linear in x and in w: its difference along any direction is the gradient's product with it."""
    rows, k, n, counts = 70, 40, 48, [30, 0, 25]
    x, w = randn(rows, k, seed=1).to(BF16), randn(3, n, k, seed=2).to(BF16)
    c, step_x, step_w = randn(rows, n, seed=3).to(BF16), randn(rows, k, seed=4).to(BF16), randn(3, n, k, seed=5).to(BF16)
    dc = group_counts(counts, dev)

    def loss(x, w):
        out = torch.empty(rows, n, device=dev)
        lpc.lpc_gemm_bf16(x.to(dev), w.to(dev), out, counts=dc)
        return float((out.cpu().double() * c.double()).sum())

    dx, dw = torch.empty(rows, k, device=dev), torch.empty(3, n, k, device=dev)
    lpc.lpc_gemm_bf16_dgrad(c.to(dev), w.to(dev), dx, counts=dc)
    lpc.lpc_gemm_bf16_wgrad(c.to(dev), x.to(dev), dw, counts=dc)
    # products of all sizes are below 2^7 in magnitude here: rows n k terms' rounding stays below 1e-3 of these sums
    assert abs(loss(step_x, w) - float((dx.cpu().double() * step_x.double()).sum())) < 1e-2
    assert abs(loss(x, step_w) - float((dw.cpu().double() * step_w.double()).sum())) < 1e-2


def test_bf16_rows_longer_than_offsets(dev):
    """Rows of 8 MiB: offsets within a tile of these pass 32 bits."""
    k, rows, n = (1 << 22) + 8, 260, 3
    x = torch.zeros(rows, k, dtype=BF16, device=dev)
    w = torch.zeros(n, k, dtype=BF16, device=dev)
    ends = torch.tensor([0, 1, k // 2, k - 1], device=dev)
    x[:, ends] = randn(rows, 4, seed=1).to(BF16).to(dev)
    w[:, ends] = randn(n, 4, seed=2).to(BF16).to(dev)
    out = Guarded((rows, n), F32, dev)
    lpc.lpc_gemm_bf16(x, w, out.t)
    xd, wd = x[:, ends].cpu().double(), w[:, ends].cpu().double()
    near(out.check(), xd @ wd.t(), xd.abs() @ wd.abs().t(), 8, F32, "long rows")
    dw = Guarded((8, k), F32, dev)
    dy = randn(rows, 8, seed=3).to(BF16)
    lpc.lpc_gemm_bf16_wgrad(dy.to(dev), x, dw.t)
    got = dw.check()
    near(got[:, ends], dy.double().t() @ xd, dy.double().abs().t() @ xd.abs(), rows, F32, "long rows' gradient")
    assert int((got != 0).sum()) <= 32


# ---------------------------------------------------------------------------
# microscaled 4-bit floats
# ---------------------------------------------------------------------------

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def mx_oracle(x):
    """(codes [..., n/2], bytes [..., n/32], values) by the definition, in 64 bits."""
    b = x.double().numpy().reshape(-1, MX)
    top = np.abs(b).max(1)
    byte = np.where(top > 0, np.frexp(top)[1] - 1 - 2 + 127, 0).clip(0)
    scale = np.ldexp(1.0, byte - 127)[:, None]
    q = np.abs(b) / scale
    index = np.zeros(q.shape, dtype=np.int64)
    for i in range(7):
        half = (GRID[i] + GRID[i + 1]) / 2
        index += (q >= half) if i % 2 else (q > half)
    code = index | (np.signbit(b) * 8)
    values = np.where(np.signbit(b), -GRID[index], GRID[index]) * scale
    code = code.reshape(*x.shape[:-1], -1, 2).astype(np.uint8)
    return (torch.from_numpy(code[..., 0] | code[..., 1] << 4), torch.from_numpy(byte.astype(np.uint8)).reshape(*x.shape[:-1], -1),
            torch.from_numpy(values).reshape(x.shape))


def edges():
    """Blocks of every magnitude, ties and their neighbours, zeros of both signs, subnormals."""
    rng = np.random.RandomState(7)
    rows = []
    for e in list(range(-149, -118)) + [-60, -10, -1, 0, 1, 2, 5, 60, 120, 125, 126, 127]:
        for top in (1.0, 1.25, 1.5, 1.999):
            b = np.ldexp(top, e) * np.append(rng.choice(np.arange(0, 65) / 64, 31), 1.0) * rng.choice([-1, 1], 32)
            rows.append(b.astype(np.float32))
    rows += [np.zeros(32, np.float32), np.full(32, -0.0, np.float32)]
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0], np.float32)
    near_ties = np.concatenate([ties, np.nextafter(ties, np.float32(0)), np.nextafter(ties, np.float32(9)), -ties])
    rows.append(near_ties)
    return torch.from_numpy(np.stack(rows))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 32), (3, 32), (7, 96), (513, 64), (1000, 1152), "edges"])
def test_mxfp4_codec(dev, shape, dtype):
    say("mxfp4 codec", shape, dtype)
    x = (edges() if shape == "edges" else randn(*shape) * torch.exp(3 * randn(shape[0], 1, seed=9))).to(dtype)
    x = x.clamp(torch.finfo(dtype).min, torch.finfo(dtype).max)  # 1.999 2^127 has no finite bf16
    codes, scales = Guarded((x.shape[0], x.shape[1] // 2), torch.uint8, dev), Guarded((x.shape[0], x.shape[1] // MX), torch.uint8, dev)
    lpc.lpc_quantize_mxfp4(x.to(dev), codes.t, scales.t)
    want = mx_oracle(x.float())
    assert torch.equal(codes.check().cpu(), want[0]) and torch.equal(scales.check().cpu(), want[1])
    for out_t in (F32, BF16):
        out = Guarded(x.shape, out_t, dev)
        lpc.lpc_dequantize_mxfp4(codes.t, scales.t, out.t)
        assert torch.equal(out.check().cpu(), want[2].to(out_t)), out_t


def mx_weights(groups, n, k, seed):
    w = randn(groups, n, k, seed=seed) * torch.exp(randn(groups, n, 1, seed=seed + 50))
    return mx_oracle(w)


def check_mxfp4(dev, rows, k, n, counts, dtype):
    say("mxfp4 product rows=%d k=%d n=%d counts=%s %s" % (rows, k, n, counts, dtype))
    groups = 1 if counts is None else len(counts)
    xc, xs, x = mx_oracle(randn(rows, k, seed=11) * torch.exp(2 * randn(rows, 1, seed=12)))
    wc, ws, w = mx_weights(groups, n, k, 13)
    where = spans(counts, rows)
    xs[where[-1][1]:] = 255  # a NaN for each of the rows that belong to no group
    out = Guarded((rows, n), dtype, dev)
    lpc.lpc_gemm_mxfp4(xc.to(dev), xs.to(dev), wc.to(dev), ws.to(dev), out.t, counts=group_counts(counts, dev))
    got = out.check().cpu()
    for g, (a, b) in enumerate(where):
        near(got[a:b], x[a:b] @ w[g].t(), x[a:b].abs() @ w[g].abs().t(), k, dtype, "group %d" % g)
    assert (got[where[-1][1]:] == 0).all()


MXFP4 = [(1, 128, 1), (1, 8192, 512), (2, 384, 130), (15, 1152, 127), (16, 256, 128), (17, 640, 1000), (33, 896, 257),
         (64, 2048, 384), (65, 1152, 129), (129, 128, 255), (257, 640, 300), (300, 1152, 1000), (777, 512, 513), (2100, 1152, 1153), (3000, 256, 3001)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,k,n", MXFP4)
def test_mxfp4_product(dev, rows, k, n, dtype):
    check_mxfp4(dev, rows, k, n, None, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,k,n,counts", [
    (1, 256, 96, [0, 1, 0]), (40, 384, 130, [0, 17, 0, 20]), (300, 640, 257, [128, 0, 172]), (300, 256, 128, [0, 0, 0]),
    (513, 896, 300, [256, 1, 255, 1]), (500, 384, 256, [-3, 200, 1000, 5]), (200, 128, 64, [50]),
    (700, 1152, 640, [3, 0, 500, 7, 40]), (3000, 640, 1300, [5, 1500, 0, 900])])
def test_mxfp4_product_groups(dev, rows, k, n, counts, dtype):
    check_mxfp4(dev, rows, k, n, counts, dtype)


# ---------------------------------------------------------------------------
# Muon
# ---------------------------------------------------------------------------

def orthogonal64(u, iterations):
    x = u / u.norm() if u.norm() > 0 else u
    wide = x.shape[0] <= x.shape[1]
    for _ in range(iterations):
        a = x @ x.t() if wide else x.t() @ x
        b = -4.7750 * a + 2.0315 * a @ a
        x = 3.4445 * x + (b @ x if wide else x @ b)
    return x


def spectra(b, rows, cols, kind, seed):
    rng = np.random.RandomState(seed)
    if kind == "normal":
        return torch.from_numpy(rng.standard_normal((b, rows, cols))).float()
    rank = max(1, min(rows, cols) // 8)
    strong = torch.from_numpy(rng.standard_normal((b, rows, rank)) @ rng.standard_normal((b, rank, cols)))
    return (strong + 0.003 * torch.from_numpy(rng.standard_normal((b, rows, cols)))).float()


def off_by(side, iterations):
    """How far (2-norm, of itself) an update may be.  For the products X, A and B are rounded to fp16 (2^-11 of an element at most,
    0.4 2^-11 in the mean).  Where x' = a x + B x, what roundings e1 of X, e2 of A and e3 of B add is B x (e1 + e3) + x (b + 2 c A)
    (2 e1 + e2) A: at a singular value of 1, where B = -2.74 and x' = 0.7, that is 0.4 2^-11 sqrt(2 2.74^2 + 0.71^2 + 1.42^2) =
    8e-4, 1.2e-3 of x', in the mean, and 5.3e-3 at most.  Later iterations multiply it by at most 1.8 (the polynomial's slope between 0.65
    and 1.2), 1.3 in the mean.  Over many rows roundings are independent and the means hold: 1.2e-3 sqrt(1 + 1.3^2 + ... + 1.3^8) =
    4e-3 for five iterations.
    A shorter side of 32 and less is computed in FP32: X = R U with R up to 3.4445^5 = 485, of 17 products of 32 terms each, so in the
    mean 0.4 2^-24 sqrt(17 32) 485 = 2.7e-4 of the largest singular values; given four times that."""
    return (4e-3 if side > 32 else 1.1e-3) * 1.8 ** max(0, iterations - 5)


def check_muon(dev, shapes, grad_t, kind="normal", copies=True, nesterov=True, iterations=5, grad_scale=None, steps=1, zero=()):
    say("muon", shapes, grad_t, kind, nesterov, iterations)
    lr, beta, decay = 0.02, 0.9, 0.1
    p = [torch.from_numpy(np.random.RandomState(100 + i).standard_normal(s) * 0.02).float() for i, s in enumerate(shapes)]
    g = [spectra(s[0] if len(s) == 3 else 1, s[-2], s[-1], kind, 200 + i).reshape(s).to(grad_t) for i, s in enumerate(shapes)]
    m = [0.5 * spectra(s[0] if len(s) == 3 else 1, s[-2], s[-1], kind, 300 + i).reshape(s) for i, s in enumerate(shapes)]
    for i in zero:
        g[i], m[i] = torch.zeros_like(g[i]), torch.zeros_like(m[i])
    scales = [0.1 + 0.3 * i for i in range(len(shapes))]
    dp, dg, dm = [], [], []
    for src, to in ((p, dp), (m, dm)):
        for t in src:
            o = Guarded(t.shape, F32, dev)
            o.t.copy_(t)
            to.append(o)
    dg = [t.to(dev) for t in g]
    dc = [Guarded(t.shape, BF16, dev) for t in p] if copies else None
    opt = lpc.Muon([o.t for o in dp], dg, [o.t for o in dm], scales=scales, copies=[o.t for o in dc] if copies else None)
    gs = None if grad_scale is None else torch.tensor([grad_scale], device=dev)
    for _ in range(steps):
        before = [o.t.cpu().clone() for o in dp], [o.t.cpu().clone() for o in dm]
        opt.step(lr=lr, beta=beta, weight_decay=decay, nesterov=nesterov, iterations=iterations, grad_scale=gs)
        for i, s in enumerate(shapes):
            flat = (-1, s[-2], s[-1])
            got_m, got_p = dm[i].check().cpu().reshape(flat), dp[i].check().cpu().reshape(flat)
            for b in range(got_p.shape[0]):
                gr = g[i].float().reshape(flat)[b] * (1.0 if grad_scale is None else np.float32(grad_scale))
                old_m, old_p = before[1][i].reshape(flat)[b], before[0][i].reshape(flat)[b]
                want_m = beta * old_m.double() + (1 - beta) * gr.double()
                # two products and a sum, and beta and 1 - beta in fp32
                assert ((got_m[b].double() - want_m).abs() <= 5 * U * (old_m.abs() + gr.abs()).double() + 1e-45).all()
                u = (1 - beta) * gr.double() + beta * want_m if nesterov else want_m
                o = orthogonal64(u, iterations)
                # the update by itself: the parameters' rounding is at most 3 u of them
                moved = old_p.double() * (1 - lr * decay) - got_p[b].double()
                off = (moved - lr * scales[i] * o).norm() / max(float(lr * scales[i] * o.norm()), 1e-30) if float(o.norm()) else moved.norm()
                own = 4 * U * float(old_p.double().norm()) / max(float(lr * scales[i] * o.norm()), 1e-30) if float(o.norm()) else 4 * U
                assert float(off) <= off_by(min(s[-2:]), iterations) + own, (i, b, float(off), own)
            if copies:
                assert torch.equal(dc[i].check().cpu(), dp[i].t.cpu().to(BF16))


MUON = [[(1, 1)], [(1, 7)], [(9, 1)], [(32, 32)], [(31, 33), (33, 31)], [(3, 32, 130)], [(5, 9000), (9000, 5)], [(2, 20000)], [(8, 8)], [(16, 1152), (1000, 16)], [(64, 64)], [(3, 5, 9)], [(65, 63)], [(127, 129), (129, 127)],
        [(2, 128, 128)], [(300, 200), (7, 500), (256, 64)], [(130, 1000)], [(1001, 131)], [(4, 96, 200), (33, 33), (2, 70, 40)],
        [(512, 512)], [(400, 700)]]


@pytest.mark.parametrize("grad_t", [F32, BF16])
@pytest.mark.parametrize("shapes", MUON, ids=str)
def test_muon(dev, shapes, grad_t):
    check_muon(dev, shapes, grad_t)


@pytest.mark.parametrize("shapes", [[(9, 520, 2100)], [(50, 300, 520)], [(50, 520, 300), (33, 33)]], ids=str)
def test_muon_large_tiles(dev, shapes):
    """Enough tiles of 256 x 256, of either product, that a round of them is not split."""
    check_muon(dev, shapes, BF16)


@pytest.mark.parametrize("shapes", [[(64, 64)], [(24, 300)], [(300, 32)], [(128, 512)], [(600, 256)], [(3, 100, 60)]], ids=str)
def test_muon_strong_directions(dev, shapes):
    check_muon(dev, shapes, F32, kind="strong")


@pytest.mark.parametrize("iterations", [1, 2, 3, 8, 10])
def test_muon_iterations(dev, iterations):
    check_muon(dev, [(40, 90), (90, 40)], F32, iterations=iterations)


def test_muon_plain_momentum_and_scale(dev):
    check_muon(dev, [(50, 60), (2, 30, 70)], BF16, nesterov=False, grad_scale=0.125, copies=False)


def test_muon_steps(dev):
    check_muon(dev, [(100, 60), (60, 100)], F32, steps=3)


def test_muon_no_update(dev):
    """Gradient and momentum of zeros: the update is zeros, and the weights only decay."""
    check_muon(dev, [(40, 60), (60, 40), (130, 130)], F32, zero=(0, 2))


@pytest.mark.parametrize("size", [1e-30, 1e-18, 1e18, 1e30])
def test_muon_norms_of_any_size(dev, size):
    """The update does not depend on the gradient's size: its squares pass fp32 on both sides."""
    u = randn(40, 70, seed=3)
    moved = []
    for by in (1.0, size):
        p, m = torch.zeros(40, 70, device=dev), torch.zeros(40, 70, device=dev)
        lpc.Muon([p], [(u * by).to(dev)], [m], scales=[1.0]).step(lr=1.0)
        moved.append(p.cpu().double())
    assert torch.isfinite(moved[1]).all()
    assert float((moved[1] - moved[0]).norm() / moved[0].norm()) <= 2 * off_by(40, 5)


def test_muon_empty_tensors(dev):
    none, some = torch.zeros(0, 5, device=dev), torch.ones(4, 4, device=dev)
    lpc.Muon([], [], []).step(lr=1.0)
    lpc.Muon([none], [none], [none]).step(lr=1.0)
    lpc.Muon([none, some], [none, some], [none, torch.zeros(4, 4, device=dev)]).step(lr=1.0)
    assert torch.isfinite(some).all() and not (some == 1).any()
