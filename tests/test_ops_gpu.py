"""The operators of include/lpc_ops.h on the GPU against plain implementations in 64 bits, through the public binding.

Tolerances.  u = 2^-24 is half a step of fp32 (2^-8: of bf16).  A sum of n fp32 terms is off by at most (n - 1) u of the
sum of their magnitudes where each addition is rounded to nearest; the matrix cores' additions are counted with twice
that.  Codes and scales have exactly one right value and are compared byte for byte."""
import numpy as np
import pytest
import torch

import oracle
from fp8_precision_allreduce_amd import lpc

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
BLOCK = 128


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lpc.lib()
    return torch.device("cuda:0")


def say(*a):
    print("[case]", *a, flush=True)


def values(codes):
    return codes.cpu().view(torch.float8_e4m3fn).double()


def quantize(x):
    """Codes and scales of fp32 rows by the oracle."""
    x = np.ascontiguousarray(x.float().cpu().numpy())
    c, s = oracle.default().quantize(x.reshape(-1))
    return torch.from_numpy(c.copy()).reshape(x.shape), torch.from_numpy(s.copy()).reshape(x.shape[0], x.shape[1] // BLOCK)


def weights(g, n, k, rng):
    w = torch.from_numpy(rng.standard_normal((g, n, k)).astype(np.float32))
    codes = torch.empty(g, n, k, dtype=torch.uint8)
    scales = torch.empty(g, -(-n // BLOCK), k // BLOCK)
    for i in range(scales.shape[1]):
        for b in range(scales.shape[2]):
            t = w[:, i * BLOCK:(i + 1) * BLOCK, b * BLOCK:(b + 1) * BLOCK]
            s = t.abs().amax((1, 2)) / 448
            scales[:, i, b] = s
            codes[:, i * BLOCK:(i + 1) * BLOCK, b * BLOCK:(b + 1) * BLOCK] = \
                (t / s[:, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, scales


def rows64(codes, scales):
    return values(codes) * scales.cpu().double().repeat_interleave(BLOCK, 1)


def tiles64(codes, scales):
    n = codes.shape[1]
    return values(codes) * scales.double().repeat_interleave(BLOCK, 1)[:, :n].repeat_interleave(BLOCK, 2)


def clamp_counts(counts, rows):
    out, left = [], rows
    for c in counts:
        c = max(0, min(c, left))
        out.append(c)
        left -= c
    return out


# ---------------------------------------------------------------------------
# product
# ---------------------------------------------------------------------------

def check_gemm(dev, rows, k, n, counts, out_t, seed=0, stream=None):
    say("gemm rows=%d k=%d n=%d counts=%s %s" % (rows, k, n, counts, out_t))
    rng = np.random.RandomState(seed)
    x, xs = quantize(torch.from_numpy(rng.standard_normal((rows, k)).astype(np.float32) *
                                      np.exp(rng.standard_normal((rows, 1))).astype(np.float32)))
    g = len(counts) if counts else 1
    w, ws = weights(g, n, k, rng)
    out = torch.full((rows, n), float("nan"), dtype=out_t, device=dev)
    dc = torch.tensor(counts, dtype=torch.int32, device=dev) if counts else None
    lpc.lpc_gemm_fp8(x.to(dev), xs.to(dev), w.to(dev), ws.to(dev), out, counts=dc)
    got = out.cpu().double()
    a, b = rows64(x, xs), tiles64(w, ws)
    at = 0
    for i, c in enumerate(clamp_counts(counts, rows) if counts else [rows]):
        want, size = a[at:at + c] @ b[i].t(), a[at:at + c].abs() @ b[i].abs().t()
        tol = size * (2 * (BLOCK + k // BLOCK) + 8) * U + (want.abs() + size * 1e-4) * HALF[out_t]
        bad = (got[at:at + c] - want).abs() > tol
        assert not bad.any() and not got[at:at + c].isnan().any(), (i, int(bad.sum()))
        at += c
    assert (got[at:] == 0).all()
    return got


GEMM = [(1, 128, 1), (1, 8192, 512), (2, 384, 130), (15, 1152, 127), (16, 256, 128), (17, 640, 1000), (33, 896, 257),
        (64, 2048, 384), (65, 1152, 129), (129, 128, 255), (257, 640, 300), (300, 1152, 1000), (777, 512, 513)]


@pytest.mark.parametrize("out_t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,k,n", GEMM)
def test_gemm(dev, rows, k, n, out_t):
    check_gemm(dev, rows, k, n, None, out_t)


@pytest.mark.parametrize("out_t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,k,n,counts", [
    (1, 256, 96, [0, 1, 0]), (40, 384, 130, [0, 17, 0, 20]), (300, 640, 257, [128, 0, 172]), (300, 256, 128, [0, 0, 0]),
    (513, 896, 300, [256, 1, 255, 1]), (500, 384, 256, [-3, 200, 1000, 5]), (200, 128, 64, [50]),
    (700, 1152, 640, [3, 0, 500, 7, 40])])
def test_gemm_groups(dev, rows, k, n, counts, out_t):
    check_gemm(dev, rows, k, n, counts, out_t)


@pytest.mark.parametrize("rows,k,n,counts", [(2100, 1152, 1152, None), (3000, 640, 1300, [5, 1500, 0, 900]),
                                             (4096, 256, 2048, None)])
def test_gemm_large_tiles(dev, rows, k, n, counts):
    check_gemm(dev, rows, k, n, counts, torch.bfloat16)


@pytest.mark.parametrize("out_t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,k,n,counts", [
    (20, 16512, 40, None), (40, 8320, 96, None), (70, 8448, 300, [33, 0, 36]), (65, 512, 8192, None),  # 32 x 32
    (33, 9216, 4160, None), (90, 256, 3300, [40, 20, 5]),                                               # 64 x 32
    (100, 8320, 4160, None), (512, 384, 1100, [1, 200, 0, 300]),                                        # 64 x 64
    (256, 896, 6500, None), (3000, 128, 700, None), (2100, 1536, 1700, [700, 0, 3, 1200])])             # large tiles
def test_gemm_kinds_of_tiles(dev, rows, k, n, counts, out_t):
    check_gemm(dev, rows, k, n, counts, out_t)


def test_gemm_long_rows_are_gathered(dev):
    """Rows of 8 MiB, more of them than a gathered decode has."""
    rows, n, k = 40, 33, 1 << 23
    say("gemm 40 rows of 8 MiB")
    x = torch.full((rows, k), 0x38, dtype=torch.uint8, device=dev)      # 1.0
    w = torch.zeros(n, k, dtype=torch.uint8, device=dev)
    w[n - 1, :] = 0x30                                                  # 0.5
    out = torch.empty(rows, n, device=dev)
    lpc.lpc_gemm_fp8(x, torch.ones(rows, k // BLOCK, device=dev), w, torch.ones(1, k // BLOCK, device=dev), out)
    want = torch.zeros(rows, n)
    want[:, n - 1] = k / 2
    assert torch.equal(out.cpu(), want)


def test_gemm_many_groups(dev):
    rng = np.random.RandomState(3)
    counts = [int(c) for c in rng.multinomial(400, np.full(130, 1 / 130))]
    check_gemm(dev, 410, 128, 20, counts, torch.float32)


def test_gemm_offsets_past_32_bits(dev):
    """A weight past 4 GiB into its array."""
    g, n, k = 5, 8192, 131072
    say("gemm 5 groups of 1 GiB")
    w = torch.zeros(g, n, k, dtype=torch.uint8, device=dev)
    ws = torch.ones(g, n // BLOCK, k // BLOCK, device=dev)
    w[4, n - 1, :] = 0x38                                     # 1.0
    x = torch.full((3, k), 0x38, dtype=torch.uint8, device=dev)
    xs = torch.ones(3, k // BLOCK, device=dev)
    out = torch.empty(3, n, device=dev)
    lpc.lpc_gemm_fp8(x, xs, w, ws, out, counts=torch.tensor([0, 1, 0, 0, 2], dtype=torch.int32, device=dev))
    want = torch.zeros(3, n)
    want[1:, n - 1] = k
    assert torch.equal(out.cpu(), want)


def test_gemm_on_another_stream_and_repeatable(dev):
    rng = np.random.RandomState(1)
    x, xs = quantize(torch.from_numpy(rng.standard_normal((300, 1152)).astype(np.float32)))
    w, ws = weights(1, 400, 1152, rng)
    t = [v.to(dev) for v in (x, xs, w, ws)]
    a, b = torch.empty(300, 400, device=dev), torch.empty(300, 400, device=dev)
    lpc.lpc_gemm_fp8(*t, a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lpc.lpc_gemm_fp8(*t, b, stream=s)
    s.synchronize()
    assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# column forms and the gradient of the weights
# ---------------------------------------------------------------------------

def columns(x, counts):
    """Column codes and scales of fp32 x by the oracle, and where each group's blocks start."""
    codes, scales, starts, at = [], [], [], 0
    for c in counts:
        starts.append(sum(s.shape[1] for s in scales))
        if c:
            wide = torch.zeros(x.shape[1], -(-c // BLOCK) * BLOCK)
            wide[:, :c] = x[at:at + c].t()
            q, s = quantize(wide)
            codes.append(q)
            scales.append(s)
        at += c
    return torch.cat(codes, 1), torch.cat(scales, 1).t().contiguous(), starts


COLS = [(1, 128, None), (127, 256, None), (128, 384, None), (129, 128, None), (300, 640, [0, 129, 0, 1, 128]),
        (500, 256, [100, 200, -5, 300]), (260, 128, [256, 4])]


def column_buffers(rows, n, groups, dev):
    p = lpc.lpc_padded_rows(rows, groups)
    return (torch.full((n, p), 0xAA, dtype=torch.uint8, device=dev), torch.full((p // BLOCK, n), -1.0, device=dev))


@pytest.mark.parametrize("in_t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,n,counts", COLS)
def test_quantize_cols(dev, rows, n, counts, in_t):
    say("cols rows=%d n=%d counts=%s %s" % (rows, n, counts, in_t))
    rng = np.random.RandomState(rows)
    y = torch.from_numpy(rng.standard_normal((rows, n)).astype(np.float32)) * \
        torch.from_numpy(np.exp(3 * rng.standard_normal((rows, 1))).astype(np.float32))
    y[:, 3] = 0                                               # a column of zeros
    y[:, 5] *= 2.0 ** -126                                    # and one below the reciprocal's range
    y[0] = 0
    y = y.to(in_t)
    used = clamp_counts(counts, rows) if counts else [rows]
    ct, st = column_buffers(rows, n, len(used), dev)
    c = torch.full((rows, n), 0xAA, dtype=torch.uint8, device=dev)
    s = torch.full((rows, n // BLOCK), -1.0, device=dev)
    dc = torch.tensor(counts, dtype=torch.int32, device=dev) if counts else None
    lpc.lpc_quantize_fp8_cols(y.to(dev), ct, st, codes=c, scales=s, counts=dc)
    wc, wst, _ = columns(y.float(), used)
    wide = wc.shape[1]
    assert torch.equal(ct.cpu()[:, :wide], wc) and torch.equal(st.cpu()[:wide // BLOCK], wst)
    assert (ct.cpu()[:, wide:] == 0xAA).all() and (st.cpu()[wide // BLOCK:] == -1).all()
    rc, rs = quantize(y.float())
    total = sum(used)
    assert torch.equal(c.cpu()[:total], rc[:total]) and torch.equal(s.cpu()[:total], rs[:total])
    assert (c.cpu()[total:] == 0xAA).all() and (s.cpu()[total:] == -1).all()
    ct2, st2 = column_buffers(rows, n, len(used), dev)
    lpc.lpc_quantize_fp8_cols(y.to(dev), ct2, st2, counts=dc)
    assert torch.equal(ct, ct2) and torch.equal(st, st2)


@pytest.mark.parametrize("rows,n,counts", COLS)
def test_requantize_cols(dev, rows, n, counts):
    say("requantize rows=%d n=%d counts=%s" % (rows, n, counts))
    rng = np.random.RandomState(rows + 1)
    x, xs = quantize(torch.from_numpy(rng.standard_normal((rows, n)).astype(np.float32)))
    used = clamp_counts(counts, rows) if counts else [rows]
    ct, st = column_buffers(rows, n, len(used), dev)
    dc = torch.tensor(counts, dtype=torch.int32, device=dev) if counts else None
    lpc.lpc_requantize_fp8_cols(x.to(dev), xs.to(dev), ct, st, counts=dc)
    held = x.view(torch.float8_e4m3fn).float() * xs.repeat_interleave(BLOCK, 1)
    wc, wst, _ = columns(held, used)
    wide = wc.shape[1]
    assert torch.equal(ct.cpu()[:, :wide], wc) and torch.equal(st.cpu()[:wide // BLOCK], wst)
    assert (ct.cpu()[:, wide:] == 0xAA).all()


WGRAD = [(1, 128, 128, None), (130, 256, 384, None), (300, 100, 37, None), (300, 384, 256, [0, 129, 0, 1, 128]),
         (1000, 640, 512, [400, 0, 590]), (700, 129, 258, [-1, 2000]), (2500, 512, 768, None)]


@pytest.mark.parametrize("rows,n,k,counts", WGRAD)
def test_wgrad(dev, rows, n, k, counts):
    say("wgrad rows=%d n=%d k=%d counts=%s" % (rows, n, k, counts))
    rng = np.random.RandomState(rows + n)
    used = clamp_counts(counts, rows) if counts else [rows]
    forms = []
    for width in (n, k):
        x = torch.from_numpy(rng.standard_normal((rows, width)).astype(np.float32))
        c, s, starts = columns(x, used)
        ct, st = column_buffers(rows, width, len(used), dev)
        ct[:, :c.shape[1]] = c.to(dev)                        # what lies past the blocks is never used
        st[:s.shape[0]] = s.to(dev)
        forms.append((ct, st, c, s))
    dw = torch.full((len(used), n, k), float("nan"), device=dev)
    dc = torch.tensor(counts, dtype=torch.int32, device=dev) if counts else None
    lpc.lpc_gemm_fp8_wgrad(*forms[0][:2], *forms[1][:2], dw, rows, counts=dc)
    a, b = [rows64(c, s.t()) for _, _, c, s in forms]
    for g, c in enumerate(used):
        lo, hi = starts[g] * BLOCK, (starts[g] + -(-c // BLOCK)) * BLOCK
        want, size = a[:, lo:hi] @ b[:, lo:hi].t(), a[:, lo:hi].abs() @ b[:, lo:hi].abs().t()
        bad = (dw[g].cpu().double() - want).abs() > size * (2 * (BLOCK + (hi - lo) // BLOCK) + 8) * U
        assert not bad.any() and not dw[g].isnan().any(), (g, int(bad.sum()))


@pytest.mark.parametrize("rows,n,k,counts", [
    (130, 1030, 1100, None), (390, 700, 900, [1, 0, 260, 100]),        # 128 x 128
    (300, 2300, 2050, None), (260, 1300, 900, [128, 3, 0, 120])])      # 256 x 128
def test_wgrad_kinds_of_tiles(dev, rows, n, k, counts):
    test_wgrad(dev, rows, n, k, counts)


def test_wgrad_without_rows(dev):
    dw = torch.full((2, 64, 128), 7.0, device=dev)
    e8, ef = torch.empty(0, dtype=torch.uint8, device=dev), torch.empty(0, device=dev)
    lpc.lpc_gemm_fp8_wgrad(e8, ef, e8, ef, dw, 0, counts=torch.zeros(2, dtype=torch.int32, device=dev))
    assert (dw == 0).all()


def test_product_gradients(dev):
    """Where every quantization is exact the two backward calls give the gradients of sum(out * dy): against autograd in
    64 bits, and against differences (the sum is linear in each operand, so a difference is its derivative)."""
    rng = np.random.RandomState(5)
    rows, k, n = 256, 256, 128

    def exact_values(*shape):                                 # E4M3 values, 448 in every block of 128 rows and columns
        v = torch.from_numpy(rng.randint(-7, 8, shape).astype(np.float64))
        i = torch.arange(shape[0])
        for c in range(0, shape[1], BLOCK):
            v[i, c + i % BLOCK] = 448
        return v

    x, dy, w = exact_values(rows, k), exact_values(rows, n), exact_values(n, k)
    code = lambda v: v.float().to(torch.float8_e4m3fn).view(torch.uint8).to(dev)  # noqa: E731
    one = lambda *s: torch.ones(*s, device=dev)  # noqa: E731
    xt, xts = column_buffers(rows, k, 1, dev)
    yt, yts = column_buffers(rows, n, 1, dev)
    yc, ys = torch.empty(rows, n, dtype=torch.uint8, device=dev), torch.empty(rows, 1, device=dev)
    lpc.lpc_quantize_fp8_cols(dy.float().to(dev), yt, yts, codes=yc, scales=ys)
    lpc.lpc_requantize_fp8_cols(code(x), one(rows, 2), xt, xts)
    dx, dw = torch.empty(rows, k, device=dev), torch.empty(n, k, device=dev)
    lpc.lpc_gemm_fp8(yc, ys, code(w).t().contiguous(), one(2, 1), dx)
    lpc.lpc_gemm_fp8_wgrad(yt, yts, xt, xts, dw, rows)
    xa, wa = x.clone().requires_grad_(), w.clone().requires_grad_()
    ((xa @ wa.t()) * dy).sum().backward()
    # whole numbers below 2^24 at every step: no rounding anywhere
    assert torch.equal(dx.cpu().double(), xa.grad) and torch.equal(dw.cpu().double(), wa.grad)
    f = lambda a, b: ((a @ b.t()) * dy).sum()  # noqa: E731
    for i, j in ((0, 0), (100, 200)):
        e = torch.zeros_like(x)
        e[i, j] = 1
        assert float(f(x + e, w) - f(x, w)) == float(dx[i, j])
        e = torch.zeros_like(w)
        e[i, j] = 1
        assert float(f(x, w + e) - f(x, w)) == float(dw[i, j])


# ---------------------------------------------------------------------------
# router
# ---------------------------------------------------------------------------

def route64(x, topk, normalize, coef, mask):
    """The definition in 64 bits, on the CPU; differentiable in x."""
    rows, e = x.shape
    allowed = (x > -float("inf"))
    valid = allowed.any(1) if mask is None else allowed.any(1) & (mask != 0)
    n = max(1, int(valid.sum()))
    safe = torch.where(allowed & valid[:, None], x, torch.full_like(x, -float("inf")))
    safe = torch.where(valid[:, None], safe, torch.zeros_like(safe))
    p = torch.softmax(safe, 1) * valid[:, None]
    order = torch.sort(safe.detach(), dim=1, descending=True, stable=True)
    which = order.indices[:, :topk]
    taken = (order.values[:, :topk] > -float("inf")) & valid[:, None]
    gates = p.gather(1, which) * taken
    if normalize:
        total = gates.sum(1, keepdim=True)
        gates = gates / torch.where(total > 0, total, torch.ones_like(total))
    counts = torch.bincount(which[taken], minlength=e)
    load = p.sum(0) / n
    share = counts.double() / (n * topk)
    return {"experts": torch.where(taken, which, torch.full_like(which, -1)), "gates": gates, "counts": counts, "load": load,
            "slope": coef * e * share / n, "loss": coef * e * (share * load).sum().reshape(1)}


def check_router(dev, x, topk, normalize, mask=None, coef=0.01, seed=0):
    say("router rows=%d experts=%d topk=%d normalize=%s mask=%s %s" % (*x.shape, topk, normalize, mask is not None, x.dtype))
    rows, e = x.shape
    rng = np.random.RandomState(seed)
    dg = torch.from_numpy(rng.standard_normal((rows, topk)).astype(np.float32))
    dl = torch.tensor([0.75])
    o = {"experts": torch.full((rows, topk), -9, dtype=torch.int32, device=dev), "gates": torch.full((rows, topk), -9.0, device=dev),
         "counts": torch.full((e,), -9, dtype=torch.int32, device=dev)}
    o.update({k: torch.full((n,), -9.0, device=dev) for k, n in (("load", e), ("slope", e), ("loss", 1))})
    xd, md = x.to(dev), None if mask is None else mask.to(dev)
    lpc.lpc_router_forward(xd, *o.values(), coef=coef, normalize=normalize, mask=md)
    dx = torch.full_like(xd, 9.0)
    lpc.lpc_router_backward(xd, o["experts"], o["slope"], dg.to(dev), dl.to(dev), dx, normalize=normalize, mask=md)
    got = {k: v.cpu() for k, v in o.items()}
    x64 = x.double().nan_to_num(nan=-float("inf"), posinf=float("inf"), neginf=-float("inf")).requires_grad_()
    want = route64(x64, topk, normalize, coef, mask)
    assert torch.equal(got["experts"].long(), want["experts"]) and torch.equal(got["counts"].long(), want["counts"])
    # exp is good to 2 units, its argument is off by half a step of a difference below `reach`, the sum has e terms
    finite = x64.detach()[torch.isfinite(x64)]
    reach = float(finite.max() - finite.min()) if finite.numel() else 0.0
    rel = (e + 2 * min(reach, 110.0) + 16) * U
    tiny = 2.0 ** -125                                       # exp of less is zero or denormal
    for key, more in (("gates", topk), ("load", rows), ("slope", 8), ("loss", rows + e)):
        w = want[key].detach()
        assert ((got[key].double() - w).abs() <= w.abs() * (rel + more * U) + tiny).all(), key
    ((want["gates"] * dg.double()).sum() + want["loss"] * 0.75).sum().backward() if rows else None
    w = x64.grad if rows and x64.grad is not None else torch.zeros_like(x64)
    w = torch.where(torch.isfinite(w), w, torch.zeros_like(w))
    up = 0.75 * float(want["slope"].max()) if e else 0.0
    size = up + 2 * dg.abs().double().sum(1, keepdim=True) if rows else 0.0
    tol = size * (rel + (e + topk + 8) * U) * 4 + w.abs() * HALF[x.dtype]
    assert ((dx.cpu().double() - w).abs() <= tol).all()
    assert (dx.cpu()[~torch.isfinite(x)] == 0).all()
    if mask is not None:
        assert (dx.cpu()[mask == 0] == 0).all() and (got["experts"][mask == 0] == -1).all()
    return got


def logits(rows, e, dtype, seed=0, holes=False):
    rng = np.random.RandomState(seed)
    x = torch.from_numpy((rng.standard_normal((rows, e)) * 2).astype(np.float32)).to(dtype)
    if holes:
        x[torch.from_numpy(rng.rand(rows, e) < 0.3)] = -float("inf")
        x[torch.from_numpy(rng.rand(rows) < 0.2)] = -float("inf")
        x[rows // 2, e // 2] = float("nan")
    return x


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("rows,e,topk", [(1, 64, 6), (1, 1, 1), (3, 2, 2), (17, 7, 3), (64, 16, 16), (65, 33, 4), (200, 60, 4),
                                         (333, 129, 8), (500, 256, 8), (70, 257, 2), (90, 1000, 16), (5000, 20, 2)])
def test_router(dev, rows, e, topk, normalize, dtype):
    check_router(dev, logits(rows, e, dtype), topk, normalize)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("rows,e,topk", [(1, 8, 2), (300, 60, 4), (100, 256, 8), (50, 300, 5)])
def test_router_masks(dev, rows, e, topk, normalize, dtype):
    x = logits(rows, e, dtype, 1, True)
    mask = torch.from_numpy((np.random.RandomState(2).rand(rows) < 0.7).astype(np.uint8))
    x[mask == 0] = float("nan")                               # what stands in a masked row does not matter
    check_router(dev, x, topk, normalize, mask)


def test_router_ties_and_extremes(dev):
    x = torch.zeros(40, 48)
    assert (check_router(dev, x, 5, True)["experts"] == torch.arange(5, dtype=torch.int32)).all()
    x[:, 20:] = torch.finfo(torch.float32).min                # masked by the lowest value: allowed, but with p = 0
    x[:10] = torch.finfo(torch.float32).min                   # such a row is uniform
    x[10:20, 3] = 1000.0
    check_router(dev, x, 8, True)
    check_router(dev, x, 8, False)
    check_router(dev, torch.full((70, 9), -float("inf")), 3, True)
    check_router(dev, torch.zeros(100, 9), 3, True, torch.zeros(100, dtype=torch.uint8))


def test_router_without_rows(dev):
    out = [torch.full((5,), 9, dtype=torch.int32, device=dev)] + [torch.full((n,), 9.0, device=dev) for n in (5, 5, 1)]
    lpc.lpc_router_forward(torch.empty(0, 5, device=dev), torch.empty(0, 2, dtype=torch.int32, device=dev),
                           torch.empty(0, 2, device=dev), *out, coef=0.1)
    assert all((t == 0).all() for t in out)


def test_router_ignores_indices_out_of_range(dev):
    x = logits(50, 12, torch.float32).to(dev)
    idx = torch.arange(50 * 3, dtype=torch.int32, device=dev).reshape(50, 3) % 12
    bad = idx.clone()
    bad[:, 1], bad[::2, 2] = 12, -(1 << 31)
    only = idx.clone()
    only[:, 1], only[::2, 2] = -1, -1
    dg, dl, slope = torch.ones(50, 3, device=dev), torch.ones(1, device=dev), torch.ones(12, device=dev)
    a, b = torch.empty_like(x), torch.empty_like(x)
    lpc.lpc_router_backward(x, bad, slope, dg, dl, a)
    lpc.lpc_router_backward(x, only, slope, dg, dl, b)
    assert torch.equal(a, b)


def test_router_gradient_against_differences(dev):
    """Central differences of the 64-bit definition; the step keeps every choice of experts."""
    x = logits(6, 10, torch.float32, 4)
    dg = torch.from_numpy(np.random.RandomState(0).standard_normal((6, 3)).astype(np.float32))
    for normalize in (True, False):
        o = [torch.empty(6, 3, dtype=torch.int32, device=dev), torch.empty(6, 3, device=dev),
             torch.empty(10, dtype=torch.int32, device=dev), *(torch.empty(n, device=dev) for n in (10, 10, 1))]
        dx = torch.empty(6, 10, device=dev)
        lpc.lpc_router_forward(x.to(dev), *o, coef=0.1, normalize=normalize)
        lpc.lpc_router_backward(x.to(dev), o[0], o[4], dg.to(dev), torch.ones(1, device=dev), dx, normalize=normalize)

        def f(v):
            r = route64(v, 3, normalize, 0.1, None)
            assert torch.equal(r["experts"], o[0].cpu().long())
            return float((r["gates"] * dg.double()).sum() + r["loss"])

        h = 1e-5
        for i in range(6):
            for j in range(10):
                d = torch.zeros(6, 10, dtype=torch.float64)
                d[i, j] = h
                # the difference is off by h^2 / 6 of the third derivative (below 20 here) and by rounding / h
                assert abs((f(x.double() + d) - f(x.double() - d)) / (2 * h) - float(dx[i, j])) < 20 * h * h + 1e-9 + 1e-5


# ---------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------

HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)


def adamw32(p, g, m, v, step, scale):
    """The step in fp32 with every operation rounded on its own, as lpc_ops.h writes it."""
    f = lambda x: torch.tensor(float(np.float32(x)))  # noqa: E731
    b1, b2 = HYPER["beta1"], HYPER["beta2"]
    g = g.float() * scale
    m = m * f(b1) + g * f(1 - b1)
    v = v * f(b2) + (g * f(1 - b2)) * g
    r = torch.from_numpy(np.sqrt(v.numpy()))                  # correctly rounded; torch's is not on every CPU
    p = p * f(1 - HYPER["lr"] * HYPER["weight_decay"]) - m * f(HYPER["lr"] / (1 - b1 ** step)) / \
        (r * f(1 / (1 - b2 ** step) ** 0.5) + f(HYPER["eps"]))
    return p, m, v, r


def adamw64(p, g, m, v, step, scale):
    b1, b2 = HYPER["beta1"], HYPER["beta2"]
    g = g.double() * float(scale)
    m, v = b1 * m.double() + (1 - b1) * g, b2 * v.double() + (1 - b2) * g * g
    d = (m / (1 - b1 ** step)) / ((v / (1 - b2 ** step)).sqrt() + HYPER["eps"])
    return p.double() * (1 - HYPER["lr"] * HYPER["weight_decay"]) - HYPER["lr"] * d


def state8(x, up):
    wide = torch.zeros(-(-x.numel() // BLOCK) * BLOCK)
    wide[:x.numel()] = x
    c, s = quantize(wide.reshape(-1, BLOCK))
    c = c.reshape(-1)[:x.numel()]
    s = s.reshape(-1)
    if up:
        c = torch.where((x > 0) & (s.repeat_interleave(BLOCK)[:x.numel()] > 0) & (c == 0), torch.ones_like(c), c)
    return c, s


def held8(c, s):
    return c.view(torch.float8_e4m3fn).float() * s.repeat_interleave(BLOCK)[:c.numel()]


SIZES = [1, 3, 127, 128, 129, 0, 4095, 4096, 4097, 20000]


@pytest.mark.parametrize("copies", [False, True])
@pytest.mark.parametrize("grad_t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw(dev, bits, grad_t, copies):
    say("adamw bits=%d %s copies=%s" % (bits, grad_t, copies))
    rng = np.random.RandomState(7)
    rand = lambda n, s: torch.from_numpy((rng.standard_normal(n) * s).astype(np.float32))  # noqa: E731
    p, m = [rand(n, 0.1) for n in SIZES], [torch.zeros(n) for n in SIZES]
    v = [torch.zeros(n) for n in SIZES]
    put = lambda ts: [t.to(dev) for t in ts]  # noqa: E731
    dp, dg = put(p), put([torch.zeros(n, dtype=grad_t) for n in SIZES])
    dcopy = put([torch.zeros(n, dtype=torch.bfloat16) for n in SIZES]) if copies else None
    if bits == 8:
        m8, r8 = [state8(t, False) for t in m], [state8(t, True) for t in v]
        dm, dms, dr, drs = put([c for c, _ in m8]), put([s for _, s in m8]), put([c for c, _ in r8]), put([s for _, s in r8])
        opt = lpc.AdamW(dp, dg, dm, dr, dms, drs, copies=dcopy)
    else:
        dm, dv = put(m), put(v)
        opt = lpc.AdamW(dp, dg, dm, dv, copies=dcopy)
    for step in (1, 2, 3):
        g = [rand(n, 10.0 ** -step).to(grad_t) for n in SIZES]
        for i, n in enumerate(SIZES):
            if n > 200:
                g[i][100:200] = 0
            dg[i].copy_(g[i])
        scale = torch.tensor([0.37]) if step != 2 else None
        opt.step(step, grad_scale=None if scale is None else scale.to(dev), **HYPER)
        sc = torch.ones(1) if scale is None else scale
        for i, n in enumerate(SIZES):
            if n == 0:
                continue
            if bits == 8:
                m[i], v[i] = held8(*m8[i]), held8(*r8[i]) ** 2
            p64 = adamw64(p[i], g[i], m[i], v[i], step, sc)
            p[i], m[i], v[i], r = adamw32(p[i], g[i], m[i], v[i], step, sc)
            assert torch.equal(dp[i].cpu(), p[i]), (step, n)
            # p: 3 roundings; the update: about 12 relative ones, of at most lr (1 - b1) / (1 - b2)^.5 (below 4 lr)
            assert ((dp[i].cpu().double() - p64).abs() <= p64.abs() * 4 * U + 4 * HYPER["lr"] * 16 * U).all()
            if copies:
                assert torch.equal(dcopy[i].cpu(), p[i].to(torch.bfloat16))
            if bits == 8:
                m8[i], r8[i] = state8(m[i], False), state8(r, True)
                for got, want in ((dm, m8[i][0]), (dms, m8[i][1]), (dr, r8[i][0]), (drs, r8[i][1])):
                    assert torch.equal(got[i].cpu(), want), (step, n)
            else:
                assert torch.equal(dm[i].cpu(), m[i]) and torch.equal(dv[i].cpu(), v[i])


def test_adamw_writes_inside_its_views(dev):
    """Tensors of odd sizes inside one buffer: what lies between them stays as it was."""
    flat = [torch.full((4096,), 0.5, device=dev) for _ in range(4)]
    codes = [torch.full((4096,), 0x31, dtype=torch.uint8, device=dev) for _ in range(2)]
    scales = [torch.full((32,), 0.1, device=dev) for _ in range(2)]
    spans, spare = [(0, 130), (512, 513), (1024, 1999)], torch.ones(4096, dtype=torch.bool)
    for a, b in spans:
        spare[a:b] = False
    cut = lambda t, d=1: [t[a // d:-(-b // d)] for a, b in spans]  # noqa: E731
    lpc.AdamW(*map(cut, flat)).step(1, **HYPER)
    lpc.AdamW(cut(flat[0]), cut(flat[1]), cut(codes[0]), cut(codes[1]), cut(scales[0], BLOCK), cut(scales[1], BLOCK)).step(1, **HYPER)
    for t, was in [(t, 0.5) for t in flat] + [(t, 0x31) for t in codes]:
        assert (t.cpu()[spare] == was).all()
    assert (flat[0].cpu()[~spare] != 0.5).all()


def test_adamw_without_tensors(dev):
    lpc.AdamW([], [], [], []).step(1, lr=0.1)
    t = torch.empty(0, device=dev)
    lpc.AdamW([t], [t], [t], [t]).step(1, lr=0.1)


# ---------------------------------------------------------------------------
# graphs and refusals on the device
# ---------------------------------------------------------------------------

def test_operators_in_a_graph(dev):
    """A captured pass of every operator, replayed between eager work, against the eager results."""
    rows, e, k, n = 300, 24, 256, 384
    rng = np.random.RandomState(11)
    x, xs = [t.to(dev) for t in quantize(torch.from_numpy(rng.standard_normal((rows, k)).astype(np.float32)))]
    w, ws = [t.to(dev) for t in weights(2, n, k, rng)]
    counts = torch.tensor([100, 190], dtype=torch.int32, device=dev)
    dy = torch.from_numpy(rng.standard_normal((rows, n)).astype(np.float32)).to(dev)
    lg = logits(rows, e, torch.float32).to(dev)
    o = {"out": torch.empty(rows, n, device=dev), "dw": torch.empty(2, n, k, device=dev), "dx": torch.empty_like(lg),
         "gates": torch.empty(rows, 2, device=dev), "loss": torch.empty(1, device=dev), "load": torch.empty(e, device=dev),
         "experts": torch.empty(rows, 2, dtype=torch.int32, device=dev)}
    cnt, slope = torch.empty(e, dtype=torch.int32, device=dev), torch.empty(e, device=dev)
    yt, yts = column_buffers(rows, n, 2, dev)
    xt, xts = column_buffers(rows, k, 2, dev)
    dg, dl = torch.ones(rows, 2, device=dev), torch.ones(1, device=dev)
    space = torch.empty(lpc.lpc_router_workspace_bytes(rows, e), dtype=torch.uint8, device=dev)
    p, g, m, v = (torch.full((5000,), c, device=dev) for c in (0.5, 0.1, 0.0, 0.0))
    opt = lpc.AdamW([p], [g], [m], [v])

    def once():
        lpc.lpc_gemm_fp8(x, xs, w, ws, o["out"], counts=counts)
        lpc.lpc_quantize_fp8_cols(dy, yt, yts, counts=counts)
        lpc.lpc_requantize_fp8_cols(x, xs, xt, xts, counts=counts)
        lpc.lpc_gemm_fp8_wgrad(yt, yts, xt, xts, o["dw"], rows, counts=counts)
        lpc.lpc_router_forward(lg, o["experts"], o["gates"], cnt, o["load"], slope, o["loss"], coef=0.01, workspace=space)
        lpc.lpc_router_backward(lg, o["experts"], slope, dg, dl, o["dx"])
        opt.step(1, lr=1e-2)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        once()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        once()
    for turn in range(3):
        lg.normal_()
        dy.normal_()
        counts.copy_(torch.tensor([50 + turn, 120], dtype=torch.int32))
        was = [t.clone() for t in (p, m, v)]
        once()
        want = {name: t.clone() for name, t in o.items()}
        stepped = [t.clone() for t in (p, m, v)]
        for t in o.values():
            t.zero_()
        for t, old in zip((p, m, v), was):
            t.copy_(old)
        graph.replay()
        torch.cuda.synchronize()
        for name, t in o.items():
            assert torch.equal(t, want[name]), (turn, name)
        assert all(torch.equal(a, b) for a, b in zip((p, m, v), stepped)), turn


def test_binding_refusals(dev):
    u8, f32 = torch.zeros(4, 128, dtype=torch.uint8, device=dev), torch.zeros(4, 1, device=dev)
    out = torch.zeros(4, 4, device=dev)
    with pytest.raises(TypeError, match="dtype"):
        lpc.lpc_gemm_fp8(u8.float(), f32, u8, f32[:1], out)
    with pytest.raises(ValueError, match="contiguous"):
        lpc.lpc_gemm_fp8(u8.t().contiguous().t(), f32, u8, f32[:1], out)
    with pytest.raises(ValueError, match="xs holds"):
        lpc.lpc_gemm_fp8(u8, f32[:3], u8, f32[:1], out)
    with pytest.raises(ValueError, match="out has shape"):
        lpc.lpc_gemm_fp8(u8, f32, u8, f32[:1], out[:3])
    with pytest.raises(ValueError, match="w has shape"):
        lpc.lpc_gemm_fp8(u8, f32, u8, f32[:1], out, counts=torch.zeros(2, dtype=torch.int32, device=dev))
    with pytest.raises(lpc.LpcError) as e:
        lpc.lpc_router_forward(torch.zeros(3, 2, device=dev), torch.zeros(3, 5, dtype=torch.int32, device=dev),
                               torch.zeros(3, 5, device=dev), torch.zeros(2, dtype=torch.int32, device=dev),
                               *(torch.zeros(n, device=dev) for n in (2, 2, 1)), coef=0.1)
    assert e.value.status_name == "LPC_ERR_SHAPE"
    with pytest.raises(lpc.LpcError) as e:
        lpc.AdamW([f32], [f32], [f32], [f32]).step(0, lr=0.1)
    assert e.value.status_name == "LPC_ERR_SHAPE"
    with pytest.raises(ValueError, match="holds"):
        lpc.AdamW([f32], [f32[:2]], [f32], [f32])


def test_binding_usual_and_other_calls_agree(dev):
    """A call that the binding checks in one expression and the same call by way of every single check (a stream given)."""
    rng = np.random.RandomState(21)
    x, xs = [t.to(dev) for t in quantize(torch.from_numpy(rng.standard_normal((70, 384)).astype(np.float32)))]
    w, ws = [t.to(dev) for t in weights(2, 200, 384, rng)]
    counts = torch.tensor([30, 35], dtype=torch.int32, device=dev)
    lg, mask = logits(70, 24, torch.bfloat16, holes=True).to(dev), (torch.rand(70, device=dev) < 0.7)
    dg, dl = torch.randn(70, 3, device=dev), torch.ones(1, device=dev)
    results = []
    for stream in (None, torch.cuda.current_stream()):
        out = torch.empty(70, 200, device=dev)
        lpc.lpc_gemm_fp8(x, xs, w, ws, out, counts=counts, stream=stream)
        o = [torch.empty(70, 3, dtype=torch.int32, device=dev), torch.empty(70, 3, device=dev),
             torch.empty(24, dtype=torch.int32, device=dev), torch.empty(24, device=dev), torch.empty(24, device=dev),
             torch.empty(1, device=dev)]
        lpc.lpc_router_forward(lg, *o, coef=0.1, mask=mask, stream=stream)
        dx = torch.empty_like(lg)
        lpc.lpc_router_backward(lg, o[0], o[4], dg, dl, dx, mask=mask, stream=stream)
        torch.cuda.synchronize()
        results.append([out, *o, dx])
    assert all(torch.equal(a, b) for a, b in zip(*results))
