"""What the products' sums hold: FP32 results keep whole numbers exactly whatever stands beside them, bf16 results go by the
cut that lpc_ops.h states, in every kernel that the sizes choose.

The data are E4M3 codes with scales of one, mostly small whole numbers with 448 among them, so that every product and every
partial sum is a whole number below 2^24: any FP32 sum of them is exact in any order, and there is one right result."""
import pytest
import torch

from fp8_precision_allreduce_amd import lpc

BLOCK, RUN = 128, 8


def exponent(v):
    """Of the power of two at or below |v|; values below 2^-6 count as 2^-6."""
    return (torch.frexp(v.abs())[1] - 1).clamp(min=-6)


def cut_sums(x, w):
    """x [r, k] times w [n, k] transposed, every product cut towards zero to a multiple of 2^(E - 13), E the largest sum of two
    exponents among the products of its run of 8 that are not zero; sums in 64 bits."""
    ex, ew = exponent(x), exponent(w)
    out = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64, device=x.device)
    for at in range(0, x.shape[1], RUN):
        e = torch.full(out.shape, -100, dtype=torch.int32, device=x.device)
        for i in range(at, at + RUN):
            both = (x[:, i, None] != 0) & (w[None, :, i] != 0)
            e = torch.maximum(e, torch.where(both, ex[:, i, None] + ew[None, :, i], torch.full_like(e, -100)))
        unit = torch.ldexp(torch.ones(out.shape, device=x.device), e - 13)
        for i in range(at, at + RUN):
            out += (torch.trunc(x[:, i, None] * w[None, :, i] / unit) * unit).double()
    return out


def whole_numbers(rows, k, gen, dev="cpu"):
    """Small whole numbers; 448 of either sign at two of each 128 elements, at places that rows share."""
    v = torch.randint(-7, 8, (rows, k), generator=gen, device=dev).float()
    sign = torch.randint(0, 2, (rows, k), generator=gen, device=dev).float() * 2 - 1
    at = torch.arange(k, device=dev) % BLOCK
    big = (at == 5) | (at == 6)
    return torch.where(big, 448 * sign, v)


def some_codes(rows, k, gen, dev="cpu"):
    """Any finite E4M3 codes, the small ones as often as the large ones."""
    c = torch.randint(0, 127, (rows, k), generator=gen, device=dev)
    c = c + 128 * torch.randint(0, 2, (rows, k), generator=gen, device=dev)
    return c.to(torch.uint8).view(torch.float8_e4m3fn).float()


def generator(seed, dev="cpu"):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


# ---------------------------------------------------------------------------
# on the CPU: the statement itself
# ---------------------------------------------------------------------------

def test_whole_numbers_show_the_cut():
    """An FP32 result by way of cut products would differ from the exact one nearly everywhere."""
    g = generator(0)
    x, w = whole_numbers(20, 256, g), whole_numbers(30, 256, g)
    exact = x.double() @ w.double().t()
    assert exact.abs().max() < 2 ** 24 and (x.double().abs() @ w.double().abs().t()).max() < 2 ** 24
    assert (cut_sums(x, w) != exact).float().mean() > 0.9


def test_cut_by_hand():
    x, w = torch.zeros(3, BLOCK), torch.ones(1, BLOCK)
    w[0, :2] = 448
    x[:, 0], x[:, 1] = 448, -448
    x[0, 2:8] = 1                                             # six ones in the run of the two large products: lost
    x[1, 8:14] = 1                                            # in another run: kept
    x[2, 2] = 60                                              # cut to a multiple of 2^(8 + 8 - 13) = 8
    assert cut_sums(x, w).tolist() == [[0], [6], [56]]


def test_bound_of_the_cut():
    """A run is off by less than 7 2^(E-13), below 2^-10 of its largest product where no code is below 2^-6."""
    g = generator(1)
    x, w = some_codes(40, RUN, g), some_codes(50, RUN, g)
    off = (cut_sums(x, w) - x.double() @ w.double().t()).abs()
    terms = x[:, None] * w[None]
    e = torch.where(terms != 0, exponent(x)[:, None] + exponent(w)[None], torch.full(terms.shape, -100, dtype=torch.int32)).amax(2)
    assert (off <= 7 * torch.ldexp(torch.ones(e.shape, dtype=torch.float64), e - 13)).all()
    normal = torch.where(x.abs() < 2.0 ** -6, torch.ones_like(x), x), torch.where(w.abs() < 2.0 ** -6, torch.ones_like(w), w)
    off = (cut_sums(*normal) - normal[0].double() @ normal[1].double().t()).abs()
    assert (off < (normal[0][:, None] * normal[1][None]).abs().amax(2).double() * 2.0 ** -10).all()


# ---------------------------------------------------------------------------
# on the GPU
# ---------------------------------------------------------------------------

@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lpc.lib()
    return torch.device("cuda:0")


def say(*a):
    print("[case]", *a, flush=True)


def codes(v):
    return v.to(torch.float8_e4m3fn).view(torch.uint8)


def product(x, w, out_t, counts=None, xs=1.0, ws=1.0):
    """x [rows, k] times w [groups, n, k], all scales xs and ws."""
    dev, (g, n, k) = x.device, w.shape
    out = torch.full((x.shape[0], n), float("nan"), dtype=out_t, device=dev)
    lpc.lpc_gemm_fp8(codes(x), torch.full((x.shape[0], k // BLOCK), xs, device=dev), codes(w),
                     torch.full((g, -(-n // BLOCK), k // BLOCK), ws, device=dev), out,
                     counts=None if counts is None else torch.tensor(counts, dtype=torch.int32, device=dev))
    return out


def grouped(f, x, w, counts):
    parts = zip(x[:sum(counts)].split(counts), w) if counts else [(x, w[0])]
    return torch.cat([f(a, b) for a, b in parts if len(a)])


# rows, k, n, counts: what the sizes choose for fp32 / bf16 results
SIZES = [(3, 1152, 200, None),                                # gathered
         (30, 512, 200, None),                                # 32 x 32 outputs
         (90, 256, 3300, [40, 0, 50]),                        # 64 x 32
         (512, 384, 1100, None),                              # 64 x 64
         (2100, 384, 1700, None),                             # large tiles, all of them split into parts
         (2560, 256, 2000, None),                             # fp32: whole large tiles
         (4096, 256, 2304, None),                             # bf16: whole large tiles
         (2900, 256, 2304, [700, 0, 3, 1200, 997])]           # short tiles at the ends of groups


@pytest.mark.gpu
@pytest.mark.parametrize("rows,k,n,counts", SIZES)
def test_fp32_results_are_exact(dev, rows, k, n, counts):
    say("exact rows=%d k=%d n=%d counts=%s" % (rows, k, n, counts))
    g = generator(rows, dev)
    x = whole_numbers(rows, k, g, dev)
    w = whole_numbers((len(counts) if counts else 1) * n, k, g, dev).view(-1, n, k)
    want = grouped(lambda a, b: a.cpu().double() @ b.cpu().double().t(), x, w, counts)
    assert torch.equal(product(x, w, torch.float32, counts)[:len(want)].cpu().double(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,k,n,counts", SIZES)
def test_bf16_results_are_the_cut_sums(dev, rows, k, n, counts):
    say("cut rows=%d k=%d n=%d counts=%s" % (rows, k, n, counts))
    g = generator(rows + 1, dev)
    x = whole_numbers(rows, k, g, dev)
    w = whole_numbers((len(counts) if counts else 1) * n, k, g, dev).view(-1, n, k)
    want = grouped(cut_sums, x, w, counts)
    assert torch.equal(product(x, w, torch.bfloat16, counts)[:len(want)], want.to(torch.bfloat16))


@pytest.mark.gpu
@pytest.mark.parametrize("rows,k,n", [(3, 1152, 200), (30, 512, 200), (512, 384, 1100), (2100, 256, 1700)])
def test_bf16_results_of_any_codes(dev, rows, k, n):
    """All magnitudes in one run: off from the cut sums by FP32's additions and one rounding to bf16."""
    say("any codes rows=%d k=%d n=%d" % (rows, k, n))
    g = generator(rows + 2, dev)
    x, w = some_codes(rows, k, g, dev), some_codes(n, k, g, dev)
    want, size = cut_sums(x, w), x.double().abs() @ w.double().abs().t()
    off = (product(x, w[None], torch.bfloat16).double() - want).abs()
    fp32 = size * (2 * (BLOCK + k // BLOCK) + 8) * 2.0 ** -24
    assert (off <= fp32 + (want.abs() + fp32) * 2.0 ** -8).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,n,k,counts", [
    (300, 100, 37, None), (390, 200, 300, [1, 0, 260, 100]),           # gathered
    (130, 1030, 1100, None), (390, 700, 900, [1, 0, 260, 100]),        # 128 x 128
    (300, 2300, 2050, None), (390, 1300, 900, [128, 3, 0, 250])])      # 256 x 128
def test_weight_gradients_are_exact(dev, rows, n, k, counts):
    say("wgrad rows=%d n=%d k=%d counts=%s" % (rows, n, k, counts))
    g = generator(rows + n, dev)
    used = counts or [rows]
    tall, blocks = lpc.lpc_padded_rows(rows, len(used)), [-(-c // BLOCK) for c in used]
    forms = []
    for width in (n, k):
        v = whole_numbers(width, tall, g, dev)
        at = 0
        for c, b in zip(used, blocks):
            v[:, at + c:at + b * BLOCK] = 0                   # a group's last block is filled up with zeros
            at += b * BLOCK
        forms.append(v)
    dw = torch.full((len(used), n, k), float("nan"), device=dev)
    one = [torch.ones(tall // BLOCK, width, device=dev) for width in (n, k)]
    lpc.lpc_gemm_fp8_wgrad(codes(forms[0]), one[0], codes(forms[1]), one[1], dw, rows,
                           counts=None if counts is None else torch.tensor(counts, dtype=torch.int32, device=dev))
    yt, xt = (v.cpu().double() for v in forms)
    at = 0
    for i, b in enumerate(blocks):
        part = slice(at, at + b * BLOCK)
        assert torch.equal(dw[i].cpu().double(), yt[:, part] @ xt[:, part].t()), i
        at += b * BLOCK


SCALES = [(1.25 * 2.0 ** -80, 1.75 * 2.0 ** -69),             # multiply to 2.1875 2^-149: rounded to 2 of a denormal's steps
          (1.25 * 2.0 ** -60, 1.75 * 2.0 ** -72),
          (1.25 * 2.0 ** -100, 1.75 * 2.0 ** -20),
          (1.25 * 2.0 ** 60, 1.5 * 2.0 ** 43),                # sums near FP32's largest
          (1.25 * 2.0 ** 120, 1.5 * 2.0 ** -120)]


@pytest.mark.gpu
@pytest.mark.parametrize("out_t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("xs,ws", SCALES)
def test_products_of_extreme_scales(dev, xs, ws, out_t):
    for rows, k, n in ((3, 128, 200), (30, 256, 200), (512, 384, 1100), (2100, 128, 1700)):
        say("scales rows=%d k=%d n=%d %g %g" % (rows, k, n, xs, ws))
        g = generator(rows, dev)
        x, w = (whole_numbers(m, k, g, dev).abs() for m in (rows, n))
        sums = x.double() @ w.double().t() if out_t == torch.float32 else cut_sums(x, w)
        want = sums * (xs * ws)
        assert want.abs().max() < 3e38
        off = (product(x, w[None], out_t, xs=xs, ws=ws).double() - want).abs()
        # the scales' product, each block's product with it and its addition; below 2^-126 half a denormal's step of each
        tol = want * (k // BLOCK + 2) * 2.0 ** -24 + k // BLOCK * 2.0 ** -125
        assert (off <= tol + (want + tol) * (2.0 ** -8 if out_t == torch.bfloat16 else 0)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("ys,xs", SCALES)
def test_weight_gradients_of_extreme_scales(dev, ys, xs):
    for rows, n, k in ((128, 100, 37), (128, 1030, 1100), (256, 2300, 2050)):
        say("scales wgrad rows=%d n=%d k=%d %g %g" % (rows, n, k, ys, xs))
        g, blocks = generator(rows, dev), rows // BLOCK
        yt, xt = (whole_numbers(m, rows, g, dev).abs() for m in (n, k))
        dw = torch.full((n, k), float("nan"), device=dev)
        lpc.lpc_gemm_fp8_wgrad(codes(yt), torch.full((blocks, n), ys, device=dev), codes(xt),
                               torch.full((blocks, k), xs, device=dev), dw, rows)
        want = (yt.double() @ xt.double().t()) * (ys * xs)
        assert ((dw.double() - want).abs() <= want * (blocks + 2) * 2.0 ** -24 + blocks * 2.0 ** -125).all()
