"""The matrix operators at what a launch can hold: calls past it are refused before anything runs, and those below it run."""
import pytest
import torch

from fp8_precision_allreduce_amd import lpc
from test_matrix_ops_gpu import BF16, MX, dev, mx_oracle, near, randn, say  # noqa: F401
from test_ops_abi_cpu import A, HIP, L, SHAPE  # noqa: F401
from test_ops_abi_cpu import BF16 as BF16_T

MOST = (1 << 23) - 512  # tiles of 256 x 256


def test_products_past_a_launch(L):  # noqa: F811
    """No device here: a call that passes the checks comes to LPC_ERR_HIP."""
    product = lambda rows, n, k: L.lpc_gemm_bf16(A, rows, k, A, n, 1, None, A, BF16_T, None)  # noqa: E731
    dgrad = lambda rows, n, k: L.lpc_gemm_bf16_dgrad(A, rows, n, A, k, 1, None, A, BF16_T, None)  # noqa: E731
    wgrad = lambda n, k: L.lpc_gemm_bf16_wgrad(A, n, A, k, 8, 1, None, A, BF16_T, None)  # noqa: E731
    mxfp4 = lambda rows, n, k: L.lpc_gemm_mxfp4(A, A, rows, k, A, A, n, 1, None, A, BF16_T, None)  # noqa: E731
    assert product(MOST * 256, 1, 8) == HIP and product((1 << 31) - 1, 1, 8) == SHAPE
    assert dgrad(MOST * 256, 8, 8) == HIP and dgrad((1 << 31) - 1, 8, 8) == SHAPE
    assert wgrad(1 << 20, 1 << 18) == HIP and wgrad(1 << 20, 1 << 19) == SHAPE
    assert mxfp4(MOST * 256, 1, 128) == HIP and mxfp4((1 << 31) - 1, 1, 128) == SHAPE


def muon_bytes(L, *rows):  # noqa: F811
    return L.lpc_muon_plan_bytes((lpc._MuonTensor * len(rows))(*[lpc._MuonTensor(A, A, A, None, *r, 1.0) for r in rows]), len(rows))


def test_muon_plans_what_its_steps_can_launch(L):  # noqa: F811
    """A plan that no step takes is refused when it is made, and a step refuses it before its first launch, which changes the momenta."""
    few = (1 << 24) - 1
    assert muon_bytes(L, (MOST, 33, 33)) and not muon_bytes(L, (MOST + 1, 33, 33))          # tiles of both products
    assert muon_bytes(L, (few, 4, 4)) and not muon_bytes(L, (few + 1, 4, 4))                # small matrices
    assert muon_bytes(L, (MOST, 33, 33), (1 << 23, 4, 4)) and not muon_bytes(L, (MOST, 33, 33), (few, 4, 4))   # all matrices
    step = lambda work: L.lpc_muon_step(A, work, 0, 0.1, 0.9, 1, 0.0, 5, None, A, 1 << 40, None)  # noqa: E731
    for field, most in (("matrices", few), ("chunks", few), ("smalls", few), ("squares", MOST), ("updates", MOST)):
        for n, status in ((most, HIP), (most + 1, SHAPE)):
            work = lpc._MuonWork(1, 1, 1, 1, 1, 64)
            setattr(work, field, n)
            assert step(work) == status, (field, n)


def room(gib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip("needs %d GiB of device memory" % gib)


def columns(n):
    return torch.tensor([0, 1, 255, 256, n // 2 - 1, n // 2, n - 257, n - 2, n - 1])


@pytest.mark.gpu
def test_bf16_few_rows_and_many_outputs(dev):  # noqa: F811
    """More tiles of 32 x 32 than a launch can have."""
    room(40)
    rows, n, k, counts = 64, (1 << 27) + 5, 8, [33, 31]
    say("bf16", rows, n, k)
    x, w = randn(rows, k, seed=1).to(BF16), torch.randn(2, n, k, device=dev).to(BF16)
    out = torch.full((rows, n), 7.0, dtype=BF16, device=dev)
    lpc.lpc_gemm_bf16(x.to(dev), w, out, counts=torch.tensor(counts, dtype=torch.int32, device=dev))
    at = columns(n)
    for g, (a, b) in enumerate(((0, 33), (33, 64))):
        xd, wd = x[a:b].double(), w[g, at.to(dev)].cpu().double()
        near(out[a:b, at.to(dev)], xd @ wd.t(), xd.abs() @ wd.abs().t(), k, BF16, "group %d" % g)


@pytest.mark.gpu
def test_mxfp4_few_rows_and_many_outputs(dev):  # noqa: F811
    room(60)
    rows, n, k, counts = 64, (1 << 27) + 5, 128, [33, 31]
    say("mxfp4", rows, n, k)
    xc, xs, x = mx_oracle(randn(rows, k, seed=1))
    at = columns(n)
    wc, ws, w = mx_oracle(randn(2, len(at), k, seed=2))
    codes = torch.zeros(2, n, k // 2, dtype=torch.uint8, device=dev)
    scales = torch.zeros(2, n, k // MX, dtype=torch.uint8, device=dev)
    codes[:, at.to(dev)], scales[:, at.to(dev)] = wc.to(dev), ws.to(dev)
    out = torch.full((rows, n), 7.0, dtype=BF16, device=dev)
    lpc.lpc_gemm_mxfp4(xc.to(dev), xs.to(dev), codes, scales, out, counts=torch.tensor(counts, dtype=torch.int32, device=dev))
    for g, (a, b) in enumerate(((0, 33), (33, 64))):
        near(out[a:b, at.to(dev)], x[a:b] @ w[g].t(), x[a:b].abs() @ w[g].abs().t(), k, BF16, "group %d" % g)
    assert not out[:, 1000:2000].any()


END = 96  # elements at each of the places looked at


@pytest.mark.gpu
def test_codec_past_a_launch(dev):  # noqa: F811
    """More lanes than a launch can have: 2^35 elements from fp32 or to bf16, 8 to a lane.  The first elements, the last, and those around each
    2^33 of them."""
    n, step = (1 << 35) + END, 1 << 33
    room(170)
    where = [slice(0, END)] + [slice(i * step + d, i * step + d + END) for i in range(1, 5) for d in (-END, 0) if i * step + d + END <= n]
    ends = randn(len(where), END, seed=1)
    c, s, v = mx_oracle(ends)
    parts = lambda w, d: slice(w.start // d, w.stop // d)  # noqa: E731
    codes, scales = torch.full((n // 2,), 0x99, dtype=torch.uint8, device=dev), torch.full((n // MX,), 9, dtype=torch.uint8, device=dev)
    x = torch.zeros(n, device=dev)
    for i, w in enumerate(where):
        x[w] = ends[i].to(dev)
    say("quantize", n)
    lpc.lpc_quantize_mxfp4(x, codes, scales)
    for i, w in enumerate(where):
        assert torch.equal(codes[parts(w, 2)].cpu(), c[i]) and torch.equal(scales[parts(w, MX)].cpu(), s[i]), i
    del x
    out = torch.full((n,), 7.0, dtype=BF16, device=dev)
    say("dequantize", n)
    lpc.lpc_dequantize_mxfp4(codes, scales, out)
    for i, w in enumerate(where):
        assert torch.equal(out[w].cpu(), v[i].to(BF16)), i
    for i in range(4):
        assert not out[i * step + END:(i + 1) * step - END].any(), i


@pytest.mark.gpu
def test_bf16_most_rows(dev):  # noqa: F811
    """As many rows as their tiles allow, 8 long: offsets of both operands and of the results pass 32 bits."""
    room(130)
    rows, k = MOST * 256, 8
    at = torch.tensor([0, 1, 255, 256, (1 << 29) - 1, 1 << 29, (1 << 30) + 77, rows - 257, rows - 256, rows - 1], device=dev)
    x, some = torch.zeros(rows, k, dtype=BF16, device=dev), randn(len(at), k, seed=1).to(BF16)
    x[at] = some.to(dev)
    for n, counts in ((1, None), (1, [1 << 29, rows - (1 << 29) - 5])):
        g = 1 if counts is None else 2
        w = randn(g, n, k, seed=2).to(BF16)
        out = torch.full((rows, n), 7.0, device=dev)
        say("bf16 product", rows, n, counts)
        lpc.lpc_gemm_bf16(x, w.to(dev), out, counts=None if counts is None else torch.tensor(counts, dtype=torch.int32, device=dev))
        for i, r in enumerate(at.tolist()):
            group = 0 if counts is None or r < counts[0] else 1
            wd = w[group].double() * (counts is None or r < sum(counts))  # the rows past the last group give zeros
            near(out[r], some[i].double() @ wd.t(), some[i].double().abs() @ wd.abs().t(), k, torch.float32, "row %d" % r)
        assert int((out != 0).sum()) <= len(at)
    del out
    dx, w = torch.full((rows, 8), 7.0, dtype=BF16, device=dev), randn(8, 8, seed=3).to(BF16)
    say("bf16 dgrad", rows)
    lpc.lpc_gemm_bf16_dgrad(x, w.to(dev), dx)
    wd = w.double()
    near(dx[at], some.double() @ wd, some.double().abs() @ wd.abs(), 8, BF16, "dgrad")
    assert int((dx != 0).any(1).sum()) <= len(at)


class Shifted:
    """Copies of tensors that start 16 bytes into a buffer (row counts and single numbers: 4), the least alignment that is taken."""

    def __init__(self, dev):
        self.dev = dev

    def __call__(self, t, by=16):
        size = t.element_size()
        buffer = torch.zeros(t.numel() + by // size, dtype=t.dtype, device=self.dev)
        view = buffer[by // size:by // size + t.numel()].view(t.shape)
        view.copy_(t)
        assert view.data_ptr() % 256 == by
        return view


@pytest.mark.gpu
@pytest.mark.parametrize("rows,k,n,counts", [(20, 128, 72, [9, 11]), (300, 384, 520, [100, 0, 150]), (2100, 128, 2056, [2100])])
def test_operands_of_the_least_alignment(dev, rows, k, n, counts):  # noqa: F811
    say("alignment", rows, k, n, counts)
    at, g = Shifted(dev), len(counts)
    same = lambda t, by=16: t.to(dev)  # noqa: E731
    x, w, dy = randn(rows, k, seed=1).to(BF16), randn(g, n, k, seed=2).to(BF16), randn(rows, n, seed=3).to(BF16)
    results = []
    for put in (same, at):
        c, q, p, d = put(torch.tensor(counts, dtype=torch.int32), 4), put(x), put(w), put(dy)
        out, dx, dw = put(torch.zeros(rows, n, dtype=BF16)), put(torch.zeros(rows, k)), put(torch.zeros(g, n, k))
        lpc.lpc_gemm_bf16(q, p, out, counts=c)
        lpc.lpc_gemm_bf16_dgrad(d, p, dx, counts=c)
        lpc.lpc_gemm_bf16_wgrad(d, q, dw, counts=c)
        codes, scales = put(torch.zeros(rows, k // 2, dtype=torch.uint8)), put(torch.zeros(rows, k // MX, dtype=torch.uint8))
        wc, ws = put(torch.zeros(g, n, k // 2, dtype=torch.uint8)), put(torch.zeros(g, n, k // MX, dtype=torch.uint8))
        lpc.lpc_quantize_mxfp4(q, codes, scales)
        lpc.lpc_quantize_mxfp4(p, wc, ws)
        served, back = put(torch.zeros(rows, n)), put(torch.zeros(rows, k, dtype=BF16))
        lpc.lpc_gemm_mxfp4(codes, scales, wc, ws, served, counts=c)
        lpc.lpc_dequantize_mxfp4(codes, scales, back)
        results.append([t.clone() for t in (out, dx, dw, codes, scales, wc, ws, served, back)])
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.gpu
def test_muon_of_the_least_alignment(dev):  # noqa: F811
    """Parameters, gradients, momenta, copies, the plan and the workspace."""
    shapes = [(3, 33, 35), (16, 300), (2, 300, 520), (9, 7)]
    same, results = (lambda t, by=16: t.to(dev)), []
    for put in (same, Shifted(dev)):
        p, g, m = ([put(randn(*s, seed=10 * i + j)) for j, s in enumerate(shapes)] for i in range(3))
        copies = [put(t.to(BF16).cpu()) for t in p]
        opt = lpc.Muon(p, g, m, copies=copies)
        if put is not same:
            opt._plan, opt._space = put(opt._plan), put(opt._space)
        say("muon", shapes)
        opt.step(lr=0.1, grad_scale=put(torch.tensor([0.5]), 4))
        results.append([t.clone() for t in p + m + copies])
    assert all(torch.equal(a, b) for a, b in zip(*results))
