"""The bf16 products, the 4-bit operators and Muon on other streams than the current one, captured in graphs, from call to call, and
one after the other as an expert's weights go through them; Muon's own memory on the CPU, with the allocator stood in for."""
import pytest
import torch

from fp8_precision_allreduce_amd import lpc
from test_ops_streams import pointer

U = 2.0 ** -24
BF16 = torch.bfloat16


def test_muon_step_keeps_its_memory_for_its_stream(monkeypatch):
    """Plan and workspace are used by a step's kernels; dropping the optimizer may not free them under a step on another stream."""
    t = lambda: torch.zeros(50, 100)  # noqa: E731
    recorded, calls, order = [], [], []
    empty = torch.empty
    monkeypatch.setattr(lpc._Args, "__call__", pointer)
    monkeypatch.setattr(lpc._Args, "many", lambda self, ts, what, dtypes, ns: [pointer(self, v) for v in ts])
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: (order.append("empty " + str(device)), empty(*a, **kw))[1])
    monkeypatch.setattr(torch.Tensor, "to", lambda self, *a, **kw: (order.append("copy"), self)[1])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, s: recorded.append((self.data_ptr(), s)))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handle)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0x10, raising=False)
    monkeypatch.setattr(lpc, "_run", lambda name, device, stream, *a: calls.append((name, stream)))
    opt = lpc.Muon([t()], [t()], [t()])
    assert order == ["empty None", "empty cuda:0", "copy"]    # the copy waits for what used the workspace's memory before
    opt.step(lr=0.1)
    assert recorded == [] and calls == [("lpc_muon_step", 0x10)]
    opt.step(lr=0.1, stream=0x20)
    both = [opt._plan.data_ptr(), opt._space.data_ptr()]
    assert recorded == [(p, 0x20) for p in both] and calls[1:] == [("lpc_muon_step", 0x20)]
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0x30)
    opt.step(lr=0.1)                                           # the current stream is another one now
    assert recorded[2:] == [(p, 0x30) for p in both]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lpc.lib()
    return torch.device("cuda:0")


class Everything:
    """One call of every operator on inputs of its own, in forms that the launchers choose differently."""

    def __init__(self, dev, seed):
        gen = torch.Generator(device=dev)
        gen.manual_seed(seed)
        self.r = lambda *s: torch.randn(*s, generator=gen, device=dev)
        self.dev, self.calls = dev, []
        for rows, k, n, counts in ((20, 512, 128, None), (300, 264, 520, [100, 0, 150]), (2100, 136, 2056, None)):
            self.product(rows, k, n, counts)
        for rows, k, n, counts in ((5, 256, 96, None), (300, 384, 520, [100, 0, 150]), (2100, 128, 2056, None)):
            self.mxfp4(rows, k, n, counts)
        self.muon([(16, 300), (40, 30), (3, 130, 200)])

    def product(self, rows, k, n, counts):
        g = 1 if counts is None else len(counts)
        x, w, dy = self.r(rows, k).to(BF16), self.r(g, n, k).to(BF16), self.r(rows, n).to(BF16)
        c = None if counts is None else torch.tensor(counts, dtype=torch.int32, device=self.dev)
        out, dx, dw = (torch.zeros(*s, device=self.dev) for s in ((rows, n), (rows, k), (g, n, k)))
        self.calls += [(lambda s: lpc.lpc_gemm_bf16(x, w, out, counts=c, stream=s), [out], [x, w]),
                       (lambda s: lpc.lpc_gemm_bf16_dgrad(dy, w, dx, counts=c, stream=s), [dx], [dy]),
                       (lambda s: lpc.lpc_gemm_bf16_wgrad(dy, x, dw, counts=c, stream=s), [dw], [x])]

    def mxfp4(self, rows, k, n, counts):
        g = 1 if counts is None else len(counts)
        x, w = self.r(rows, k), self.r(g, n, k).to(BF16)
        c = None if counts is None else torch.tensor(counts, dtype=torch.int32, device=self.dev)
        new = lambda *s: torch.zeros(*s, dtype=torch.uint8, device=self.dev)  # noqa: E731
        xc, xs, wc, ws, out, back = new(rows, k // 2), new(rows, k // 32), new(g, n, k // 2), new(g, n, k // 32), self.r(rows, n), self.r(rows, k)
        self.calls += [(lambda s: lpc.lpc_quantize_mxfp4(x, xc, xs, stream=s), [xc, xs], [x]),
                       (lambda s: lpc.lpc_quantize_mxfp4(w, wc, ws, stream=s), [wc, ws], [w]),
                       (lambda s: lpc.lpc_gemm_mxfp4(xc, xs, wc, ws, out, counts=c, stream=s), [out], []),
                       (lambda s: lpc.lpc_dequantize_mxfp4(xc, xs, back, stream=s), [back], [])]

    def muon(self, shapes):
        p, g, m = ([self.r(*s) for s in shapes] for _ in range(3))
        copies = [t.to(BF16) for t in p]
        start = [(t, t.clone()) for t in p + m]

        def step(s, opt=lpc.Muon(p, g, m, copies=copies)):
            for t, was in start:
                t.copy_(was)
            opt.step(lr=0.1, weight_decay=0.1, stream=s)

        self.calls.append((step, p + m + copies, g))

    def run(self, stream=None):
        for call, _, _ in self.calls:
            call(stream)

    def outputs(self):
        return [t.clone() for _, ts, _ in self.calls for t in ts]

    def change_inputs(self):
        for _, _, ts in self.calls:
            for t in ts:
                t.mul_(-0.75)


def same(a, b):
    return len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.gpu
def test_the_same_bits_every_time(dev):
    a, b = Everything(dev, 1), Everything(dev, 1)
    a.run()
    b.run()
    first = a.outputs()
    assert same(first, b.outputs()) and all(torch.isfinite(t.float()).all() for t in first)
    for _ in range(3):
        a.run()
        assert same(first, a.outputs())


@pytest.mark.gpu
def test_graph_replays_match_eager(dev):
    """Replays see the inputs as they are, and eager work and other graphs between them change nothing."""
    e, other = Everything(dev, 2), Everything(dev, 3)
    side = torch.cuda.Stream()
    graphs = []
    for x in (e, other):
        with torch.cuda.stream(side):
            x.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            x.run()
        graphs.append(g)
    for _ in range(4):
        e.change_inputs()
        e.run()
        torch.cuda.synchronize()
        want = e.outputs()
        for _, ts, _ in e.calls:
            for t in ts:
                t.zero_()
        graphs[1].replay()
        graphs[0].replay()
        torch.cuda.synchronize()
        assert same(want, e.outputs())


@pytest.mark.gpu
def test_two_streams_at_once(dev):
    xs, streams = [Everything(dev, s) for s in (4, 5)], [torch.cuda.Stream() for _ in range(2)]
    want = []
    for x in xs:
        x.run()
        want.append(x.outputs())
        for _, ts, _ in x.calls:
            for t in ts:
                t.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                x.run()
    torch.cuda.synchronize()
    assert all(same(w, x.outputs()) for w, x in zip(want, xs))
    for i in (0, 1):  # a stream that is given: as a handle and as an object
        s = streams[i].cuda_stream if i else streams[i]
        for call, outs, _ in xs[i].calls[:-1]:  # (the optimizer's restart is eager work of the current stream)
            call(s)
    torch.cuda.synchronize()
    assert all(same(w, x.outputs()) for w, x in zip(want, xs))


@pytest.mark.gpu
def test_an_experts_weights_from_step_to_answer(dev):
    """Forward, both gradients, the update and the 4-bit product, each from what the one before gave, against 64 bits throughout.
    Every step is compared by itself on its real inputs, so that tolerances are those of one operator."""
    torch.manual_seed(7)
    rows, k, n, experts, splits = 200, 256, 128, 3, [90, 0, 100]
    x, target = torch.randn(rows, k, device=dev).to(BF16), torch.randn(rows, n, device=dev)
    w = torch.randn(experts, n, k, device=dev) * k ** -0.5
    copy, m, dw = w.to(BF16), torch.zeros_like(w), torch.empty_like(w)
    counts = torch.tensor(splits, dtype=torch.int32, device=dev)
    opt = lpc.Muon([w], [dw], [m], copies=[copy])
    out, dx = torch.empty(rows, n, device=dev), torch.empty(rows, k, device=dev)
    codes, scales = torch.empty(experts, n, k // 2, dtype=torch.uint8, device=dev), torch.empty(experts, n, k // 32, dtype=torch.uint8, device=dev)
    xc, xs = torch.empty(rows, k // 2, dtype=torch.uint8, device=dev), torch.empty(rows, k // 32, dtype=torch.uint8, device=dev)
    held, xh, served = torch.empty(experts, n, k, device=dev), torch.empty(rows, k, device=dev), torch.empty(rows, n, device=dev)
    spans = [(0, 90), (90, 90), (90, 190)]

    def near(got, want, size, terms):
        assert ((got.double() - want).abs() <= size * 2 * terms * U + want.abs() * U).all()

    for step in range(3):
        used = copy.double()
        lpc.lpc_gemm_bf16(x, copy, out, counts=counts)
        dy = ((out - target) * (1.0 / rows)).to(BF16)
        lpc.lpc_gemm_bf16_dgrad(dy, copy, dx, counts=counts)
        lpc.lpc_gemm_bf16_wgrad(dy, x, dw, counts=counts)
        before, momentum = w.double().clone(), m.double().clone()
        opt.step(lr=0.01, beta=0.9)
        for g, (a, b) in enumerate(spans):
            xd, dd, wd = x[a:b].double(), dy[a:b].double(), used[g]
            near(out[a:b], xd @ wd.t(), xd.abs() @ wd.abs().t(), k)
            near(dx[a:b], dd @ wd, dd.abs() @ wd.abs(), n)
            near(dw[g], dd.t() @ xd, dd.abs().t() @ xd.abs(), b - a + 1)
            mu = 0.9 * momentum[g] + 0.1 * dw[g].double()
            u = 0.9 * mu + 0.1 * dw[g].double()
            if float(u.norm()) == 0:
                assert torch.equal(w[g].double(), before[g])
                continue
            o = u / u.norm()
            for _ in range(5):
                s = o @ o.t()
                o = 3.4445 * o + (-4.7750 * s + 2.0315 * s @ s) @ o
            want = 0.01 * 0.2 * k ** 0.5 * o
            # an update is off by 4e-3 of itself at most, and the sum is rounded
            assert float((before[g] - w[g].double() - want).norm()) <= 4e-3 * float(want.norm()) + 2 * U * float(before[g].norm())
        assert (out[190:] == 0).all() and (dx[190:] == 0).all() and torch.equal(copy, w.to(BF16))
        lpc.lpc_quantize_mxfp4(w, codes, scales)
        lpc.lpc_dequantize_mxfp4(codes, scales, held)
        lpc.lpc_quantize_mxfp4(x, xc, xs)
        lpc.lpc_dequantize_mxfp4(xc, xs, xh)
        # in units of the scale the largest is in [4, 8): between 4 and 6 a value is off by 1 at most, and one of up to 8 becomes 6
        top = w.reshape(-1, 32).abs().amax(1, keepdim=True)
        assert ((held - w).reshape(-1, 32).abs() <= top / 4).all()
        lpc.lpc_gemm_mxfp4(xc, xs, codes, scales, served, counts=counts)
        for g, (a, b) in enumerate(spans):
            near(served[a:b], xh[a:b].double() @ held[g].double().t(), xh[a:b].double().abs() @ held[g].double().abs().t(), k)
