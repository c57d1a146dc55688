"""The operators' own device memory (the router's workspace, AdamW's plan) where a call runs on a stream that is not the
current one: on the CPU with the allocator and the entry points stood in for, and on the GPU."""
import contextlib

import pytest
import torch

from fp8_precision_allreduce_amd import lpc

ROWS, EXPERTS, TOPK = 1000, 60, 4


class Streams:
    """Stands in for torch.cuda's streams: which one is current when something is allocated."""

    def __init__(self, monkeypatch):
        self.current, self.allocated = "current", []
        empty = torch.empty

        @contextlib.contextmanager
        def enter(s):
            was, self.current = self.current, s
            yield
            self.current = was

        def record(*a, device=None, **kw):
            self.allocated.append(self.current)
            return empty(*a, **kw)

        monkeypatch.setattr(torch.cuda, "stream", enter)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handle)
        monkeypatch.setattr(torch, "empty", record)
        monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)


def pointer(self, t, *_):
    self.device = 0
    return t.data_ptr()


def router_buffers(dev):
    return [torch.zeros(ROWS, TOPK, dtype=torch.int32, device=dev), torch.zeros(ROWS, TOPK, device=dev),
            torch.zeros(EXPERTS, dtype=torch.int32, device=dev), torch.zeros(EXPERTS, device=dev),
            torch.zeros(EXPERTS, device=dev), torch.zeros(1, device=dev)]


def test_router_workspace_is_of_the_streams_pool(monkeypatch):
    """A workspace of another stream's pool may still be read or written by that stream's earlier calls."""
    out, x = router_buffers("cpu"), torch.zeros(ROWS, EXPERTS)
    assert lpc.lpc_router_workspace_bytes(ROWS, EXPERTS) > 0
    streams, calls = Streams(monkeypatch), []
    monkeypatch.setattr(lpc._Args, "__call__", pointer)
    monkeypatch.setattr(lpc, "_run", lambda name, device, stream, *a: calls.append((name, stream)))
    lpc.lpc_router_forward(x, *out, coef=0.1, stream=0x5000)
    assert calls == [("lpc_router_forward", 0x5000)] and streams.allocated == [0x5000]
    lpc.lpc_router_forward(x, *out, coef=0.1)
    assert calls[1:] == [("lpc_router_forward", None)] and streams.allocated[1:] == ["current"]


def test_adamw_step_keeps_its_plan_for_its_stream(monkeypatch):
    """The plan is read by a step's kernel; dropping the optimizer may not free it under a step on another stream."""
    t = lambda: torch.zeros(5000)  # noqa: E731
    recorded, calls = [], []
    monkeypatch.setattr(lpc._Args, "__call__", pointer)
    monkeypatch.setattr(lpc._Args, "many", lambda self, ts, what, dtypes, ns: [pointer(self, v) for v in ts])
    monkeypatch.setattr(torch.Tensor, "to", lambda self, *a, **kw: self)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, s: recorded.append((self.data_ptr(), s)))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handle)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0x10, raising=False)
    monkeypatch.setattr(lpc, "_run", lambda name, device, stream, *a: calls.append(stream))
    opt = lpc.AdamW([t()], [t()], [t()], [t()])
    opt.step(1, lr=0.1)
    assert recorded == [] and calls in ([0x10], [None])
    opt.step(2, lr=0.1, stream=0x20)
    assert recorded == [(opt._plan.data_ptr(), 0x20)] and calls[1:] == [0x20]
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0x30)
    opt.step(3, lr=0.1)                                       # the current stream is another one now
    assert recorded[1:] == [(opt._plan.data_ptr(), 0x30)]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lpc.lib()
    return torch.device("cuda:0")


@pytest.mark.gpu
def test_router_on_given_streams_agrees(dev):
    """Calls in turn on three streams, each without a workspace, with a different input each: no call sees another's."""
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.manual_seed(3)
    xs = [torch.randn(ROWS, EXPERTS, device=dev) for _ in range(12)]
    want, got = [], []
    for x in xs:
        want.append(router_buffers(dev))
        lpc.lpc_router_forward(x, *want[-1], coef=0.1)
    got = [router_buffers(dev) for _ in xs]
    torch.cuda.synchronize()
    for i, x in enumerate(xs):
        s = streams[i % 3]
        lpc.lpc_router_forward(x, *got[i], coef=0.1, stream=s if i % 2 else s.cuda_stream)
        lpc.lpc_router_forward(x, *router_buffers(dev), coef=0.1)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.gpu
def test_adamw_plan_outlives_its_optimizer_under_a_step(dev):
    """While a step waits on another stream, what is allocated after its optimizer is gone is not its plan."""
    side = torch.cuda.Stream()
    p, g, m, v = (torch.full((50_000,), c, device=dev) for c in (0.5, 0.1, 0.0, 0.0))
    big = torch.empty(1 << 30, dtype=torch.uint8, device=dev)
    want = p.clone()
    lpc.AdamW([want], [g], [m.clone()], [v.clone()]).step(1, lr=1e-2)
    opt = lpc.AdamW([p], [g], [m], [v])
    size, plan = opt._plan.numel(), opt._plan.data_ptr()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(200):
            big.zero_()
    opt.step(1, lr=1e-2, stream=side)
    del opt
    after = torch.empty(size, dtype=torch.uint8, device=dev)  # never written
    assert not side.query()                                   # the step has not run yet
    assert after.data_ptr() != plan
    torch.cuda.synchronize()
    assert torch.equal(p, want)
