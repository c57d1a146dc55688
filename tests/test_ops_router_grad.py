"""The router's gradient element by element, in every layout that the number of experts chooses, each element within the
rounding of its own terms; and, on the CPU, that a gradient with a term left out or misplaced is outside of that.

u = 2^-24 is half a step of fp32.  A probability's relative error: exp good to 2 units (4 u) of an argument that is off by
u |x - top|, the same for every term of the sum, experts - 1 additions, a quotient and a product."""
import numpy as np
import pytest
import torch

from fp8_precision_allreduce_amd import lpc

U = 2.0 ** -24
TINY = 2.0 ** -125                                            # exp of less is zero or denormal
# 16 lanes with 1, 2, 4, 8 and 16 experts each, 64 lanes with 16; whole vectors of four and not
LAYOUTS = [(40, 5, 2), (40, 16, 4), (33, 27, 3), (33, 32, 8), (50, 50, 4), (50, 64, 6), (40, 101, 8), (40, 128, 16),
           (70, 201, 5), (70, 256, 8), (30, 333, 16), (30, 1000, 4), (30, 1024, 8)]


def inputs(rows, e, topk, dtype, kind, seed=0):
    """Logits, the chosen experts (some slots empty), gradients and slope.  `kind`: which of them are not zero."""
    r = np.random.RandomState(seed)
    f = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32))  # noqa: E731
    x = (2 * f(rows, e)).to(dtype)
    x[torch.from_numpy(r.rand(rows, e) < 0.1)] = -float("inf")
    x[3] = -float("inf")
    which = torch.sort(x.float(), dim=1, descending=True, stable=True)[1][:, :topk].to(torch.int32)
    which[~(x.float().gather(1, which.long()) > -float("inf"))] = -1
    mask = torch.ones(rows, dtype=torch.uint8)
    mask[5], mask[rows - 1] = 0, 0
    which[mask == 0] = -1
    dg = f(rows, topk) if kind != "loss" else torch.zeros(rows, topk)
    slope = f(e).abs() + 0.1 if kind != "gates" else torch.zeros(e)
    return x, which, mask, dg, slope, torch.tensor([0.75])


def gradient(x, which, mask, dg, slope, dloss, normalize, mistake=None):
    """(gradient, tolerance) of sum(gates dg) + dloss sum(p slope) by each logit, in 64 bits; `mistake`: a planted one."""
    x, dg, up = x.double(), dg.double(), dloss.double() * slope.double()
    rows, e = x.shape
    topk = which.shape[1]
    allowed = (x > -float("inf")) & (mask != 0)[:, None]
    top = torch.where(allowed, x, -float("inf")).amax(1, keepdim=True).clamp(min=-1e30)
    p = torch.where(allowed, (x - top).exp(), 0.0)
    p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
    reach = torch.where(allowed, top - x, 0.0).amax(1, keepdim=True).clamp(max=110.0)
    rel = (2 * reach + 8 + e + 2) * U
    taken = which >= 0
    at = which.long().clamp(min=0)
    spread = lambda v: torch.zeros_like(p).scatter_add(1, at, torch.where(taken, v, 0.0))  # noqa: E731
    picked = torch.where(taken, p.gather(1, at), 0.0)
    if mistake == "slope of the next expert":
        up = up.roll(1)
    if mistake == "no balance loss":
        up = torch.zeros_like(up)
    if mistake == "gate of the next slot":
        dg = dg.roll(1, 1)
    dot_of = lambda v: (p * v).sum(1, keepdim=True)  # noqa: E731
    if normalize:
        gates = picked / picked.sum(1, keepdim=True).clamp(min=1e-300)
        inner, inner_size = (gates * dg).sum(1, keepdim=True), (gates * dg.abs()).sum(1, keepdim=True)
        direct = spread(gates * (dg - inner))
        rel_gate = 2 * rel + (topk + 2) * U                   # a quotient of p and a sum of topk of them
        off = spread(gates * ((dg.abs() + inner_size) * (rel_gate + 3 * U) + inner_size * (rel_gate + (topk + 1) * U)))
        slopes = up.expand_as(p)
    else:
        direct, off = torch.zeros_like(p), torch.zeros_like(p)
        slopes = up + spread(dg)
    if mistake == "zero where not chosen":
        slopes = torch.where(spread(torch.ones_like(dg)) > 0, slopes, 0.0)
    dot, size = dot_of(slopes), dot_of(slopes.abs())
    if mistake == "no mean over the experts":
        dot = torch.zeros_like(dot)
    if mistake == "no gates":
        direct = torch.zeros_like(p)
        dot = dot if normalize else dot_of(up.expand_as(p))
        slopes = slopes if normalize else up.expand_as(p)
    dx = p * (slopes - dot) + direct
    # slopes: a product and a sum; dot: e products and additions of terms each off by rel; then a difference, a product, a sum
    tol = off + p * ((slopes.abs() + size) * (rel + 5 * U) + size * (rel + (e + 4) * U)) + dx.abs() * U
    return dx, tol + TINY * (1 + slopes.abs() + size)


def within(got, want, tol, dtype):
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0      # of the result's one rounding to bf16
    return (got.double() - want).abs() <= tol + (want.abs() + tol) * half


KINDS = ["both", "loss", "gates"]
MISTAKES = {"both": ["no balance loss", "no gates"], "gates": ["no gates", "gate of the next slot"],
            "loss": ["no balance loss", "slope of the next expert", "no mean over the experts", "zero where not chosen"]}


def case(rows, e, topk, dtype, kind):
    print("[case] rows=%d experts=%d topk=%d %s %s" % (rows, e, topk, dtype, kind), flush=True)
    return inputs(rows, e, topk, dtype, kind, seed=e)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("rows,e,topk", LAYOUTS)
def test_formula_and_what_the_tolerance_tells_apart(rows, e, topk, normalize, dtype):
    for kind in KINDS:
        a = case(rows, e, topk, dtype, kind)
        want, tol = gradient(*a, normalize)
        x, which, mask, dg, slope, dloss = a
        xa = x.double().requires_grad_()
        ok = (x > -float("inf")) & (mask != 0)[:, None]
        rows_on = ok.any(1)
        p = torch.zeros(rows, e, dtype=torch.float64)
        p[rows_on] = torch.softmax(torch.where(ok, xa, -float("inf"))[rows_on], 1)
        gates = torch.where(which >= 0, p.gather(1, which.long().clamp(min=0)), 0.0)
        if normalize:
            gates = gates / gates.sum(1, keepdim=True).clamp(min=1e-300)
        ((gates * dg.double()).sum() + dloss.double()[0] * (p * slope.double()).sum()).backward()
        auto = torch.where(ok, xa.grad, 0.0)
        assert torch.allclose(want, auto, rtol=1e-11, atol=1e-13)
        for mistake in MISTAKES[kind]:
            wrong = gradient(*a, normalize, mistake)[0].to(dtype)
            assert not within(wrong, want, tol, dtype).all(), (kind, mistake)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("rows,e,topk", LAYOUTS)
def test_gradient(rows, e, topk, normalize, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    for kind in KINDS:
        x, which, mask, dg, slope, dloss = a = case(rows, e, topk, dtype, kind)
        want, tol = gradient(*a, normalize)
        dx = torch.full((rows, e), 9.0, dtype=dtype, device="cuda:0")
        lpc.lpc_router_backward(*(t.to("cuda:0") for t in (x, which, slope, dg, dloss)), dx, normalize=normalize,
                                mask=mask.to("cuda:0"))
        got = dx.cpu()
        bad = ~within(got, want, tol, dtype)
        assert not bad.any(), (kind, int(bad.sum()), float(((got.double() - want).abs() / tol).max()))
        assert (got[~(x > -float("inf"))] == 0).all() and (got[mask == 0] == 0).all()
