"""Muon's iterations by themselves, for every number of them and for updates of full and of low rank, against 64 bits.

beta 0 without Nesterov makes m = g and u = g exactly, and parameters of zeros with lr and scale 1 become -X, rounded once: what is
compared is X alone, on the update that the kernel itself takes.

a = 3.4445 is what an iteration multiplies a small singular value by, and the most that it multiplies a rounding error in a direction that
the update does not have."""
import numpy as np
import pytest
import torch

from fp8_precision_allreduce_amd import lpc
from test_matrix_ops_gpu import F32, U, Guarded, dev, orthogonal64, say  # noqa: F401

pytestmark = pytest.mark.gpu
A = 3.4445


def update(rows, cols, kind, seed=0):
    """Exactly of the rank that its name says: products of small whole numbers are exact."""
    rng = np.random.RandomState(seed)
    short, long = min(rows, cols), max(rows, cols)
    if kind.startswith("rank"):
        u = rng.randint(-9, 10, (short, int(kind[4:]))).astype(float) @ rng.randint(-9, 10, (int(kind[4:]), long))
    elif kind == "repeated":
        u = np.repeat(rng.standard_normal(((short + 3) // 4, long)), 4, 0)[:short]
    elif kind == "strong":  # a few directions that hide the rest
        u = rng.standard_normal((short, 2)) @ rng.standard_normal((2, long)) + 0.003 * rng.standard_normal((short, long))
    else:
        u = rng.standard_normal((short, long))
    return torch.from_numpy(u if rows <= cols else u.T.copy()).float()


def iterated(dev, g, iterations):  # noqa: F811
    """The kernel's X of one matrix."""
    p, m = Guarded(g.shape, F32, dev), Guarded(g.shape, F32, dev)
    p.t.zero_()
    m.t.zero_()
    lpc.Muon([p.t], [g.to(dev)], [m.t], scales=[1.0]).step(lr=1.0, beta=0.0, nesterov=False, iterations=iterations)
    assert torch.equal(m.check().cpu(), g)
    return -p.check().cpu().double()


def off(got, want):
    return float((got - want).norm() / want.norm())


SMALL = [(4, 64), (16, 16), (16, 1152), (24, 300), (32, 130), (300, 32), (64, 4), (1152, 16), (5, 20000)]
KINDS = ["rank1", "rank3", "repeated", "strong", "normal"]


@pytest.mark.parametrize("iterations", range(1, 11))
@pytest.mark.parametrize("kind", KINDS)
def test_short_sides(dev, kind, iterations):  # noqa: F811
    """A side of 32 and less.  All is 64 bits from u on, and X is rounded to FP32: U.  The update's 64-bit A = U U^T is off by the roundings of
    at most 200 additions in a row, and each iteration's three products of 32 terms add 100 of what is then there: 300 2^-53 in all.
    X = R U where R takes A's eigenvalue l = s^2 to x(s) / s, which is a^n at 0: between 0 and l it changes by a^n / l at most, so that
    d in A changes X by d s a^n / l = d a^n / s, and where s < a^-n, as R is flat there, by d a^2n."""
    for rows, cols in SMALL:
        g = update(rows, cols, kind)
        say("muon", rows, cols, kind, iterations)
        s = torch.linalg.svdvals(g.double() / g.double().norm())
        least = max(float(s[s > 1e-9].min()), A ** -iterations)
        got = off(iterated(dev, g, iterations), orthogonal64(g.double(), iterations))
        assert got <= U + 300 * 2.0 ** -53 * A ** iterations / least, (rows, cols, got)


def strong_and_weak(side, other, weak, seed=0):
    """One element of 1 and, in rows and columns of their own, a block of norm `weak` whose singular values are alike."""
    u = torch.zeros(side, other, dtype=torch.float64)
    block = torch.from_numpy(np.linalg.qr(np.random.RandomState(seed).standard_normal((other - 1, side - 1)))[0].T.copy())
    u[0, 0], u[1:, 1:] = 1.0, block * (weak / (side - 1) ** 0.5)
    return u.float()


@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("iterations", range(1, 7))
def test_weak_directions_keep_22_bits(dev, iterations, turned):  # noqa: F811
    """Longer sides than 32: X is held in 22 bits at every iteration.  What an iteration adds to a block of singular values s of 1e-3 at
    most by products is b s^2 = 4.8e-6 of it, 2^-11 of which counts for each of the three roundings to fp16 in it.  The rest of the block
    is a X: two halves of 11 bits leave 2^-22 of an element, and FP32's steps to it (the product by 1/1024, the low half's, their sum, by
    a, and the sum with the product) 5 U.  The start is rounded to FP32 and to the halves, the result once."""
    for side, other in ((40, 90), (64, 64), (130, 300)):
        g = strong_and_weak(side, other, 1e-3 * (side - 1) ** 0.5 / A ** iterations)
        g = g.T.contiguous() if turned else g
        say("muon", tuple(g.shape), iterations)
        got, want = iterated(dev, g, iterations), orthogonal64(g.double(), iterations)
        bound = iterations * (2.0 ** -22 + 5 * U + 3 * 2.0 ** -11 * 4.8e-6) + 2.0 ** -22 + 2 * U
        assert off(got[1:, 1:], want[1:, 1:]) <= bound, (side, other, off(got[1:, 1:], want[1:, 1:]), bound)
        assert (got[0, 1:] == 0).all() and (got[1:, 0] == 0).all()


@pytest.mark.parametrize("iterations", range(1, 11))
@pytest.mark.parametrize("kind", KINDS + ["rank40"])
def test_long_sides(dev, kind, iterations):  # noqa: F811
    """Longer sides than 32, updates of any rank.  Products of operands in fp16 leave X of singular values of 1 off by 1.2e-3 of itself in the mean and
    by 5.3e-3 at most (off_by in test_matrix_ops_gpu has the sum), and a later iteration multiplies that by 1.3 in the mean.  Means hold
    where roundings are independent: not where rows are the same or one multiple of each other.  Directions that the update does not have
    get 2^-22 of it from X's two halves at most, times a at each iteration."""
    each = 5.3e-3 if kind in ("rank1", "repeated") else 1.2e-3
    bound = each * sum(1.3 ** (2 * i) for i in range(iterations)) ** 0.5 + 2.0 ** -22 * A ** iterations
    for rows, cols in ((33, 33), (40, 90), (130, 64), (128, 512), (300, 200), (450, 700)):
        g = update(rows, cols, kind)
        say("muon", rows, cols, kind, iterations)
        want = orthogonal64(g.double().to(dev), iterations).cpu()
        got = off(iterated(dev, g, iterations), want)
        assert got <= bound, (rows, cols, got, bound)
