"""Infinities in the projection with adapters come out as the formulas have them (GPU).

An infinity in a factor, a token or a gradient makes an infinity, or NaN where two of them meet or one meets a zero, of
exactly the elements that the formulas in 64 bits make so, and leaves the bits of all others as they were.  (The rows
that pad an adapter's to a multiple of 32 take no part: an infinite factor times their zeros is no NaN of the gradients.)
"""

import numpy as np
import pytest
import torch

from grouped_nf4_expert_b200 import build, e4b
from oracle import adapters as oa
from test_gpu_adapters import Case, f64, serve, train

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="session", autouse=True)
def _built():
    build.build()
    e4b.lib()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def same(got, good, want, what):
    got, good = f64(got), f64(good)
    finite = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), "%s: %d NaN, expected %d" % (
        what, np.isnan(got).sum(), np.isnan(want).sum())
    at = np.isinf(want)
    assert np.array_equal(got[at], want[at]), what
    assert np.array_equal(got[finite], good[finite]), what


def put(c, where):
    """One infinity in `where`, in adapter 0 or its first token ("+": beside factors of one sign, so that the sums that
    it enters are infinite and not NaN)."""
    t = int(np.flatnonzero(c.ids.cpu().numpy() == 0)[0])
    if where[0] == "A":
        c.A[0, 3, 5] = INF
    elif where[0] == "B":
        c.B[0, 2, 3] = -INF
    elif where[0] == "x":
        c.x[t, 5] = INF
    elif where[:2] == "dY":
        c.dY[t, 2] = -INF


def case(T, r, where):
    c = Case(T, 64, 72, 2, r, "runs", seed=600)
    c.ids[0] = 0
    c.nf4.fill_(0xff)  # weights of one sign, none zero: an infinite token has infinite base products
    if where.endswith("+"):
        c.A.abs_()
        c.B.abs_()
    if where in ("A+", "B+"):  # p (A) and dY, or q (B) and x, of one sign as well
        c.x.abs_()
        c.dY.abs_()
    return c


def results(c):
    """What the formulas in 64 bits give."""
    with np.errstate(invalid="ignore"):
        m = c.ref()
        y, _ = oa.project(**m)
        dx, _, dA, dB = oa.project_backward(m["x"], m["ids"], f64(c.dY), m["W"], m["A"], m["B"], m["scale"])
    return y, dx, dA, dB


@pytest.mark.parametrize("where", ["A", "B", "x", "x+"])
@pytest.mark.parametrize("T,r", [(1, 8), (7, 24), (16, 64), (20, 8), (90, 40), (256, 64), (300, 24), (700, 64)])
def test_serving(T, r, where):
    good, c = serve(case(T, r, where)).y.clone(), case(T, r, where)
    put(c, where)
    same(serve(c).y, good, results(c)[0], "y")


@pytest.mark.parametrize("where", ["x", "x+", "dY", "dY+", "A", "A+", "B", "B+"])
@pytest.mark.parametrize("T,r", [(40, 8), (300, 24), (700, 64)])
def test_training(T, r, where):
    good, c = train(case(T, r, where)), case(T, r, where)
    put(c, where)
    pj = train(c)
    for name, want in zip(("y", "dx", "dA", "dB"), results(c)):
        same(getattr(pj, name), getattr(good, name), want, name)
