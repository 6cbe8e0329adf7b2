"""What the projection with adapters keeps between its two low-rank products (GPU).

p and q are held in 32 bits, at worst as two bf16 values: a cut of less than 2^-7 (the last place), and what it left
rounded by 2^-9 of that last place, 2^-16 together.  The
inputs make the ranks cancel in pairs (A's rows of a pair are equal but for one value, B's columns are opposite), and
for the adapter gradients the tokens too, while the frozen matrix is next to nothing; so an error of p stands out that
bf16's last place would hide otherwise.  Bounds as in ``test_gpu_adapters.py``, with 2^-16 in the place of bf16's 2^-8
where p or q is held:

    e_p       = 2^-16 |p*| + (K + 4) 2^-23 s |A| |x|
    |y - y*| <= (1 + u) (sum_j |B_j| e_p + (K + 2 r + 4) 2^-23 (|W| |x| + |B| |p|)) + u |y*|,  u = 2^-8

(2 r: a pair is two products and additions).  Tokens whose x and dY are zero add exact zeros to the adapter gradients,
so only the others count as additions there.
"""

import numpy as np
import pytest
import torch

from closeness import check
from grouped_nf4_expert_b200 import build, e4b
from oracle import adapters as oa
from test_gpu_adapters import F, U, Case, f64, serve, train

pytestmark = pytest.mark.gpu

PAIR = 2.0 ** -16


@pytest.fixture(scope="session", autouse=True)
def _built():
    build.build()
    e4b.lib()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def cancelling(T, K, N, n, r, seed, live=None):
    """A case whose ranks, and (live: that many tokens, the rest zero) whose tokens, cancel in pairs."""
    c = Case(T, K, N, n, r, "one" if n == 1 else "runs", seed=seed)
    c.absmax *= 2.0 ** -24
    c.A[:, 1::2] = c.A[:, 0::2]
    c.A[:, 1::2, 0] *= -1.0
    c.B[:, :, 1::2] = -c.B[:, :, 0::2]
    if live is not None:
        c.x[live:], c.dY[live:] = 0, 0
        half = live // 2
        c.x[half:live] = c.x[:half]
        c.x[half:live, 1] *= -1.0
        c.dY[half:live] = -c.dY[:half]
        c.dY[half:live, 1] *= -1.0
    return c


def reference(c):
    """(value, bound) of y, and of the gradients."""
    m = c.ref()
    ab = {k: (np.abs(v) if k != "ids" else v) for k, v in m.items()}
    dY = f64(c.dY)
    y, p = oa.project(**m)
    y_abs, p_abs = oa.project(**ab)
    dx, q, dA, dB = oa.project_backward(m["x"], m["ids"], dY, m["W"], m["A"], m["B"], m["scale"])
    dx_abs, q_abs, dA_abs, dB_abs = oa.project_backward(ab["x"], m["ids"], np.abs(dY), ab["W"], ab["A"], ab["B"],
                                                        ab["scale"])
    e_p = PAIR * np.abs(p) + (c.K + 4) * F * p_abs
    e_q = PAIR * np.abs(q) + (c.N + 4) * F * q_abs
    t = int((np.abs(m["x"]).sum(1) + np.abs(dY).sum(1) > 0).sum())
    ey, edx, edA, edB = np.zeros_like(y), np.zeros_like(dx), np.zeros_like(dA), np.zeros_like(dB)
    for a in range(c.n):
        rows = np.flatnonzero(m["ids"] == a)
        ey[rows] = e_p[rows] @ ab["B"][a].T
        edx[rows] = e_q[rows] @ ab["A"][a]
        edA[a] = e_q[rows].T @ ab["x"][rows]
        edB[a] = np.abs(dY[rows]).T @ e_p[rows]
    out = {}
    for name, v, e, m_, v_abs in (("y", y, ey, c.K + 2 * c.r, y_abs), ("dx", dx, edx, c.N + 2 * c.r, dx_abs),
                                  ("dA", dA, edA, 2 * t, dA_abs), ("dB", dB, edB, 2 * t, dB_abs)):
        out[name] = (v, (1 + U) * (e + (m_ + 4) * F * v_abs) + U * np.abs(v))
    return out


# every form of the serving call: up to 16 tokens, up to 256, and above
@pytest.mark.parametrize("shape", [(1, 64, 264, 1, 8), (5, 64, 136, 3, 24), (12, 128, 264, 4, 64), (16, 64, 72, 2, 40),
                                   (20, 64, 136, 3, 8), (100, 128, 264, 5, 40), (256, 64, 520, 7, 64),
                                   (300, 64, 264, 5, 24), (700, 128, 136, 3, 64), (1111, 64, 4096, 8, 16)],
                         ids=lambda s: "-".join(map(str, s)))
def test_serving(shape):
    c = cancelling(*shape, seed=200)
    check(serve(c).y, *reference(c)["y"], "y")


# few rows and many (with the reduction split over clusters), ranks padded and not
@pytest.mark.parametrize("shape", [(24, 64, 64, 1, 8), (24, 64, 72, 1, 24), (60, 64, 128, 1, 64), (40, 128, 64, 1, 40),
                                   (300, 64, 136, 1, 16), (2500, 64, 136, 1, 32), (2500, 64, 72, 1, 64)],
                         ids=lambda s: "-".join(map(str, s)))
def test_training(shape):
    c = cancelling(*shape, seed=201, live=16)
    pj, want = train(c), reference(c)
    for name in ("y", "dx", "dA", "dB"):
        check(getattr(pj, name), *want[name], name)


def test_the_buffers_hold_a_value_and_what_its_cut_left():
    c = Case(100, 192, 136, 3, 24, "zipf", seed=202)
    pj = train(c)
    order, m = pj.order.cpu().numpy(), c.ref()
    _, p = oa.project(**m)
    _, q, _, _ = oa.project_backward(m["x"], m["ids"], f64(c.dY), m["W"], m["A"], m["B"], m["scale"])
    ab = {k: np.abs(v) if k != "ids" else v for k, v in m.items()}
    _, p_abs = oa.project(**ab)
    _, q_abs, _, _ = oa.project_backward(ab["x"], m["ids"], np.abs(f64(c.dY)), ab["W"], ab["A"], ab["B"], ab["scale"])
    rows = np.flatnonzero((order < c.T) & (np.arange(order.size) < int(pj.offsets[c.n])))
    for pairs, high, want, want_abs, m_ in ((pj._p_pairs, pj.p, p, p_abs, c.K), (pj._q_pairs, pj.q, q, q_abs, c.N)):
        two = f64(pairs)[rows]
        e = (m_ + 4) * F * want_abs[order[rows]]
        w = want[order[rows]]
        check(two.sum(1), w, PAIR * np.abs(w) + (1 + U) * e, "pair")
        check(f64(high)[rows], w, 2 * U * np.abs(w) + (1 + U) * e, "cut value")


@pytest.mark.parametrize("T,r", [(90, 8), (300, 40), (2500, 24)])
def test_what_the_buffers_held_does_not_matter(T, r):
    c = Case(T, 64, 136, 4, r, "zipf", seed=203)
    want, pj = train(c), e4b.Projection(c.dims, T)
    for t in (pj._p_pairs, pj._q_pairs, pj.ws[256:].view(torch.bfloat16)):
        t.fill_(float("nan"))
    pj.e4b_adapter_group(c.ids)
    pj.e4b_multi_lora_fwd(c.x, c.base(), c.adapters())
    pj.e4b_multi_lora_dgrad(c.dY, c.base(), c.adapters())
    pj.e4b_multi_lora_wgrad(c.x, c.dY)
    for name in ("y", "dx", "dA", "dB"):
        assert torch.equal(getattr(pj, name), getattr(want, name)), name
