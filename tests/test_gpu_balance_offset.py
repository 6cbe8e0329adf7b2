"""The balance loss and its gradient for logits far from zero (GPU).

A common offset of a token's logits changes its probabilities by nothing, so the error of the balance term must not
grow with it.  With H = 2^-24 and m the row's maximum, a probability exp(l - m) / sum is off by at most
r = (2.3 |l - m| + E + 16) H of itself (the head of ``test_gpu_balance.py``), and with f the experts' shares and
b = c_b / (S' n_s)

    |d - d*| <= p b (f_j + sum_e p f_e) (2 r + (E + 16) H)

without a term in |lse|.  Only the z term's own value 2 c_z lse p / n is off by H |lse| (lse is one float32).
"""

import numpy as np
import pytest
import torch

from closeness import check
from grouped_nf4_expert_b200 import build, e4b
from oracle import balance as ob
from test_gpu_balance import H, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="session", autouse=True)
def _built():
    build.build()
    e4b.lib()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def gradient(E, k, logits, ids, seq, mask, cb, cz):
    """(gradient, bound, probabilities) in 64 bits."""
    l64, off = logits.double().cpu().numpy(), seq.cpu().tolist()
    _, _, _, counts, _, n_s, lse, grad = ob.balance_loss(l64, ids.cpu().numpy(), k, off, mask.cpu().numpy(), cb, cz)
    T, S = l64.shape[0], len(off) - 1
    top = l64.max(1, keepdims=True)
    ex = np.exp(l64 - top)
    p = ex / ex.sum(1, keepdims=True) * mask.cpu().numpy()[:, None]
    f = E * counts / (k * np.maximum(n_s, 1)[:, None])
    s = np.searchsorted(np.array(off[1:]), np.arange(T), side="right").clip(max=S - 1)
    b = cb / (max(1, (n_s > 0).sum()) * np.maximum(n_s, 1))[s][:, None]
    r = (2.3 * (top - l64) + E + 16) * H
    r_row = (p * r).sum(1, keepdims=True) + r
    bound = p * b * (f[s] + (p * f[s]).sum(1, keepdims=True)) * (2 * r_row + (E + 16) * H)
    bound += p * 2 * cz / max(1, n_s.sum()) * (np.abs(lse)[:, None] * (2 * r + (E + 20) * H) + r)
    return grad, 1.01 * bound + 1e-37, p


@pytest.mark.parametrize("offset", [0.0, 50.0, -1000.0, 1000.0, 3e4])
@pytest.mark.parametrize("shape", [(40, 16, 2, 3, 0.9), (33, 8, 2, 1, 1.0), (60, 65, 4, 2, 1.0), (50, 128, 8, 4, 0.8),
                                   (30, 512, 8, 2, 1.0), (20, 1021, 8, 1, 1.0)], ids=lambda s: "-".join(map(str, s)))
def test_offset_logits(shape, offset):
    T, E, k, S, keep = shape
    logits, ids, seq, mask = make(T, E, k, S, keep, seed=300)
    logits += offset + torch.linspace(-3, 3, T, device="cuda")[:, None]  # tokens of different offsets
    for cb, cz in ((0.7, 0.0), (0.7, 0.3)):
        b, d = run(E, k, logits, ids, seq, mask, cb, cz)
        want, bound, p = gradient(E, k, logits, ids, seq, mask, cb, cz)
        check(d, want, bound, "gradient")
        if cz == 0.0:  # a row of the balance term's gradient sums to 0
            check(d.double().sum(1), np.zeros(T), bound.sum(1), "row sums")
