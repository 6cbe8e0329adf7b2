"""The balance loss where its blocks and warps go round more than once (GPU; the reference is pinned on the CPU).

Batches above what one wave of blocks holds at a time: a block's range takes several rounds, a warp's run of the
gradient several steps, and the join reads more records of a sequence than it has lanes for.  With the sums' depth D
(the additions that a value passes through, not the tokens) the bounds of ``test_gpu_balance.py`` are, H = 2^-24:

    |P - P*| <= (r + D H) P*,  |balance - balance*| <= (r + (D + E + S + 8) H) balance*,  r = (2.3 |l - m| + E + 16) H

D: a lane's rounds (at most T / 2368 + 1: a wave of 296 blocks holds 2368 tokens or more), 5 shuffles, 8 warps, a
quarter of 592 records, 2 shuffles, 8 warps.
"""

import numpy as np
import pytest
import torch

from closeness import check
from grouped_nf4_expert_b200 import build, e4b
from oracle import balance as ob
from test_gpu_balance import H, make, run

CB, CZ = 0.7, 0.3


def dense(logits, ids, k, offsets, mask, cb, cz):
    """``oracle.balance.balance_loss`` over whole arrays (finite logits, ids in range, every token in a sequence)."""
    T, E = logits.shape
    S = len(offsets) - 1
    mask = np.asarray(mask).astype(bool)
    seq = np.searchsorted(np.asarray(offsets[1:]), np.arange(T), side="right")
    top = logits.max(1, keepdims=True)
    ex = np.exp(logits - top)
    tot = ex.sum(1, keepdims=True)
    p, lse = ex / tot * mask[:, None], np.where(mask, (top + np.log(tot))[:, 0], 0.0)
    n_s = np.bincount(seq[mask], minlength=S)
    counts = np.bincount((seq[mask, None] * E + ids[mask]).ravel(), minlength=S * E).reshape(S, E)
    psum = np.zeros((S, E))
    for s in range(S):
        psum[s] = p[offsets[s]:offsets[s + 1]].sum(0)
    n_seq, n = max(1, (n_s > 0).sum()), max(1, n_s.sum())
    safe = np.maximum(n_s, 1)[:, None]
    f = E * counts / (k * safe)
    balance, z = float((f * psum / safe).sum() / n_seq), float((lse ** 2).sum() / n)
    w = (cb / (n_seq * safe))[seq]
    scale = p * (w * (f[seq] + (p * f[seq]).sum(1, keepdims=True)) + 2 * cz / n * np.abs(lse)[:, None])
    grad = p * (w * (f[seq] - (p * f[seq]).sum(1, keepdims=True)) + 2 * cz / n * lse[:, None])
    return (cb * balance + cz * z, balance, z, counts, psum, n_s, lse, grad), (top - logits), scale, p * 2 * cz / n


def test_the_reference_is_the_oracle():
    logits, ids, seq, mask = [t.cpu() for t in _make_cpu(60, 12, 3, 5, 0.8)]
    args = (logits.double().numpy(), ids.numpy().astype(np.int64), 3, seq.tolist(), mask.numpy(), CB, CZ)
    got, want = dense(*args)[0], ob.balance_loss(*args)
    for g, w in zip(got, want):
        np.testing.assert_allclose(g, w, rtol=1e-12, atol=1e-15)


def _make_cpu(T, E, k, S, keep):
    g = torch.Generator().manual_seed(9)
    logits = torch.randn((T, E), generator=g) * 2
    cuts = torch.sort(torch.randint(0, T + 1, (S - 1,), generator=g)).values
    seq = torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.tensor([T])])
    return logits, torch.topk(logits, k, dim=1).indices, seq, (torch.rand(T, generator=g) < keep).to(torch.uint8)


@pytest.fixture(scope="module")
def built():
    build.build()
    e4b.lib()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


# (T, E, k, S, kept share): several rounds a block with ragged sequences and a mask; one sequence of more records than
# a block's lanes; two blocks an SM, rows off the vector width and on it; more slots than a lane holds and over 2048
# ids in a range; many short sequences, several in every range
@pytest.mark.gpu
@pytest.mark.parametrize("case", [
    (30011, 256, 8, 37, 0.9), (40000, 64, 6, 1, 1.0), (131072, 64, 6, 64, 0.97), (5000, 1021, 8, 3, 0.9),
    (9001, 1024, 32, 1, 0.95), (200003, 8, 8, 5, 0.9), (200003, 3, 3, 2, 1.0), (170000, 16, 5, 1, 1.0),
    (50000, 128, 8, 900, 0.9), (4096, 128, 8, 512, 1.0), (60001, 60, 4, 11, 0.5),
], ids=lambda c: "-".join(map(str, c)))
def test_large_batches(built, case):
    T, E, k, S, keep = case
    logits, ids, seq, mask = make(T, E, k, S, keep, seed=400)
    b, d = run(E, k, logits, ids, seq, mask, CB, CZ)
    (loss, bal, z, counts, psum, n_s, lse, grad), spread, scale, zp = dense(
        logits.double().cpu().numpy(), ids.cpu().numpy().astype(np.int64), k, seq.cpu().tolist(), mask.cpu().numpy(),
        CB, CZ)
    D = T / 2368 + 1 + 5 + 8 + 148 + 2 + 8
    r_el = (2.3 * spread + E + 16) * H
    r = r_el.max()
    assert np.array_equal(b.counts.cpu().numpy(), counts) and b.tokens.cpu().tolist() == n_s.tolist()
    assert b._tokens.cpu().tolist()[S:] == [int(n_s.sum()), int((n_s > 0).sum())]
    check(b.prob_sum, psum, (r + D * H) * psum + 1e-30, "probability sums")
    lmax = np.abs(lse).max()
    check(b.lse, lse, lmax * H * 2 + 2 * r, "lse")
    t_b = (r + (D + E + S + 8) * H) * bal
    t_z = 2 * lmax * (r + lmax * H + 4 * H) + (D + S + 8) * H * z
    check(b.loss, np.array([loss, bal, z]),
          np.array([CB * t_b + CZ * t_z + 4 * H * (CB * bal + CZ * z), t_b, t_z]) + 1e-30, "loss")
    bound = scale * (2 * r_el + (np.abs(lse)[:, None] + E + 16) * H) + zp * (np.abs(lse)[:, None] * H + r_el)
    check(d, grad, 1.01 * bound + 1e-37, "gradient")
    start = torch.linspace(-1e-3, 1e-3, T * E, device="cuda").view(T, E)
    total = start.clone()
    b.e4b_balance_bwd(logits, total, seq, mask, balance_coef=CB, z_coef=CZ, accumulate=True)
    live = mask.bool()
    assert torch.equal(total[live], (start + d)[live]) and torch.equal(total[~live], start[~live])
