"""Oracle of the router's balance loss, float64, one sequence at a time.

Pinned by ``tests/test_oracle_adapters.py`` (closed values and differences).
"""

from __future__ import annotations

import numpy as np


def _softmax(row):
    """(probabilities, logsumexp); a row of -inf alone has neither (zeros, -inf)."""
    m = row.max()
    if m == -np.inf:
        return np.zeros_like(row), -np.inf
    e = np.exp(row - m)
    return e / e.sum(), m + np.log(e.sum())


def balance_loss(logits, ids, k, offsets, mask, c_b, c_z):
    """loss, balance, z, counts [S, E], prob_sum [S, E], n_s [S], lse [T], d loss / d logits [T, E]."""
    T, E = logits.shape
    S = len(offsets) - 1
    counts, psum, n_s = np.zeros((S, E), dtype=np.int64), np.zeros((S, E)), np.zeros(S, dtype=np.int64)
    lse, grad, probs = np.zeros(T), np.zeros((T, E)), np.zeros((T, E))
    seqs = [[t for t in range(offsets[s], offsets[s + 1]) if mask[t]] for s in range(S)]
    n_seq, n = sum(1 for q in seqs if q), sum(len(q) for q in seqs)
    z = 0.0
    for s, q in enumerate(seqs):
        n_s[s] = len(q)
        for t in q:
            probs[t], lse[t] = _softmax(logits[t])
            psum[s] += probs[t]
            if lse[t] != -np.inf:
                z += lse[t] ** 2 / n
            for e in ids[t]:
                if 0 <= e < E:
                    counts[s, e] += 1
    balance = 0.0
    for s, q in enumerate(seqs):
        if not q:
            continue
        f = E * counts[s] / (k * len(q))
        balance += float(f @ psum[s]) / len(q) / n_seq
        for t in q:
            grad[t] = c_b / (n_seq * len(q)) * probs[t] * (f - probs[t] @ f)
            if lse[t] != -np.inf:
                grad[t] += 2.0 * c_z / n * lse[t] * probs[t]
    return c_b * balance + c_z * z, balance, z, counts, psum, n_s, lse, grad
