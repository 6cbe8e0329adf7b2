"""Oracle of the NF4 projection with the adapters of many requests, float64, one adapter at a time.

Each function returns its results and, where asked, the sums of absolute values that bound the
rounding errors of a float32 evaluation.  Pinned by ``tests/test_oracle_adapters.py``.
"""

from __future__ import annotations

import numpy as np


def project(x, ids, W, A, B, scale):
    """``y = x W^T`` plus, for tokens with ``0 <= ids < n``, ``s[a] (x A[a]^T) B[a]^T``.

    x [T, K], ids [T], W [N, K], A [n, r, K], B [n, N, r], scale [n].  Returns (y [T, N], p [T, r]); p is
    zero for tokens without an adapter.
    """
    y = x @ W.T
    p = np.zeros((x.shape[0], A.shape[1]))
    for a in range(A.shape[0]):
        rows = np.flatnonzero(np.asarray(ids) == a)
        if rows.size:
            p[rows] = scale[a] * (x[rows] @ A[a].T)
            y[rows] += p[rows] @ B[a].T
    return y, p


def project_backward(x, ids, dY, W, A, B, scale):
    """Gradients of ``sum(dY * y)``: (dx [T, K], q [T, r], dA [n, r, K], dB [n, N, r])."""
    dx = dY @ W
    q = np.zeros((x.shape[0], A.shape[1]))
    dA, dB = np.zeros(A.shape), np.zeros(B.shape)
    for a in range(A.shape[0]):
        rows = np.flatnonzero(np.asarray(ids) == a)
        if rows.size:
            p = scale[a] * (x[rows] @ A[a].T)
            q[rows] = scale[a] * (dY[rows] @ B[a])
            dx[rows] += q[rows] @ A[a]
            dA[a] = q[rows].T @ x[rows]
            dB[a] = dY[rows].T @ p
    return dx, q, dA, dB


def group(ids, n):
    """(rows of each group, padded starts): the tokens sorted by adapter (stable), each adapter's rows at a
    multiple of 32, the tokens without an adapter (ids outside [0, n)) last."""
    ids = np.asarray(ids)
    members = [np.flatnonzero(ids == a) for a in range(n)]
    members.append(np.flatnonzero((ids < 0) | (ids >= n)))
    starts, at = [], 0
    for a in range(n):
        starts.append(at)
        at += -(-members[a].size // 32) * 32
    starts += [at, at + members[n].size]
    return members, np.array(starts)
