"""Pins of the adapter and balance oracles: dense formulas, closed values, and gradients by differences (CPU)."""

import numpy as np
import pytest

from oracle import adapters as oa
from oracle import balance as ob


def _case(seed, T=7, K=6, N=5, n=3, r=2):
    g = np.random.default_rng(seed)
    ids = np.array([0, 2, -1, 2, 0, 5, 2])[:T]
    return (g.standard_normal((T, K)), ids, g.standard_normal((N, K)), g.standard_normal((n, r, K)),
            g.standard_normal((n, N, r)), g.uniform(0.5, 2, n))


def test_projection_is_the_per_token_matrix():
    x, ids, W, A, B, s = _case(1)
    y, _ = oa.project(x, ids, W, A, B, s)
    for t, a in enumerate(ids):
        M = W + (s[a] * B[a] @ A[a] if 0 <= a < 3 else 0.0)
        np.testing.assert_allclose(y[t], M @ x[t], rtol=1e-12, atol=1e-12)


def _numeric(f, v, eps=1e-6):
    g = np.zeros(v.shape)
    for i in np.ndindex(v.shape):
        o = v[i]
        v[i] = o + eps
        hi = f()
        v[i] = o - eps
        lo = f()
        v[i] = o
        g[i] = (hi - lo) / (2 * eps)
    return g


def test_projection_gradients_by_differences():
    x, ids, W, A, B, s = _case(2)
    dY = np.random.default_rng(3).standard_normal((7, 5))
    dx, q, dA, dB = oa.project_backward(x, ids, dY, W, A, B, s)
    f = lambda: float((dY * oa.project(x, ids, W, A, B, s)[0]).sum())  # noqa: E731
    for got, v in ((dx, x), (dA, A), (dB, B)):
        np.testing.assert_allclose(got, _numeric(f, v), rtol=1e-6, atol=1e-7)
    assert np.all(dA[1] == 0) and np.all(dB[1] == 0)  # an adapter with no tokens


def test_group_is_stable_and_padded():
    members, starts = oa.group([1, 0, 1, -1, 9, 1], 3)
    assert [m.tolist() for m in members] == [[1], [0, 2, 5], [], [3, 4]]
    assert starts.tolist() == [0, 32, 64, 64, 66]


def test_balance_closed_values():
    # uniform logits and even counts: balance is 1, z is log(E)^2, the gradient of the balance is 0
    T, E, k = 8, 4, 2
    logits = np.zeros((T, E))
    ids = np.array([[t % 4, (t + 1) % 4] for t in range(T)])
    loss, bal, z, counts, psum, n_s, lse, grad = ob.balance_loss(logits, ids, k, [0, T], np.ones(T), 0.5, 0.25)
    assert abs(bal - 1.0) < 1e-12 and abs(z - np.log(4) ** 2) < 1e-12 and abs(loss - 0.5 - 0.25 * z) < 1e-12
    assert counts.tolist() == [[4, 4, 4, 4]] and n_s.tolist() == [8]
    np.testing.assert_allclose(grad, 2 * 0.25 / 8 * np.log(4) / 4, rtol=1e-12)
    # everything on one expert: balance is E
    far = np.full((T, E), -200.0)
    far[:, 2] = 0.0
    assert abs(ob.balance_loss(far, np.full((T, 1), 2), 1, [0, T], np.ones(T), 1.0, 0.0)[1] - E) < 1e-9


@pytest.mark.parametrize("offsets", [[0, 9], [0, 4, 4, 9], [1, 3, 8]])
def test_balance_gradient_by_differences(offsets):
    g = np.random.default_rng(5)
    logits = g.standard_normal((9, 5))
    logits[3, 1] = -np.inf
    ids = np.stack([g.permutation(5)[:2] for _ in range(9)])
    mask = np.array([1, 1, 0, 1, 1, 1, 0, 1, 1])
    grad = ob.balance_loss(logits, ids, 2, offsets, mask, 0.7, 0.3)[-1]
    f = lambda: ob.balance_loss(logits, ids, 2, offsets, mask, 0.7, 0.3)[0]  # noqa: E731
    finite = np.isfinite(logits)
    num = np.zeros((9, 5))
    for i in np.argwhere(finite):
        i, o = tuple(i), logits[tuple(i)]
        logits[i] = o + 1e-6
        hi = f()
        logits[i] = o - 1e-6
        lo = f()
        logits[i] = o
        num[i] = (hi - lo) / 2e-6
    np.testing.assert_allclose(grad, num, rtol=1e-6, atol=1e-9)


def test_balance_rows_without_probabilities():
    logits = np.full((3, 4), -np.inf)
    logits[1] = [0.0, 1.0, -np.inf, 2.0]
    ids = np.array([[0], [3], [9]])
    loss, bal, z, counts, psum, n_s, lse, grad = ob.balance_loss(logits, ids, 1, [0, 3], np.ones(3), 1.0, 1.0)
    assert np.isfinite([loss, bal, z]).all() and np.isfinite(grad).all()
    assert counts.tolist() == [[1, 0, 0, 1]] and lse[0] == -np.inf and np.all(grad[0] == 0)
