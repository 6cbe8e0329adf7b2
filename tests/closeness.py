"""Comparison of a computed array with an expected one, element by element."""

import numpy as np


def check(got, want, tol, what):
    """Every element of ``got`` within ``tol`` of ``want``: an element that is NaN, or not within it, fails."""
    got, want, tol = (np.asarray(v.detach().double().cpu().numpy() if hasattr(v, "detach") else v, dtype=np.float64)
                      for v in (got, want, tol))
    assert got.shape == want.shape, "%s: shape %s, expected %s" % (what, got.shape, want.shape)
    tol = np.broadcast_to(tol, want.shape)
    off = ~(np.abs(got - want) <= tol)
    if off.any():
        i = tuple(np.argwhere(off)[0])
        raise AssertionError("%s: %d of %d off (%d NaN), first at %s: %r, expected %r within %.3g" % (
            what, off.sum(), off.size, np.isnan(got).sum(), i, float(got[i]), float(want[i]), tol[i]))
