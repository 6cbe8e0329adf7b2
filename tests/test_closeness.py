"""The comparison that the GPU tests use must not let anything pass (CPU)."""

import numpy as np
import pytest
import torch

from closeness import check


def test_values_within_the_bound_pass():
    check(torch.tensor([1.0, 2.0]), np.array([1.0, 2.5]), np.array([0.0, 0.5]), "v")
    check(np.zeros((2, 0)), np.zeros((2, 0)), 0.0, "empty")


@pytest.mark.parametrize("got", [[1.0, float("nan")], [float("nan")] * 2, [1.0, float("inf")], [1.0, 2.1]])
def test_nan_and_far_values_fail(got):
    with pytest.raises(AssertionError, match="v: "):
        check(torch.tensor(got), np.array([1.0, 2.0]), np.array([0.05, 0.05]), "v")


def test_an_undefined_bound_fails():
    with pytest.raises(AssertionError):
        check(np.array([1.0]), np.array([1.0]), np.array([float("nan")]), "v")


def test_another_shape_fails():
    with pytest.raises(AssertionError, match="shape"):
        check(np.zeros(3), np.zeros((3, 1)), 1.0, "v")
