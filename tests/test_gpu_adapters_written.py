"""The projection's oracle tests once more, with a comparison that NaN cannot pass (GPU).

The outputs are filled with NaN ahead of the calls, so an element that a call leaves unwritten, and a NaN that it
computes, has to fail: ``abs(nan - want) > tol`` is false, ``not abs(nan - want) <= tol`` is true.
"""

import pytest
import torch

import closeness
import test_gpu_adapters as base
from grouped_nf4_expert_b200 import build, e4b

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="session", autouse=True)
def _built():
    build.build()
    e4b.lib()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.fixture(autouse=True)
def _strict(monkeypatch):
    monkeypatch.setattr(base, "check", closeness.check)


def _id(s):
    return "-".join(map(str, s))


@pytest.mark.parametrize("shape", base.SERVE, ids=_id)
def test_serve(shape):
    base.test_serve(shape)


@pytest.mark.parametrize("shape", base.test_serve_wide.pytestmark[0].args[1], ids=_id)
def test_serve_wide(shape):
    base.test_serve_wide(shape)


@pytest.mark.parametrize("shape", base.TRAIN, ids=_id)
def test_train(shape):
    base.test_train(shape)


@pytest.mark.parametrize("name", ["test_more_padding_than_the_unit_was_chosen_for", "test_offsets_past_32_bits",
                                  "test_gradient_offsets_past_32_bits", "test_as_used_with_the_expert_block"])
def test_others(name):
    getattr(base, name)()


def test_an_unwritten_output_fails():
    # the comparison in place is the strict one: a call that writes nothing does not pass
    c = base.Case(3, 64, 72, 2, 8)
    y, tol, _ = base.bounds(c)
    pj = e4b.Projection(c.dims, c.T, train=False)
    pj.y.fill_(float("nan"))
    with pytest.raises(AssertionError, match="216 NaN"):
        base.check(pj.y, y, tol, "y")
