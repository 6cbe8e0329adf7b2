"""The balance gradient ahead of its forward is refused (GPU)."""

import pytest
import torch

from grouped_nf4_expert_b200 import build, e4b
from test_gpu_balance import make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="session", autouse=True)
def _built():
    build.build()
    e4b.lib()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def test_the_gradient_ahead_of_the_forward_is_refused():
    logits, ids, seq, mask = make(30, 8, 2, 3, 1.0)
    b, d = e4b.RouterBalance(8, 2, 30, 3), torch.full((30, 8), 7.0, device="cuda")
    n0 = e4b.e4b_launch_count()
    for accumulate in (False, True):
        with pytest.raises(ValueError, match="call e4b_balance_fwd first"):
            b.e4b_balance_bwd(logits, d, seq, mask, accumulate=accumulate)
    with pytest.raises(TypeError, match="logits: dtype"):  # a forward that was refused is none
        b.e4b_balance_fwd(logits.double(), ids, seq, mask)
    with pytest.raises(ValueError, match="call e4b_balance_fwd first"):
        b.e4b_balance_bwd(logits, d, seq, mask)
    assert e4b.e4b_launch_count() == n0 and bool((d == 7.0).all())
    b.e4b_balance_fwd(logits, ids, seq, mask, 0.7, 0.3)
    b.e4b_balance_bwd(logits, d, seq, mask, 0.7, 0.3)
    assert torch.equal(d, run(8, 2, logits, ids, seq, mask, 0.7, 0.3)[1])
