"""The waits inside a launch of the operators end at their limit (GPU).

A block's wait is for a counter in the workspace that earlier blocks of the launch raise.  A counter far below zero
cannot be raised far enough, so the wait ends at its limit (2 s) and the call reports it; after the workspace is
initialised again the object works as before.
"""

import pytest
import torch

from grouped_nf4_expert_b200 import build, e4b
from test_gpu_adapters import Case, serve
from test_gpu_balance import make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="session", autouse=True)
def _built():
    build.build()
    e4b.lib()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def header(ws):
    """The workspace's error code, site and block, and its two counters."""
    return ws[:20].view(torch.int32)


def runs_out(obj, call, site):
    header(obj.ws)[3] = -(1 << 20)
    call()
    assert obj.check_device_error() == e4b.E4B_ERR_DEVICE_TIMEOUT
    assert header(obj.ws)[:2].tolist() == [e4b.E4B_ERR_DEVICE_TIMEOUT, site]
    e4b.e4b_workspace_init(obj.ws)
    assert obj.check_device_error() == e4b.E4B_OK
    call()
    assert obj.check_device_error() == e4b.E4B_OK
    assert header(obj.ws).tolist() == [0] * 5


@pytest.mark.parametrize("T,site", [(5, 640), (20, 641)])
def test_a_projection_that_waits_for_p(T, site):
    c = Case(T, 256, 136, 3, 16, "zipf", seed=500)
    want = serve(c).y.clone()
    pj, base, ad = e4b.Projection(c.dims, c.T, train=False), c.base(), c.adapters()
    runs_out(pj, lambda: pj.e4b_multi_lora_serve_fwd(c.ids, c.x, base, ad), site)
    assert torch.equal(pj.y, want)


def test_a_join_that_waits_for_its_records():
    logits, ids, seq, mask = make(3000, 64, 4, 3, 0.9, seed=501)
    want = run(64, 4, logits, ids, seq, mask, 0.7, 0.3)[0]
    b = e4b.RouterBalance(64, 4, 3000, 3)
    runs_out(b, lambda: b.e4b_balance_fwd(logits, ids, seq, mask, 0.7, 0.3), 700)
    assert torch.equal(b.loss, want.loss) and torch.equal(b.counts, want.counts)
