"""Batches of up to 256 tokens take p in a launch of its own where the GPU needs less time that way (GPU).

The sizes are ones where a call takes less than the host needs for two launches; what the host needs is not part of
the choice (replayed from a graph it is nothing).
"""

import pytest
import torch

from closeness import check
from grouped_nf4_expert_b200 import build, e4b
from test_gpu_adapters import Case, bounds

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="session", autouse=True)
def _built():
    build.build()
    e4b.lib()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("shape", [(57, 4096, 4096, 32, 32), (17, 2048, 4096, 32, 32), (128, 4096, 4096, 32, 32),
                                   (256, 4096, 1024, 64, 64)], ids=lambda s: "-".join(map(str, s)))
def test_p_in_a_launch_of_its_own(shape):
    c = Case(*shape, "zipf", seed=700)
    pj, base, ad = e4b.Projection(c.dims, c.T, train=False), c.base(), c.adapters()
    e4b.e4b_profiler_read()
    e4b.e4b_profiler_enable(True)
    try:
        pj.e4b_multi_lora_serve_fwd(c.ids, c.x, base, ad)
    finally:
        e4b.e4b_profiler_enable(False)
    assert {k: n for k, (n, _) in e4b.e4b_profiler_read().items()} == {"adapter_low_rank": 1, "adapter_split": 1}
    y, tol, _ = bounds(c)
    check(pj.y, y, tol, "y")
    want, g = pj.y.clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            pj.e4b_multi_lora_serve_fwd(c.ids, c.x, base, ad)
    for _ in range(3):
        pj.y.fill_(float("nan"))
        g.replay()
        assert torch.equal(pj.y, want)
    assert pj.check_device_error() == e4b.E4B_OK
