"""The router's balance loss against its float64 oracle (GPU).

Bounds.  f = 2^-24 is half a last place of float32.  A probability is 2^(log2(e) (l - m)) / sum: the subtraction is
off by f |l - m|, the product and its constant by 1.3 f |l - m|, the exponential by 4 f, the inverse and the product
with it by 2 f; the sum by the same on average (the average of |l - m| is at most log E) and by its additions, E f at
most.  So its relative error is at most r = (2.3 |l - m| + E + 16) f (with three experts 4 + 2 + 6.4 + 3 < 19, and more
experts add to the right side what they add to the left).  Sums over T tokens add T f.  The counts are whole numbers.
With b = c_b / (S' n_s), and lse off by f |lse| and r:

    |P - P*| <= (r + T f) P*,   |balance - balance*| <= (r + (T + E + S + 8) f) balance*
    |d - d*| <= p (b (f_j + sum_e p f_e) + 2 c_z |lse| / n) (2 r + (|lse| + E + 16) f)
"""

import numpy as np
import pytest
import torch

from grouped_nf4_expert_b200 import build, e4b
from oracle import balance as ob

pytestmark = pytest.mark.gpu

H = 2.0 ** -24


@pytest.fixture(scope="session", autouse=True)
def _built():
    build.build()
    e4b.lib()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def make(T, E, k, S, keep, seed=0):
    g = torch.Generator().manual_seed(77 + seed)
    logits = torch.randn((T, E), generator=g) * 2
    ids = torch.topk(logits, k, dim=1).indices.to(torch.int32).contiguous()
    cuts = torch.sort(torch.randint(0, T + 1, (S - 1,), generator=g)).values
    seq = torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.tensor([T])]).to(torch.int32)
    mask = (torch.rand(T, generator=g) < keep).to(torch.uint8)
    return [t.cuda() for t in (logits, ids, seq, mask)]


def run(E, k, logits, ids, seq, mask, cb=0.7, cz=0.3, dloss=None, d=None):
    T, S = logits.shape[0], (1 if seq is None else seq.numel() - 1)
    b = e4b.RouterBalance(E, k, T, S)
    for t in (b.counts, b._tokens, b.lse, b.loss, b.prob_sum, b.ws[256:]):
        t.fill_(85)
    b.e4b_balance_fwd(logits, ids, seq, mask, balance_coef=cb, z_coef=cz)
    out = torch.full((T, E), float("nan"), device="cuda") if d is None else d
    b.e4b_balance_bwd(logits, out, seq, mask, balance_coef=cb, z_coef=cz, dloss=dloss, accumulate=d is not None)
    assert b.check_device_error() == e4b.E4B_OK
    return b, out


def reference(E, k, logits, ids, seq, mask, cb=0.7, cz=0.3):
    T = logits.shape[0]
    return ob.balance_loss(logits.double().cpu().numpy(), ids.cpu().numpy(), k,
                           [0, T] if seq is None else seq.cpu().tolist(),
                           np.ones(T) if mask is None else mask.cpu().numpy(), cb, cz)


def compare(b, d, want, E, k, logits, cb=0.7, cz=0.3, up=1.0):
    loss, bal, z, counts, psum, n_s, lse, grad = want
    T, S = logits.shape[0], counts.shape[0]
    l64 = logits.double().cpu().numpy()
    fin = np.where(np.isfinite(l64), l64, 0.0)
    spread = (fin.max(1, keepdims=True) - fin).max() if T else 0.0
    r = (2.3 * spread + E + 16) * H
    assert np.array_equal(b.counts.cpu().numpy(), counts)
    assert b.tokens.cpu().tolist() == n_s.tolist()
    assert b._tokens.cpu().tolist()[S:] == [int(n_s.sum()), int((n_s > 0).sum())]
    np.testing.assert_array_less(np.abs(b.prob_sum.double().cpu().numpy() - psum), (r + T * H) * psum + 1e-30)
    got = b.loss.double().cpu().numpy()
    t_b = (r + (T + E + S + 8) * H) * bal
    lmax = np.abs(lse[np.isfinite(lse)]).max() if np.isfinite(lse).any() else 0.0
    t_z = 2 * lmax * (r + lmax * H + 4 * H) + (T + S + 8) * H * z
    assert abs(got[1] - bal) <= t_b + 1e-30 and abs(got[2] - z) <= t_z + 1e-30
    assert abs(got[0] - loss) <= abs(cb) * t_b + abs(cz) * t_z + 4 * H * (abs(cb) * bal + abs(cz) * z) + 1e-30
    # the gradient, with every term's absolute value
    n, n_seq = max(1, n_s.sum()), max(1, (n_s > 0).sum())
    g = d.double().cpu().numpy()
    bound = np.zeros_like(grad)
    starts = want_offsets
    for s in range(S):
        if n_s[s] == 0:
            continue
        f = E * counts[s] / (k * n_s[s])
        for t in range(starts[s], starts[s + 1]):
            if lse[t] == 0.0 and not grad[t].any():
                continue
            if lse[t] == -np.inf:
                continue
            p = np.exp(l64[t] - lse[t])
            bound[t] = p * (cb / (n_seq * n_s[s]) * (f + p @ f) + 2 * cz / n * abs(lse[t]))
            bound[t] *= 2 * r + (abs(lse[t]) + E + 16) * H
            bound[t] += p * 2 * cz / n * (abs(lse[t]) * H + r)  # the error of lse itself
    assert np.all(np.abs(g - up * grad) <= up * bound * 1.01 + 1e-37), np.abs(g - up * grad).max()


want_offsets = None


def both(E, k, logits, ids, seq, mask, **kw):
    global want_offsets
    want_offsets = [0, logits.shape[0]] if seq is None else seq.cpu().tolist()
    b, d = run(E, k, logits, ids, seq, mask, **kw)
    compare(b, d, reference(E, k, logits, ids, seq, mask), E, k, logits)
    return b, d


# (T, E, k, S, kept share): one token; expert counts off the vector width and around the lane groups
CASES = [(1, 1, 1, 1, 1.0), (1, 128, 8, 1, 1.0), (2, 3, 2, 2, 1.0), (5, 7, 3, 1, 0.5), (16, 128, 8, 1, 1.0),
         (33, 8, 2, 4, 0.9), (100, 60, 4, 3, 1.0), (255, 64, 6, 7, 0.8), (300, 65, 2, 300, 1.0), (257, 130, 8, 5, 0.9),
         (513, 256, 8, 9, 0.97), (700, 333, 5, 2, 1.0), (300, 512, 8, 3, 0.9), (200, 1024, 32, 4, 0.9),
         (150, 1021, 8, 2, 1.0), (3001, 16, 2, 11, 0.9), (4096, 128, 8, 1, 1.0), (50, 20, 3, 64, 1.0)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_balance(case):
    T, E, k, S, keep = case
    both(E, k, *make(T, E, k, S, keep))


def test_whole_batch_without_offsets_or_mask():
    logits, ids, seq, mask = make(130, 24, 2, 1, 1.0)
    both(24, 2, logits, ids, None, None)


def test_masked_everything_and_empty_sequences():
    logits, ids, seq, mask = make(40, 16, 2, 6, 1.0)
    b, d = both(16, 2, logits, ids, torch.tensor([0, 0, 10, 10, 10, 40, 40], dtype=torch.int32, device="cuda"), mask)
    b, d = run(16, 2, logits, ids, seq, torch.zeros_like(mask))
    assert b.loss.tolist() == [0.0, 0.0, 0.0] and not b.counts.any() and not d.any()


def test_tokens_outside_every_sequence_are_left_out():
    logits, ids, seq, mask = make(60, 16, 2, 3, 0.9)
    b, d = both(16, 2, logits, ids, torch.tensor([5, 20, 20, 48], dtype=torch.int32, device="cuda"), mask)
    assert not d[:5].any() and not d[48:].any()


def test_values_in_masked_places_are_not_read_into_the_result():
    logits, ids, seq, mask = make(70, 32, 4, 3, 0.7, seed=2)
    b0, d0 = run(32, 4, logits, ids, seq, mask)
    bad = logits.clone()
    off = mask == 0
    bad[off] = float("nan")
    bad[torch.nonzero(off)[0]] = float("inf")
    ids2 = ids.clone()
    ids2[off] = 10 ** 6
    b1, d1 = run(32, 4, bad, ids2, seq, mask)
    assert torch.equal(b0.loss, b1.loss) and torch.equal(b0.counts, b1.counts) and torch.equal(d0, d1)


def test_rows_of_minus_infinity():
    logits, ids, seq, mask = make(50, 12, 2, 2, 1.0, seed=3)
    logits[7] = float("-inf")
    logits[20, :11] = float("-inf")
    logits[30, 3] = torch.finfo(torch.float32).min
    both(12, 2, logits, ids, seq, mask)


def test_ids_outside_the_experts_are_not_counted():
    logits, ids, seq, mask = make(30, 9, 3, 2, 1.0, seed=4)
    ids[3, 0], ids[4, 1] = -1, 9
    both(9, 3, logits, ids, seq, mask)


def test_accumulates_and_scales():
    logits, ids, seq, mask = make(90, 40, 4, 3, 0.8, seed=5)
    _, d = run(40, 4, logits, ids, seq, mask)
    up = torch.tensor([-2.0], device="cuda")
    _, d2 = run(40, 4, logits, ids, seq, mask, dloss=up)
    assert torch.equal(d2, -2.0 * d)  # a power of two scales exactly
    start = torch.randn_like(d)
    keep = start.clone()
    _, d3 = run(40, 4, logits, ids, seq, mask, d=start)
    live = mask.bool()
    assert torch.equal(d3[live], (keep + d)[live]) and torch.equal(d3[~live], keep[~live])


def test_repeated_and_captured_calls_give_the_same_bits():
    logits, ids, seq, mask = make(2000, 128, 8, 5, 0.9, seed=6)
    b0, d0 = run(128, 8, logits, ids, seq, mask)
    b, d = e4b.RouterBalance(128, 8, 2000, 5), torch.empty_like(d0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.e4b_balance_fwd(logits, ids, seq, mask, 0.7, 0.3)
        b.e4b_balance_bwd(logits, d, seq, mask, 0.7, 0.3)
    for _ in range(3):
        g.replay()
        assert torch.equal(b.loss, b0.loss) and torch.equal(d, d0) and torch.equal(b.counts, b0.counts)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    b.e4b_balance_fwd(logits, ids, seq, mask, 0.7, 0.3, stream=st)
    st.synchronize()
    assert torch.equal(b.loss, b0.loss)


def test_no_tokens():
    b = e4b.RouterBalance(8, 2, 0, 3)
    for t in (b.counts, b._tokens, b.prob_sum, b.loss):
        t.fill_(9)
    n0 = e4b.e4b_launch_count()
    seq = torch.zeros(4, dtype=torch.int32, device="cuda")
    b.e4b_balance_fwd(None, None, seq)
    b.e4b_balance_bwd(None, None, seq)
    assert e4b.e4b_launch_count() == n0
    assert not b.counts.any() and not b._tokens.any() and not b.prob_sum.any() and not b.loss.any()


def test_the_binding_refuses_before_any_launch():
    logits, ids, seq, mask = make(30, 8, 2, 3, 1.0)
    b = e4b.RouterBalance(8, 2, 30, 3)
    n0 = e4b.e4b_launch_count()
    with pytest.raises(TypeError, match="logits: dtype"):
        b.e4b_balance_fwd(logits.double(), ids, seq)
    with pytest.raises(ValueError, match="seq_offsets: required"):
        b.e4b_balance_fwd(logits, ids)
    with pytest.raises(ValueError, match="seq_offsets: 3 elements, the call needs 4"):
        b.e4b_balance_fwd(logits, ids, seq[:3])
    with pytest.raises(TypeError, match="token_mask: dtype"):
        b.e4b_balance_fwd(logits, ids, seq, mask.bool())
    with pytest.raises(ValueError, match="d_logits: a tensor is required"):
        b.e4b_balance_bwd(logits, None, seq)
    with pytest.raises(ValueError, match="topk_ids: .* elements"):
        b.e4b_balance_fwd(logits, ids[:10], seq)
    with pytest.raises(e4b.E4BError, match="E4B_ERR_INVALID_ARG"):
        b.e4b_balance_fwd(logits, ids, seq, balance_coef=float("nan"))
    assert e4b.e4b_launch_count() == n0


def test_as_used_in_a_training_step():
    # routing, the block's forward and input gradient, the router's gradient, and the balance gradient on top
    from grouped_nf4_expert_b200 import device as dv
    from grouped_nf4_expert_b200 import inputs
    cfg = inputs.CONFIGS["tiny"]
    d = dv.upload(inputs.make_problem(cfg))
    blk = e4b.Block(dv.dims_of(cfg), cfg.T)
    blk.e4b_route_permute(d.logits, d.x, gather=False)
    blk.e4b_grouped_nf4_lora_fwd(d.base(), d.lora(), x=d.x)
    blk.e4b_grouped_nf4_lora_dgrad(d.base(), d.lora(), d.dY)
    alone = torch.empty((cfg.T, cfg.E), device="cuda")
    blk.e4b_router_backward(d.dY, alone)
    total = alone.clone()
    b = e4b.RouterBalance(cfg.E, cfg.top_k, cfg.T)
    b.e4b_balance_fwd(d.logits, blk.topk_ids, balance_coef=0.01, z_coef=0.001)
    b.e4b_balance_bwd(d.logits, total, balance_coef=0.01, z_coef=0.001, accumulate=True)
    assert torch.equal(b.counts[0], blk.counts)  # the router's own counts
    want = reference(cfg.E, cfg.top_k, d.logits, blk.topk_ids, None, None, 0.01, 0.001)
    got = (total.double() - alone.double()).cpu().numpy()
    # the sum is rounded once more, by half a last place of the router's gradient
    assert np.all(np.abs(got - want[-1]) <= 2 * H * np.abs(total.double().cpu().numpy()) + 1e-4 * np.abs(want[-1]).max())
    assert blk.check_device_error() == e4b.E4B_OK


def test_calls_on_several_streams_at_once():
    # the joining blocks of a launch wait only for blocks of it that come before them
    cases = [make(T, E, 4, S, 0.9, seed=T) + [E] for T, E, S in ((5000, 64, 3), (3000, 512, 40), (20000, 16, 1),
                                                                 (2000, 1000, 200))]
    want = [run(c[4], 4, *c[:4]) for c in cases]
    objs = [(e4b.RouterBalance(c[4], 4, c[0].shape[0], c[2].numel() - 1), torch.empty_like(c[0]), torch.cuda.Stream())
            for c in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for (logits, ids, seq, mask, _E), (b, d, st) in zip(cases, objs):
            b.e4b_balance_fwd(logits, ids, seq, mask, 0.7, 0.3, stream=st)
            b.e4b_balance_bwd(logits, d, seq, mask, 0.7, 0.3, stream=st)
    torch.cuda.synchronize()
    for (w, wd), (b, d, _st) in zip(want, objs):
        assert torch.equal(b.loss, w.loss) and torch.equal(d, wd) and b.check_device_error() == e4b.E4B_OK


def test_what_a_call_launches():
    logits, ids, seq, mask = make(500, 64, 4, 3, 1.0)
    b, d = e4b.RouterBalance(64, 4, 500, 3), torch.empty_like(logits)
    e4b.e4b_profiler_read()
    e4b.e4b_profiler_enable(True)
    try:
        b.e4b_balance_fwd(logits, ids, seq, mask)
        b.e4b_balance_bwd(logits, d, seq, mask)
    finally:
        e4b.e4b_profiler_enable(False)
    assert {k: n for k, (n, _) in e4b.e4b_profiler_read().items()} == {"balance_fwd": 1, "balance_bwd": 1}


def test_what_a_workspace_held_does_not_matter():
    logits, ids, seq, mask = make(700, 60, 4, 5, 0.9)
    w, wd = run(60, 4, logits, ids, seq, mask)
    b, d = e4b.RouterBalance(60, 4, 700, 5), torch.empty_like(logits)
    b.ws[256:].fill_(0xff)
    b.e4b_balance_fwd(logits, ids, seq, mask, 0.7, 0.3)
    b.e4b_balance_bwd(logits, d, seq, mask, 0.7, 0.3)
    assert torch.equal(b.loss, w.loss) and torch.equal(b.counts, w.counts) and torch.equal(d, wd)
