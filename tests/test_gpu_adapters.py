"""The NF4 projection with adapters of many requests against its float64 oracle (GPU).

Bounds, per element.  bf16 rounds by at most u = 2^-8 of a value.  The kernels round p (or q) to bf16, sum in
float32 (each of the m products and additions off by at most one last place, 2^-23 of the running sum, which the
sum of absolute values bounds) and round the result once:

    |y - y*| <= (1 + u) (sum_j |B_j| e_p + (m + 4) 2^-23 (|W| |x| + |B| |p|)) + u |y*|
    e_p       = u |p*| + (K + 4) 2^-23 s |A| |x|

and the same with the roles swapped for dx, dA and dB.
"""

import ctypes

import numpy as np
import pytest
import torch

import oracle
from grouped_nf4_expert_b200 import build, e4b
from oracle import adapters as oa

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
F = 2.0 ** -23


@pytest.fixture(scope="session", autouse=True)
def _built():
    build.build()
    e4b.lib()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def f64(t):
    return t.detach().double().cpu().numpy()


class Case:
    def __init__(self, T, K, N, n, r, mix="zipf", seed=0, device="cuda"):
        g = torch.Generator().manual_seed(1000 + seed)
        self.T, self.K, self.N, self.n, self.r = T, K, N, n, r
        if mix == "each":
            ids = torch.randperm(n, generator=g)[torch.arange(T) % n]
        elif mix == "one":
            ids = torch.full((T,), n - 1)
        elif mix == "none":
            ids = torch.where(torch.arange(T) % 2 == 0, -1, n)
        elif mix == "runs":
            ids = torch.sort(torch.randint(0, n, (T,), generator=g)).values.flip(0)
        else:  # popular and rare adapters, a tenth of the tokens with none
            w = torch.arange(1, n + 1, dtype=torch.float32) ** -1.1
            ids = torch.multinomial(w, T, replacement=True, generator=g)
            ids = torch.where(torch.rand(T, generator=g) < 0.1, torch.full_like(ids, -1), ids)
        bf = torch.bfloat16
        self.ids = ids.to(torch.int32).to(device)
        self.x = torch.randn((T, K), generator=g).to(bf).to(device)
        self.dY = torch.randn((T, N), generator=g).to(bf).to(device)
        self.nf4 = torch.randint(0, 256, (N, K // 2), generator=g).to(torch.uint8).to(device)
        self.absmax = ((torch.rand((N, K // 64), generator=g) + 0.5) * 2 * K ** -0.5).to(device)
        self.A = (torch.randn((n, r, K), generator=g) * K ** -0.5).to(bf).to(device)
        self.B = (torch.randn((n, N, r), generator=g) * 0.1).to(bf).to(device)
        self.scale = (torch.rand(n, generator=g) + 0.5).to(device)
        self.dims = e4b.ProjDims(K=K, N=N, n_adapters=n, r=r)

    def base(self):
        return e4b.nf4_matrix(self.nf4, self.absmax)

    def adapters(self):
        return e4b.adapter_factors(self.A, self.B, self.scale)

    def ref(self):
        W = oracle.dequantize_nf4_matrix(self.nf4.cpu().numpy(), self.absmax.cpu().numpy())
        return dict(x=f64(self.x), ids=self.ids.cpu().numpy(), W=W, A=f64(self.A), B=f64(self.B),
                    scale=f64(self.scale))


def bounds(c):
    """y*, its bound, and a function for the gradients."""
    m = c.ref()
    ab = {k: (np.abs(v) if k != "ids" else v) for k, v in m.items()}
    y, p = oa.project(**m)
    y_abs, p_abs = oa.project(**ab)
    e_p = U * np.abs(p) + (c.K + 4) * F * p_abs
    prop = np.zeros_like(y)
    for a in range(c.n):
        rows = np.flatnonzero(m["ids"] == a)
        prop[rows] = e_p[rows] @ ab["B"][a].T
    y_tol = (1 + U) * (prop + (c.K + c.r + 4) * F * y_abs) + U * np.abs(y)

    def grads():
        dY = f64(c.dY)
        dx, q, dA, dB = oa.project_backward(m["x"], m["ids"], dY, m["W"], m["A"], m["B"], m["scale"])
        dx_abs, q_abs, dA_abs, dB_abs = oa.project_backward(ab["x"], m["ids"], np.abs(dY), ab["W"], ab["A"], ab["B"],
                                                            ab["scale"])
        e_q = U * np.abs(q) + (c.N + 4) * F * q_abs
        dx_e, dA_e, dB_e = np.zeros_like(dx), np.zeros_like(dA), np.zeros_like(dB)
        for a in range(c.n):
            rows = np.flatnonzero(m["ids"] == a)
            dx_e[rows] = e_q[rows] @ ab["A"][a]
            dA_e[a] = e_q[rows].T @ ab["x"][rows]
            dB_e[a] = np.abs(dY[rows]).T @ e_p[rows]
        t = c.T + 4
        return ((dx, (1 + U) * (dx_e + (c.N + c.r + 4) * F * dx_abs) + U * np.abs(dx)),
                (dA, (1 + U) * (dA_e + (t + c.N) * F * dA_abs) + U * np.abs(dA)),
                (dB, (1 + U) * (dB_e + (t + c.K) * F * dB_abs) + U * np.abs(dB)))

    return y, y_tol, grads


def check(got, want, tol, what):
    got = f64(got)
    assert got.shape == want.shape, what
    off = np.abs(got - want) > tol
    assert not off.any(), "%s: %d of %d off, worst %.3g against %.3g" % (
        what, off.sum(), off.size, np.abs(got - want)[off].max(), tol[off].min())


def serve(c, **kw):
    pj = e4b.Projection(c.dims, c.T, train=False, **kw)
    pj.y.fill_(float("nan"))
    pj.e4b_multi_lora_serve_fwd(c.ids, c.x, c.base(), c.adapters())
    assert pj.check_device_error() == e4b.E4B_OK
    return pj


def train(c, **kw):
    pj = e4b.Projection(c.dims, c.T, **kw)
    for t in (pj.y, pj.dx, pj.dA, pj.dB):
        t.fill_(float("nan"))
    pj.e4b_adapter_group(c.ids)
    pj.e4b_multi_lora_fwd(c.x, c.base(), c.adapters())
    pj.e4b_multi_lora_dgrad(c.dY, c.base(), c.adapters())
    pj.e4b_multi_lora_wgrad(c.x, c.dY)
    assert pj.check_device_error() == e4b.E4B_OK
    return pj


# (T, K, N, n, r, mix): one token; odd batches around the tile sizes; narrow and ragged N; ranks that are not a
# power of two; every adapter its own token; one adapter for all; no adapters at all
SERVE = [
    (1, 64, 8, 1, 8, "one"), (1, 512, 264, 5, 16, "zipf"), (3, 192, 136, 3, 24, "each"), (7, 2048, 64, 4, 64, "zipf"),
    (8, 128, 1000, 8, 8, "each"), (9, 256, 128, 40, 16, "each"), (15, 448, 72, 2, 40, "zipf"),
    (16, 1024, 256, 16, 16, "each"), (17, 320, 200, 6, 32, "zipf"), (31, 576, 128, 31, 8, "each"),
    (33, 256, 512, 4, 56, "runs"), (57, 512, 520, 64, 64, "zipf"), (64, 256, 128, 3, 16, "none"),
    (65, 384, 256, 1, 16, "one"), (100, 256, 264, 100, 8, "each"), (129, 512, 384, 7, 48, "zipf"),
    (200, 128, 1024, 1024, 8, "zipf"), (256, 256, 256, 32, 32, "zipf"), (257, 192, 328, 5, 16, "zipf"),
    (300, 256, 512, 300, 8, "each"), (513, 64, 136, 9, 64, "runs"), (777, 512, 256, 16, 24, "zipf"),
    (1111, 256, 520, 8, 16, "runs"), (2049, 128, 264, 3, 8, "zipf"),
]


@pytest.mark.parametrize("shape", SERVE, ids=lambda s: "-".join(map(str, s)))
def test_serve(shape):
    c = Case(*shape)
    y, tol, _ = bounds(c)
    check(serve(c).y, y, tol, "y")


TRAIN = [
    (1, 64, 8, 1, 8, "one"), (2, 128, 72, 3, 16, "each"), (16, 64, 64, 4, 8, "each"), (40, 192, 136, 5, 24, "zipf"),
    (100, 256, 128, 100, 8, "each"), (129, 320, 264, 4, 64, "runs"), (255, 128, 512, 6, 40, "zipf"),
    (300, 256, 200, 2, 16, "none"), (777, 512, 256, 16, 24, "zipf"), (1500, 128, 136, 1, 48, "one"),
    (600, 1024, 1032, 2, 64, "runs"), (2500, 1024, 520, 1, 32, "one"), (1300, 2048, 264, 3, 16, "zipf"),
]


@pytest.mark.parametrize("shape", TRAIN, ids=lambda s: "-".join(map(str, s)))
def test_train(shape):
    c = Case(*shape)
    y, tol, grads = bounds(c)
    pj = train(c)
    check(pj.y, y, tol, "y")
    for got, (want, t), what in zip((pj.dx, pj.dA, pj.dB), grads(), ("dx", "dA", "dB")):
        check(got, want, t, what)
    # adapters without tokens: exact zeros
    used = np.isin(np.arange(c.n), c.ids.cpu().numpy())
    assert np.all(f64(pj.dA)[~used] == 0) and np.all(f64(pj.dB)[~used] == 0)


@pytest.mark.parametrize("T,n,mix", [(1, 1, "one"), (5, 3, "zipf"), (100, 7, "zipf"), (1024, 64, "zipf"),
                                     (2000, 1024, "zipf"), (4097, 5, "runs"), (64, 4, "none")])
def test_group(T, n, mix):
    c = Case(T, 64, 8, n, 8, mix)
    pj = e4b.Projection(c.dims, T)
    pj.order.fill_(-7)
    pj.e4b_adapter_group(c.ids)
    members, starts = oa.group(c.ids.cpu().numpy(), n)
    order, offsets = pj.order.cpu().numpy(), pj.offsets.cpu().numpy()
    assert np.array_equal(offsets, starts)
    want = np.full(order.shape, T)
    for m, s in zip(members, starts):
        want[s:s + m.size] = m
    assert np.array_equal(order, want)


def test_a_bad_value_stays_with_its_request():
    # an adapter of infinities, one of NaN and a token of NaN: every other request's rows, and the other
    # adapters' gradients, are what they were without them
    c = Case(90, 256, 136, 5, 16, "zipf", seed=3)
    good_s, good_t = serve(c).y.clone(), train(c)
    ids = c.ids.cpu().numpy()
    victim = int(np.flatnonzero(ids == 0)[0])
    c.A[1], c.B[2] = float("nan"), float("inf")
    c.x[victim, 5] = float("nan")
    c.dY[victim, 3] = float("inf")
    ok = torch.tensor(((ids == 0) | (ids > 2) | (ids < 0)) & (np.arange(90) != victim))
    bad_t = train(c)
    for got, want in ((serve(c).y, good_s), (bad_t.y, good_t.y), (bad_t.dx, good_t.dx)):
        assert torch.equal(got.cpu()[ok], want.cpu()[ok])
        assert not torch.isfinite(got.float()).all()
    for a in (3, 4):
        assert torch.equal(bad_t.dA[a], good_t.dA[a]) and torch.equal(bad_t.dB[a], good_t.dB[a])


def test_repeated_calls_give_the_same_bits():
    c = Case(300, 512, 264, 9, 32, "zipf", seed=4)
    a, b = train(c), train(c)
    for name in ("y", "dx", "dA", "dB"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name
    s1, s2 = serve(c), serve(c)
    assert torch.equal(s1.y, s2.y)


@pytest.mark.parametrize("T", [1, 20, 90, 400])
def test_another_stream_and_a_graph(T):
    c = Case(T, 256, 264, 6, 16, "zipf", seed=5)
    want = serve(c).y.clone()
    base, ad = c.base(), c.adapters()
    st = torch.cuda.Stream()
    pj = e4b.Projection(c.dims, T, train=False)
    st.wait_stream(torch.cuda.current_stream())
    pj.e4b_multi_lora_serve_fwd(c.ids, c.x, base, ad, stream=st)
    st.synchronize()
    assert torch.equal(pj.y, want)
    pj.y.zero_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pj.e4b_multi_lora_serve_fwd(c.ids, c.x, base, ad)
    for _ in range(3):
        g.replay()
    assert torch.equal(pj.y, want)
    # new inputs and another mix of adapters in the same buffers
    d = Case(T, 256, 264, 6, 16, "each", seed=6)
    c.ids.copy_(d.ids)
    c.x.copy_(d.x)
    g.replay()
    assert torch.equal(pj.y, serve(c).y)


def test_training_step_captured():
    c = Case(200, 256, 136, 4, 16, "zipf", seed=7)
    want = train(c)
    pj = e4b.Projection(c.dims, c.T)
    base, ad = c.base(), c.adapters()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pj.e4b_adapter_group(c.ids)
        pj.e4b_multi_lora_fwd(c.x, base, ad)
        pj.e4b_multi_lora_dgrad(c.dY, base, ad)
        pj.e4b_multi_lora_wgrad(c.x, c.dY)
    g.replay()
    g.replay()
    for name in ("y", "dx", "dA", "dB"):
        assert torch.equal(getattr(pj, name), getattr(want, name)), name


def test_graphs_that_share_a_workspace():
    # a serving and a training graph over one object's buffers, replayed in turn
    c = Case(150, 256, 136, 5, 24, "zipf", seed=9)
    want, want_t = serve(c).y.clone(), train(c)
    pj = e4b.Projection(c.dims, c.T)
    base, ad = c.base(), c.adapters()
    gs, gt = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(gs):
        pj.e4b_multi_lora_serve_fwd(c.ids, c.x, base, ad)
    with torch.cuda.graph(gt):
        pj.e4b_adapter_group(c.ids)
        pj.e4b_multi_lora_fwd(c.x, base, ad)
        pj.e4b_multi_lora_dgrad(c.dY, base, ad)
    for _ in range(3):
        gt.replay()
        assert torch.equal(pj.y, want_t.y) and torch.equal(pj.dx, want_t.dx)
        gs.replay()
        assert torch.equal(pj.y, want)
    assert pj.check_device_error() == e4b.E4B_OK


def test_a_graph_of_two_launches_under_one_another():
    c = Case(256, 4096, 4096, 32, 32, "zipf", seed=60)
    want = serve(c).y.clone()
    pj, base, ad = e4b.Projection(c.dims, c.T, train=False), c.base(), c.adapters()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            pj.e4b_multi_lora_serve_fwd(c.ids, c.x, base, ad)
    for _ in range(3):
        pj.y.zero_()
        g.replay()
        assert torch.equal(pj.y, want)
    assert pj.check_device_error() == e4b.E4B_OK


@pytest.mark.parametrize("T", [5, 14, 60, 256, 300])
def test_a_chain_of_launches_under_one_another(T):
    # every projection reads what the one before it wrote; launches may start early, reads may not
    cases = [Case(T, K, N, n, 16, "zipf", seed=70 + i) for i, (K, N, n) in enumerate(
        ((2048, 4096, 4), (4096, 1024, 40), (1024, 128, 3), (128, 4096, 7), (4096, 2048, 32)))]
    first = cases[0].x
    steps = [(e4b.Projection(c.dims, T, train=False), c) for c in cases]
    args = [(c.base(), c.adapters()) for c in cases]

    def run(sync):
        x = first
        for (pj, c), (base, ad) in zip(steps, args):
            pj.e4b_multi_lora_serve_fwd(c.ids, x, base, ad)
            if sync:
                torch.cuda.synchronize()
            x = pj.y
        return x

    want = run(True).clone()
    for _ in range(30):
        for pj, _c in steps:
            pj.y.fill_(float("nan"))
        assert torch.equal(run(False), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(False)
        y = run(False)
    for _ in range(5):
        g.replay()
        assert torch.equal(y, want)


@pytest.mark.parametrize("T,n", [(7, 3), (60, 5), (300, 5), (700, 40)])
def test_what_a_workspace_held_does_not_matter(T, n):
    # a workspace full of NaN behind its header
    c = Case(T, 320, 264, n, 24, "zipf", seed=95)
    want, want_t = serve(c).y.clone(), train(c)
    pj = e4b.Projection(c.dims, c.T)
    pj.ws[256:].fill_(0xff)
    pj.e4b_multi_lora_serve_fwd(c.ids, c.x, c.base(), c.adapters())
    assert torch.equal(pj.y, want)
    for t in (pj.p, pj.q):
        t.fill_(float("nan"))
    pj.ws[256:].fill_(0xff)
    pj.e4b_adapter_group(c.ids)
    pj.e4b_multi_lora_fwd(c.x, c.base(), c.adapters())
    pj.e4b_multi_lora_dgrad(c.dY, c.base(), c.adapters())
    pj.e4b_multi_lora_wgrad(c.x, c.dY)
    for k in ("y", "dx", "dA", "dB"):
        assert torch.equal(getattr(pj, k), getattr(want_t, k)), k


@pytest.mark.parametrize("shape", [(5, 512, 264, 6, 16), (60, 512, 264, 6, 16), (256, 4096, 4096, 32, 32),
                                   (300, 512, 264, 6, 16)], ids=lambda s: "-".join(map(str, s)))
def test_inputs_written_between_calls(shape):
    # the same buffers filled with another batch ahead of each call, on the stream: each call sees its own batch, its
    # own adapters and its own matrix
    batches = [Case(*shape, "zipf", seed=90 + i) for i in range(4)]
    want = [serve(b).y.clone() for b in batches]
    c = Case(*shape, "zipf", seed=90)
    pj, base, ad = e4b.Projection(c.dims, c.T, train=False), c.base(), c.adapters()
    for i in (1, 3, 0, 2, 2, 1, 0, 3):
        b = batches[i]
        for name in ("ids", "x", "nf4", "absmax", "A", "B", "scale"):
            getattr(c, name).copy_(getattr(b, name))
        pj.e4b_multi_lora_serve_fwd(c.ids, c.x, base, ad)
        pj.e4b_multi_lora_serve_fwd(c.ids, c.x, base, ad)
        assert torch.equal(pj.y, want[i])


def test_more_padding_than_the_unit_was_chosen_for():
    # three groups of 97 tokens take 353 rows where 339 were expected: units of 352 rows, the last one alone in its own
    c = Case(291, 128, 16384, 2, 16, "runs", seed=80)
    ids = torch.arange(291) % 3
    ids[ids == 2] = -1
    c.ids = ids.to(torch.int32).cuda()
    y, tol, _ = bounds(c)
    check(serve(c).y, y, tol, "y")


def test_calls_on_several_streams_at_once():
    # each with an object of its own: blocks that wait inside one launch wait only for earlier blocks of it
    cases = [Case(T, 1024, 2048, 8, 16, "zipf", seed=20 + i) for i, T in enumerate((3, 16, 60, 200, 256, 300))]
    cases.append(Case(256, 4096, 4096, 32, 32, "zipf", seed=60))
    want = [serve(c).y.clone() for c in cases]
    objs = [(e4b.Projection(c.dims, c.T, train=False), c.base(), c.adapters(), torch.cuda.Stream()) for c in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, (pj, base, ad, st) in zip(cases, objs):
            pj.e4b_multi_lora_serve_fwd(c.ids, c.x, base, ad, stream=st)
    torch.cuda.synchronize()
    for w, (pj, *_rest) in zip(want, objs):
        assert torch.equal(pj.y, w) and pj.check_device_error() == e4b.E4B_OK


def test_calls_of_several_host_threads():
    # sizes that need different amounts of shared memory, launched from threads of their own
    import threading
    cases = [Case(300, 128, 72, n, 8, "zipf", seed=40 + i) for i, n in enumerate((3, 900, 40, 600))]
    cases += [Case(T, 256, 264, 5, 8, "zipf", seed=50 + i) for i, T in enumerate((20, 250, 130, 256))]
    want = [serve(c).y.clone() for c in cases]
    bad = []

    def work(c, w):
        try:
            pj, base, ad, st = e4b.Projection(c.dims, c.T, train=False), c.base(), c.adapters(), torch.cuda.Stream()
            torch.cuda.synchronize()
            for _ in range(200):
                pj.e4b_multi_lora_serve_fwd(c.ids, c.x, base, ad, stream=st)
            st.synchronize()
            if not torch.equal(pj.y, w):
                bad.append((c.T, c.n))
        except Exception as e:  # noqa: BLE001 (told below, with its case)
            bad.append((c.T, c.n, repr(e)))

    threads = [threading.Thread(target=work, args=a) for a in zip(cases, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad


def test_offsets_past_32_bits():
    # y holds 2^31 elements and more: the last tokens' rows against the formula in 64 bits
    T, N = 16400, 131080
    c = Case(1, 64, N, 3, 8, "one", seed=30)
    g = torch.Generator().manual_seed(4)
    c.T, c.ids = T, torch.randint(-1, 3, (T,), generator=g).to(torch.int32).cuda()
    c.x = torch.randn((T, 64), generator=g).to(torch.bfloat16).cuda()
    y = serve(c).y
    rows = [0, 7, 16000, 16384, T - 2, T - 1]
    m = c.ref()
    m["x"], m["ids"] = m["x"][rows], m["ids"][rows]
    want, p = oa.project(**m)
    ab = {k: (np.abs(v) if k != "ids" else v) for k, v in m.items()}
    want_abs, p_abs = oa.project(**ab)
    e_p = U * np.abs(p) + (64 + 4) * F * p_abs
    prop = np.stack([e_p[i] @ ab["B"][a].T if 0 <= a < 3 else np.zeros(N) for i, a in enumerate(m["ids"])])
    check(y[torch.tensor(rows).cuda()], want, (1 + U) * (prop + (64 + 8 + 4) * F * want_abs) + U * np.abs(want), "y")


def test_gradient_offsets_past_32_bits():
    # x, dx and the rows of the weight gradients' inputs, likewise
    T, K = 16400, 131136
    c = Case(1, K, 8, 3, 8, "one", seed=31)
    g = torch.Generator().manual_seed(5)
    c.T, c.ids = T, torch.randint(-1, 3, (T,), generator=g).to(torch.int32).cuda()
    c.x = torch.randint(-3, 4, (T, K), dtype=torch.int8, device="cuda").to(torch.bfloat16)
    c.dY = torch.randn((T, 8), generator=g).to(torch.bfloat16).cuda()
    pj = train(c)
    rows, cols = [0, 7, 16000, 16384, T - 2, T - 1], [0, 1, 63, 65536, K - 2, K - 1]
    m, ids = c.ref(), c.ids.cpu().numpy()
    dY = f64(c.dY)
    q = np.zeros((T, c.r))
    q_abs = np.zeros((T, c.r))
    for a in range(c.n):
        q[ids == a] = m["scale"][a] * dY[ids == a] @ m["B"][a]
        q_abs[ids == a] = m["scale"][a] * np.abs(dY[ids == a]) @ np.abs(m["B"][a])
    e_q = U * np.abs(q) + (8 + 4) * F * q_abs
    xc = f64(c.x[:, torch.tensor(cols).cuda()])
    for a in range(c.n):
        of = ids == a
        want = q[of].T @ xc[of]
        tol = ((1 + U) * (e_q[of].T @ np.abs(xc[of]) + (T + 4 + 8) * F * (q_abs[of].T @ np.abs(xc[of])))
               + U * np.abs(want))
        check(pj.dA[a][:, torch.tensor(cols).cuda()], want, tol, "dA")
    A = np.stack([m["A"][a] if 0 <= a < 3 else np.zeros_like(m["A"][0]) for a in ids[rows]])
    dx = dY[rows] @ m["W"] + np.einsum("tr,trk->tk", q[rows], A)
    dx_abs = np.abs(dY[rows]) @ np.abs(m["W"]) + np.einsum("tr,trk->tk", q_abs[rows], np.abs(A))
    e = np.einsum("tr,trk->tk", e_q[rows], np.abs(A)) + (8 + 8 + 4) * F * dx_abs
    check(pj.dx[torch.tensor(rows).cuda()], dx, (1 + U) * e + U * np.abs(dx), "dx")


@pytest.mark.parametrize("shape,kernels", [
    ((1, 256, 136, 3, 8, "one"), {"adapter_gemv": 1}),
    ((16, 256, 136, 3, 8, "zipf"), {"adapter_gemv": 1}),
    ((9, 4096, 4096, 3, 8, "zipf"), {"adapter_split": 1}),
    ((17, 256, 136, 3, 8, "zipf"), {"adapter_split": 1}),
    ((256, 256, 136, 3, 8, "zipf"), {"adapter_split": 1}),
    ((256, 4096, 4096, 32, 32, "zipf"), {"adapter_low_rank": 1, "adapter_split": 1}),
    ((257, 256, 136, 3, 8, "zipf"), {"adapter_group": 1, "adapter_proj_x": 1, "adapter_fwd": 1}),
])
def test_what_a_serving_call_launches(shape, kernels):
    c = Case(*shape)
    pj = e4b.Projection(c.dims, c.T, train=False)
    e4b.e4b_profiler_read()
    e4b.e4b_profiler_enable(True)
    try:
        pj.e4b_multi_lora_serve_fwd(c.ids, c.x, c.base(), c.adapters())
    finally:
        e4b.e4b_profiler_enable(False)
    assert {k: n for k, (n, _) in e4b.e4b_profiler_read().items()} == kernels


@pytest.mark.parametrize("shape", [
    # one share of K and more, the blocks of p before the products and beside them, two token tiles of the warp
    # products over several row blocks, forward units of 96 to 256 rows, both widths of the input gradient
    (9, 4096, 4096, 3, 24, "zipf"), (30, 512, 8200, 5, 16, "zipf"), (30, 2048, 1024, 30, 64, "each"),
    (250, 1024, 2056, 40, 64, "zipf"), (120, 4096, 264, 3, 32, "runs"), (12, 1024, 4104, 12, 40, "each"),
    (400, 2048, 4096, 4, 16, "runs"), (700, 512, 12800, 6, 8, "zipf"),
    # units of three parts, the third of 64 to 128 rows, ranks padded and not, an adapter over all of them, none at all
    (1111, 256, 4096, 8, 16, "runs"), (260, 128, 16384, 1, 64, "one"), (262, 192, 18000, 2, 24, "zipf"),
    (300, 320, 16384, 2, 40, "runs"), (340, 128, 16392, 1, 8, "zipf"), (270, 64, 16384, 2, 8, "none"),
    # p in a launch of its own
    (256, 4096, 4096, 32, 32, "zipf"), (200, 2048, 18952, 100, 64, "each"),
], ids=lambda s: "-".join(map(str, s)))
def test_serve_wide(shape):
    c = Case(*shape)
    y, tol, _ = bounds(c)
    check(serve(c).y, y, tol, "y")


def test_rows_behind_the_last_token_stay():
    # buffers larger than the call: what lies behind the T tokens is left as it was
    c = Case(37, 128, 136, 3, 8, "zipf")
    big = torch.full((64, 136), 3.0, dtype=torch.bfloat16, device="cuda")
    pj = e4b.Projection(c.dims, c.T)
    ref = ctypes.byref
    e4b._check(e4b.lib().e4b_multi_lora_serve_fwd(ref(pj._dims_c), c.T, c.ids.data_ptr(), c.x.data_ptr(),
                                                  ref(c.base()), ref(c.adapters()), big.data_ptr(), pj._ws_p,
                                                  pj._ws_n, e4b._stream(None)), "serve")
    assert torch.equal(big[:37], serve(c).y) and bool((big[37:] == 3.0).all())


def test_no_tokens():
    d = e4b.ProjDims(K=64, N=72, n_adapters=3, r=8)
    c = Case(4, 64, 72, 3, 8)
    pj = e4b.Projection(d, 0)
    n0 = e4b.e4b_launch_count()
    pj.e4b_adapter_group(None)
    pj.e4b_multi_lora_serve_fwd(None, None, c.base(), c.adapters())
    pj.e4b_multi_lora_fwd(None, c.base(), c.adapters())
    pj.e4b_multi_lora_dgrad(None, c.base(), c.adapters())
    pj.dA.fill_(1.0)
    pj.dB.fill_(1.0)
    pj.e4b_multi_lora_wgrad(None, None)
    assert e4b.e4b_launch_count() == n0
    assert not pj.dA.any() and not pj.dB.any()


def test_the_binding_refuses_before_any_launch():
    c = Case(20, 128, 136, 3, 8)
    pj = e4b.Projection(c.dims, 20)
    so = e4b.Projection(c.dims, 20, train=False)
    base, ad = c.base(), c.adapters()
    n0 = e4b.e4b_launch_count()
    with pytest.raises(TypeError, match="ids: dtype"):
        pj.e4b_multi_lora_serve_fwd(c.ids.long(), c.x, base, ad)
    with pytest.raises(ValueError, match="x: .* elements, the call needs"):
        pj.e4b_multi_lora_serve_fwd(c.ids, c.x[:19], base, ad)
    with pytest.raises(ValueError, match="x: must be contiguous"):
        pj.e4b_multi_lora_fwd(c.x.t(), base, ad)
    with pytest.raises(ValueError, match="ids: must be a CUDA tensor"):
        pj.e4b_adapter_group(c.ids.cpu())
    with pytest.raises(ValueError, match="a tensor is required"):
        pj.e4b_multi_lora_wgrad(c.x, None)
    with pytest.raises(TypeError, match="base: an Nf4Matrix"):
        pj.e4b_multi_lora_serve_fwd(c.ids, c.x, ad, ad)
    with pytest.raises(TypeError, match="adapters: AdapterFactors"):
        pj.e4b_multi_lora_serve_fwd(c.ids, c.x, base, None)
    with pytest.raises(ValueError, match="base.nf4: .* the dims need"):
        pj.e4b_multi_lora_fwd(c.x, e4b.nf4_matrix(c.nf4[:1], c.absmax), ad)
    with pytest.raises(ValueError, match="adapters.scale: .* the dims need"):
        pj.e4b_multi_lora_dgrad(c.dY, base, e4b.adapter_factors(c.A, c.B, c.scale[:2]))
    with pytest.raises(ValueError, match="train=False"):
        so.e4b_adapter_group(c.ids)
    with pytest.raises(e4b.E4BError, match="E4B_ERR_INVALID_ARG"):  # x off its 16-byte alignment
        off = torch.zeros(20 * 128 + 8, dtype=torch.bfloat16, device="cuda")[1:20 * 128 + 1]
        pj.e4b_multi_lora_serve_fwd(c.ids, off.view(20, 128), base, ad)
    assert e4b.e4b_launch_count() == n0


def test_as_used_with_the_expert_block():
    # one decode step of several requests: the adapted projection feeds the expert block's serving call
    from grouped_nf4_expert_b200 import device as dv
    from grouped_nf4_expert_b200 import inputs
    cfg = inputs.CONFIGS["tiny"]
    prob = inputs.make_problem(cfg)
    d = dv.upload(prob)
    c = Case(cfg.T, 128, cfg.H, 4, 8, "each", seed=8)
    pj = serve(c)
    blk = e4b.Block(dv.dims_of(cfg), cfg.T)
    blk.e4b_moe_serve_fwd(d.logits, pj.y, d.base(), d.lora())
    y, tol, _ = bounds(c)
    check(pj.y, y, tol, "projection")
    prob.x = pj.y.view(torch.int16).cpu().numpy().view(np.uint16)
    f = lambda b: inputs.bits_to_f32(b).astype(np.float64)  # noqa: E731
    ex = oracle.Experts(prob.gate_up_nf4, prob.gate_up_absmax, prob.down_nf4, prob.down_absmax, f(prob.A_gu),
                        f(prob.B_gu), f(prob.A_d), f(prob.B_d))
    want = oracle.moe_forward(f(prob.x), prob.logits, ex, cfg.top_k, cfg.alpha)["y"]
    got = f64(blk.y)
    assert np.abs(got - want).max() <= 1e-2 * np.abs(want).max()


def test_training_calls_out_of_order_are_refused():
    c = Case(40, 64, 72, 3, 8)
    pj, n0 = e4b.Projection(c.dims, c.T), e4b.e4b_launch_count()
    with pytest.raises(ValueError, match="call e4b_adapter_group first"):
        pj.e4b_multi_lora_fwd(c.x, c.base(), c.adapters())
    with pytest.raises(ValueError, match="call e4b_adapter_group first"):
        pj.e4b_multi_lora_dgrad(c.dY, c.base(), c.adapters())
    assert e4b.e4b_launch_count() == n0
    pj.e4b_adapter_group(c.ids)
    pj.e4b_multi_lora_fwd(c.x, c.base(), c.adapters())
    with pytest.raises(ValueError, match="call e4b_multi_lora_dgrad first"):
        pj.e4b_multi_lora_wgrad(c.x, c.dY)
    pj.e4b_multi_lora_dgrad(c.dY, c.base(), c.adapters())
    pj.e4b_multi_lora_wgrad(c.x, c.dY)
    pj.e4b_adapter_group(c.ids)  # another step: its forward and input gradient come first again
    with pytest.raises(ValueError, match="call e4b_multi_lora_fwd, e4b_multi_lora_dgrad first"):
        pj.e4b_multi_lora_wgrad(c.x, c.dY)
    with pytest.raises(ValueError, match="train=False"):
        e4b.Projection(c.dims, c.T, train=False).e4b_adapter_group(c.ids)
