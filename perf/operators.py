"""Performance cases of the operators beside the expert block: an NF4 projection with the low-rank
adapters of many requests at once, and the router's balance loss with its per-expert counts.

``run`` computes either the operators' plain form (elementary torch operations in float32) or, with
``own`` set, the calls a user's program makes of ``grouped_nf4_expert_b200.e4b``.  ``exact`` evaluates
the operators' definitions in float64.

Projection, for token t with adapter a = ids[t] (any id outside [0, n) means none):

    y[t] = W x[t] + s[a] B[a] (A[a] x[t])         W[i, j] = bf16(level[code[i, j]] * absmax[i, j // 64])

and, trained, with q[t] = s[a] dY[t] B[a] and p[t] = s[a] A[a] x[t]:

    dx[t] = dY[t] W + q[t] A[a]      dA[a] = sum_t q[t]^T x[t]      dB[a] = sum_t dY[t]^T p[t]

Balance loss over sequences s (token ranges), tokens with mask 0 left out, p = softmax(logits):

    f[s, e] = E * count[s, e] / (k * n_s)          P[s, e] = sum_t p[t, e] / n_s
    balance = mean over the sequences with tokens of sum_e f P
    z       = mean over the tokens of logsumexp(logits)^2
    loss    = c_b * balance + c_z * z              (counts are piecewise constant: no gradient through f)
"""

import math

import torch

own = False

LEVELS = (-1.0, -0.6961928009986877, -0.5250730514526367, -0.39491748809814453, -0.28444138169288635,
          -0.18477343022823334, -0.09105003625154495, 0.0, 0.07958029955625534, 0.16093020141124725,
          0.24611230194568634, 0.33791524171829224, 0.44070982933044434, 0.5626170039176941,
          0.7229568362236023, 1.0)

_COST = 2 * 16384 * 4096 * 14336  # flops of the largest listed projection
_ELEMS = 131072 * 64              # logits of the largest listed balance loss


def listed():
    def serve(name, T, K, N, n, r, mix):
        return {"name": name, "op": "serve", "T": T, "K": K, "N": N, "n": n, "r": r, "mix": mix}

    def train(name, T, K, N, n, r, mix):
        return {"name": name, "op": "train", "T": T, "K": K, "N": N, "n": n, "r": r, "mix": mix}

    def balance(name, T, E, k, S, keep, grad):
        return {"name": name, "op": "balance", "T": T, "E": E, "k": k, "S": S, "keep": keep, "grad": grad}

    return [
        # one token of one request: pure latency (the block's model width H = 2048)
        serve("serve_1", 1, 2048, 4096, 8, 16, "each"),
        # the decode workload's batch: 16 requests, every one with an adapter of its own
        serve("serve_16", 16, 2048, 4096, 16, 16, "each"),
        # a narrow projection (keys or values), odd batch, some requests without an adapter
        serve("serve_57_narrow", 57, 2048, 512, 64, 64, "some"),
        # a full decode batch over popular and rare adapters
        serve("serve_256", 256, 4096, 4096, 32, 32, "zipf"),
        # a mixed batch: prefill pieces of a few ragged requests
        serve("serve_1111", 1111, 2048, 4096, 8, 16, "runs"),
        # the largest prefill, at the widest projection of the repository's layers (4096 -> 14336)
        serve("serve_16384", 16384, 4096, 14336, 64, 16, "runs"),
        # a training step of a few adapters over one base, at the training workload's width and rank
        train("train_8192", 8192, 2048, 2048, 4, 64, "runs"),
        # a small ragged training step: tokens of 16 adapters interleaved, rank not a power of two
        train("train_777", 777, 512, 2048, 16, 24, "zipf"),
        # router statistics of a decode batch (counts and loss, no gradient)
        balance("balance_16", 16, 128, 8, 1, 1.0, False),
        # the training workload's router: 8192 tokens, 128 experts, top-8, whole-batch loss
        balance("balance_8192", 8192, 128, 8, 1, 1.0, True),
        # per-sequence loss over ragged sequences with padding tokens, many experts
        balance("balance_seq", 30011, 256, 8, 37, 0.9, True),
        # the largest: a long batch of many sequences
        balance("balance_131072", 131072, 64, 6, 64, 0.97, True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["serve", "serve", "serve", "train", "balance"])
    if op == "balance":
        E = rng.choice([8, 60, 64, 100, 128, 160, 256, 512, 1024])
        T = min(_spread(rng, 1, 131072), _ELEMS // E)
        return {"op": op, "T": T, "E": E, "k": rng.randint(1, min(E, 8)), "S": rng.randint(1, max(1, min(64, T))),
                "keep": rng.choice([1.0, 0.9, 0.5]), "grad": rng.random() < 0.75}
    K = 64 * _spread(rng, 4, 128)
    N = 8 * _spread(rng, 16, 1792)
    n = _spread(rng, 1, 64)
    r = 8 * rng.randint(1, 8)
    top = 16384 if op == "serve" else 8192
    # the dense low-rank terms of the plain form and the three training products count too
    unit = 2 * (K * N + n * r * (K + N)) * (1 if op == "serve" else 3)
    T = max(1, min(_spread(rng, 1, top), _COST // unit))
    return {"op": op, "T": T, "K": K, "N": N, "n": n, "r": r, "mix": rng.choice(["each", "some", "zipf", "runs"])}


def _ids(case, g, device):
    T, n, mix = case["T"], case["n"], case["mix"]
    if mix == "each":  # every request an adapter of its own, while there are enough
        base = torch.randperm(n, generator=g, device=device)
        ids = base[torch.arange(T, device=device) % n]
    elif mix == "some":  # a tenth of the tokens without an adapter
        ids = torch.randint(0, n, (T,), generator=g, device=device)
        ids = torch.where(torch.rand(T, generator=g, device=device) < 0.1, torch.full_like(ids, -1), ids)
    elif mix == "zipf":  # a few popular adapters
        w = torch.arange(1, n + 1, device=device, dtype=torch.float32) ** -1.1
        ids = torch.multinomial(w, T, replacement=True, generator=g)
    else:  # runs of tokens: each request's tokens stand together
        m = max(1, min(2 * n, T))
        cuts = torch.sort(torch.randint(0, T, (m - 1,), generator=g, device=device)).values if m > 1 else \
            torch.zeros(0, dtype=torch.int64, device=device)
        req = torch.searchsorted(cuts, torch.arange(T, device=device), right=True)
        ids = torch.randint(0, n, (m,), generator=g, device=device)[req]
    return ids.to(torch.int32)


def _weights(N, K, g, device):
    """NF4 codes and block scales of a normal weight matrix (scale 1 / sqrt(K))."""
    levels = torch.tensor(LEVELS, device=device)
    mids = (levels[1:] + levels[:-1]) / 2
    packed = torch.empty((N, K // 2), dtype=torch.uint8, device=device)
    absmax = torch.empty((N, K // 64), dtype=torch.float32, device=device)
    for i in range(0, N, 4096):
        w = torch.randn((min(4096, N - i), K), generator=g, device=device) * K ** -0.5
        a = w.view(w.shape[0], -1, 64).abs().amax(-1)
        c = torch.bucketize((w.view(w.shape[0], -1, 64) / a[..., None]).view(w.shape), mids).to(torch.uint8)
        packed[i:i + 4096] = c[:, 0::2] * 16 + c[:, 1::2]
        absmax[i:i + 4096] = a
    return packed, absmax


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(1000003 * seed + 17)
    st = {"case": dict(case)}
    T = case["T"]
    bf = torch.bfloat16
    if case["op"] == "balance":
        E, k, S = case["E"], case["k"], case["S"]
        # log probabilities of a skewed router plus noise, as a partly balanced router gives
        bias = -0.5 * torch.log1p(torch.arange(E, device=dev, dtype=torch.float32))
        st["logits"] = bias[torch.randperm(E, generator=g, device=dev)] + torch.randn((T, E), generator=g, device=dev)
        st["ids"] = torch.topk(st["logits"], k, dim=1).indices.to(torch.int32).contiguous()
        cuts = torch.sort(torch.randint(0, T + 1, (S - 1,), generator=g, device=dev)).values
        st["seq"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), T)]).to(torch.int32)
        st["mask"] = (torch.rand(T, generator=g, device=dev) < case["keep"]).to(torch.uint8)
        st["dloss"] = torch.ones(1, device=dev)
        if own:
            from grouped_nf4_expert_b200 import e4b
            st["bal"] = e4b.RouterBalance(E, k, T, S)
            st["d_logits"] = torch.empty((T, E), device=dev)
        return st
    K, N, n, r = case["K"], case["N"], case["n"], case["r"]
    st["ids"] = _ids(case, g, dev)
    st["x"] = torch.randn((T, K), generator=g, device=dev).to(bf)
    st["packed"], st["absmax"] = _weights(N, K, g, dev)
    st["A"] = (torch.randn((n, r, K), generator=g, device=dev) * K ** -0.5).to(bf)
    st["B"] = (torch.randn((n, N, r), generator=g, device=dev) * 0.05).to(bf)
    st["scale"] = torch.rand(n, generator=g, device=dev) * 1.5 + 0.5
    if case["op"] == "train":
        st["dY"] = torch.randn((T, N), generator=g, device=dev).to(bf)
    if own:
        from grouped_nf4_expert_b200 import e4b
        st["proj"] = e4b.Projection(e4b.ProjDims(K=K, N=N, n_adapters=n, r=r), T, train=case["op"] == "train")
        st["base"] = e4b.nf4_matrix(st["packed"], st["absmax"])
        st["adapters"] = e4b.adapter_factors(st["A"], st["B"], st["scale"])
    return st


# ---------------------------------------------------------------------------- plain form


def _dequant(packed, absmax):
    levels = torch.tensor(LEVELS, device=packed.device)
    c = torch.stack([packed >> 4, packed & 15], dim=-1).view(packed.shape[0], -1).to(torch.int64)
    w = levels[c].view(absmax.shape[0], absmax.shape[1], 64) * absmax[..., None]
    return w.to(torch.bfloat16).float().view(packed.shape[0], -1)


def _plain_projection(st):
    c = st["case"]
    T, K, N, n, r = c["T"], c["K"], c["N"], c["n"], c["r"]
    W = _dequant(st["packed"], st["absmax"])
    x, A, B = st["x"].float(), st["A"].float(), st["B"].float()
    # every adapter's low-rank product side by side, kept where it is the token's own
    mine = (st["ids"][:, None] == torch.arange(n, device=x.device, dtype=torch.int32)).float() * st["scale"]
    p = ((x @ A.view(n * r, K).t()).view(T, n, r) * mine[:, :, None]).view(T, n * r)
    Bt = B.permute(0, 2, 1).reshape(n * r, N)
    y = (x @ W.t() + p @ Bt).to(torch.bfloat16)
    if c["op"] == "serve":
        return y
    dY = st["dY"].float()
    q = ((dY @ Bt.t()).view(T, n, r) * mine[:, :, None]).view(T, n * r)
    dx = dY @ W + q @ A.view(n * r, K)
    dA = q.t() @ x
    dB = (dY.t() @ p).view(N, n, r).permute(1, 0, 2)
    return y, dx.to(torch.bfloat16), dA.view(n, r, K).to(torch.bfloat16), dB.contiguous().to(torch.bfloat16)


C_BALANCE, C_Z = 0.01, 0.001


def _plain_balance(st):
    c = st["case"]
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    logits, mask = st["logits"], st["mask"].float()
    dev = logits.device
    top = logits.amax(1, keepdim=True)
    ex = torch.exp(logits - top)
    tot = ex.sum(1, keepdim=True)
    p = ex / tot
    lse = (top + torch.log(tot))[:, 0]
    seq = torch.searchsorted(st["seq"][1:].contiguous(), torch.arange(T, device=dev, dtype=torch.int32), right=True)
    member = (seq[None, :] == torch.arange(S, device=dev)[:, None]).float() * mask  # [S, T]
    chosen = torch.zeros((T, E), device=dev).scatter_(1, st["ids"].long(), 1.0)
    # 0/1 products: whole numbers far below 2^24
    counts = member @ chosen
    n_s = member.sum(1)
    full = (n_s > 0).float()
    safe = n_s.clamp(min=1.0)
    f = E * counts / (k * safe[:, None])
    P = (member @ p) / safe[:, None]
    n_seq = full.sum().clamp(min=1.0)
    n_tok = n_s.sum().clamp(min=1.0)
    balance = (f * P).sum() / n_seq
    z = (mask * lse * lse).sum() / n_tok
    loss = torch.stack([C_BALANCE * balance + C_Z * z, balance, z])
    out = (loss, counts.to(torch.int32), n_s.to(torch.int32))
    if not c["grad"]:
        return out
    ft = f[seq]
    wt = (1.0 / (safe * n_seq))[seq][:, None]
    d = C_BALANCE * wt * p * (ft - (p * ft).sum(1, keepdim=True)) + (2.0 * C_Z / n_tok) * lse[:, None] * p
    return out + (st["dloss"] * d * mask[:, None],)


def run(state):
    c = state["case"]
    if not own:
        return _plain_balance(state) if c["op"] == "balance" else _plain_projection(state)
    if c["op"] == "balance":
        b = state["bal"]
        b.e4b_balance_fwd(state["logits"], state["ids"], seq_offsets=state["seq"], token_mask=state["mask"],
                          balance_coef=C_BALANCE, z_coef=C_Z)
        if not c["grad"]:
            return b.loss, b.counts, b.tokens
        b.e4b_balance_bwd(state["logits"], state["d_logits"], seq_offsets=state["seq"], token_mask=state["mask"],
                          balance_coef=C_BALANCE, z_coef=C_Z, dloss=state["dloss"])
        return b.loss, b.counts, b.tokens, state["d_logits"]
    pj = state["proj"]
    if c["op"] == "serve":
        pj.e4b_multi_lora_serve_fwd(state["ids"], state["x"], state["base"], state["adapters"])
        return pj.y
    pj.e4b_adapter_group(state["ids"])
    pj.e4b_multi_lora_fwd(state["x"], state["base"], state["adapters"])
    pj.e4b_multi_lora_dgrad(state["dY"], state["base"], state["adapters"])
    pj.e4b_multi_lora_wgrad(state["x"], state["dY"])
    return pj.y, pj.dx, pj.dA, pj.dB


def work(case):
    T = case["T"]
    if case["op"] == "balance":
        E, k, S = case["E"], case["k"], case["S"]
        fwd = 4 * T * E + 4 * T * k + T + 4 * (S + 1) + 4 * S * E + 4 * S + 12
        bwd = 4 * T * E + 4 if case["grad"] else 0  # the gradient's write; the logits are counted once
        return {"bytes": fwd + bwd, "flops": T * E * (12 if case["grad"] else 5)}
    K, N, n, r = case["K"], case["N"], case["n"], case["r"]
    used = min(n, T)
    base = N * K // 2 + N * (K // 64) * 4
    lora = used * r * (K + N) * 2 + 4 * n
    fwd_bytes = base + lora + 2 * T * (K + N) + 4 * T
    fwd_flops = 2 * T * (K * N + r * (K + N))
    if case["op"] == "serve":
        return {"bytes": fwd_bytes, "flops": fwd_flops}
    return {"bytes": fwd_bytes + 2 * T * (K + N) + n * r * (K + N) * 2,
            "flops": 2 * fwd_flops + 2 * T * r * (K + N)}


# ---------------------------------------------------------------------------- definitions in float64


def _exact_projection(case, st):
    n = case["n"]
    codes = st["packed"].long()
    table = torch.tensor(LEVELS, dtype=torch.float32, device=codes.device)
    # the stored weight: one float32 product of level and block scale, rounded to bf16 by definition
    hi, lo = table[codes // 16], table[codes % 16]
    scale = torch.repeat_interleave(st["absmax"], 32, dim=1)
    W = torch.empty((case["N"], case["K"]), dtype=torch.float64, device=codes.device)
    W[:, 0::2] = (hi * scale).bfloat16().double()
    W[:, 1::2] = (lo * scale).bfloat16().double()
    x = st["x"].double()
    y = torch.matmul(x, W.T)
    train = case["op"] == "train"
    if train:
        dY = st["dY"].double()
        dx = torch.matmul(dY, W)
        dA = torch.zeros((n, case["r"], case["K"]), dtype=torch.float64, device=x.device)
        dB = torch.zeros((n, case["N"], case["r"]), dtype=torch.float64, device=x.device)
    del W
    for a in range(n):
        rows = torch.nonzero(st["ids"] == a)[:, 0]
        if rows.numel() == 0:
            continue
        A, B, s = st["A"][a].double(), st["B"][a].double(), st["scale"][a].double()
        low = s * torch.matmul(x[rows], A.T)
        y[rows] += torch.matmul(low, B.T)
        if train:
            back = s * torch.matmul(dY[rows], B)
            dx[rows] += torch.matmul(back, A)
            dA[a] = torch.einsum("tr,tk->rk", back, x[rows])
            dB[a] = torch.einsum("tn,tr->nr", dY[rows], low)
    return (y, dx, dA, dB) if train else y


def _exact_balance(case, st):
    E, k, S, T = case["E"], case["k"], case["S"], case["T"]
    logits = st["logits"].double()
    ends = st["seq"].tolist()
    keep = st["mask"].bool()
    prob = torch.softmax(logits, dim=1)
    lse = torch.logsumexp(logits, dim=1)
    counts = torch.zeros((S, E), dtype=torch.int32, device=logits.device)
    tokens = torch.zeros(S, dtype=torch.int32, device=logits.device)
    spans = [torch.arange(ends[s], ends[s + 1], device=logits.device) for s in range(S)]
    spans = [v[keep[v]] for v in spans]
    n_seq = max(1, sum(1 for v in spans if v.numel()))
    n_tok = max(1, sum(v.numel() for v in spans))
    grad = torch.zeros((T, E), dtype=torch.float64, device=logits.device)
    balance = torch.zeros((), dtype=torch.float64, device=logits.device)
    z = torch.zeros((), dtype=torch.float64, device=logits.device)
    for s, v in enumerate(spans):
        if v.numel() == 0:
            continue
        tokens[s] = v.numel()
        counts[s] = torch.bincount(st["ids"][v].reshape(-1).long(), minlength=E).to(torch.int32)
        f = counts[s].double() * E / (k * v.numel())
        balance += torch.dot(f, prob[v].mean(0)) / n_seq
        z += lse[v].square().sum() / n_tok
        pull = f[None, :] - torch.matmul(prob[v], f)[:, None]
        grad[v] = (C_BALANCE / (n_seq * v.numel()) * pull + 2 * C_Z / n_tok * lse[v][:, None]) * prob[v]
    loss = torch.stack([C_BALANCE * balance + C_Z * z, balance, z])
    if not case["grad"]:
        return loss, counts, tokens
    return loss, counts, tokens, grad * st["dloss"].double()


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_balance(case, st) if case["op"] == "balance" else _exact_projection(case, st)
