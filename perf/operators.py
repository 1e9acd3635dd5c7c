"""Operators of the mixture-of-experts layer on packed 4-bit weights: what is timed, on which
inputs, and the plain statement of each operator that the kernels are held to.

Three operators, each through the calls a user makes (``own``) or in elementary torch operations:

* ``route``: the top-k softmax router of M tokens over E experts, with the (token, choice) slots
  listed by expert;
* ``experts``: 4-bit products whose weight each row picks from a stack of experts;
* ``moe``: the whole layer, router to weighted sum of the experts' gated MLPs.
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = "bf16", "fp32"
DTYPES = {BF16: torch.bfloat16, F32: torch.float32}


# ---- cases -----------------------------------------------------------------------------------

def _route(M, E, k, dtype, normalize=True, masked=0):
    return dict(op="route", M=M, E=E, k=k, dtype=dtype, normalize=normalize, masked=masked)


def _experts(M, E, k, N, K, bs, dtype, zp=False, bias=False, per_slot=False, empty=0):
    return dict(op="experts", M=M, E=E, k=k, N=N, K=K, bs=bs, dtype=dtype, zp=zp, bias=bias,
                per_slot=per_slot, empty=empty)


def _moe(M, E, k, H, I, bs, dtype, zp=False, bias=False, normalize=True):
    return dict(op="moe", M=M, E=E, k=k, H=H, I=I, bs=bs, dtype=dtype, zp=zp, bias=bias,
                normalize=normalize)


def listed():
    return [
        # One token of a decode step: latency alone.
        dict(name="route_one", **_route(1, 128, 8, F32)),
        # A mixed batch with some experts switched off (masked by -inf), probabilities kept.
        dict(name="route_batch_masked", **_route(501, 60, 6, BF16, normalize=False, masked=5)),
        # A long prompt or a packed batch of them.
        dict(name="route_prompt", **_route(32768, 128, 8, BF16)),
        # The first projection of one decode token's experts.
        dict(name="experts_one", **_experts(1, 64, 8, 1536, 2560, 32, BF16)),
        # fp32 activations, zero points, bias, padding tokens without an expert, sizes that fill
        # no tile: a small batch of an exported model.
        dict(name="experts_ragged_fp32",
             **_experts(13, 24, 3, 1000, 1111, 32, F32, zp=True, bias=True, empty=2)),
        # The second projection of a prompt's experts: every slot has its own row.
        dict(name="experts_prompt",
             **_experts(2048, 32, 4, 2560, 1024, 128, BF16, per_slot=True)),
        # One decode token through the whole layer, many narrow experts.
        dict(name="moe_one", **_moe(1, 128, 8, 2560, 768, 32, BF16)),
        # One decode token, few wide experts, fp32 activations and zero points.
        dict(name="moe_one_fp32", **_moe(1, 8, 2, 1024, 2048, 32, F32, zp=True)),
        # A decode batch: most experts have one or two tokens.
        dict(name="moe_batch", **_moe(16, 128, 8, 2560, 768, 32, BF16)),
        # A few concurrent requests, odd widths, biases.
        dict(name="moe_few_ragged", **_moe(5, 20, 4, 1000, 520, 64, BF16, zp=True, bias=True)),
        # A short prompt: every expert's weights are read for a few tokens each.
        dict(name="moe_short_prompt", **_moe(192, 64, 6, 2560, 1408, 128, BF16, zp=True)),
        # A long prompt: large products.
        dict(name="moe_prompt", **_moe(4096, 128, 8, 2560, 768, 32, BF16)),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width over the logarithm of lo..hi: mostly multiples of 64, sometimes odd."""
    n = _log_int(rng, lo, hi)
    return n if rng.random() < 0.3 else max(64, n // 64 * 64)


def draw(rng):
    op = rng.choice(("route", "experts", "experts", "moe", "moe", "moe"))
    E = _log_int(rng, 4, 256)
    k = rng.randint(1, min(8, E))
    bs = rng.choice((16, 32, 32, 64, 128, 256))
    dtype = rng.choice((BF16, BF16, F32))
    if op == "route":
        return _route(_log_int(rng, 1, 32768), E, k, dtype, normalize=rng.random() < 0.7,
                      masked=rng.choice((0, 0, E // 8)))
    # fp32 activations belong to small batches; bf16 ones to every length.
    M = _log_int(rng, 1, 64 if dtype == F32 else 4096)
    zp, bias = rng.random() < 0.4, rng.random() < 0.3
    most = 4096 * 8 * 3 * 2560 * 768  # multiply-adds of the largest listed case
    wide = 128 * 3 * 2560 * 768       # weights of the largest listed case
    while True:
        H, I = _width(rng, 256, 4096), _width(rng, 128, 2816)
        if op == "experts" and M * k * H * I <= most and E * H * I <= wide:
            N, K = (H, I) if rng.random() < 0.5 else (I, H)
            return _experts(M, E, k, N, K, bs, dtype, zp=zp, bias=bias,
                            per_slot=rng.random() < 0.5, empty=rng.choice((0, M // 6)))
        if op == "moe" and M * k * 3 * H * I <= most and E * 3 * H * I <= wide:
            return _moe(M, E, k, H, I, bs, dtype, zp=zp, bias=bias,
                        normalize=rng.random() < 0.7)
        M = max(1, M // 2)


# ---- inputs ----------------------------------------------------------------------------------

def _weight(g, E, N, K, bs, dtype, zp):
    """A stack of E weights in the MatMulNBits storage: uniform codes, scales of a trained
    layer's size, and zero points or none (8). The scales have the activations' type."""
    nb = -(-K // bs)
    B = torch.randint(0, 256, (E, N, nb, bs // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.rand(E, N, nb, generator=g, device="cuda") * 0.015 + 0.005).to(dtype)
    # Trained codes are centred: zero points lie around the middle of 0..15.
    z = None
    if zp:
        lo, hi = (torch.randint(6, 11, (E, N, (nb + 1) // 2), generator=g, device="cuda",
                                dtype=torch.uint8) for _ in range(2))
        z = lo | (hi << 4)
    return dict(B=B, s=s, z=z, E=E, N=N, K=K, bs=bs)


def _bias(g, E, N):
    return torch.randn(E, N, generator=g, device="cuda") * 0.02


def _logits(g, M, E, dtype):
    """Router logits: spread over the tokens, with experts that are liked more than others."""
    liked = torch.randn(E, generator=g, device="cuda") * 0.3
    return (torch.randn(M, E, generator=g, device="cuda") + liked).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, M, E, k, dt = case, case["M"], case["E"], case["k"], DTYPES[case["dtype"]]
    st = dict(case)
    if c["op"] == "route":
        st["logits"] = _logits(g, M, E, dt)
        if c["masked"]:
            off = torch.randperm(E, generator=g, device="cuda")[:min(c["masked"], E - 1)]
            st["logits"][:, off] = -math.inf
        return st
    if c["op"] == "experts":
        ws = {"w": _weight(g, E, c["N"], c["K"], c["bs"], dt, c["zp"])}
        shape = (M, k, c["K"]) if c["per_slot"] else (M, c["K"])
        st["A"] = torch.randn(*shape, generator=g, device="cuda").to(dt)
        st["bias"] = _bias(g, E, c["N"]) if c["bias"] else None
        table = _logits(g, M, E, torch.float32).topk(k, dim=1).indices.to(torch.int32)
        if c["empty"]:  # padding tokens: no expert
            table[torch.randperm(M, generator=g, device="cuda")[:c["empty"]]] = -1
        st["table"] = table
    else:
        H, I = c["H"], c["I"]
        ws = {"gate": _weight(g, E, I, H, c["bs"], dt, c["zp"]),
              "up": _weight(g, E, I, H, c["bs"], dt, c["zp"]),
              "down": _weight(g, E, H, I, c["bs"], dt, c["zp"])}
        st["X"] = torch.randn(M, H, generator=g, device="cuda").to(dt)
        st["logits"] = _logits(g, M, E, torch.float32)
        st["bg"], st["bu"], st["bd"] = ((_bias(g, E, I), _bias(g, E, I), _bias(g, E, H))
                                        if c["bias"] else (None, None, None))
    if own:  # a program packs its weights once, when it loads them
        import int4_weight_only_matmulnbits_gb300 as mnb
        ws = {n: mnb.mnb_prepack_experts(w["B"], w["s"], w["z"], w["N"], w["K"], w["bs"])
              for n, w in ws.items()}
    st.update(ws)
    return st


# ---- plain form ------------------------------------------------------------------------------

def _plain_route(logits, k, normalize):
    x = logits.float()
    x = torch.where(torch.isnan(x), -math.inf, x)
    top, experts = torch.sort(x, dim=1, descending=True, stable=True)
    top, experts = top[:, :k], experts[:, :k]
    p = torch.exp(top - top[:, :1])
    all_p = torch.exp(x - top[:, :1])
    weights = p / (p if normalize else all_p).sum(1, keepdim=True)
    chosen = top > -math.inf
    weights = torch.where(chosen, weights, 0.0)
    experts = torch.where(chosen, experts, -1).to(torch.int32)
    return weights, experts


def _lists(experts, E):
    """Slots by expert: offsets [E + 1] and the slots in that order, those without one last."""
    e = experts.flatten().long()
    key = torch.where((e >= 0) & (e < E), e, E)
    order = torch.sort(key, stable=True).indices
    offsets = torch.searchsorted(key[order], torch.arange(E + 1, device=key.device))
    return key, offsets.to(torch.int32), order.to(torch.int32)


def _dequant(B, s, z, K):
    """(q - z) * s in 32 bits for any leading shape: B [.., nb, bs/2] -> [.., K]."""
    q = torch.stack((B & 15, B >> 4), -1).flatten(-2).float()
    if z is None:
        zero = torch.full_like(s, 8.0, dtype=torch.float32)
    else:
        zero = torch.stack((z & 15, z >> 4), -1).flatten(-2)[..., :s.shape[-1]].float()
    w = (q - zero.unsqueeze(-1)) * s.float().unsqueeze(-1)
    return w.flatten(-2)[..., :K]


def _plain_products(A, w, key, bias):
    """Rows A [P, K] through the expert each names in key [P] (E: none) -> [P, N] in 32 bits."""
    P, E, K = A.shape[0], w["E"], w["K"]
    some = (key < E).unsqueeze(1)
    e = key.clamp(max=E - 1)
    if P <= E:  # fewer rows than experts: only the weights the rows name
        z = None if w["z"] is None else w["z"][e]
        y = torch.bmm(_dequant(w["B"][e], w["s"][e], z, K), A.unsqueeze(2)).squeeze(2)
    else:       # each expert's rows side by side, padded to the longest list
        order = torch.sort(key, stable=True).indices
        first = torch.searchsorted(key[order], torch.arange(E + 1, device=key.device))
        room = max(1, int((first[1:] - first[:-1]).max()))
        rank = torch.empty_like(key)
        rank[order] = torch.arange(P, device=key.device) - first[key[order]]
        rank = rank.clamp(max=room - 1)
        rows = A.new_zeros(E * room, K)
        rows.index_add_(0, e * room + rank, torch.where(some, A, 0.0))
        full = torch.bmm(rows.view(E, room, K),
                         _dequant(w["B"], w["s"], w["z"], K).transpose(1, 2))
        y = full.view(E * room, -1)[e * room + rank]
    if bias is not None:
        y = y + bias[e]
    return torch.where(some, y, 0.0)


def _plain(st):
    k, E, M = st["k"], st["E"], st["M"]
    if st["op"] == "route":
        weights, experts = _plain_route(st["logits"], k, st["normalize"])
        _, offsets, order = _lists(experts, E)
        return weights, experts, offsets, order
    if st["op"] == "experts":
        A = st["A"].float()
        A = A.view(M * k, -1) if st["per_slot"] else A.repeat_interleave(k, 0)
        key, _, _ = _lists(st["table"], E)
        y = _plain_products(A, st["w"], key, st["bias"])
        return y.view(M, k, -1).to(st["A"].dtype)
    X = st["X"].float().repeat_interleave(k, 0)
    weights, experts = _plain_route(st["logits"], k, st["normalize"])
    key, _, _ = _lists(experts, E)
    g = _plain_products(X, st["gate"], key, st["bg"])
    u = _plain_products(X, st["up"], key, st["bu"])
    y = _plain_products(g / (1 + torch.exp(-g)) * u, st["down"], key, st["bd"])
    return (y.view(M, k, -1) * weights.unsqueeze(2)).sum(1).to(st["X"].dtype)


def run(state):
    if not own:
        return _plain(state)
    import int4_weight_only_matmulnbits_gb300 as mnb
    st = state
    if st["op"] == "route":
        r = mnb.mnb_moe_route(st["logits"], st["k"], normalize=st["normalize"])
        return r.weights, r.experts, r.offsets, r.order
    if st["op"] == "experts":
        return mnb.mnb_matmul_experts(st["A"], st["w"], st["table"], st["bias"])
    return mnb.mnb_moe(st["X"], st["logits"], st["gate"], st["up"], st["down"], st["k"],
                       normalize=st["normalize"], bias_gate=st["bg"], bias_up=st["bu"],
                       bias_down=st["bd"])


# ---- what a pass has to read, write and compute --------------------------------------------------

def _distinct(M, E, k):
    """Experts that M tokens of _logits' distribution name: the mean of a few trials."""
    if M * k >= 40 * E:
        return float(E)
    g = torch.Generator().manual_seed(1)
    n = 0
    for _ in range(8):
        x = torch.randn(M, E, generator=g) + torch.randn(E, generator=g) * 0.3
        n += x.topk(k, dim=1).indices.unique().numel()
    return n / 8


def work(case):
    c, M, E, k = case, case["M"], case["E"], case["k"]
    es = 2 if c["dtype"] == BF16 else 4
    if c["op"] == "route":
        return {"bytes": M * E * es + M * k * 12 + (E + 1) * 4, "flops": 4 * M * E}
    rows = M - c.get("empty", 0)
    d = _distinct(rows, E, k)

    def weight(N, K):
        nb = -(-K // c["bs"])
        return N * (K / 2 + nb * es + (nb / 2 if c["zp"] else 0) + (4 if c["bias"] else 0))

    if c["op"] == "experts":
        a = rows * (k if c["per_slot"] else 1) * c["K"] * es
        return {"bytes": d * weight(c["N"], c["K"]) + a + M * k * (c["N"] * es + 4),
                "flops": 2 * rows * k * c["N"] * c["K"]}
    H, I = c["H"], c["I"]
    return {"bytes": d * (2 * weight(I, H) + weight(H, I)) + 2 * M * H * es + M * E * 4,
            "flops": 6 * M * k * H * I}


# ---- the definition in 64 bits --------------------------------------------------------------------

def _codes64(w, e):
    """Expert e's matrix [N, K] in 64 bits, element by element of the definition."""
    K, bs = w["K"], w["bs"]
    i = torch.arange(K, device="cuda")
    byte = w["B"][e].reshape(w["N"], -1)[:, i // 2].long()
    q = (byte >> (4 * (i % 2))) & 15
    b = i // bs
    z = 8 if w["z"] is None else (w["z"][e].long()[:, b // 2] >> (4 * (b % 2))) & 15
    return (q - z).double() * w["s"][e].double()[:, b]


def _choice64(logits, k, normalize):
    """Choices (expert, weight) by repeated maximum, on the host in 64 bits."""
    x = logits.double().cpu().numpy().copy()
    rows = np.arange(x.shape[0])
    best = x.max(1, keepdims=True)
    p = np.exp(x - best)
    total = p.sum(1)
    experts = np.empty((x.shape[0], k), np.int64)
    weights = np.zeros((x.shape[0], k))
    for j in range(k):
        i = x.argmax(1)
        ok = x[rows, i] > -np.inf
        experts[:, j] = np.where(ok, i, -1)
        weights[:, j] = np.where(ok, p[rows, i], 0)
        x[rows, i] = -np.inf
    weights /= weights.sum(1, keepdims=True) if normalize else total[:, None]
    return experts, weights


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    M, E, k = st["M"], st["E"], st["k"]
    if st["op"] == "route":
        _, weights = _choice64(st["logits"], k, st["normalize"])
        return torch.from_numpy(weights), None, None, None
    if st["op"] == "experts":
        table = st["table"].long().cpu()
        A = st["A"].double()
        y = torch.zeros(M, k, st["N"], device="cuda", dtype=torch.float64)
        for e in range(E):
            m, j = (t.cuda() for t in torch.nonzero(table == e, as_tuple=True))
            if len(m):
                rows = A[m, j] if st["per_slot"] else A[m]
                y[m, j] = rows @ _codes64(st["w"], e).T
                if st["bias"] is not None:
                    y[m, j] += st["bias"][e].double()
        return y
    experts, weights = (torch.from_numpy(v) for v in _choice64(st["logits"], k, st["normalize"]))
    X = st["X"].double()
    y = torch.zeros(M, st["H"], device="cuda", dtype=torch.float64)
    bias = lambda b, e: 0.0 if b is None else b[e].double()  # noqa: E731
    for e in range(E):
        m, j = torch.nonzero(experts == e, as_tuple=True)
        if len(m):
            w = weights[m, j].cuda().unsqueeze(1)
            m = m.cuda()
            g = X[m] @ _codes64(st["gate"], e).T + bias(st["bg"], e)
            u = X[m] @ _codes64(st["up"], e).T + bias(st["bu"], e)
            h = g * torch.sigmoid(g) * u
            y[m] += w * (h @ _codes64(st["down"], e).T + bias(st["bd"], e))
    return y
