"""Operators of the attention block around the 4-bit projections: what is timed, on which inputs,
and the plain statement of each operator that the kernels are held to.

Four operators, each through the calls a user makes (``own``) or in elementary torch operations:

* ``table``: cosines and sines of rotary positions, frequencies scaled for long contexts or not;
* ``rope``: norms of queries and keys for each head, with the position rotation in the same pass;
* ``append``: the same on the rows of the fused q, k, v projection, with keys and values going
  into a paged cache;
* ``attend``: attention of each sequence's new tokens over its pages of the cache.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "fp32"
DTYPES = {BF16: torch.bfloat16, F32: torch.float32}
EPS = 1e-6


# ---- cases -----------------------------------------------------------------------------------

def _table(n, rot, base, factor=1.0, original=0.0, low=1.0, high=32.0, magnitude=1.0):
    return dict(op="table", n=n, rot=rot, base=base, factor=factor, original=original, low=low,
                high=high, magnitude=magnitude)


def _rope(T, hq, hk, D, dtype, rot=None, interleaved=False, norm=True, positions=40960):
    return dict(op="rope", T=T, hq=hq, hk=hk, D=D, dtype=dtype, rot=rot or D,
                interleaved=interleaved, norm=norm, positions=positions)


def _append(news, lens, hq, hk, D, page, dtype, rot=None, interleaved=False, norm=True):
    """news, lens: tokens that each sequence adds, and its length with them, as texts."""
    return dict(op="append", news=_text(news), lens=_text(lens), hq=hq, hk=hk, D=D, page=page,
                dtype=dtype, rot=rot or D, interleaved=interleaved, norm=norm)


def _attend(news, lens, hq, hk, D, page, dtype, window=0):
    return dict(op="attend", news=_text(news), lens=_text(lens), hq=hq, hk=hk, D=D, page=page,
                dtype=dtype, window=window)


def _text(values):
    return ",".join(str(v) for v in values)


def _ints(text):
    return [int(v) for v in text.split(",")]


def _spread(n, lo, hi):
    """n lengths over the logarithm of lo..hi, in no order of size."""
    return [int(lo * (hi / lo) ** (((i * 37) % n + 0.5) / n)) for i in range(n)]


def listed():
    return [
        # The tables of a model of 40960 positions, made when it is loaded.
        dict(name="table_plain", **_table(40960, 128, 1e6)),
        # Tables for a context stretched four and a half times, by the parts of the spectrum.
        dict(name="table_stretched", **_table(147457, 128, 1e6, factor=4.5, original=32768.0,
                                              magnitude=1.15)),
        # One token of a decode step, into a caller's own cache: latency alone.
        dict(name="rope_one", **_rope(1, 32, 8, 128, BF16)),
        # A prompt of an fp32 model with neighbouring pairs rotated in half of each head.
        dict(name="rope_prompt_fp32", **_rope(16411, 16, 8, 64, F32, rot=32, interleaved=True,
                                              norm=False)),
        # One token of a decode step: norms, rotation and the cache in one go.
        dict(name="append_one", **_append([1], [2001], 32, 8, 128, 16, BF16)),
        # A decode batch of sequences of every length.
        dict(name="append_batch", **_append([1] * 64, _spread(64, 100, 16000), 32, 8, 128, 16,
                                            BF16)),
        # Three prompts of a step, one of them the second half of a longer one.
        dict(name="append_prompt", **_append([9000, 5123, 2261], [9000, 11123, 2261], 32, 8, 128,
                                             64, BF16)),
        # One decode token over a few thousand: latency.
        dict(name="attend_one", **_attend([1], [4097], 32, 8, 128, 16, BF16)),
        # The same of a small fp32 model.
        dict(name="attend_one_fp32", **_attend([1], [2049], 16, 8, 128, 16, F32)),
        # A decode batch: the cache is read once.
        dict(name="attend_batch", **_attend([1] * 64, _spread(64, 500, 32000), 32, 8, 128, 16,
                                            BF16)),
        # A chunk of a long prompt beside seven decoding sequences, odd lengths.
        dict(name="attend_chunk", **_attend([515] + [1] * 7, [17003] + _spread(7, 300, 9000), 32,
                                            8, 128, 32, BF16)),
        # Whole prompts: large products.
        dict(name="attend_prompt", **_attend([9000, 5123, 2261], [9000, 5123, 2261], 32, 8, 128,
                                             64, BF16)),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _pairs(news, lens, window):
    """Attended (query, key) pairs of a batch, and the keys that any query attends."""
    pairs = keys = 0
    for n, L in zip(news, lens):
        w = min(window or L, L)
        full = min(n, L - w + 1)  # queries that attend a whole window, the last ones
        ramp = n - full           # the others, from position L - n on, attend all before them
        pairs += ramp * (L - n) + ramp * (ramp + 1) // 2 + full * w
        keys += min(L, n + w - 1)
    return pairs, keys


def draw(rng):
    op = rng.choice(("table", "rope", "append", "append", "attend", "attend", "attend", "attend"))
    if op == "table":
        rot = rng.choice((16, 32, 64, 80, 96, 128))
        most = 147457 * 128
        n = _log_int(rng, 1000, most // rot)
        if rng.random() < 0.5:
            return _table(n, rot, rng.choice((1e4, 5e5, 1e6)))
        return _table(n, rot, rng.choice((1e4, 5e5, 1e6)), factor=rng.uniform(1.5, 16),
                      original=rng.choice((0.0, 4096.0, 8192.0)), low=rng.choice((1.0, 1.0, 2.0)),
                      high=rng.choice((4.0, 32.0)), magnitude=rng.choice((1.0, 1.2)))
    D = rng.choice((64, 128, 128))
    dtype = rng.choice((BF16, BF16, BF16, F32))
    hk = rng.choice((1, 2, 4, 8, 8))
    hq = hk * rng.choice((1, 2, 3, 4, 4, 5, 7, 8))
    rot, inter, norm = rng.choice((D, D, D // 2)), rng.random() < 0.3, rng.random() < 0.7
    if op == "rope":
        T = _log_int(rng, 1, 16384)
        while T > 1 and T * (hq + hk) * D > 16000 * 24 * 64:
            T = (T + 1) // 2
        return _rope(T, hq, hk, D, dtype, rot, inter, norm)
    page = rng.choice((16, 16, 32, 64, 128, 256))
    window = rng.choice((0, 0, 0, _log_int(rng, 1, 8192))) if op == "attend" else 0
    B = _log_int(rng, 1, 64)
    kind = rng.choice(("decode", "decode", "few", "mixed", "prompts"))
    if kind in ("mixed", "prompts"):
        B = min(B, 16)
    lens = [_log_int(rng, 1, 32000) for _ in range(B)]
    if kind == "decode":
        news = [1] * B
    elif kind == "few":      # drafted tokens to verify
        news = [min(L, rng.randint(1, 9)) for L in lens]
    elif kind == "mixed":    # a chunk or two among decoding sequences, some with nothing new
        news = [min(L, rng.choice((0, 1, 1, _log_int(rng, 2, 2048)))) for L in lens]
        news[0] = max(1, news[0])
    else:
        lens = [min(L, 8192) for L in lens]
        news = list(lens)
    while True:
        pairs, keys = _pairs(news, lens, window)
        flops, rows = 4 * pairs * hq * D, sum(news) * (hq + 2 * hk) * D
        # fp32 activations belong to small batches; bf16 ones to every length.
        if (flops <= (2e10 if dtype == F32 else 9e11) and rows <= 16384 * 48 * 128
                and keys * hk * D <= 460000 * 8 * 128):
            break
        news = [max(min(n, 1), n // 2) for n in news]
        lens = [max(n, 1, (L + 1) // 2) for n, L in zip(news, lens)]
    if op == "append":
        return _append(news, lens, hq, hk, D, page, dtype, rot, inter, norm)
    return _attend(news, lens, hq, hk, D, page, dtype, window)


# ---- inputs ----------------------------------------------------------------------------------

def _positions_table(n, rot):
    """The cosines and sines a program holds: from angles in 64 bits."""
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    a = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * 1e6 ** (-2 * i / rot)
    return torch.cos(a).float(), torch.sin(a).float()


def _gammas(g, c):
    if not c["norm"]:
        return None, None
    return tuple(1 + 0.2 * torch.randn(c["D"], generator=g, device="cuda") for _ in range(2))


def _pages(g, c, lens):
    """A cache with pages in no order and some to spare, and the table of each sequence's pages."""
    page, B = c["page"], len(lens)
    need = [-(-L // page) for L in lens]
    total = sum(need) + B + 3
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    width = max(need) + 1
    table = torch.full((B, width), -1, dtype=torch.int32)
    at, order = 0, order.cpu()
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    shape = (total, c["hk"], page, c["D"])
    k, v = (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(
        DTYPES[c["dtype"]]) for _ in range(2))
    return k, v, table.cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = case
    st = dict(c)
    if c["op"] == "table":
        # Other inputs for another seed: a base that differs in its last digits.
        st["base"] = c["base"] * (1 + (seed % 1009) * 1e-6)
        st["frequencies"] = torch.tensor(_frequencies(dict(c, base=st["base"])),
                                         dtype=torch.float64)
        return st
    dt, D, hq, hk = DTYPES[c["dtype"]], c["D"], c["hq"], c["hk"]
    if c["op"] == "attend":
        news, lens = _ints(c["news"]), _ints(c["lens"])
        k, v, table = _pages(g, c, lens)
        # Heads that look at a few tokens and heads that look at many.
        gain = torch.exp(torch.linspace(-0.7, 1.4, hq, device="cuda"))[:, None]
        st["q"] = (torch.randn(sum(news), hq, D, generator=g, device="cuda") * gain).to(dt)
        _batch(st, k, v, table, news, lens)
        return st
    T = c["T"] if c["op"] == "rope" else sum(_ints(c["news"]))
    # The fused projection's rows: the operators read them where they are.
    st["rows"] = torch.randn(T, (hq + 2 * hk) * D, generator=g, device="cuda").to(dt)
    st["gq"], st["gk"] = _gammas(g, c)
    if c["op"] == "rope":
        st["positions"] = torch.randint(0, c["positions"], (T,), generator=g, device="cuda",
                                        dtype=torch.int32)
        cos, sin = _positions_table(c["positions"], c["rot"])
    else:
        news, lens = _ints(c["news"]), _ints(c["lens"])
        k, v, table = _pages(g, c, lens)
        _batch(st, k, v, table, news, lens)
        cos, sin = _positions_table(max(max(lens), 2), c["rot"])
    st["cos"], st["sin"] = cos, sin
    if own:
        import int4_weight_only_matmulnbits_gb300 as mnb
        st["rope"] = mnb.RopeTable(cos, sin)
    return st


def _batch(st, k, v, table, news, lens):
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    st.update(k=k, v=v, table=table, starts_list=starts, lens_list=lens,
              starts=torch.tensor(starts, dtype=torch.int32, device="cuda"),
              lengths=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    if own:
        import int4_weight_only_matmulnbits_gb300 as mnb
        st["cache"] = mnb.KvCache(k, v)
        st["batch"] = mnb.KvBatch(st["starts"], st["lengths"], table)


def _frequencies(c):
    """Angle per position of each pair: plain, all slowed by a factor, or slowed by parts (the
    fast ones not, the slow ones whole, a ramp over the turns within the original length)."""
    out = []
    for i in range(c["rot"] // 2):
        f = c["base"] ** (-2.0 * i / c["rot"])
        keep = 0.0
        if c["original"]:
            turns = c["original"] * f / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - c["low"]) / (c["high"] - c["low"])))
        out.append((1 - keep) * f / c["factor"] + keep * f)
    return out


# ---- plain form ------------------------------------------------------------------------------

def _norm_rotate(x, gamma, cos, sin, rot, interleaved):
    """x [T, H, D] in 32 bits; cos, sin [T, rot / 2] of the rows' positions."""
    if gamma is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma
    r, rest = x[..., :rot], x[..., rot:]
    c, s = cos[:, None], sin[:, None]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((r, rest), -1)


def _split(st):
    hq, hk, D = st["hq"], st["hk"], st["D"]
    rows = st["rows"].view(-1, hq + 2 * hk, D)
    return rows[:, :hq], rows[:, hq:hq + hk], rows[:, hq + hk:]


def _places(st):
    """Position, page and place in the page of each new token."""
    news = [b - a for a, b in zip(st["starts_list"], st["starts_list"][1:])]
    seq = torch.repeat_interleave(torch.arange(len(news), device="cuda"),
                                  torch.tensor(news, device="cuda"), output_size=sum(news))
    pos = (torch.arange(sum(news), device="cuda") - st["starts"].long()[seq + 1]
           + st["lengths"].long()[seq])
    return pos, st["table"].long()[seq, pos // st["page"]], pos % st["page"]


def _plain_attend(st):
    q, hk, D = st["q"], st["hk"], st["D"]
    G = st["hq"] // hk
    out = torch.empty_like(q)
    for b, L in enumerate(st["lens_list"]):
        t0, t1 = st["starts_list"][b:b + 2]
        n = t1 - t0
        if n == 0:
            continue
        pages = st["table"][b, :-(-L // st["page"])].long()
        keys, values = (x[pages].transpose(0, 1).reshape(hk, -1, D)[:, :L].float()
                        for x in (st["k"], st["v"]))
        rows = q[t0:t1].float().view(n, hk, G, D).permute(1, 2, 0, 3)  # [hk, G, n, D]
        p, j = torch.arange(L - n, L, device="cuda")[:, None], torch.arange(L, device="cuda")
        hidden = j > p
        if st["window"]:
            hidden |= j <= p - st["window"]
        # All heads of a short sequence at a time, else the queries of one key head.
        for h in range(0, hk, hk if hk * G * n * L < 1 << 28 else 1):
            h1 = hk if hk * G * n * L < 1 << 28 else h + 1
            r, k, v = rows[h:h1], keys[h:h1, None], values[h:h1, None]
            s = (r @ k.transpose(-1, -2)) * (1 / math.sqrt(D))
            s.masked_fill_(hidden, -math.inf)
            s = torch.exp(s - s.amax(-1, keepdim=True))
            o = (s @ v) / s.sum(-1, keepdim=True)
            out[t0:t1].view(n, hk, G, D)[:, h:h1] = o.permute(2, 0, 1, 3).to(q.dtype)
    return out


def _plain(st):
    if st["op"] == "attend":
        return _plain_attend(st)
    if st["op"] == "table":
        n = torch.arange(st["n"], device="cuda", dtype=torch.float64)
        a = n[:, None] * st["frequencies"].cuda()
        return (torch.cos(a) * st["magnitude"]).float(), (torch.sin(a) * st["magnitude"]).float()
    q, k, v = _split(st)
    dt = q.dtype
    if st["op"] == "rope":
        cos, sin = st["cos"][st["positions"].long()], st["sin"][st["positions"].long()]
    else:
        pos, page, at = _places(st)
        cos, sin = st["cos"][pos], st["sin"][pos]
    q = _norm_rotate(q.float(), st["gq"], cos, sin, st["rot"], st["interleaved"]).to(dt)
    k = _norm_rotate(k.float(), st["gk"], cos, sin, st["rot"], st["interleaved"]).to(dt)
    if st["op"] == "rope":
        return q, k
    st["k"][page, :, at] = k
    st["v"][page, :, at] = v
    return q, st["k"], st["v"]


def run(state):
    st = state
    if not own:
        return _plain(st)
    import int4_weight_only_matmulnbits_gb300 as mnb
    if st["op"] == "table":
        r = mnb.mnb_rope_table(st["frequencies"], st["n"], magnitude=st["magnitude"])
        return r.cos, r.sin
    if st["op"] == "attend":
        return mnb.mnb_paged_attention(st["q"], st["cache"], st["batch"], window=st["window"])
    q, k, v = _split(st)
    if st["op"] == "rope":
        return mnb.mnb_qk_norm_rope(q, k, st["rope"], st["positions"], gamma_q=st["gq"],
                                    gamma_k=st["gk"], eps=EPS, interleaved=st["interleaved"])
    q = mnb.mnb_cache_append(q, k, v, st["cache"], st["batch"], st["rope"], gamma_q=st["gq"],
                             gamma_k=st["gk"], eps=EPS, interleaved=st["interleaved"])
    return q, st["k"], st["v"]


# ---- what a pass has to read, write and compute --------------------------------------------------

def work(case):
    c = case
    if c["op"] == "table":
        return {"bytes": c["n"] * c["rot"] * 4, "flops": c["n"] * c["rot"] * 20}
    es, D, hq, hk = (2 if c["dtype"] == BF16 else 4), c["D"], c["hq"], c["hk"]
    if c["op"] == "rope":
        n = c["T"] * (hq + hk) * D
        return {"bytes": 2 * n * es + c["T"] * (4 + c["rot"] * 4), "flops": 8 * n}
    news, lens = _ints(c["news"]), _ints(c["lens"])
    T = sum(news)
    if c["op"] == "append":
        n = T * (hq + 2 * hk) * D
        return {"bytes": 2 * n * es + T * c["rot"] * 4 + 12 * len(lens), "flops": 8 * n}
    pairs, keys = _pairs(news, lens, c["window"])
    return {"bytes": 2 * keys * hk * D * es + 2 * T * hq * D * es
            + 4 * (keys // c["page"] + 2 * len(lens)), "flops": 4 * pairs * hq * D}


# ---- the definition in 64 bits --------------------------------------------------------------------

def _turned64(x, gamma, cos, sin, rot, interleaved):
    """Norm and rotation of x [T, H, D], pair by pair as a complex product."""
    x = x.double()
    if gamma is not None:
        x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * gamma.double()
    i = torch.arange(rot // 2, device=x.device)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    z = torch.complex(x[..., ia], x[..., ib]) * torch.complex(cos.double(), sin.double())[:, None]
    y = x.clone()
    y[..., ia], y[..., ib] = z.real, z.imag
    return y


def _attend64(st):
    q, D, page = st["q"], st["D"], st["page"]
    G = st["hq"] // st["hk"]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    for b, L in enumerate(st["lens_list"]):
        t0, t1 = st["starts_list"][b:b + 2]
        j = torch.arange(L, device="cuda")
        where = st["table"][b].long()[j // page]
        for h in range(st["hk"]):
            keys, values = (x[where, h, j % page].double() for x in (st["k"], st["v"]))
            for head in range(h * G, h * G + G):
                for r0 in range(t0, t1, 2048):
                    r1 = min(t1, r0 + 2048)
                    p = L - t1 + torch.arange(r0, r1, device="cuda")
                    back = p[:, None] - j
                    seen = (back >= 0) & (back < (st["window"] or L))
                    s = q[r0:r1, head].double() @ keys.T / math.sqrt(D)
                    w = torch.softmax(torch.where(seen, s, -math.inf), 1)
                    out[r0:r1, head] = w @ values
    return out


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    if st["op"] == "attend":
        return _attend64(st)
    if st["op"] == "table":
        angle = torch.outer(torch.arange(st["n"], dtype=torch.float64, device="cuda"),
                            torch.tensor(_frequencies(st), dtype=torch.float64, device="cuda"))
        z = torch.polar(torch.full_like(angle, st["magnitude"]), angle)
        return z.real, z.imag
    q, k, v = _split(st)
    pos = st["positions"].long() if st["op"] == "rope" else _places(st)[0]
    args = (st["cos"][pos], st["sin"][pos], st["rot"], st["interleaved"])
    q, k = _turned64(q, st["gq"], *args), _turned64(k, st["gk"], *args)
    if st["op"] == "rope":
        return q, k
    kc, vc = st["k"].double(), st["v"].double()
    for b, L in enumerate(st["lens_list"]):
        t0, t1 = st["starts_list"][b:b + 2]
        j = torch.arange(L - (t1 - t0), L, device="cuda")
        where = st["table"][b].long()[j // st["page"]]
        kc[where, :, j % st["page"]] = k[t0:t1]
        vc[where, :, j % st["page"]] = v[t0:t1].double()
    return q, kc, vc
