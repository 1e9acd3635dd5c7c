"""The attention block's operators on the GPU against their 64-bit definitions
(tests/attn_reference.py, with bounds counted from the kernels' roundings)."""
import math

import pytest
import torch

import int4_weight_only_matmulnbits_gb300 as mnb
from tests import attn_reference as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    mnb.build_library()
    mnb.load()
    return torch.device("cuda:0")


@pytest.fixture(autouse=True)
def no_wait_ran_out(dev):
    yield
    assert mnb.mnb_fault_status() == 0


def within(got, want, bound):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), "not finite"
    over = ((got - want).abs() / bound).max().item()
    assert over <= 1, f"error {over:.3g} of its bound"


def tables(n, rot, base=1e4):
    f = torch.tensor(ref.frequencies(rot, base), dtype=torch.float64)
    a = torch.arange(n, dtype=torch.float64)[:, None] * f
    return torch.cos(a).float(), torch.sin(a).float()


# ---- tables --------------------------------------------------------------------------------------

@pytest.mark.parametrize("rot,first,n,mag", [
    (128, 0, 4096, 1.0), (64, 2 ** 31 - 1000, 999, 1.0), (6, 12345, 77, 1.15), (2, 0, 1, 0.7),
    (256, 1 << 20, 300, 1.0), (80, 999_983, 501, 3.0)])
def test_tables(dev, rot, first, n, mag):
    """Within 2^-22 of themselves: the angle is kept to 2^-53 of frequency times position, sine and
    cosine round a few times in fp32, the magnitude once."""
    f = mnb.mnb_rope_frequencies(rot, 1e6, factor=3.0, original=4096.0)
    t = mnb.mnb_rope_table(f, n, first=first, magnitude=mag, device=dev)
    a = torch.arange(first, first + n, dtype=torch.float64)[:, None] * f
    slack = 2.0 ** -52 * (a + 1) * mag  # of the angle: the reference's product rounds as well
    for got, want in ((t.cos, torch.cos(a) * mag), (t.sin, torch.sin(a) * mag)):
        assert got.shape == (n, rot // 2) and got.dtype == F32
        within(got, want, 2.0 ** -22 * want.abs() + 4 * slack + 1e-30)


def test_tables_of_odd_frequencies(dev):
    """Negative, large and zero frequencies, and near multiples of a quarter turn."""
    f = torch.tensor([-0.3, 7.0, 0.0, math.pi / 2, -math.pi, 1e3], dtype=torch.float64)
    t = mnb.mnb_rope_table(f, 2000, device=dev)
    a = torch.arange(2000, dtype=torch.float64)[:, None] * f
    slack = 2.0 ** -50 * (a.abs() + 1)
    within(t.cos, torch.cos(a), 2.0 ** -22 * torch.cos(a).abs() + slack)
    within(t.sin, torch.sin(a), 2.0 ** -22 * torch.sin(a).abs() + slack)


# ---- norms and rotation --------------------------------------------------------------------------

def rows(g, T, n, D, dtype, layout="plain", spread=1.0):
    """[T, n, D] values in one of the layouts a projection may leave: plain, slices of wider rows,
    head-major, or off 16 bytes by one element."""
    x = (torch.randn(T, n, D, generator=g) * spread).to(dtype)
    if layout == "plain":
        return x.cuda()
    if layout == "slice":
        wide = torch.full((T, n + 3, D), NAN, dtype=dtype, device="cuda")
        wide[:, 1:n + 1] = x.cuda()
        return wide[:, 1:n + 1]
    if layout == "head_major":
        return x.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    flat = torch.full((T * n * D + 1,), NAN, dtype=dtype, device="cuda")
    flat[1:] = x.flatten().cuda()
    return flat[1:].view(T, n, D)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,hq,hk,D,rot,inter,norm,layout", [
    (1, 32, 8, 128, 128, False, True, "slice"), (1, 1, 1, 2, 2, True, True, "plain"),
    (5, 16, 8, 128, 64, False, True, "slice"), (7, 3, 1, 64, 64, True, True, "plain"),
    (33, 4, 2, 80, 80, False, True, "plain"), (3, 2, 2, 96, 32, True, False, "head_major"),
    (4, 5, 5, 256, 256, False, True, "plain"), (6, 6, 2, 64, 16, False, False, "odd"),
    (9, 2, 1, 30, 10, False, True, "plain"), (2, 4, 4, 128, 128, True, True, "odd"),
    (3, 40, 8, 32, 32, False, True, "slice"), (2, 3, 3, 254, 254, True, True, "plain")])
def test_norm_and_rotation(dev, T, hq, hk, D, rot, inter, norm, layout, dtype):
    g = torch.Generator().manual_seed(T * 1000 + D)
    q, k = rows(g, T, hq, D, dtype, layout, 3.0), rows(g, T, hk, D, dtype, layout)
    gq, gk = (1 + 0.3 * torch.randn(D, generator=g) for _ in range(2)) if norm else (None, None)
    cos, sin = tables(50, rot)
    pos = torch.randint(0, 50, (T,), generator=g, dtype=torch.int32)
    if T > 3:
        pos[1], pos[2], pos[3] = -1, 50, 2 ** 31 - 1  # no such position: zeros
    up = lambda t: None if t is None else t.to(dev)  # noqa: E731
    yq, yk = mnb.mnb_qk_norm_rope(q, k, mnb.RopeTable(up(cos), up(sin)), up(pos), gamma_q=up(gq),
                                  gamma_k=up(gk), eps=1e-5, interleaved=inter)
    for x, gamma, y in ((q, gq, yq), (k, gk, yk)):
        want, mag = ref.norm_rotate(x.cpu(), gamma, 1e-5, cos, sin, pos, inter)
        within(y, want, ref.norm_rotate_bound(want, mag, D, dtype, norm))
        if T > 3:
            assert not y[1:4].any()


@pytest.mark.parametrize("D,layout", [(128, "slice"), (64, "plain"), (30, "odd")])
def test_norm_and_rotation_in_place(dev, D, layout):
    """In place equals apart, bit for bit; what lies around the rows stays."""
    g = torch.Generator().manual_seed(5)
    q, k = rows(g, 11, 6, D, BF16, layout), rows(g, 11, 2, D, BF16, layout)
    r = mnb.RopeTable(*(t.to(dev) for t in tables(64, D)))
    pos = torch.arange(11, dtype=torch.int32, device=dev)
    gamma = torch.rand(D, generator=g).to(dev)
    yq, yk = mnb.mnb_qk_norm_rope(q, k, r, pos, gamma_q=gamma, gamma_k=gamma)
    zq, zk = mnb.mnb_qk_norm_rope(q, k, r, pos, gamma_q=gamma, gamma_k=gamma, out_q=q, out_k=k)
    assert zq is q and zk is k and torch.equal(yq, q) and torch.equal(yk, k)


def test_one_of_a_kind(dev):
    """Queries alone, a norm of one side only, a norm without rotation, nothing at all."""
    g = torch.Generator().manual_seed(6)
    q, k = rows(g, 4, 3, 64, F32), rows(g, 4, 1, 64, F32)
    cos, sin = tables(9, 64)
    r, pos = mnb.RopeTable(cos.to(dev), sin.to(dev)), torch.tensor([0, 8, 3, 3], dtype=torch.int32)
    gamma = torch.rand(64, generator=g)
    yq, none = mnb.mnb_qk_norm_rope(q, None, r, pos.to(dev))
    assert none is None
    want, mag = ref.norm_rotate(q.cpu(), None, 1e-6, cos, sin, pos, False)
    within(yq, want, ref.norm_rotate_bound(want, mag, 64, F32, False))
    yq, yk = mnb.mnb_qk_norm_rope(q, k, None, None, gamma_k=gamma.to(dev))
    assert torch.equal(yq, q)
    want, mag = ref.norm_rotate(k.cpu(), gamma, 1e-6, None, None, pos, False)
    within(yk, want, ref.norm_rotate_bound(want, mag, 64, F32, True))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("inter,norm", [(False, True), (True, False)])
def test_many_rows_equal_few(dev, inter, norm, dtype):
    """Thousands of rows (several heads a group of lanes) bit for bit as the same rows in small
    calls, for odd counts of heads."""
    g = torch.Generator().manual_seed(7)
    T, hq, hk, D = 4801, 29, 7, 128
    qkv = torch.randn(T, hq + 2 * hk, D, generator=g).to(dtype).to(dev)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    r = mnb.RopeTable(*(t.to(dev) for t in tables(4900, 64)))
    pos = torch.randint(0, 4900, (T,), generator=g, dtype=torch.int32).to(dev)
    gamma = torch.rand(D, generator=g).to(dev) if norm else None
    kw = dict(gamma_q=gamma, gamma_k=gamma, interleaved=inter)
    yq, yk = mnb.mnb_qk_norm_rope(q, k, r, pos, **kw)
    # Three sequences, the second one with nothing new, 40 rows behind the last.
    starts, lens = [0, 4000, 4000, T - 40], [4000, 5, 861]
    ps = 256
    _, table, pages, _ = make_batch(g, [4000, 0, 761], lens, ps)
    cache = make_cache(g, pages, hk, ps, D, dtype)
    k0, v0 = cache.k.clone(), cache.v.clone()
    out = torch.full_like(yq, 7.0)
    mnb.mnb_cache_append(q, k, v, cache, on_gpu(starts, lens, table), r, out=out, **kw)
    assert torch.all(out[T - 40:] == 7.0)
    for a in range(0, T, 1000):
        zq, zk = mnb.mnb_qk_norm_rope(q[a:a + 50], k[a:a + 50], r, pos[a:a + 50], **kw)
        assert torch.equal(zq, yq[a:a + 50]) and torch.equal(zk, yk[a:a + 50])
    where = torch.tensor([p for _, p, _, _ in ref.places(starts, lens, table, ps, pages, T)],
                         dtype=torch.int32).to(dev)
    zq, zk = mnb.mnb_qk_norm_rope(q[:T - 40], k[:T - 40], r, where, **kw)
    assert torch.equal(out[:T - 40], zq)
    for t, _, page, at in ref.places(starts, lens, table, ps, pages, T):
        k0[page, :, at], v0[page, :, at] = zk[t], v[t]
    assert torch.equal(cache.k, k0) and torch.equal(cache.v, v0)


def test_rows_of_zeros_and_a_row_of_nan(dev):
    q = torch.zeros(3, 2, 128, device=dev, dtype=BF16)
    q[1, 1, 5] = NAN
    gamma = torch.ones(128, device=dev)
    y, _ = mnb.mnb_qk_norm_rope(q, None, None, None, gamma_q=gamma)
    assert not y[0].any() and not y[2].any() and not y[1, 0].any() and y[1, 1].isnan().all()


# ---- appending -----------------------------------------------------------------------------------

def make_cache(g, pages, H, ps, D, dtype, layout="heads_first", fill=None):
    """Pages [pages, H, ps, D] with heads or tokens first in memory, or keys and values beside one
    another."""
    if layout == "tokens_first":
        k, v = (torch.empty(pages, ps, H, D, dtype=dtype, device="cuda").transpose(1, 2)
                for _ in range(2))
    elif layout == "beside":
        both = torch.empty(pages, 2, H, ps, D, dtype=dtype, device="cuda")
        k, v = both[:, 0], both[:, 1]
    else:
        k, v = (torch.empty(pages, H, ps, D, dtype=dtype, device="cuda") for _ in range(2))
    for t in (k, v):
        t.copy_(torch.randn(t.shape, generator=g).to(dtype) if fill is None else
                torch.full(t.shape, fill, dtype=dtype))
    return mnb.KvCache(k, v)


def make_batch(g, news, lens, ps, spare=3, width=None, rows_behind=0):
    need = [-(-max(L, 0) // ps) for L in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), width or max(need + [1])), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    return starts, table, pages, starts[-1] + rows_behind


def on_gpu(starts, lens, table):
    i = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    return mnb.KvBatch(i(starts), i(lens), table.cuda())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("news,lens,hq,H,D,rot,inter,norm,ps,layout,cl", [
    ([1], [1], 4, 2, 128, 128, False, True, 16, "slice", "heads_first"),
    ([1], [2001], 32, 8, 128, 128, False, True, 16, "slice", "heads_first"),
    ([1, 0, 3, 17, 0], [33, 5, 3, 64, 0], 6, 2, 64, 32, True, True, 32, "plain", "tokens_first"),
    ([5, 1], [49, 16], 3, 1, 80, 80, False, False, 16, "plain", "beside"),
    ([40], [40], 2, 2, 30, 30, False, True, 16, "odd", "tokens_first"),
    ([1] * 70, list(range(1, 71)), 2, 1, 64, 64, False, True, 48, "slice", "heads_first"),
    ([2, 9], [700, 9], 8, 8, 256, 128, False, True, 1024, "plain", "heads_first")])
def test_append(dev, news, lens, hq, H, D, rot, inter, norm, ps, layout, cl, dtype):
    g = torch.Generator().manual_seed(len(news) * 100 + D)
    starts, table, pages, T = make_batch(g, news, lens, ps, rows_behind=2)
    cache = make_cache(g, pages, H, ps, D, dtype, cl)
    q, k, v = (rows(g, T, n, D, dtype, layout) for n in (hq, H, H))
    gq, gk = (1 + 0.3 * torch.randn(D, generator=g) for _ in range(2)) if norm else (None, None)
    cos, sin = tables(max(lens) + 1, rot)
    up = lambda t: None if t is None else t.to(dev)  # noqa: E731
    k0, v0 = cache.k.clone(), cache.v.clone()
    out = torch.full((T, hq, D), 7.0, dtype=dtype, device=dev)
    y = mnb.mnb_cache_append(q, k, v, cache, on_gpu(starts, lens, table),
                             mnb.RopeTable(up(cos), up(sin)), gamma_q=up(gq), gamma_k=up(gk),
                             interleaved=inter, out=out)
    assert y is out and torch.all(out[starts[-1]:] == 7.0)
    pl = ref.places(starts, lens, table, ps, pages, T)
    pos = torch.tensor([p for _, p, _, _ in pl])
    n = starts[-1]
    want, mag = ref.norm_rotate(q.cpu()[:n], gq, 1e-6, cos, sin, pos, inter)
    within(out[:n], want, ref.norm_rotate_bound(want, mag, D, dtype, norm))
    want, mag = ref.norm_rotate(k.cpu()[:n], gk, 1e-6, cos, sin, pos, inter)
    bound = ref.norm_rotate_bound(want, mag, D, dtype, norm)
    untouched = torch.ones(cache.k.shape, dtype=torch.bool)
    for t, _, page, at in pl:
        within(cache.k[page, :, at], want[t], bound[t])
        assert torch.equal(cache.v[page, :, at], v[t])
        untouched[page, :, at] = False
    untouched = untouched.to(dev)
    assert torch.equal(cache.k[untouched], k0[untouched])
    assert torch.equal(cache.v[untouched], v0[untouched])


@pytest.mark.parametrize("D", [64, 30])
def test_append_with_arrays_that_make_no_sense(dev, D):
    """Pages that do not exist, positions past the table of pages or of angles, lengths below the
    new tokens: such tokens append nothing, and nothing else is touched."""
    g = torch.Generator().manual_seed(8)
    cache = make_cache(g, 4, 2, 16, D, BF16)
    table = torch.tensor([[0, -1], [9, 4], [1, 2], [3, 3], [2 ** 31 - 1, -2 ** 31]],
                         dtype=torch.int32)
    starts, lens = [0, 2, 4, 7, 9, 11], [18, 17, 40, 1, -5]
    q, k, v = (rows(g, 11, n, D, BF16) for n in (4, 2, 2))
    r = mnb.RopeTable(*(t.to(dev) for t in tables(39, D)))
    k0, v0 = cache.k.clone(), cache.v.clone()
    y = mnb.mnb_cache_append(q, k, v, cache, on_gpu(starts, lens, table), r)
    # Only sequence 3's second token has a place: page 3, 0.
    k1, v1 = cache.k.clone(), cache.v.clone()
    assert torch.equal(v1[3, :, 0], v[8]) and torch.equal(k1[3, :, 0], k[8])  # angle 0
    k1[3, :, 0], v1[3, :, 0] = k0[3, :, 0], v0[3, :, 0]
    assert torch.equal(k0, k1) and torch.equal(v0, v1)
    assert not y[6].any() and not y[7].any() and not y[9:].any()  # positions 39, -1, -7, -6
    assert torch.isfinite(y.float()).all()


def test_append_without_queries_or_rotation(dev):
    g = torch.Generator().manual_seed(9)
    starts, table, pages, T = make_batch(g, [3, 2], [20, 2], 16)
    cache = make_cache(g, pages, 2, 16, 64, F32)
    k, v = rows(g, T, 2, 64, F32, "slice"), rows(g, T, 2, 64, F32, "slice")
    assert mnb.mnb_cache_append(None, k, v, cache, on_gpu(starts, [20, 2], table)) is None
    for t, _, page, at in ref.places(starts, [20, 2], table, 16, pages, T):
        assert torch.equal(cache.k[page, :, at], k[t]) and torch.equal(cache.v[page, :, at], v[t])


# ---- attention -----------------------------------------------------------------------------------

def attend(g, news, lens, hq, H, D, ps, dtype, *, window=0, scale=None, layout="plain",
           cl="heads_first", spread=1.0, rows_behind=0, dirty=False):
    starts, table, pages, T = make_batch(g, news, lens, ps, rows_behind=rows_behind)
    cache = make_cache(g, pages, H, ps, D, dtype, cl)
    q = rows(g, T, hq, D, dtype, layout, spread)
    k, v = cache.k.cpu(), cache.v.cpu()
    if dirty:  # every place that holds no token of a sequence: NaN and infinities
        used = torch.zeros(pages, ps, dtype=torch.bool)
        for b, L in enumerate(lens):
            for j in range(L):
                used[table[b, j // ps], j % ps] = True
        junk = torch.tensor([NAN, math.inf, -math.inf])[torch.randint(0, 3, k.shape, generator=g)]
        for t in (cache.k, cache.v):
            t.copy_(torch.where(used[:, None, :, None], t.cpu(), junk.to(dtype)))
    out = torch.full((T, hq, D), 7.0, dtype=dtype, device="cuda")
    y = mnb.mnb_paged_attention(q, cache, on_gpu(starts, lens, table), scale=scale, window=window,
                                out=out)
    assert y is out
    n = starts[-1]
    assert torch.all(out[n:] == 7.0), "rows of no sequence"
    want, bound = ref.attend(q.cpu()[:n], k, v, starts, lens, table,
                             D ** -0.5 if scale is None else scale, window)
    within(out[:n], want, bound)
    return out


CASES = [
    # news, lens, q heads, key heads, page size
    ([1], [1], 1, 1, 16), ([1], [17], 4, 2, 16), ([1], [1000], 32, 8, 16),
    ([2, 1, 4], [2, 700, 130], 8, 2, 32), ([1] * 9, [1, 16, 64, 65, 129, 300, 31, 2, 500], 8, 8, 16),
    ([7, 0, 3], [50, 0, 3], 15, 3, 48), ([5], [200], 7, 1, 256), ([16, 33], [16, 95], 6, 2, 64),
    ([1, 1], [4000, 5], 16, 1, 16), ([3], [130], 40, 2, 128), ([100], [100], 4, 2, 16),
    ([65, 1, 140], [321, 77, 140], 8, 2, 32), ([257], [300], 5, 1, 16), ([300], [1000], 2, 1, 1024),
    # One sequence and few, of few rows: clusters of 16 and 8 blocks, and more units than fit them.
    ([8], [200], 16, 8, 16), ([4], [1030], 30, 15, 16), ([1, 1, 1], [700, 16, 90], 12, 4, 16),
    ([2], [333], 8, 1, 16), ([1], [2500], 64, 32, 16), ([0, 1], [5, 999], 8, 8, 64),
    ([16], [900], 4, 1, 16), ([17], [900], 4, 1, 16), ([2], [64], 4, 2, 16), ([3], [640], 4, 2, 16),
]


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 128), (F32, 64)])
@pytest.mark.parametrize("news,lens,hq,H,ps", CASES)
def test_attention(dev, news, lens, hq, H, ps, dtype, D):
    g = torch.Generator().manual_seed(sum(lens) + D)
    attend(g, news, lens, hq, H, D, ps, dtype, rows_behind=1)


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 128), (F32, 64)])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 257])
def test_attention_over_a_window(dev, window, dtype, D):
    g = torch.Generator().manual_seed(window)
    attend(g, [1, 130, 9, 1], [400, 290, 9, 1], 4, 2, D, 16, dtype, window=window, dirty=True)


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 64)])
@pytest.mark.parametrize("layout,cl", [("slice", "tokens_first"), ("head_major", "beside")])
def test_attention_layouts(dev, layout, cl, dtype, D):
    g = torch.Generator().manual_seed(3)
    attend(g, [1, 30, 70], [90, 30, 200], 8, 4, D, 32, dtype, layout=layout, cl=cl)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("news,lens", [([1, 1, 3], [33, 127, 65]), ([90, 1, 200], [111, 7, 201])])
def test_what_no_token_wrote_does_not_matter(dev, news, lens, dtype):
    """NaN and infinities in every place past a sequence's end, and in pages of no sequence."""
    g = torch.Generator().manual_seed(4)
    attend(g, news, lens, 8, 2, 128, 64, dtype, dirty=True)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0, 1e-30])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scales(dev, scale, dtype):
    g = torch.Generator().manual_seed(11)
    attend(g, [1, 70], [300, 150], 4, 2, 64, 16, dtype, scale=scale, spread=0.3)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_peaked_and_far_apart_scores(dev, dtype):
    """Scores of hundreds: one key takes all, the running maximum jumps."""
    g = torch.Generator().manual_seed(12)
    attend(g, [1, 40], [500, 300], 4, 1, 128, 16, dtype, spread=20.0)


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 128)])
@pytest.mark.parametrize("n", [3, 150])
def test_values_that_are_not_finite_reach_only_who_attends_them(dev, n, dtype, D):
    """A NaN value at one token and an infinite key at another: the rows before them are as if they
    were not there, the rows from the NaN on are not finite."""
    g = torch.Generator().manual_seed(13)
    L, H, hq, ps = 260, 2, 4, 16
    starts, table, pages, T = make_batch(g, [n], [L], ps)
    cache = make_cache(g, pages, H, ps, D, dtype)
    q = rows(g, T, hq, D, dtype)
    batch = on_gpu(starts, [L], table)
    clean = mnb.mnb_paged_attention(q, cache, batch)
    bad = L - 2  # the last row but one is the first to attend it
    page, at = int(table[0, bad // ps]), bad % ps
    cache.v[page, :, at, 3] = NAN
    page, at = int(table[0, (L - 1) // ps]), (L - 1) % ps
    cache.k[page, :, at] = math.inf
    cache.v[page, :, at] = -math.inf
    y = mnb.mnb_paged_attention(q, cache, batch)
    assert torch.equal(y[:n - 2], clean[:n - 2])
    assert not torch.isfinite(y[n - 2:, :, 3].float()).any()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [1, 100])
def test_pages_that_do_not_exist_and_empty_rows(dev, n, dtype):
    """Holes in the table are not attended; rows without a key (all pages missing, a length below
    the new tokens) are zeros."""
    g = torch.Generator().manual_seed(14)
    D, H, hq, ps = 64, 2, 4, 16
    news, lens = [n, n, n, n], [200, 230, 120, max(n // 2, 0)]
    starts, table, pages, T = make_batch(g, news, lens, ps)
    cache = make_cache(g, pages, H, ps, D, dtype)
    table[0, 3], table[0, 5], table[1, :], table[2, 0] = -1, pages, -7, 2 ** 31 - 1
    q = rows(g, T, hq, D, dtype)
    y = mnb.mnb_paged_attention(q, cache, on_gpu(starts, lens, table))
    want, bound = ref.attend(q.cpu(), cache.k.cpu(), cache.v.cpu(), starts, lens, table, D ** -0.5)
    within(y, want, bound)
    assert not y[n:2 * n].any() and not y[3 * n:4 * n - lens[3]].any()
    # Whole pages of one window missing.
    y = mnb.mnb_paged_attention(q, cache, on_gpu(starts, lens, table), window=5)
    want, bound = ref.attend(q.cpu(), cache.k.cpu(), cache.v.cpu(), starts, lens, table, D ** -0.5,
                             5)
    within(y, want, bound)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [1, 40])
def test_arrays_that_make_no_sense(dev, n, dtype):
    """Starts that decrease, overlap or lie outside, lengths of any size, pages of any number: some
    result or other, nothing outside the buffers."""
    g = torch.Generator().manual_seed(28)
    B, T, ps = 9, 3 * n, 16
    cache = make_cache(g, 6, 2, ps, 64, dtype)
    q = rows(g, T, 4, 64, dtype)
    for starts in ([0, T] * 5, [T, 0] * 5, [-5, T + 99] * 5, [2 ** 31 - 1, -2 ** 31] * 5):
        lens = [int(x) for x in torch.randint(-50, 200, (B,), generator=g)]
        lens[3], lens[4] = 2 ** 31 - 1, -2 ** 31
        table = torch.randint(-3, 9, (B, 5), generator=g, dtype=torch.int32)
        table[0, 0], table[1, 1] = 2 ** 31 - 1, -2 ** 31
        for window in (0, 7):
            guard = torch.full((T + 8, 4, 64), 7.0, dtype=dtype, device=dev)
            batch = on_gpu(starts, lens, table)
            mnb.mnb_paged_attention(q, cache, batch, window=window, out=guard[4:T + 4])
            mnb.mnb_cache_append(None, rows(g, T, 2, 64, dtype), rows(g, T, 2, 64, dtype), cache,
                                 batch)
            assert torch.all(guard[:4] == 7.0) and torch.all(guard[T + 4:] == 7.0)


def test_broadcast_queries(dev):
    """Queries without a stride of their own between heads or tokens (expanded views)."""
    g = torch.Generator().manual_seed(29)
    for n in (1, 90):
        starts, table, pages, T = make_batch(g, [n], [200], 16)
        cache = make_cache(g, pages, 2, 16, 64, BF16)
        one = torch.randn(T, 1, 64, generator=g).to(BF16).to(dev).expand(T, 4, 64)
        tok = torch.randn(1, 4, 64, generator=g).to(BF16).to(dev).expand(T, 4, 64)
        for q in (one, tok):
            batch = on_gpu(starts, [200], table)
            assert torch.equal(mnb.mnb_paged_attention(q, cache, batch),
                               mnb.mnb_paged_attention(q.contiguous(), cache, batch))


def test_more_sequences_than_a_round_of_the_plan(dev):
    g = torch.Generator().manual_seed(30)
    lens = [5 + i % 3 for i in range(1100)]
    attend(g, [5 if i % 7 else 0 for i in range(1100)], lens, 4, 1, 64, 16, BF16)


def test_lengths_past_the_table(dev):
    """Keys past the last page of a row of the table are not attended; nothing else is read."""
    g = torch.Generator().manual_seed(15)
    starts, table, pages, T = make_batch(g, [2, 1], [64, 64], 16)
    cache = make_cache(g, pages, 2, 16, 64, BF16)
    q = rows(g, T, 2, 64, BF16)
    for long in (2 ** 31 - 1, 70, 65):
        y = mnb.mnb_paged_attention(q, cache, on_gpu(starts, [64, long], table))
        want, bound = ref.attend(q.cpu(), cache.k.cpu(), cache.v.cpu(), starts, [64, long], table,
                                 64 ** -0.5)
        within(y, want, bound)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,window", [(5, 0), (5, 20), (5, 1000), (90, 0), (90, 30), (90, 300)])
def test_positions_past_the_table(dev, n, window, dtype):
    """Rows whose own positions lie past the table's pages attend the keys that it does hold, as
    far as their windows reach them."""
    g = torch.Generator().manual_seed(31)
    lens = [150, 2 ** 30, 128 + n // 2]
    _, table, pages, T = make_batch(g, [n] * 3, [128] * 3, 16)
    cache = make_cache(g, pages, 2, 16, 64, dtype)
    q, starts = rows(g, T, 4, 64, dtype), [0, n, 2 * n, 3 * n]
    y = mnb.mnb_paged_attention(q, cache, on_gpu(starts, lens, table), window=window)
    want, bound = ref.attend(q.cpu(), cache.k.cpu(), cache.v.cpu(), starts, lens, table, 64 ** -0.5,
                             window)
    within(y, want, bound)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("news,lens,hq,window", [([1], [9001], 4, 0), ([16], [6007], 4, 0),
                                                 ([7, 4, 2, 9], [135, 24, 9000, 700], 5, 0),
                                                 ([150], [5003], 4, 0), ([150], [5003], 4, 900)])
def test_lone_long_sequences_over_one_key_head(dev, news, lens, hq, window, dtype):
    g = torch.Generator().manual_seed(35)
    attend(g, news, lens, hq, 1, 128, 32, dtype, window=window)


@pytest.mark.parametrize("hq,D", [(16, 128), (24, 128), (8, 64)])
def test_what_shared_memory_held_before(dev, hq, D):
    """Masked blocks that are a CTA's first, after a kernel that leaves NaN all over the SMs."""
    g = torch.Generator().manual_seed(34)
    news, lens = [7, 708, 9, 5, 1, 2, 1, 0, 57], [7, 908, 4312, 2428, 11, 2, 10, 90, 57]
    starts, table, pages, T = make_batch(g, news, lens, 64)
    cache = make_cache(g, pages, 8, 64, D, BF16)
    q, batch = rows(g, T, hq, D, BF16), on_gpu(starts, lens, table)
    want, bound = ref.attend(q.cpu(), cache.k.cpu(), cache.v.cpu(), starts, lens, table, D ** -0.5)
    for _ in range(6):
        torch.full((1 << 26,), math.nan, device=dev)
        within(mnb.mnb_paged_attention(q, cache, batch), want, bound)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window", [2 ** 30, 2 ** 31 - 1026, 2 ** 31 - 1, 2 ** 31, 2 ** 63 - 1])
def test_windows_past_every_position(dev, window, dtype):
    """The largest windows, with rows that stand before the first position (they attend nothing)."""
    g = torch.Generator().manual_seed(33)
    for news, lens in ([3, 1, 90], [1, 50, 60]), ([2000], [7]):
        attend(g, news, lens, 4, 2, 64, 16, dtype, window=window)


def test_tables_that_are_slices_of_wider_ones(dev):
    g = torch.Generator().manual_seed(32)
    starts, table, pages, T = make_batch(g, [1, 70], [90, 100], 16, width=9)
    cache = make_cache(g, pages, 2, 16, 64, BF16)
    q, batch = rows(g, T, 4, 64, BF16), on_gpu(starts, [90, 100], table)
    wide = torch.full((2, 40), -1, dtype=torch.int32, device=dev)
    wide[:, 3:12] = batch.table
    part = mnb.KvBatch(batch.starts, batch.lengths, wide[:, 3:12])
    assert torch.equal(mnb.mnb_paged_attention(q, cache, batch),
                       mnb.mnb_paged_attention(q, cache, part))


@pytest.mark.parametrize("n", [1, 80])
def test_offsets_past_32_bits(dev, n):
    """A cache of 4.3 G elements: pages whose bytes and elements lie past 2^32."""
    g = torch.Generator().manual_seed(16)
    pages, H, ps, D = 2 ** 18 + 2 ** 10, 8, 16, 128
    k, v = (torch.empty(pages, H, ps, D, dtype=BF16, device=dev) for _ in range(2))
    assert k.numel() > 2 ** 32
    table = torch.tensor([[pages - 1, 0, 2 ** 17 + 3, pages - 2, 5, 2 ** 18 - 1, 7]],
                         dtype=torch.int32)
    small = [torch.randn(7, H, ps, D, generator=g).to(BF16) for _ in range(2)]
    for t, s in zip((k, v), small):
        t[table[0].long().to(dev)] = s.to(dev)
    cache, L = mnb.KvCache(k, v), 100
    q = rows(g, n, 16, D, BF16)
    y = mnb.mnb_paged_attention(q, cache, on_gpu([0, n], [L], table))
    want, bound = ref.attend(q.cpu(), *small, [0, n], [L],
                             torch.arange(7, dtype=torch.int32)[None], D ** -0.5)
    within(y, want, bound)
    kn, vn = rows(g, n, H, D, BF16), rows(g, n, H, D, BF16)
    mnb.mnb_cache_append(None, kn, vn, cache, on_gpu([0, n], [L], table))
    for t, p, _, at in ref.places([0, n], [L], table, ps, pages, n):
        page = int(table[0, p // ps])
        assert torch.equal(k[page, :, at], kn[t]) and torch.equal(v[page, :, at], vn[t])


def test_many_sequences(dev):
    """More sequences than a warp looks over at a time, some without new tokens; results do not
    depend on who else is in the batch (up to the order of sums)."""
    g = torch.Generator().manual_seed(17)
    lens = [int(x) for x in torch.randint(1, 90, (333,), generator=g)]
    news = [int(x) for x in torch.randint(0, 3, (333,), generator=g)]
    news = [min(a, b) for a, b in zip(news, lens)]
    attend(g, news, lens, 4, 2, 64, 16, BF16)


@pytest.mark.parametrize("news,lens", [([1] * 5, [900, 33, 257, 1, 64]),
                                       ([150, 1, 70], [900, 33, 257])])
def test_repeated_calls_are_bitwise_equal(dev, news, lens):
    g = torch.Generator().manual_seed(18)
    starts, table, pages, T = make_batch(g, news, lens, 16)
    cache = make_cache(g, pages, 2, 16, 128, BF16)
    q, batch = rows(g, T, 8, 128, BF16), on_gpu(starts, lens, table)
    first = mnb.mnb_paged_attention(q, cache, batch)
    for _ in range(20):
        assert torch.equal(first, mnb.mnb_paged_attention(q, cache, batch))


# ---- together, streams and graphs ----------------------------------------------------------------

def test_a_layer_step_by_step(dev):
    """A prompt and two decode steps through 4-bit projections, norms, rotation, cache, attention
    and the output projection, against the 64-bit definitions fed with each step's own inputs."""
    from int4_weight_only_matmulnbits_gb300.workloads import make_problem
    g = torch.Generator().manual_seed(19)
    hidden, hq, H, D, ps = 256, 4, 2, 64, 16
    probs = [make_problem(1, n, hidden, 32, dtype=BF16, seed=30 + i)
             for i, n in enumerate((hq * D, H * D, H * D))]
    po = make_problem(1, hidden, hq * D, 32, dtype=BF16, seed=40)
    pack = lambda p: mnb.mnb_prepack(p.B.to(dev), p.scales.to(dev), None, p.N, p.K, 32)  # noqa: E731
    ws, wo = [pack(p) for p in probs], pack(po)
    gq, gk = (1 + 0.2 * torch.randn(D, generator=g) for _ in range(2))
    rope = mnb.mnb_rope_table(mnb.mnb_rope_frequencies(D, 1e6), 256, device=dev)
    cache = make_cache(g, 20, H, ps, D, BF16, fill=NAN)
    table = torch.randperm(20, generator=g).to(torch.int32).view(2, 10)
    lens = [0, 0]
    for news in ([70, 33], [1, 1], [1, 1]):
        T = sum(news)
        lens = [a + b for a, b in zip(lens, news)]
        starts = [0, news[0], T]
        x = torch.randn(T, hidden, generator=g).to(BF16).to(dev)
        q, k, v = (mnb.mnb_matmul(x, w).view(T, -1, D) for w in ws)
        batch = on_gpu(starts, lens, table)
        y = mnb.mnb_cache_append(q, k, v, cache, batch, rope, gamma_q=gq.to(dev),
                                 gamma_k=gk.to(dev))
        a = mnb.mnb_paged_attention(y, cache, batch)
        o = mnb.mnb_matmul(a.view(T, -1), wo)
        pl = ref.places(starts, lens, table, ps, 20, T)
        pos = torch.tensor([p for _, p, _, _ in pl])
        cos, sin = rope.cos.cpu(), rope.sin.cpu()
        want, mag = ref.norm_rotate(q.cpu(), gq, 1e-6, cos, sin, pos, False)
        within(y, want, ref.norm_rotate_bound(want, mag, D, BF16, True))
        want, mag = ref.norm_rotate(k.cpu(), gk, 1e-6, cos, sin, pos, False)
        bound = ref.norm_rotate_bound(want, mag, D, BF16, True)
        for t, _, page, at in pl:
            within(cache.k[page, :, at], want[t], bound[t])
        want, bound = ref.attend(y.cpu(), cache.k.cpu(), cache.v.cpu(), starts, lens, table,
                                 D ** -0.5)
        within(a, want, bound)
        assert torch.isfinite(o.float()).all()


@pytest.mark.parametrize("news", [[1, 1, 1], [40, 1, 20]])
def test_captured_and_replayed(dev, news):
    """Append and attention captured once; replayed, two graphs at a time on two streams, with
    rows, lengths and pages that change between replays."""
    hq, H, D, ps, B = 8, 2, 128, 16, 3
    T, made = sum(news), []
    for i in range(2):
        g = torch.Generator().manual_seed(20 + i)
        cache = make_cache(g, 60, H, ps, D, BF16)
        rope = mnb.mnb_rope_table(mnb.mnb_rope_frequencies(D, 1e6), 512, device=dev)
        qkv = torch.zeros(T, hq + 2 * H, D, dtype=BF16, device=dev)
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)  # noqa: E731
        batch = mnb.KvBatch(i32(B + 1), i32(B), i32(B, 18))
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + H], qkv[:, hq + H:]
        step = lambda q=q, k=k, v=v, cache=cache, batch=batch, rope=rope: (  # noqa: E731
            lambda y: (y, mnb.mnb_paged_attention(y, cache, batch)))(
                mnb.mnb_cache_append(q, k, v, cache, batch, rope))
        graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            step()
        st.synchronize()
        with torch.cuda.graph(graph, stream=st):
            y, a = step()
        made.append((g, cache, rope, qkv, batch, graph, st, y, a))
    for turn in range(3):
        plans = []
        for g, cache, rope, qkv, batch, graph, st, y, a in made:
            lens = [max(n, int(x)) for n, x in zip(news, torch.randint(1, 280, (B,), generator=g))]
            used = list(news)
            if turn == 2:
                used[1] = 0  # a padded batch: rows behind the last sequence
            starts = [0]
            for n in used:
                starts.append(starts[-1] + n)
            table = torch.randperm(60, generator=g)[:54].to(torch.int32).view(B, 18)
            qkv.copy_(torch.randn(qkv.shape, generator=g).to(BF16))
            batch.starts.copy_(torch.tensor(starts, dtype=torch.int32))
            batch.lengths.copy_(torch.tensor(lens, dtype=torch.int32))
            batch.table.copy_(table)
            plans.append((starts, lens, table))
        torch.cuda.synchronize()
        for *_, graph, st, y, a in made:
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        for (starts, lens, table), (g, cache, rope, qkv, batch, graph, st, y, a) in zip(plans, made):
            n = starts[-1]
            want, bound = ref.attend(y.cpu()[:n], cache.k.cpu(), cache.v.cpu(), starts, lens,
                                     table, D ** -0.5)
            within(a[:n], want, bound)


def test_on_a_stream_of_its_own(dev):
    """stream= runs the call, its outputs and its workspace there; two streams at once."""
    g = torch.Generator().manual_seed(25)
    jobs = []
    for i in range(2):
        starts, table, pages, T = make_batch(g, [1, 60], [500, 90], 16)
        jobs.append((make_cache(g, pages, 2, 16, 64, BF16), rows(g, T, 4, 64, BF16),
                     on_gpu(starts, [500, 90], table), torch.cuda.Stream(), (starts, table)))
    torch.cuda.synchronize()
    outs = [[] for _ in jobs]
    for _ in range(10):
        for out, (cache, q, batch, st, _) in zip(outs, jobs):
            out.append(mnb.mnb_paged_attention(q, cache, batch, stream=st))
    torch.cuda.synchronize()
    for out, (cache, q, batch, st, (starts, table)) in zip(outs, jobs):
        want, bound = ref.attend(q.cpu(), cache.k.cpu(), cache.v.cpu(), starts, [500, 90], table,
                                 64 ** -0.5)
        for y in out:
            within(y, want, bound)


def test_without_programmatic_launch(dev):
    g = torch.Generator().manual_seed(26)
    mnb.mnb_set_programmatic_launch(False)
    try:
        attend(g, [1, 50], [100, 60], 4, 2, 64, 16, BF16)
    finally:
        mnb.mnb_set_programmatic_launch(True)


# ---- calls that a plain step does not make -------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("news,lens,T", [
    ([1, 6], [40, 100], 4), ([3, 20, 9], [50, 21, 70], 5), ([2] * 40 + [7], [30] * 40 + [90], 83),
    ([3, 200, 90], [50, 300, 700], 260), ([300], [1000], 150), ([150, 9, 100], [150, 60, 100], 152)])
def test_the_first_rows_of_a_step(dev, news, lens, T, window, dtype):
    """A call of the first T rows of a step whose starts go on past them: every row is placed as in
    the whole step, by appending and by attention alike."""
    g = torch.Generator().manual_seed(T + window)
    hq, H, D, ps = 8, 2, 64, 16
    starts, table, pages, whole = make_batch(g, news, lens, ps)
    assert T < whole
    q, k, v = (rows(g, whole, n, D, dtype) for n in (hq, H, H))
    cache, batch = make_cache(g, pages, H, ps, D, dtype), on_gpu(starts, lens, table)
    k0, v0 = cache.k.clone(), cache.v.clone()
    y = mnb.mnb_paged_attention(q[:T], cache, batch, window=window)
    want, bound = ref.attend(q.cpu(), k0.cpu(), v0.cpu(), starts, lens, table, D ** -0.5, window)
    within(y, want[:T], bound[:T])
    mnb.mnb_cache_append(None, k[:T], v[:T], cache, batch)
    for t, _, page, at in ref.places(starts, lens, table, ps, pages, T):
        k0[page, :, at], v0[page, :, at] = k[t], v[t]
    assert torch.equal(cache.k, k0) and torch.equal(cache.v, v0)


@pytest.mark.parametrize("f,n,first", [(-1e-11, 3000, 0), (-7e-11, 3000, 0), (1e-13, 3000, 0),
                                       (-1e-13, 500, 2 ** 31 - 1000), (-1e-9, 500, 1 << 20),
                                       (3e-17, 500, 2 ** 30), (-0.7, 2000, 0)])
def test_tables_of_small_and_negative_frequencies(dev, f, n, first):
    """Relative to themselves but for what the angle is off: 2^-52 of it (two products of doubles),
    and 2^-65 of a turn for each position."""
    t = mnb.mnb_rope_table(torch.tensor([f], dtype=torch.float64), n, first=first, device=dev)
    p = torch.arange(first, first + n, dtype=torch.float64)[:, None]
    a = p * f
    slack = 2.0 ** -52 * a.abs() + p * (2 * math.pi * 2.0 ** -65)
    slack += 2.0 ** -53 * a.abs()  # the reference's product
    within(t.cos, torch.cos(a), 2.0 ** -22 * torch.cos(a).abs() + slack + 1e-45)
    within(t.sin, torch.sin(a), 2.0 ** -22 * torch.sin(a).abs() + slack + 1e-45)


def test_other_threads_run_while_a_call_waits(dev):
    """A launch that finds the stream's queue full blocks until the GPU catches up; the process's
    other Python threads go on meanwhile. (The stream is held by a host function that sleeps.)"""
    import ctypes
    import threading
    import time
    hold = 0.5
    driver = ctypes.CDLL("libcuda.so.1")
    sleep = ctypes.cast(ctypes.CDLL(None).usleep, ctypes.c_void_p)
    q = torch.zeros(1, 1, 64, dtype=BF16, device=dev)
    y = torch.empty_like(q)
    gamma = torch.ones(64, device=dev)
    call = lambda: mnb.mnb_qk_norm_rope(q, None, None, None, gamma_q=gamma, out_q=y)  # noqa: E731
    call()
    torch.cuda.synchronize()
    beats, stop = [], threading.Event()

    def beat():
        while not stop.is_set():
            beats.append(time.perf_counter())
            time.sleep(0.002)
    other = threading.Thread(target=beat)
    other.start()
    try:
        stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        assert driver.cuLaunchHostFunc(stream, sleep, ctypes.c_void_p(int(hold * 1e6))) == 0
        start = at = time.perf_counter()
        longest = 0.0
        while at - start < hold:
            call()
            now = time.perf_counter()
            longest, at = max(longest, now - at), now
    finally:
        stop.set()
        other.join()
        torch.cuda.synchronize()
    assert longest > hold / 2, "no call had to wait"
    beats = [b for b in beats if start <= b <= at]
    gaps = [b - a for a, b in zip([start] + beats, beats + [at])]
    assert max(gaps) < hold / 4, f"the other thread stood still for {max(gaps):.3f} s"


FINE, FINER = 2.0 ** -9, 2.0 ** -18  # 1 + FINE + FINER: each bf16 part of it holds one of the three


def one_sequence_per_row(q, k, v, scale):
    """Attention of q [n, heads, D], each row a sequence of its own over k, v [n or 1, keys, D] of
    one key head."""
    n, L, D = q.shape[0], k.shape[1], q.shape[2]
    ps = -(-L // 16) * 16
    pad = lambda x: torch.nn.functional.pad(x, (0, 0, 0, ps - L))[:, None].cuda()  # noqa: E731
    table = torch.arange(n, dtype=torch.int32)[:, None] if k.shape[0] == n else torch.zeros(
        n, 1, dtype=torch.int32)
    return mnb.mnb_paged_attention(q.cuda(), mnb.KvCache(pad(k), pad(v)),
                                   on_gpu(list(range(n + 1)), [L] * n, table), scale=scale)


@pytest.mark.parametrize("G", [1, 4, 16])
@pytest.mark.parametrize("D", [64, 128])
def test_the_low_bits_of_fp32_keys(dev, D, G):
    """Two keys whose scores differ by bits past the 16th alone, in some of the elements, blown up
    by the scale: row t, which holds element t alone, sees them as 1 apart where they differ. All
    products and sums are exact in 24 bits."""
    g = torch.Generator().manual_seed(D + G)
    bit = torch.randint(0, 2, (D,), generator=g).float()
    k = torch.full((1, 2, D), 1 + FINE)
    k[0, 0] += bit * FINER
    q = torch.eye(D)[:, None].expand(D, G, D).contiguous()
    v = torch.tensor([1.0, 0.0])[None, :, None].expand(1, 2, D).contiguous()
    y = one_sequence_per_row(q, k, v, 1 / FINER).double().cpu()
    want = torch.sigmoid(bit.double())
    # The exponential to 2^-21, the roundings of weight, sum, quotient and product.
    assert ((y - want[:, None, None]).abs() <= 2.0 ** -20).all()


@pytest.mark.parametrize("G", [1, 4, 16])
@pytest.mark.parametrize("D", [64, 128])
def test_the_low_bits_of_fp32_queries(dev, D, G):
    """The same with the low bits in the rows: element t has them, element t + 1 does not; one key
    takes the even elements, the other the odd ones."""
    t = torch.arange(D)
    q = torch.zeros(D, G, D)
    q[t, :, t], q[t, :, (t + 1) % D] = 1 + FINE + FINER, 1 + FINE
    even = (t % 2 == 0).float()
    k = torch.stack((even, 1 - even))[None]
    v = torch.tensor([1.0, 0.0])[None, :, None].expand(1, 2, D).contiguous()
    y = one_sequence_per_row(q, k, v, 1 / FINER).double().cpu()
    want = torch.sigmoid(torch.where(t % 2 == 0, 1.0, -1.0).double())
    assert ((y - want[:, None, None]).abs() <= 2.0 ** -20).all()


@pytest.mark.parametrize("G", [1, 4, 16])
@pytest.mark.parametrize("D", [64, 128])
def test_products_of_the_middle_bits(dev, D, G):
    """(1 + 2^-9)^2 against 1 + 2^-8: the product of both factors' second parts is what differs."""
    t = torch.arange(D)
    q = torch.zeros(D, G, D)
    q[t, :, t], q[t, :, (t + 1) % D] = 1 + FINE, 1.0
    k = torch.zeros(D, 2, D)
    k[t, 0, t], k[t, 1, (t + 1) % D] = 1 + FINE, 1 + 2 * FINE
    v = torch.tensor([1.0, 0.0])[None, :, None].expand(D, 2, D).contiguous()
    y = one_sequence_per_row(q, k, v, 1 / FINER).double().cpu()
    assert ((y - torch.sigmoid(torch.tensor(1.0).double())).abs() <= 2.0 ** -20).all()


@pytest.mark.parametrize("G", [1, 4, 16])
@pytest.mark.parametrize("D", [64, 128])
def test_the_low_bits_of_fp32_values(dev, D, G):
    """One key attended with weight 1, at every place of a step in turn (the others' scores are
    200 below): its value comes back, 24 bits of it."""
    g = torch.Generator().manual_seed(D * G)
    n = 64
    q = torch.zeros(n, G, D)
    q[..., 0] = 1.0
    k, v = torch.zeros(n, n, D), torch.randn(n, n, D, generator=g)
    k[..., 0] = -200.0
    i = torch.arange(n)
    k[i, i, 0] = 0.0
    y = one_sequence_per_row(q, k, v, 1.0).double().cpu()
    want = v[i, i].double()[:, None].expand(n, G, D)
    # Three parts to 2^-25 and their sum to 2^-23; e^-200 counts for nothing in 24 bits.
    assert ((y - want).abs() <= 2.0 ** -22 * want.abs()).all()


@pytest.mark.parametrize("G", [1, 4, 16])
@pytest.mark.parametrize("D", [64, 128])
def test_the_low_bits_of_fp32_weights(dev, D, G):
    """Weights 1 and 1 - 2^-9 - 2^-18 of opposite values, at every pair of neighbouring places of a
    step: what is left of the sum is their difference, 2^-18 of which are the weight's third part."""
    n = 64
    w = 1 - FINE - FINER
    q = torch.zeros(n, G, D)
    q[..., 0] = 1.0
    k, v = torch.zeros(n, n, D), torch.zeros(n, n, D)
    k[..., 0] = -200.0
    i = torch.arange(n)
    k[i, i, 0], k[i, (i + 1) % n, 0] = 0.0, math.log(w)
    v[i, i], v[i, (i + 1) % n] = 1.0, -1.0
    y = one_sequence_per_row(q, k, v, 1.0).double().cpu()
    want = (1 - w) / (1 + w)
    # The exponential to 2^-21, over a sum of 2; without the third part it would be 2^-19 off.
    assert ((y - want).abs() <= 2.0 ** -21).all()


@pytest.mark.parametrize("news,lens,hq,H,D", [
    ([1], [2049], 16, 8, 128), ([4], [300], 2, 2, 64), ([1] * 12, [900] * 12, 8, 2, 128),
    ([16], [16], 4, 2, 64), ([40], [1000], 4, 2, 128), ([130], [130], 8, 1, 64),
    ([33, 60], [700, 2000], 6, 2, 128)])
@pytest.mark.parametrize("spread", [1.0, 4.0])
def test_fp32_attention_is_as_exact_as_fp32_arithmetic(dev, news, lens, hq, H, D, spread):
    """The error's mean square against 64 bits, beside that of the same attention in elementary fp32
    operations. Three bf16 parts a factor come out at up to 1.4 times the plain error when the
    kernel's arithmetic is followed on the CPU, two parts at 20 times and more."""
    g = torch.Generator().manual_seed(len(news) + D)
    starts, table, pages, T = make_batch(g, news, lens, 16)
    cache = make_cache(g, pages, H, 16, D, F32)
    q = rows(g, T, hq, D, F32, spread=spread)
    y = mnb.mnb_paged_attention(q, cache, on_gpu(starts, lens, table)).cpu()
    want, _ = ref.attend(q.cpu(), cache.k.cpu(), cache.v.cpu(), starts, lens, table, D ** -0.5)
    plain = torch.empty_like(y)
    for b, L in enumerate(lens):
        g_ = table[b].long()
        k, v = (x.cpu()[g_].transpose(1, 2).reshape(-1, H, D)[:L].repeat_interleave(hq // H, 1)
                for x in (cache.k, cache.v))
        for t in range(starts[b], starts[b + 1]):
            p = L - (starts[b + 1] - t) + 1
            s = (q[t].cpu()[None] * k[:p]).sum(-1) * D ** -0.5
            w = torch.exp(s - s.amax(0))
            plain[t] = (w[..., None] * v[:p]).sum(0) / w.sum(0)[:, None]
    rms = lambda x: (x.double() - want).pow(2).mean().sqrt().item()  # noqa: E731
    assert rms(y) <= 4 * rms(plain), f"{rms(y):.3g}, plain fp32 {rms(plain):.3g}"


@pytest.mark.parametrize("hq,D", [(16, 128), (24, 128), (8, 64)])
def test_what_the_kernel_itself_left_in_shared_memory(dev, hq, D):
    """Masked blocks that are a CTA's first, after the same kernel has filled every stage of every
    SM's ring with the NaN of another cache."""
    g = torch.Generator().manual_seed(34)
    news, lens = [7, 708, 9, 5, 1, 2, 1, 0, 57], [7, 908, 4312, 2428, 11, 2, 10, 90, 57]
    starts, table, pages, T = make_batch(g, news, lens, 64)
    cache = make_cache(g, pages, 8, 64, D, BF16)
    q, batch = rows(g, T, hq, D, BF16), on_gpu(starts, lens, table)
    want, bound = ref.attend(q.cpu(), cache.k.cpu(), cache.v.cpu(), starts, lens, table, D ** -0.5)
    # 4000 tokens of 8 key heads: each CTA takes more blocks of keys than its ring holds.
    starts2, table2, pages2, T2 = make_batch(g, [4000], [4000], 64)
    nan = make_cache(g, pages2, 8, 64, D, BF16, fill=NAN)
    q2, batch2 = rows(g, T2, hq, D, BF16), on_gpu(starts2, [4000], table2)
    for _ in range(6):
        assert mnb.mnb_paged_attention(q2, nan, batch2).isnan().all()
        within(mnb.mnb_paged_attention(q, cache, batch), want, bound)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window", [1, 16, 100, 700])
def test_many_sequences_over_a_window(dev, window, dtype):
    """More sequences and units than clusters take, a few tokens each."""
    g = torch.Generator().manual_seed(window + 40)
    lens = [int(x) for x in torch.randint(3, 900, (45,), generator=g)]
    attend(g, [1 + i % 3 for i in range(45)], lens, 8, 2, 128, 16, dtype, window=window, dirty=True)


@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("chunk,L", [(100, 700), (150, 150)])
def test_a_chunk_among_many_decoding_sequences(dev, chunk, L, window):
    """So many sequences that the chunk goes through the kernel for few rows as well."""
    g = torch.Generator().manual_seed(chunk)
    lens = [int(x) for x in torch.randint(1, 400, (63,), generator=g)]
    attend(g, [1] * 40 + [chunk] + [1] * 23, lens[:40] + [L] + lens[40:], 4, 2, 128, 16, BF16,
           window=window, dirty=True)


@pytest.mark.parametrize("n,new", [(1, 4864), (160, 16)])
def test_runs_of_blocks_longer_than_a_wait(dev, n, new):
    """154 M positions (pages that repeat), so that a CTA of the tensor-core kernel goes through
    blocks without a mask, or with one tile alone, for more than the second after which other waits
    give up. Four keys of a page take all the weight (the others' underflows to 0)."""
    g = torch.Generator().manual_seed(41)
    hq, D, ps, repeats = 8, 128, 1 << 16, 2344
    L = repeats * ps - 40000
    hot = torch.tensor([70, 20001, 30011, 65535])
    u = torch.randn(D, generator=g)
    u /= u.norm()
    k = torch.zeros(1, 1, ps, D)
    k[0, 0, hot] = u * 40
    q = (u * 34 + 0.3 * torch.randn(n * new, hq, D, generator=g)).to(BF16).to(dev)
    cache = mnb.KvCache(k.to(BF16).to(dev), torch.randn(k.shape, generator=g).to(BF16).to(dev))
    starts = list(range(0, n * new + 1, new))
    y = mnb.mnb_paged_attention(q, cache, on_gpu(starts, [L] * n,
                                                 torch.zeros(n, repeats, dtype=torch.int32)))
    assert mnb.mnb_fault_status() == 0
    keys, values = (x[0, 0, hot.to(dev)].double().cpu() for x in (cache.k, cache.v))
    for t in torch.randint(0, n * new, (40,), generator=g).tolist():
        p = L - (new - t % new)
        times = (p + 1) // ps + (hot <= p % ps).double() * ((p + 1) % ps > 0)
        qt = q[t].double().cpu()
        s = qt @ keys.T * D ** -0.5
        assert (s > 105).all()  # e^-105 is below the smallest number
        w = times * torch.exp(s - s.amax(-1, keepdim=True))
        w /= w.sum(-1, keepdim=True)
        want, spread = w @ values, w @ values.abs()
        # As ref.attend counts them, with an addition for each time that a key counts.
        dw = (D + 8) * 2.0 ** -23 * (qt.abs() @ keys.abs().T).amax() * D ** -0.5 + 2.0 ** -20
        rel = 2 * dw + ref.BF16_U + (4 * repeats + 16) * 2.0 ** -23
        within(y[t], want, rel * (spread + want.abs()) + ref.BF16_U * want.abs() + 1e-30)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,new,repeats", [(1, 4864, 16), (1, 4864, 64), (304, 1, 64)])
def test_sums_of_millions_of_keys(dev, n, new, repeats, D):
    """The mean of ones over 1 M and 4 M keys (pages that repeat), on the tensor-core kernel and, a
    row a sequence, on the streaming one: 1, unless the sums lose half of bf16's step below it,
    2^-9. (Weights are rounded to bf16, 2^-9 either way, which a million of them average out.)"""
    g = torch.Generator().manual_seed(42)
    hq, ps = 8, 1 << 16
    cache = mnb.KvCache(*(x.to(BF16).to(dev) for x in (torch.randn(1, 1, ps, D, generator=g),
                                                       torch.ones(1, 1, ps, D))))
    q = (0.2 * torch.randn(n * new, hq, D, generator=g)).to(BF16).to(dev)
    batch = on_gpu(list(range(0, n * new + 1, new)), [repeats * ps] * n,
                   torch.zeros(n, repeats, dtype=torch.int32))
    y = mnb.mnb_paged_attention(q, cache, batch)
    assert torch.all(y == 1), f"{y.float().min().item()} .. {y.float().max().item()}"


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 150_000])
def test_sums_put_aside_between_runs(dev, window, D):
    """Runs of 512 blocks and more whose maxima keep growing, in units that CTAs share: 210 000 keys
    that get longer, shuffled pages, some of which are missing."""
    g = torch.Generator().manual_seed(43)
    hq, ps, L, T = 8, 64, 210_000, 5000
    pages = -(-L // ps)
    table = torch.randperm(pages, generator=g).to(torch.int32)[None].clone()
    table[0, 100:120], table[0, 2000] = -1, pages
    k, v = (torch.randn(pages * ps, D, generator=g) for _ in range(2))
    k *= torch.linspace(0.1, 2.5, pages * ps)[:, None]
    there = ((table[0] >= 0) & (table[0] < pages)).repeat_interleave(ps)[:L].to(dev)
    k, v = k.to(BF16).to(dev), v.to(BF16).to(dev)  # by position
    cache = make_cache(g, pages, 1, ps, D, BF16, fill=NAN)
    for x, y in ((cache.k, k), (cache.v, v)):
        for i, page in enumerate(table[0].tolist()):
            if 0 <= page < pages:
                x[page, 0] = y[i * ps:(i + 1) * ps]
    q = rows(g, T, hq, D, BF16)
    y = mnb.mnb_paged_attention(q, cache, on_gpu([0, T], [L], table), window=window)
    for t in [0, 1, T - 1] + torch.randint(0, T, (25,), generator=g).tolist():
        p = L - T + t
        j = torch.arange(L, device=dev)
        on = there & (j <= p) & ((j > p - window) if window else True)
        kd, vd, qt = k[:L][on].double(), v[:L][on].double(), q[t].double()
        s = qt @ kd.T * D ** -0.5
        w = torch.softmax(s, -1)
        want, spread = w @ vd, w @ vd.abs()
        # As ref.attend counts them; 2^-11 for what additions cut off.
        ds = (D + 8) * 2.0 ** -23 * (qt.abs() @ kd.abs().T).amax(-1) * D ** -0.5
        rel = 2 * (ds + 2.0 ** -21 + 3 * ref.F32_U) + ref.BF16_U + 2.0 ** -11
        bound = rel[:, None] * (spread + want.abs())
        within(y[t], want.cpu(), (bound + ref.BF16_U * (want.abs() + bound)).cpu())


def test_calls_from_several_threads(dev):
    """Threads with streams of their own, whose calls overlap on the host and on the GPU: every
    result as alone."""
    import threading
    jobs = []
    for i, (news, lens, dtype) in enumerate([([1, 1], [900, 70], BF16), ([130, 3], [300, 40], BF16),
                                             ([1] * 40, [50] * 40, BF16), ([9], [700], F32)]):
        g = torch.Generator().manual_seed(50 + i)
        starts, table, pages, T = make_batch(g, news, lens, 16)
        cache = make_cache(g, pages, 2, 16, 128, dtype)
        q, batch = rows(g, T, 8, 128, dtype), on_gpu(starts, lens, table)
        gamma = torch.rand(128, generator=g).to(dev)

        def step(q=q, cache=cache, batch=batch, gamma=gamma):
            y, _ = mnb.mnb_qk_norm_rope(q, None, None, None, gamma_q=gamma)
            return mnb.mnb_paged_attention(y, cache, batch)
        jobs.append((step, step(), torch.cuda.Stream(), []))
    torch.cuda.synchronize()

    def work(step, stream, out):
        with torch.cuda.stream(stream):
            for _ in range(100):
                out.append(step())
    threads = [threading.Thread(target=work, args=(step, stream, out))
               for step, _, stream, out in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for _, alone, _, out in jobs:
        assert len(out) == 100 and all(torch.equal(y, alone) for y in out)


@pytest.mark.parametrize("news,lens", [([1], [300]), ([1] * 40, [90] * 40), ([150], [200])])
def test_results_beside_the_queries(dev, news, lens):
    """q and out as slices of one matrix's rows."""
    g = torch.Generator().manual_seed(44)
    starts, table, pages, T = make_batch(g, news, lens, 16)
    cache, batch = make_cache(g, pages, 2, 16, 128, BF16), on_gpu(starts, lens, table)
    both = torch.full((T, 18, 128), 7.0, dtype=BF16, device=dev)
    both[:, 1:9] = rows(g, T, 8, 128, BF16)
    q, out = both[:, 1:9], both[:, 9:17]
    want = mnb.mnb_paged_attention(q.contiguous(), cache, batch)
    before = q.clone()
    assert mnb.mnb_paged_attention(q, cache, batch, out=out) is out
    assert torch.equal(out, want) and torch.equal(q, before)
    assert torch.all(both[:, 0] == 7.0) and torch.all(both[:, 17] == 7.0)
