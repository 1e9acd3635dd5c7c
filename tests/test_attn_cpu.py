"""The attention block's entry points on the host: frequencies, and refusals that come before any
device work (fake device addresses; nothing is dereferenced)."""
import ctypes
import math

import pytest
import torch

import int4_weight_only_matmulnbits_gb300 as mnb
from int4_weight_only_matmulnbits_gb300 import binding as b
from tests import attn_reference as ref

F32, BF16 = b.MNB_F32, b.MNB_BF16
BIG = 2 ** 31
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module")
def lib():
    mnb.build_library()
    return mnb.load()


# Fake device addresses, 16 GiB apart.
Q, K, V, QO, KO, COS, SIN, POS, GQ, GK, CK, CV, STA, LEN, TAB, WS = (
    0x7000_0000_0000 + i * (1 << 34) for i in range(16))


def by(s):
    return None if s is None else ctypes.byref(s)


def heads(p, n=4, ts=None, hs=64, reserved=0):
    return b.HeadsC(p or None, n * 64 if ts is None else ts, hs, n, reserved)


def rope(cos=COS, sin=SIN, positions=100, rot=64, inter=0):
    return b.RopeC(cos or None, sin or None, positions, rot, inter)


def cache(k=CK, v=CV, pages=8, ps=16, H=2, D=64, dt=BF16, **over):
    c = b.KvCacheC(k or None, v or None, pages, H * ps * D, ps * D, D, H * ps * D, ps * D, D, ps,
                   H, D, dt)
    for n, x in over.items():
        setattr(c, n, x)
    return c


def batch(s=STA, l=LEN, t=TAB, n=2, pages=4, stride=None):
    return b.KvBatchC(s or None, l or None, t or None, n, pages,
                      pages if stride is None else stride)


@pytest.mark.parametrize("args", [(128, 1e6), (64, 1e4, 8.0), (80, 5e5, 4.0, 8192.0, 1.0, 4.0),
                                  (2, 10.0), (256, 1e6, 4.5, 32768.0, 1.0, 32.0)])
def test_frequencies(args):
    names = ("factor", "original", "low", "high")
    got = mnb.mnb_rope_frequencies(*args[:2], **dict(zip(names, args[2:])))
    want = torch.tensor(ref.frequencies(*args), dtype=torch.float64)
    assert got.shape == want.shape and torch.all((got - want).abs() <= 1e-14 * want)


def test_frequencies_by_parts_keep_the_fast_and_slow_the_slow():
    plain = mnb.mnb_rope_frequencies(128, 1e6)
    got = mnb.mnb_rope_frequencies(128, 1e6, factor=4.0, original=32768.0, low=1.0, high=32.0)
    turns = 32768.0 * plain / (2 * math.pi)
    assert torch.equal(got[turns >= 32], plain[turns >= 32])
    assert torch.equal(got[turns <= 1], plain[turns <= 1] / 4)
    assert torch.all((got <= plain) & (got >= plain / 4))


@pytest.mark.parametrize("change", [
    dict(rot=0), dict(rot=3), dict(rot=258), dict(base=0.0), dict(base=-1.0), dict(base=INF),
    dict(factor=0.0), dict(factor=NAN), dict(original=-1.0), dict(original=INF),
    dict(original=10.0, low=2.0, high=2.0), dict(original=10.0, low=-1.0),
    dict(original=10.0, high=NAN)])
def test_frequency_refusals(lib, change):
    a = dict(dict(rot=64, base=1e4, factor=2.0, original=0.0, low=1.0, high=32.0), **change)
    out = (ctypes.c_double * 256)()
    assert lib.mnb_rope_frequencies(a["rot"], a["base"], a["factor"], a["original"], a["low"],
                                    a["high"], out) == b.MNB_ERR_SHAPE
    assert lib.mnb_rope_frequencies(64, 1e4, 1.0, 0.0, 1.0, 32.0, None) == b.MNB_ERR_NULL


@pytest.mark.parametrize("change,status", [
    (dict(f=0), b.MNB_ERR_NULL), (dict(cos=0), b.MNB_ERR_NULL), (dict(sin=0), b.MNB_ERR_NULL),
    (dict(rot=1), b.MNB_ERR_SHAPE), (dict(rot=0), b.MNB_ERR_SHAPE),
    (dict(rot=300), b.MNB_ERR_SHAPE), (dict(first=-1), b.MNB_ERR_SHAPE),
    (dict(n=0), b.MNB_ERR_SHAPE), (dict(first=BIG - 10), b.MNB_ERR_SHAPE),
    (dict(mag=NAN), b.MNB_ERR_SHAPE), (dict(mag=1e300), b.MNB_ERR_SHAPE),
    (dict(value=INF), b.MNB_ERR_SHAPE), (dict(cos=COS + 2), b.MNB_ERR_ALIGN),
    (dict(sin=COS + 4), b.MNB_ERR_ALIAS)])
def test_table_refusals(lib, change, status):
    a = dict(dict(f=1, value=0.5, rot=64, first=0, n=100, mag=1.0, cos=COS, sin=SIN), **change)
    f = (ctypes.c_double * 256)(*([0.5] * 31 + [a["value"]] + [0.5] * 200))
    assert lib.mnb_rope_table(f if a["f"] else None, a["rot"], a["first"], a["n"], a["mag"],
                              a["cos"] or None, a["sin"] or None, None) == status


def norm_rope(lib, q=None, k=0, T=10, D=64, dt=BF16, gq=GQ, gk=GK, eps=1e-6, r=0, pos=POS, qo=None,
              ko=0):
    q = heads(Q) if q is None else q
    qo = heads(QO) if qo is None else qo
    k = heads(K, 2) if k == 0 else k
    ko = heads(KO, 2) if ko == 0 else ko
    r = rope() if r == 0 else r
    return lib.mnb_qk_norm_rope(by(q or None), by(k), T, D, dt, gq or None, gk or None, eps, by(r),
                                pos or None, by(qo or None), by(ko), None)


@pytest.mark.parametrize("change,status", [
    (dict(q=False), b.MNB_ERR_NULL), (dict(qo=False), b.MNB_ERR_NULL),
    (dict(k=None), b.MNB_ERR_NULL), (dict(ko=None), b.MNB_ERR_NULL),
    (dict(r=None), b.MNB_ERR_NULL), (dict(pos=0), b.MNB_ERR_NULL),
    (dict(q=heads(0)), b.MNB_ERR_NULL), (dict(r=rope(cos=0)), b.MNB_ERR_NULL),
    (dict(T=0), b.MNB_ERR_SHAPE), (dict(T=BIG), b.MNB_ERR_SHAPE), (dict(D=63), b.MNB_ERR_SHAPE),
    (dict(D=0), b.MNB_ERR_SHAPE), (dict(eps=-1.0), b.MNB_ERR_SHAPE),
    (dict(eps=NAN), b.MNB_ERR_SHAPE), (dict(eps=INF), b.MNB_ERR_SHAPE),
    (dict(q=heads(Q, 0)), b.MNB_ERR_SHAPE), (dict(q=heads(Q, ts=-1)), b.MNB_ERR_SHAPE),
    (dict(q=heads(Q, reserved=1)), b.MNB_ERR_SHAPE),
    (dict(qo=heads(QO, 2)), b.MNB_ERR_SHAPE), (dict(ko=heads(KO, 4)), b.MNB_ERR_SHAPE),
    (dict(r=rope(rot=66)), b.MNB_ERR_SHAPE), (dict(r=rope(rot=0)), b.MNB_ERR_SHAPE),
    (dict(r=rope(rot=31)), b.MNB_ERR_SHAPE), (dict(r=rope(positions=0)), b.MNB_ERR_SHAPE),
    (dict(r=rope(inter=2)), b.MNB_ERR_SHAPE),
    (dict(D=258, q=heads(Q, hs=258, ts=1032), k=None, ko=None,
          qo=heads(QO, hs=258, ts=1032)), b.MNB_ERR_UNSUPPORTED),
    (dict(dt=3), b.MNB_ERR_DTYPE), (dict(q=heads(Q + 1)), b.MNB_ERR_ALIGN),
    (dict(dt=F32, k=heads(K + 2, 2)), b.MNB_ERR_ALIGN), (dict(gq=GQ + 2), b.MNB_ERR_ALIGN),
    (dict(pos=POS + 1), b.MNB_ERR_ALIGN), (dict(r=rope(sin=SIN + 2)), b.MNB_ERR_ALIGN),
    (dict(qo=heads(Q + 128)), b.MNB_ERR_ALIAS), (dict(qo=heads(K)), b.MNB_ERR_ALIAS),
    (dict(ko=heads(QO + 2, 2)), b.MNB_ERR_ALIAS), (dict(qo=heads(POS)), b.MNB_ERR_ALIAS),
    (dict(qo=heads(COS)), b.MNB_ERR_ALIAS), (dict(ko=heads(GK, 2)), b.MNB_ERR_ALIAS),
    (dict(qo=heads(QO, ts=64)), b.MNB_ERR_ALIAS), (dict(qo=heads(QO, hs=32)), b.MNB_ERR_ALIAS),
    (dict(qo=heads(QO, ts=0)), b.MNB_ERR_ALIAS)])
def test_norm_rope_refusals(lib, change, status):
    assert norm_rope(lib, **change) == status


def test_rows_of_one_matrix_do_not_overlap(lib):
    """Slices of a fused row are apart although their ends interleave; the call gets as far as the
    device."""
    row = 8 * 64
    q, k = heads(Q, 4, ts=row), heads(Q + 4 * 128, 2, ts=row)
    assert norm_rope(lib, q=q, k=k, qo=q, ko=k) in (b.MNB_ERR_DEVICE, b.MNB_ERR_CUDA)
    assert norm_rope(lib, q=q, k=k, qo=heads(Q + 6 * 128, 2 + 2, ts=row),
                     ko=k) == b.MNB_ERR_ALIAS  # past the row, into the next one's q


def append(lib, q=None, k=None, v=None, T=10, gq=GQ, gk=GK, eps=1e-6, r=0, c=None, bt=None,
           qo=None):
    q = heads(Q) if q is None else q
    qo = heads(QO) if qo is None else qo
    k = heads(K, 2) if k is None else k
    v = heads(V, 2) if v is None else v
    c, bt = cache() if c is None else c, batch() if bt is None else bt
    return lib.mnb_cache_append(by(q or None), by(k or None), by(v or None), T, gq or None,
                                gk or None, eps, by(rope() if r == 0 else r), by(c or None),
                                by(bt or None), by(qo or None), None)


CACHES = [
    (dict(c=False), b.MNB_ERR_NULL), (dict(bt=False), b.MNB_ERR_NULL),
    (dict(c=cache(k=0)), b.MNB_ERR_NULL), (dict(c=cache(v=0)), b.MNB_ERR_NULL),
    (dict(bt=batch(s=0)), b.MNB_ERR_NULL), (dict(bt=batch(l=0)), b.MNB_ERR_NULL),
    (dict(bt=batch(t=0)), b.MNB_ERR_NULL), (dict(c=cache(dt=7)), b.MNB_ERR_DTYPE),
    (dict(c=cache(pages=0)), b.MNB_ERR_SHAPE), (dict(c=cache(pages=BIG)), b.MNB_ERR_SHAPE),
    (dict(c=cache(ps=8)), b.MNB_ERR_SHAPE), (dict(c=cache(ps=24)), b.MNB_ERR_SHAPE),
    (dict(c=cache(H=0)), b.MNB_ERR_SHAPE), (dict(c=cache(k_token_stride=32)), b.MNB_ERR_SHAPE),
    (dict(c=cache(v_page_stride=0)), b.MNB_ERR_SHAPE),
    (dict(c=cache(v_head_stride=-64)), b.MNB_ERR_SHAPE),
    (dict(bt=batch(n=0)), b.MNB_ERR_SHAPE), (dict(bt=batch(pages=0)), b.MNB_ERR_SHAPE),
    (dict(bt=batch(stride=3)), b.MNB_ERR_SHAPE),
    (dict(bt=batch(pages=BIG // 16)), b.MNB_ERR_SHAPE),
    (dict(T=0), b.MNB_ERR_SHAPE), (dict(T=BIG), b.MNB_ERR_SHAPE),
    (dict(c=cache(k=CK + 1)), b.MNB_ERR_ALIGN), (dict(bt=batch(s=STA + 2)), b.MNB_ERR_ALIGN),
    (dict(bt=batch(t=TAB + 1)), b.MNB_ERR_ALIGN), (dict(c=cache(k=CV)), b.MNB_ERR_ALIAS)]


@pytest.mark.parametrize("change,status", CACHES + [
    (dict(q=False), b.MNB_ERR_NULL), (dict(qo=False), b.MNB_ERR_NULL),
    (dict(k=False), b.MNB_ERR_NULL), (dict(v=False), b.MNB_ERR_NULL),
    (dict(k=heads(K, 4)), b.MNB_ERR_SHAPE), (dict(v=heads(V, 1)), b.MNB_ERR_SHAPE),
    (dict(qo=heads(QO, 5)), b.MNB_ERR_SHAPE), (dict(eps=-1.0), b.MNB_ERR_SHAPE),
    (dict(c=cache(D=258)), b.MNB_ERR_UNSUPPORTED), (dict(c=cache(D=63)), b.MNB_ERR_SHAPE),
    (dict(r=rope(rot=128)), b.MNB_ERR_SHAPE), (dict(k=heads(K + 1, 2)), b.MNB_ERR_ALIGN),
    (dict(k=heads(CK, 2)), b.MNB_ERR_ALIAS), (dict(v=heads(CV + 256, 2)), b.MNB_ERR_ALIAS),
    (dict(qo=heads(CK)), b.MNB_ERR_ALIAS), (dict(qo=heads(K)), b.MNB_ERR_ALIAS),
    (dict(qo=heads(V)), b.MNB_ERR_ALIAS), (dict(qo=heads(TAB)), b.MNB_ERR_ALIAS),
    (dict(gk=CK + 4), b.MNB_ERR_ALIAS), (dict(bt=batch(l=CV)), b.MNB_ERR_ALIAS)])
def test_append_refusals(lib, change, status):
    assert append(lib, **change) == status


def attention(lib, q=None, T=10, c=None, bt=None, scale=0.125, window=0, o=None, ws=WS,
              ws_bytes=1 << 30):
    q = heads(Q) if q is None else q
    o = heads(QO) if o is None else o
    c, bt = cache() if c is None else c, batch() if bt is None else bt
    return lib.mnb_paged_attention(by(q or None), T, by(c or None), by(bt or None), scale, window,
                                   by(o or None), ws or None, ws_bytes, None)


@pytest.mark.parametrize("change,status", CACHES + [
    (dict(q=False), b.MNB_ERR_NULL), (dict(o=False), b.MNB_ERR_NULL), (dict(ws=0), b.MNB_ERR_NULL),
    (dict(q=heads(Q, 3), o=heads(QO, 3)), b.MNB_ERR_SHAPE), (dict(o=heads(QO, 2)), b.MNB_ERR_SHAPE),
    (dict(scale=NAN), b.MNB_ERR_SHAPE), (dict(scale=INF), b.MNB_ERR_SHAPE),
    (dict(window=-1), b.MNB_ERR_SHAPE), (dict(ws_bytes=16), b.MNB_ERR_SHAPE),
    (dict(c=cache(D=80), o=heads(QO, ts=320, hs=80)), b.MNB_ERR_UNSUPPORTED),
    (dict(c=cache(D=256), o=heads(QO, ts=1024, hs=256)), b.MNB_ERR_UNSUPPORTED),
    (dict(q=heads(Q + 2)), b.MNB_ERR_ALIGN), (dict(o=heads(QO + 8)), b.MNB_ERR_ALIGN),
    (dict(q=heads(Q, ts=260)), b.MNB_ERR_ALIGN), (dict(o=heads(QO, ts=512, hs=68)), b.MNB_ERR_ALIGN),
    (dict(c=cache(k=CK + 8)), b.MNB_ERR_ALIGN),
    (dict(c=cache(v_token_stride=66)), b.MNB_ERR_ALIGN), (dict(ws=WS + 16), b.MNB_ERR_ALIGN),
    (dict(o=heads(Q)), b.MNB_ERR_ALIAS), (dict(o=heads(CK)), b.MNB_ERR_ALIAS),
    (dict(ws=CV), b.MNB_ERR_ALIAS), (dict(ws=QO), b.MNB_ERR_ALIAS),
    (dict(o=heads(QO, ts=128)), b.MNB_ERR_ALIAS), (dict(o=heads(TAB)), b.MNB_ERR_ALIAS)])
def test_attention_refusals(lib, change, status):
    assert attention(lib, **change) == status


def test_workspace_size_of_refused_arguments(lib):
    size = lambda T=10, hq=4, c=None, bt=None: lib.mnb_paged_attention_workspace_size(  # noqa: E731
        T, hq, by(c or cache()), by(bt or batch()))
    assert size() > 0 and size() % 4 == 0
    assert size(T=0) == size(hq=3) == size(c=cache(D=96)) == size(bt=batch(n=0)) == 0
    assert lib.mnb_paged_attention_workspace_size(10, 4, None, by(batch())) == 0


def test_valid_calls_get_as_far_as_the_device(lib):
    """What the refusals vary is in order: on a machine without the GPU the device check ends it."""
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    for st in (norm_rope(lib), append(lib), attention(lib), norm_rope(lib, k=None, ko=None),
               norm_rope(lib, r=None, pos=0), append(lib, q=False, qo=False, r=None),
               norm_rope(lib, qo=heads(Q), ko=heads(K, 2)), append(lib, qo=heads(Q)),
               attention(lib, window=5, scale=-1.0)):
        assert st in (b.MNB_ERR_DEVICE, b.MNB_ERR_CUDA)


def test_binding_refuses_what_it_cannot_describe():
    t = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        mnb.mnb_qk_norm_rope(t, None, None, None)  # not on a GPU
    with pytest.raises(ValueError):
        mnb.mnb_rope_table(torch.zeros(3), 10)     # not float64
    with pytest.raises(ValueError):
        mnb.mnb_paged_attention(t, mnb.KvCache(t, t), mnb.KvBatch(t, t, t))


def test_frequencies_by_parts_ramp_over_the_turns_and_not_over_the_index():
    """What the header says of the other ramp in use, with its formulas: a caller who needs it can
    tell that these are not its frequencies."""
    rot, base, original, factor, low, high = 128, 1e6, 32768.0, 4.0, 1.0, 32.0
    plain = mnb.mnb_rope_frequencies(rot, base)
    here = mnb.mnb_rope_frequencies(rot, base, factor=factor, original=original, low=low, high=high)
    d = lambda n: rot * math.log(original / (2 * math.pi * n)) / (2 * math.log(base))  # noqa: E731
    first, last = math.floor(d(high)), math.ceil(d(low))
    r = ((last - torch.arange(rot // 2, dtype=torch.float64)) / (last - first)).clamp(0, 1)
    there = (1 - r) * plain / factor + r * plain
    apart = (here / there - 1).abs()
    assert int((apart > 0.01).sum()) == 16 and int(apart.argmax()) == 32
    assert abs(float(here[32] / plain[32]) - 0.352) < 5e-4
    assert abs(float(there[32] / plain[32]) - 0.603) < 5e-4
    assert torch.equal(here[:first + 1], plain[:first + 1])
    assert torch.equal(here[last:], plain[last:] / factor)


def test_attention_between_slices_of_one_matrix(lib):
    """Rows of q and of the result side by side in one matrix: apart, although their ends interleave;
    not so where they share an element, or the workspace lies among the rows of q."""
    row = 8 * 64
    q, o = heads(Q, 4, ts=row), heads(Q + 4 * 128, 4, ts=row)
    assert attention(lib, q=q, o=o) in (b.MNB_ERR_DEVICE, b.MNB_ERR_CUDA)
    assert attention(lib, q=o, o=q) in (b.MNB_ERR_DEVICE, b.MNB_ERR_CUDA)
    assert attention(lib, q=q, o=heads(Q + 4 * 128 - 16, 4, ts=row)) == b.MNB_ERR_ALIAS
    assert attention(lib, q=q, o=heads(Q + 5 * 128, 4, ts=row)) == b.MNB_ERR_ALIAS  # the next row's
    assert attention(lib, q=q, ws=Q + 256) == b.MNB_ERR_ALIAS
    assert attention(lib, q=q, o=q) == b.MNB_ERR_ALIAS
