"""GPU parity of the mixture-of-experts operators (mnb_moe_route, mnb_matmul_experts, mnb_moe)
against their definition in 64 bits (moe_reference.py)."""
import copy
import dataclasses
import math
import threading

import pytest
import torch

import int4_weight_only_matmulnbits_gb300 as mnb
from int4_weight_only_matmulnbits_gb300 import binding

from . import moe_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    mnb.build_library()
    mnb.load()
    return torch.device("cuda:0")


def stack(g, E, N, K, bs, sdt, zp, bias):
    """(B, scales, zero points, bias) of E seeded weights, on the CPU."""
    nb = -(-K // bs)
    B = torch.randint(0, 256, (E, N, nb, bs // 2), generator=g, dtype=torch.uint8)
    s = (torch.rand(E, N, nb, generator=g) * 0.015 + 0.005).to(sdt)
    z = (torch.randint(0, 256, (E, N, (nb + 1) // 2), generator=g, dtype=torch.uint8)
         if zp else None)
    b = torch.randn(E, N, generator=g) * 0.05 if bias else None
    return B, s, z, b


def to(dev, *ts):
    return [None if t is None else t.to(dev) for t in ts]


def pack(dev, w, N, K, bs):
    B, s, z, b = to(dev, *w)
    return mnb.mnb_prepack_experts(B, s, z, N, K, bs), b, ref.dequant(B, s, z, K)


# ---- packing -------------------------------------------------------------------------------

@pytest.mark.parametrize("bs", [16, 32, 256])
@pytest.mark.parametrize("E,N,K", [(1, 1, 1), (3, 16, 64), (2, 33, 130), (5, 48, 257)])
@pytest.mark.parametrize("zp", [False, True])
def test_pack_is_the_padded_stack(dev, bs, E, N, K, zp):
    """The packed stack is mnb_prepack's of the E * Np rows with zero padding."""
    g = torch.Generator().manual_seed(bs + N)
    B, s, z, _ = to(dev, *stack(g, E, N, K, bs, F32, zp, False))
    w = mnb.mnb_prepack_experts(B, s, z, N, K, bs)
    Np = -(-N // 16) * 16
    pad = lambda t: None if t is None else torch.nn.functional.pad(
        t, (0, 0) * (t.dim() - 2) + (0, Np - N)).reshape(E * Np, *t.shape[2:]).contiguous()
    plain = mnb.mnb_prepack(pad(B), pad(s), pad(z), E * Np, K, bs)
    assert torch.equal(w.packed_scales, plain.packed_scales)
    assert torch.equal(w.packed_b, plain.packed_b)
    assert (z is None) == (w.packed_zp is None)
    if zp:
        assert torch.equal(w.packed_zp, plain.packed_zp)
    # Row factors: powers of two that bring the largest scale into 2^14 .. 2^15.
    fac, most = w.packed_rows[:-E].view(E, Np), w.packed_rows[-E:]
    assert torch.equal(most, s.abs().amax((1, 2)))
    assert (torch.frexp(fac).mantissa == 0.5).all()
    top = s.abs().amax(2) * fac[:, :N]
    assert ((top >= 2.0 ** 14) & (top < 2.0 ** 15)).all()


# ---- router --------------------------------------------------------------------------------

def check_route(logits, k, normalize):
    r = mnb.mnb_moe_route(logits, k, normalize=normalize)
    w, e, off, order = ref.route(logits, k, normalize)
    assert torch.equal(r.experts.cpu().long(), e)
    assert torch.equal(r.offsets.cpu().long(), off)
    assert torch.equal(r.order.cpu().long(), order)
    # exp within 2 steps, a sum of E terms, a division: (E + 8) 2^-24.
    E = logits.shape[1]
    assert ((r.weights.cpu().double() - w).abs() <= (E + 8) * 2.0 ** -24 * w + 1e-37).all()
    return r


@pytest.mark.parametrize("M,E,k", [(1, 1, 1), (1, 128, 8), (2, 7, 7), (5, 33, 4), (31, 64, 6),
                                   (32, 128, 8), (33, 8, 2), (100, 256, 8), (257, 60, 5),
                                   (3, 1024, 32), (700, 16, 3)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("normalize", [True, False])
def test_route(dev, M, E, k, dtype, normalize):
    g = torch.Generator().manual_seed(M * 7 + E)
    check_route(torch.randn(M, E, generator=g).to(dtype).to(dev), k, normalize)


@pytest.mark.parametrize("E", [4, 60, 64, 96, 128, 200, 256])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_route_alignment(dev, E, dtype):
    """Rows that start off the piece a lane loads give what aligned ones do, ties included."""
    g = torch.Generator().manual_seed(E)
    x = (torch.randint(-8, 8, (9, E), generator=g) / 4).to(dtype).to(dev)
    want = check_route(x, 4, True)
    for off in (1, 2, 4):
        room = torch.zeros(9 * E + off, dtype=dtype, device=dev)
        y = room[off:].view(9, E)
        y.copy_(x)
        assert all(torch.equal(a, b) for a, b in zip(want, mnb.mnb_moe_route(y, 4)))


@pytest.mark.parametrize("M", [4, 300])
@pytest.mark.parametrize("normalize", [True, False])
def test_route_ties(dev, M, normalize):
    """Few distinct values, both zeros among them: the lowest index wins."""
    g = torch.Generator().manual_seed(5)
    values = torch.tensor([-1.0, -0.0, 0.0, 0.5])
    x = values[torch.randint(0, 4, (M, 48), generator=g)]
    check_route(x.to(dev), 6, normalize)
    check_route(x.to(BF16).to(dev), 6, normalize)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("normalize", [True, False])
def test_route_masks_and_extremes(dev, dtype, normalize):
    """-inf and NaN are masked (some, all but few, all), the lowest finite value is not;
    +inf takes the whole weight."""
    E, k = 40, 5
    x = torch.randn(8, E, generator=torch.Generator().manual_seed(3)).to(dtype)
    x[0, ::2] = -math.inf
    x[1, 1:] = math.nan
    x[2] = -math.inf
    x[3, 3:] = -math.inf
    x[3, 1] = math.nan
    x[4] = torch.finfo(dtype).min
    x[5, 7] = x[5, 30] = math.inf
    x[6] = torch.finfo(dtype).max
    r = check_route(x.to(dev), k, normalize)
    assert (r.experts[2] == -1).all() and (r.weights[2] == 0).all()
    assert r.experts[1].tolist() == [0, -1, -1, -1, -1]
    assert r.experts[5, :2].tolist() == [7, 30] and r.weights[5, :2].tolist() == [0.5, 0.5]


@pytest.mark.parametrize("M,E,k", [(4099, 128, 8), (20000, 64, 2), (9000, 256, 8)])
def test_route_many_rows(dev, M, E, k):
    """Long inputs against torch's stable sort (the choice is exact)."""
    g = torch.Generator().manual_seed(M)
    x = torch.randn(M, E, generator=g).to(BF16).to(dev)
    x[::17, : E // 2] = -math.inf
    x[5::1000] = -math.inf
    r = mnb.mnb_moe_route(x, k)
    top, idx = torch.sort(x.double(), dim=1, descending=True, stable=True)
    idx = torch.where(top > -math.inf, idx, -1)[:, :k]
    assert torch.equal(r.experts.long(), idx)
    p = torch.exp(top[:, :k] - top[:, :1]).nan_to_num(0.0)
    w = (p / p.sum(1, keepdim=True)).nan_to_num(0.0)
    assert ((r.weights.double() - w).abs() <= (E + 8) * 2.0 ** -24 * w + 1e-37).all()
    key = torch.where(idx < 0, E, idx).flatten()
    assert torch.equal(r.order.long(), torch.sort(key, stable=True).indices)
    assert torch.equal(r.offsets.long(),
                       torch.searchsorted(torch.sort(key).values, torch.arange(E + 1, device=dev)))
    again = mnb.mnb_moe_route(x, k)
    assert all(torch.equal(a, b) for a, b in zip(r, again))


@pytest.mark.parametrize("M,E,k", [(12160, 128, 8), (12300, 128, 8), (400000, 64, 8),
                                   (24000, 64, 8), (1400, 1000, 8), (1600, 1000, 8),
                                   (130, 1024, 32), (3000, 1024, 32), (3200000, 3, 1)])
@pytest.mark.parametrize("masked", [False, True])
def test_route_lists_of_many_slots(dev, M, E, k, masked):
    """Either way of summing the sort's counts, on both sides of where the choice changes;
    slots without an expert come last."""
    g = torch.Generator(device=dev).manual_seed(M)
    x = torch.randn(M, E, generator=g, device=dev).to(BF16)
    if masked:
        x[:, E // 2:] = -math.inf
        x[3::7] = -math.inf
    r = mnb.mnb_moe_route(x, k)
    key = torch.where(r.experts < 0, E, r.experts).flatten()
    assert torch.equal(r.order.long(), torch.sort(key, stable=True).indices)
    assert torch.equal(r.offsets.long(), torch.searchsorted(
        torch.sort(key).values, torch.arange(E + 1, device=dev, dtype=torch.int32)))
    assert ((r.experts < 0) == (r.weights == 0)).all()


# ---- products --------------------------------------------------------------------------------

def run_experts(dev, M, E, k, N, K, bs, dtype, *, sdt=None, zp=False, bias=False,
                per_slot=False, table=None, seed=0):
    g = torch.Generator().manual_seed(seed)
    w, b, W = pack(dev, stack(g, E, N, K, bs, sdt or dtype, zp, bias), N, K, bs)
    A = torch.randn(*((M, k, K) if per_slot else (M, K)), generator=g).to(dtype).to(dev)
    if table is None:
        table = torch.randint(0, E, (M, k), generator=g, dtype=torch.int32)
    table = table.to(dev)
    room = torch.full((M + 1, k, N), 77.0, dtype=dtype, device=dev)
    Y = mnb.mnb_matmul_experts(A, w, table, b, out=room[:M])
    assert (room[M:] == 77.0).all()
    a = A.double() if per_slot else A.double().unsqueeze(1).expand(M, k, K)
    R, err = ref.products(a, W, table, b, dtype)
    what = f"M{M} E{E} k{k} N{N} K{K} bs{bs}"
    ref.check(Y, R, err, what)
    none = (table < 0) | (table >= E)
    assert (Y[none] == 0).all()
    assert torch.equal(Y, mnb.mnb_matmul_experts(A, w, table, b)), "not reproducible"
    return Y


@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("zp", [False, True])
def test_experts_tails(dev, bs, dtype, zp):
    """Ragged N and K, one expert to many, few slots to many, both row forms."""
    i = 0
    for N, K in ((1, 1), (7, bs + 1), (33, 72), (129, 257), (80, 640)):
        for M, k, E in ((1, 1, 1), (1, 8, 12), (3, 2, 5), (17, 4, 6), (70, 3, 4)):
            i += 1
            run_experts(dev, M, E, k, N, K, bs, dtype, zp=zp, bias=i % 2 == 0,
                        per_slot=i % 3 == 0, seed=100 * bs + i)


@pytest.mark.parametrize("adt,sdt", [(F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("M", [2, 90])
def test_experts_mixed_scale_types(dev, adt, sdt, M):
    for bs, zp in ((16, True), (32, False), (64, True)):
        run_experts(dev, M, 3, 2, 96, 512, bs, adt, sdt=sdt, zp=zp, bias=True, seed=bs + M)


@pytest.mark.parametrize("M", [6, 150])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_experts_empty_and_repeated(dev, M, dtype):
    """Rows without an expert (-1 and other indices outside), one expert named twice in a row,
    experts nobody names, and tables that are all empty or all one expert."""
    E, k = 9, 4
    g = torch.Generator().manual_seed(M)
    t = torch.randint(0, E, (M, k), generator=g, dtype=torch.int32)
    t[t == 3] = 4
    t[1] = -1
    t[2] = torch.tensor([5, 5, 5, -7], dtype=torch.int32)
    t[3, 1], t[4, 2] = E, 2 ** 31 - 1
    for per_slot in (False, True):
        run_experts(dev, M, E, k, 70, 320, 32, dtype, bias=True, table=t, per_slot=per_slot)
        run_experts(dev, M, E, k, 70, 320, 32, dtype, table=torch.full_like(t, -1),
                    per_slot=per_slot)
        run_experts(dev, M, E, k, 70, 320, 32, dtype, table=torch.full_like(t, 6),
                    per_slot=per_slot)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,k,E,N,K", [(1, 8, 64, 768, 2560), (9, 2, 8, 512, 1024),
                                       (40, 6, 24, 208, 1111), (400, 4, 16, 264, 704),
                                       (700, 8, 5, 136, 2048), (33, 1, 1, 1000, 4096)])
def test_experts_larger(dev, M, k, E, N, K, dtype):
    run_experts(dev, M, E, k, N, K, 32, dtype, zp=N % 3 == 0, bias=M > 8, per_slot=k % 2 == 0,
                seed=M)


def test_experts_wide_magnitudes(dev):
    """Rows of very different size, values beyond the range of fp16, zeros and one large value
    among small ones: each row is as exact as the others."""
    for M, dtype in ((5, F32), (5, BF16), (130, F32), (130, BF16)):
        g = torch.Generator().manual_seed(M)
        E, k, N, K, bs = 4, 2, 64, 512, 32
        w, _, W = pack(dev, stack(g, E, N, K, bs, F32, True, False), N, K, bs)
        A = torch.randn(M, K, generator=g) * 10.0 ** torch.randint(-20, 15, (M, 1), generator=g)
        A[1] = 0
        A[2] = torch.randn(K, generator=g) * 1e-3
        A[2, 17] = 3e6
        A = A.to(dtype).to(dev)
        t = torch.randint(0, E, (M, k), generator=g, dtype=torch.int32).to(dev)
        R, err = ref.products(A.double().unsqueeze(1).expand(M, k, K), W, t, None, dtype)
        ref.check(mnb.mnb_matmul_experts(A, w, t), R, err, f"M{M} {dtype}")


@pytest.mark.parametrize("M", [3, 140])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -60, 2.0 ** 20])
@pytest.mark.parametrize("code", [0x00, 0xFF])
def test_experts_largest_scales(dev, M, dtype, size, code):
    """Scales of 2^80, the largest that the products take, with every term of one sign and
    every code at its end: no sum on the way overflows, whatever the activations' size."""
    E, k, N = 3, 2, 40
    for K, bs in ((2560, 32), (16384, 128)):
        B = torch.full((E, N, K // bs, bs // 2), code, dtype=torch.uint8)
        z = torch.full((E, N, (K // bs + 1) // 2), 0xFF - code, dtype=torch.uint8)
        s = torch.full((E, N, K // bs), 2.0 ** 80, dtype=dtype)
        for zp in (None, z):
            w, _, W = pack(dev, (B, s, zp, None), N, K, bs)
            A = torch.full((M, K), size, dtype=dtype, device=dev)
            t = torch.randint(0, E, (M, k), dtype=torch.int32).to(dev)
            R, err = ref.products(A.double().unsqueeze(1).expand(M, k, K), W, t, None, dtype)
            ref.check(mnb.mnb_matmul_experts(A, w, t), R, err, f"K{K}")


# ---- the layer ---------------------------------------------------------------------------------

def layer_inputs(dev, M, E, k, H, I, bs, dtype, *, sdt=None, zp=False, bias=False, seed=0,
                 bs_down=None):
    g = torch.Generator().manual_seed(seed)
    ws = [pack(dev, stack(g, E, N, K, b, sdt or dtype, zp, bias), N, K, b)
          for N, K, b in ((I, H, bs), (I, H, bs), (H, I, bs_down or bs))]
    X = torch.randn(M, H, generator=g).to(dtype).to(dev)
    logits = torch.randn(M, E, generator=g).to(dev)
    return X, logits, ws


def run_layer(dev, X, logits, ws, k, normalize=True, what=""):
    (wg, bg, Wg), (wu, bu, Wu), (wd, bd, Wd) = ws
    M, H = X.shape
    room = torch.full((M + 1, H), 77.0, dtype=X.dtype, device=dev)
    kw = dict(normalize=normalize, bias_gate=bg, bias_up=bu, bias_down=bd)
    Y = mnb.mnb_moe(X, logits, wg, wu, wd, k, out=room[:M], **kw)
    assert (room[M:] == 77.0).all()
    weights, experts, _, _ = ref.route(logits, k, normalize)
    R, err = ref.layer(X, weights, experts.to(dev), Wg, Wu, Wd, bg, bu, bd, X.dtype)
    ref.check(Y, R, err, what)
    assert torch.equal(Y, mnb.mnb_moe(X, logits, wg, wu, wd, k, **kw)), "not reproducible"
    return Y


@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("zp", [False, True])
def test_layer_tails(dev, bs, dtype, zp):
    i = 0
    for H, I in ((1, 1), (bs + 1, 7), (130, 72), (200, 257)):
        for M, k, E in ((1, 1, 1), (1, 4, 9), (5, 2, 3), (20, 3, 6), (65, 2, 4)):
            i += 1
            x = layer_inputs(dev, M, E, k, H, I, bs, dtype, zp=zp, bias=i % 2 == 0, seed=bs + i)
            run_layer(dev, *x, k, normalize=i % 3 != 0, what=f"M{M} E{E} k{k} H{H} I{I} bs{bs}")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,k,E,H,I,bs", [(1, 8, 128, 1024, 512, 32), (16, 8, 64, 512, 768, 32),
                                          (33, 4, 20, 1000, 520, 64), (150, 6, 16, 640, 352, 128),
                                          (600, 8, 8, 512, 256, 32), (300, 2, 40, 264, 136, 16)])
def test_layer_larger(dev, M, k, E, H, I, bs, dtype):
    x = layer_inputs(dev, M, E, k, H, I, bs, dtype, zp=M % 2 == 0, bias=M > 100, seed=M,
                     bs_down=32)
    run_layer(dev, *x, k, what=f"M{M}")


@pytest.mark.parametrize("M", [3, 140])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_layer_scale_outliers(dev, M, dtype):
    """One block of each expert's three weights is 64 times as large as the others, and small
    activations with one large one: the bounds that values are scaled by lie far above them."""
    E, k, H, I, bs = 6, 2, 320, 256, 32
    g = torch.Generator().manual_seed(M)
    ws = []
    for N, K in ((I, H), (I, H), (H, I)):
        B, s, z, b = stack(g, E, N, K, bs, dtype, False, False)
        s[:, N // 3, 1] *= 64
        ws.append(pack(dev, (B, s, z, b), N, K, bs))
    X = torch.randn(M, H, generator=g) * 0.05
    X[:, 7] = 20
    logits = torch.randn(M, E, generator=g).to(dev)
    run_layer(dev, X.to(dtype).to(dev), logits, ws, k, what="outliers")


@pytest.mark.parametrize("M", [3, 140])
@pytest.mark.parametrize("factor", [1, 16])
def test_layer_outliers_cost_no_bits(dev, M, factor):
    """Scales of a block `factor` times the others, met by zero activations: what is left keeps
    its precision. Norm-wise: the output's rounding to bf16 is at most 2^-8 of each element; the
    roundings of weights and hidden values (2^-11 each, twice) have random signs and grow no
    more than what they belong to: 2^-8 + 4 2^-11 of the result's norm."""
    E, k, H, I, bs = 6, 2, 1024, 768, 32
    g = torch.Generator().manual_seed(M)
    ws = []
    for N, K in ((I, H), (I, H), (H, I)):
        B, s, z, b = stack(g, E, N, K, bs, BF16, False, False)
        s[:, N // 3, 1] *= factor
        ws.append(pack(dev, (B, s, z, b), N, K, bs))
    X = (torch.randn(M, H, generator=g) * 0.05).to(BF16).to(dev)
    X[:, 32:64] = 0
    logits = torch.randn(M, E, generator=g).to(dev)
    weights, experts, _, _ = ref.route(logits, k, True)
    R, _ = ref.layer(X, weights, experts.to(dev), *[W for _, _, W in ws], None, None, None, BF16)
    err = mnb.mnb_moe(X, logits, *[w for w, _, _ in ws], k).double() - R
    plain = torch.arange(H, device=dev) != H // 3  # the row with the large scale has its own size
    assert err[:, plain].norm() <= (2.0 ** -8 + 4 * 2.0 ** -11) * R[:, plain].norm()


@pytest.mark.parametrize("M", [3, 140])
@pytest.mark.parametrize("factor", [64, 256, 1024])
def test_layer_large_outliers_cost_no_bits(dev, M, factor):
    """The same with larger blocks, at the width of a real layer."""
    E, k, H, I, bs = 6, 2, 2560, 768, 32
    g = torch.Generator().manual_seed(M)
    ws = []
    for N, K in ((I, H), (I, H), (H, I)):
        B, s, z, b = stack(g, E, N, K, bs, BF16, False, False)
        s[:, N // 3, 1] *= factor
        ws.append(pack(dev, (B, s, z, b), N, K, bs))
    X = (torch.randn(M, H, generator=g) * 0.05).to(BF16).to(dev)
    X[:, 32:64] = 0
    logits = torch.randn(M, E, generator=g).to(dev)
    weights, experts, _, _ = ref.route(logits, k, True)
    R, _ = ref.layer(X, weights, experts.to(dev), *[W for _, _, W in ws], None, None, None, BF16)
    err = mnb.mnb_moe(X, logits, *[w for w, _, _ in ws], k).double() - R
    plain = torch.arange(H, device=dev) != H // 3
    assert err[:, plain].norm() <= (2.0 ** -8 + 4 * 2.0 ** -11) * R[:, plain].norm()


@pytest.mark.parametrize("M", [3, 140])
@pytest.mark.parametrize("gate", [-10.0, -20.0, -40.0])
def test_layer_small_hidden_rows_keep_their_bits(dev, M, gate):
    """Gates far below zero: SiLU makes every hidden value, and with it the result, up to 2^52
    times smaller, and no less precise. Norm-wise as above, and a rounding of the gate sums (at
    most 2^-11 of some 0.1, of random sign) moves SiLU by as much of itself."""
    E, k, H, I, bs = 6, 2, 1024, 768, 32
    g = torch.Generator().manual_seed(M)
    ws = [pack(dev, stack(g, E, N, K, bs, BF16, False, False), N, K, bs)
          for N, K in ((I, H), (I, H), (H, I))]
    X = (torch.randn(M, H, generator=g) * 0.05).to(BF16).to(dev)
    logits = torch.randn(M, E, generator=g).to(dev)
    bg = torch.full((E, I), gate, device=dev)
    weights, experts, _, _ = ref.route(logits, k, True)
    R, _ = ref.layer(X, weights, experts.to(dev), *[W for _, _, W in ws], bg, None, None, BF16)
    err = mnb.mnb_moe(X, logits, *[w for w, _, _ in ws], k, bias_gate=bg).double() - R
    assert err.norm() <= (2.0 ** -8 + 5 * 2.0 ** -11) * R.norm()


@pytest.mark.parametrize("M", [3, 12, 140])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_layer_masked_tokens(dev, M, dtype):
    """Tokens with fewer experts than choices, with none at all, and a batch without any."""
    X, logits, ws = layer_inputs(dev, M, 10, 4, 96, 160, 32, dtype, bias=True, seed=M)
    logits[0] = -math.inf
    logits[1, 2:] = -math.inf
    logits[2, ::2] = math.nan
    Y = run_layer(dev, X, logits, ws, 4, what="masked")
    assert (Y[0] == 0).all()
    Y = run_layer(dev, X, torch.full_like(logits, -math.inf), ws, 4, what="all masked")
    assert (Y == 0).all()


@pytest.mark.parametrize("M", [4, 140])
def test_layer_all_tokens_one_expert(dev, M):
    X, logits, ws = layer_inputs(dev, M, 6, 2, 128, 192, 32, BF16, seed=M)
    logits[:, 4] += 50
    logits[:, 1] += 40
    run_layer(dev, X, logits, ws, 2, what="skewed")


@pytest.mark.parametrize("M", [9, 140])
@pytest.mark.parametrize("H", [128, 2560])
@pytest.mark.parametrize("gap", [20.0, 60.0, 150.0, math.inf])
@pytest.mark.parametrize("normalize", [True, False])
def test_layer_negligible_weights(dev, M, H, gap, normalize):
    """Chosen experts whose weight is tiny, underflows, or is exactly 0 beside a logit of +inf
    add (next to) nothing: their weighted hidden rows vanish, the tokens' rows do not."""
    X, logits, ws = layer_inputs(dev, M, 6, 2, H, 192, 32, BF16, seed=M + H)
    logits[:, 4] += gap
    run_layer(dev, X, logits, ws, 2, normalize, what=f"H{H} gap {gap}")


@pytest.mark.parametrize("M", [9, 140])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H", [128, 2560])
@pytest.mark.parametrize("bias", [False, True])
def test_layer_zero_experts(dev, M, dtype, H, bias):
    """Experts whose scales are all zero in one of the three weights, or in all of them."""
    E, k, I, bs = 6, 2, 192, 32
    g = torch.Generator().manual_seed(M + H)
    ws = []
    for i, (N, K) in enumerate(((I, H), (I, H), (H, I))):
        B, s, z, b = stack(g, E, N, K, bs, dtype, False, bias)
        s[i] = s[4] = 0
        ws.append(pack(dev, (B, s, z, b), N, K, bs))
    X = torch.randn(M, H, generator=g).to(dtype).to(dev)
    run_layer(dev, X, torch.randn(M, E, generator=g).to(dev), ws, k, what=f"H{H}")


@pytest.mark.parametrize("M", [9, 140])
@pytest.mark.parametrize("H", [128, 2560])
@pytest.mark.parametrize("bias_down", [False, True])
def test_layer_hidden_rows_vanish(dev, M, H, bias_down):
    """Gates so negative that SiLU underflows: hidden rows of zeros under ordinary weights."""
    X, logits, ws = layer_inputs(dev, M, 6, 2, H, 192, 32, BF16, bias=True, seed=M + H)
    (wg, bg, Wg), (wu, bu, Wu), (wd, bd, Wd) = ws
    bg[1::2] = -400.0
    run_layer(dev, X, logits, ((wg, bg, Wg), (wu, bu, Wu), (wd, bd if bias_down else None, Wd)),
              2, what=f"H{H}")


@pytest.mark.parametrize("M", [3, 140])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate,up", [(-50.0, 1e38), (50.0, 1e36), (-85.0, 1e37), (1e36, 50.0)])
def test_layer_range_of_the_gated_product(dev, M, dtype, gate, up):
    """gate * up is beyond fp32, or near its end, where silu(gate) * up is not."""
    X, logits, ((wg, bg, Wg), (wu, bu, Wu), (wd, bd, Wd)) = layer_inputs(
        dev, M, 5, 2, 128, 96, 32, dtype, bias=True, seed=M)
    bg[:] = gate
    bu[:] = up
    Y = run_layer(dev, X, logits, ((wg, bg, Wg), (wu, bu, Wu), (wd, bd, Wd)), 2,
                  what=f"{gate} {up}")
    # Norm-wise: 2^-8 of the output, four roundings of 2^-11 as above, and SiLU moved by a
    # rounding of the gate sums (2^-11 of some 0.7).
    weights, experts, _, _ = ref.route(logits, 2, True)
    R, _ = ref.layer(X, weights, experts.to(dev), Wg, Wu, Wd, bg, bu, bd, dtype)
    assert (Y.double() - R).norm() <= (2.0 ** -8 + 5 * 2.0 ** -11) * R.norm()


@pytest.mark.parametrize("M", [1, 9, 170])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_layer_many_experts(dev, M, dtype):
    """As many choices as the operators take, of nearly as many experts."""
    X, logits, ws = layer_inputs(dev, M, 1000, 32, 72, 40, 32, dtype, seed=M)
    run_layer(dev, X, logits, ws, 32, what=f"M{M}")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_layer_many_counts(dev, dtype):
    """Enough slots and experts for the sort's counts to be summed by a launch of their own."""
    X, logits, ws = layer_inputs(dev, 420, 1000, 32, 72, 40, 32, dtype, seed=1)
    logits[5] = -math.inf
    run_layer(dev, X, logits, ws, 32, what="many counts")


@pytest.mark.parametrize("M", [1, 7])
def test_long_rows(dev, M):
    """Rows too long for the streaming kernel's shared memory: bf16 ones go to the tensor cores
    at any number of slots, fp32 ones are refused."""
    K, N, bs = 66000, 20, 32
    g = torch.Generator().manual_seed(M)
    w, _, W = pack(dev, stack(g, 2, N, K, bs, BF16, False, False), N, K, bs)
    A = torch.randn(M, K, generator=g).to(BF16).to(dev)
    t = torch.randint(0, 2, (M, 1), generator=g, dtype=torch.int32).to(dev)
    R, err = ref.products(A.double().unsqueeze(1), W, t, None, BF16)
    ref.check(mnb.mnb_matmul_experts(A, w, t), R, err, "product")
    with pytest.raises(mnb.MnbError) as e:
        mnb.mnb_matmul_experts(A.float(), w, t)
    assert e.value.status == binding.MNB_ERR_UNSUPPORTED
    X, logits, ws = layer_inputs(dev, M, 2, 1, 24, K, bs, BF16, seed=M)
    run_layer(dev, X, logits, ws, 1, what="layer")
    packed = [w for w, _, _ in ws]
    with pytest.raises(mnb.MnbError) as e:
        mnb.mnb_moe(X.float(), logits, *packed, 1)
    assert e.value.status == binding.MNB_ERR_UNSUPPORTED


@pytest.mark.parametrize("M", [1, 7, 140])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_layer_is_its_parts(dev, M, dtype):
    """The operators together: router, gate and up products, SiLU in torch, down product and
    weighted sum give the layer's result."""
    E, k, H, I = 12, 3, 256, 320
    X, logits, ((wg, bg, _), (wu, bu, _), (wd, bd, _)) = layer_inputs(
        dev, M, E, k, H, I, 32, dtype, bias=True, seed=M)
    r = mnb.mnb_moe_route(logits.to(BF16).float(), k)
    g = mnb.mnb_matmul_experts(X, wg, r.experts, bg).float()
    u = mnb.mnb_matmul_experts(X, wu, r.experts, bu).float()
    h = (torch.nn.functional.silu(g) * u).to(dtype)
    y = mnb.mnb_matmul_experts(h, wd, r.experts, bd).float()
    Y = mnb.mnb_moe(X, logits.to(BF16), wg, wu, wd, k, bias_gate=bg, bias_up=bu, bias_down=bd)
    parts = (r.weights.unsqueeze(2) * y).sum(1)
    # Both are within a few roundings of the activations' type of the exact layer.
    u = {F32: 1e-5, BF16: 2.0 ** -6}[dtype]
    assert (Y.float() - parts).norm() <= u * parts.norm()


@pytest.mark.parametrize("M", [2, 140])
def test_layer_rows_do_not_mix(dev, M):
    """A token with infinite or NaN activations spoils its own row only."""
    X, logits, ((wg, _, _), (wu, _, _), (wd, _, _)) = layer_inputs(
        dev, M, 5, 2, 128, 96, 32, BF16, seed=M)
    Y = mnb.mnb_moe(X, logits, wg, wu, wd, 2)
    bad = X.clone()
    bad[0, 3] = math.inf
    bad[0, 9] = math.nan
    Z = mnb.mnb_moe(bad, logits, wg, wu, wd, 2)
    assert not torch.isfinite(Z[0]).any()
    assert torch.equal(Y[1:], Z[1:])


@pytest.mark.parametrize("dtype,per_slot", [(BF16, True), (BF16, False), (F32, True)])
def test_experts_offsets_past_32_bits(dev, dtype, per_slot):
    """More than 2^31 elements of activations by slot, and of outputs: sampled rows."""
    M, k, E, bs = 70000, 8, 12, 32
    g = torch.Generator().manual_seed(1)
    gd = torch.Generator(device=dev).manual_seed(1)
    t = torch.randint(-1, E, (M, k), generator=gd, device=dev, dtype=torch.int32)
    for N, K in ((16, 4096), (4096, 64)):
        w, b, W = pack(dev, stack(g, E, N, K, bs, dtype, False, True), N, K, bs)
        A = torch.randn(*((M, k, K) if per_slot else (M, K)), generator=gd, device=dev,
                        dtype=dtype)
        Y = mnb.mnb_matmul_experts(A, w, t, b)
        m = torch.tensor([0, 1, 33333, 65535, 65536, M - 2, M - 1], device=dev)
        a = A[m].double() if per_slot else A[m].double().unsqueeze(1).expand(len(m), k, K)
        R, err = ref.products(a, W, t[m], b, dtype)
        ref.check(Y[m], R, err, f"N{N} K{K}")
        del A, Y


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_layer_offsets_past_32_bits(dev, dtype):
    """More than 2^31 hidden values, and as many down sums: sampled tokens."""
    M, k, E, bs = 70000, 8, 12, 32
    for H, I in ((64, 4096), (4096, 64)):
        _, _, ws = layer_inputs(dev, 1, E, k, H, I, bs, dtype, bias=True, seed=H)
        gd = torch.Generator(device=dev).manual_seed(H)
        X = torch.randn(M, H, generator=gd, device=dev, dtype=dtype)
        logits = torch.randn(M, E, generator=gd, device=dev)
        logits[33333, 3:] = -math.inf
        (wg, bg, Wg), (wu, bu, Wu), (wd, bd, Wd) = ws
        Y = mnb.mnb_moe(X, logits, wg, wu, wd, k, bias_gate=bg, bias_up=bu, bias_down=bd)
        m = torch.tensor([0, 1, 33333, 65535, 65536, M - 2, M - 1], device=dev)
        weights, experts, _, _ = ref.route(logits[m], k, True)
        R, err = ref.layer(X[m], weights, experts.to(dev), Wg, Wu, Wd, bg, bu, bd, dtype)
        ref.check(Y[m], R, err, f"H{H} I{I}")
        del X, Y


@pytest.mark.parametrize("M", [5, 140])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("off", [1, 2, 3])
def test_rows_off_alignment(dev, M, dtype, off):
    """Activations, logits and outputs that start off the 16 bytes (and off pairs) that whole
    tensors start on give what aligned ones do."""
    E, k, H, I = 9, 3, 128, 96
    X, logits, ws = layer_inputs(dev, M, E, k, H, I, 32, dtype, seed=M)
    packed = [w for w, _, _ in ws]

    def shifted(t):
        y = torch.empty(t.numel() + off, dtype=t.dtype, device=dev)[off:].view(t.shape)
        return y.copy_(t)

    r = mnb.mnb_moe_route(logits, k)
    Y = mnb.mnb_moe(X, logits, *packed, k)
    P = mnb.mnb_matmul_experts(X, packed[0], r.experts)
    out = shifted(torch.zeros_like(Y))
    assert torch.equal(mnb.mnb_moe(shifted(X), shifted(logits), *packed, k, out=out), Y)
    out = shifted(torch.zeros_like(P))
    assert torch.equal(
        mnb.mnb_matmul_experts(shifted(X), packed[0], shifted(r.experts), out=out), P)


# ---- streams and graphs --------------------------------------------------------------------------

@pytest.mark.parametrize("M", [1, 12, 140])
def test_captured_and_replayed(dev, M):
    """Captured once, replayed on new inputs, two graphs on two streams at a time."""
    k = 4
    made = []
    for i in range(2):
        X, logits, ws = layer_inputs(dev, M, 16, k, 256, 192, 32, BF16, seed=M + i)
        packed = [w for w, _, _ in ws]
        mnb.mnb_moe(X, logits, *packed, k)
        torch.cuda.synchronize()
        graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=st):
            Y = mnb.mnb_moe(X, logits, *packed, k)
            r = mnb.mnb_moe_route(logits, k)
            P = mnb.mnb_matmul_experts(X, packed[0], r.experts)
        made.append((X, logits, packed, graph, st, Y, r, P))
    for turn in range(3):
        for X, logits, *_ in made:
            X.copy_(torch.randn_like(X))
            logits.copy_(torch.randn_like(logits))
        torch.cuda.synchronize()
        for *_, graph, st, Y, r, P in made:
            with torch.cuda.stream(st):
                for _ in range(5):
                    graph.replay()
        torch.cuda.synchronize()
        for X, logits, packed, graph, st, Y, r, P in made:
            assert torch.equal(Y, mnb.mnb_moe(X, logits, *packed, k))
            now = mnb.mnb_moe_route(logits, k)
            assert all(torch.equal(a, b) for a, b in zip(r, now))
            assert torch.equal(P, mnb.mnb_matmul_experts(X, packed[0], now.experts))


@pytest.mark.parametrize("M", [2, 140])
def test_other_stream(dev, M):
    k = 2
    X, logits, ws = layer_inputs(dev, M, 8, k, 256, 192, 32, BF16, seed=M)
    packed = [w for w, _, _ in ws]
    Y = mnb.mnb_moe(X, logits, *packed, k)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    outs = [mnb.mnb_moe(X, logits, *packed, k, stream=st) for _ in range(8)]
    st.synchronize()
    assert all(torch.equal(o, Y) for o in outs)


def test_calls_at_once(dev):
    """Two threads, each on a stream of its own, with calls of either kernel in flight."""
    k = 2
    X, logits, ws = layer_inputs(dev, 140, 8, k, 256, 192, 32, BF16)
    packed = [w for w, _, _ in ws]
    want = {M: mnb.mnb_moe(X[:M], logits[:M], *packed, k) for M in (1, 7, 140)}
    torch.cuda.synchronize()
    got, errors = [], []

    def work(sizes):
        try:
            st = torch.cuda.Stream()
            outs = [(M, mnb.mnb_moe(X[:M], logits[:M], *packed, k, stream=st))
                    for _ in range(20) for M in sizes]
            st.synchronize()
            got.extend(outs)
        except Exception as e:  # noqa: BLE001 (reported below)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(s,)) for s in ((1, 140), (140, 7))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and len(got) == 80
    assert all(torch.equal(Y, want[M]) for M, Y in got)


def test_copied_and_replaced_stacks(dev):
    """A copy of a packed stack is a packed weight of its own (its header has to be registered,
    as any restored weight's), and a stack keeps what it was made with."""
    g = torch.Generator().manual_seed(1)
    (a, _, Wa), (b, _, Wb) = (pack(dev, stack(g, 3, 32, 64, 32, F32, True, False), 32, 64, 32)
                              for _ in range(2))
    A = torch.randn(4, 64, generator=g).to(dev)
    t = torch.randint(0, 3, (4, 2), generator=g, dtype=torch.int32).to(dev)
    Ya, Yb = mnb.mnb_matmul_experts(A, a, t), mnb.mnb_matmul_experts(A, b, t)
    other = copy.deepcopy(a)
    with pytest.raises(mnb.MnbError) as e:
        mnb.mnb_matmul_experts(A, other, t)
    assert e.value.status == binding.MNB_ERR_LAYOUT
    mnb.mnb_packed_register(other.packed_b, mnb.mnb_packed_read_header(other.packed_b))
    assert torch.equal(mnb.mnb_matmul_experts(A, other, t), Ya)
    mnb.mnb_packed_forget(other.packed_b)
    with pytest.raises(dataclasses.FrozenInstanceError):
        a.packed_scales = b.packed_scales
    c = dataclasses.replace(a, packed_b=b.packed_b, packed_scales=b.packed_scales,
                            packed_zp=b.packed_zp, packed_rows=b.packed_rows)
    assert torch.equal(mnb.mnb_matmul_experts(A, c, t), Yb)


def test_wrong_descriptions_are_refused(dev):
    """A stack described with another division of its rows, a single weight passed as a stack
    and a stack of another N are turned down on the host; a stack as the single weight that its
    header says it is, and one known by a registered header, are taken."""
    E, N, K, bs = 8, 64, 128, 32
    g = torch.Generator().manual_seed(2)
    B, s, _, _ = to(dev, *stack(g, E, N, K, bs, F32, False, False))
    w = mnb.mnb_prepack_experts(B, s, None, N, K, bs)
    plain = mnb.mnb_prepack(B.view(1, E * N, -1, bs // 2), s.view(E * N, -1), None, E * N, K, bs)
    A = torch.randn(2, K, generator=g).to(dev)
    t = torch.zeros(2, 1, dtype=torch.int32, device=dev)
    Y = torch.zeros(2, 1, 2 * N, device=dev)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=dev)
    lib = mnb.load()

    def call(c):
        return lib.mnb_matmul_experts(A.data_ptr(), 0, c, t.data_ptr(), 2, 1, Y.data_ptr(),
                                      binding.MNB_F32, ws.data_ptr(), ws.numel(), None)

    def described(packed, E, N):
        return binding.ExpertsC(packed.packed_b.data_ptr(), packed.packed_scales.data_ptr(), None,
                                w.packed_rows.data_ptr(), None, E, N, K, bs, binding.MNB_F32)

    for packed, e, n in ((w, 16, 32), (w, 4, 128), (w, 1, 512), (w, 8, 60), (plain, 8, 64),
                         (plain, 1, 512)):
        assert call(described(packed, e, n)) == binding.MNB_ERR_LAYOUT, (e, n)
        assert b"stack" in lib.mnb_last_error_string()
    assert call(described(w, 8, 64)) == 0
    whole = mnb.PackedWeight(w.packed_b, w.packed_scales, None, E * N, K, bs, F32)
    assert torch.equal(mnb.mnb_matmul(A, whole), mnb.mnb_matmul(A, plain))
    want = mnb.mnb_matmul_experts(A, w, t)
    mnb.mnb_packed_register(w.packed_b, mnb.mnb_packed_read_header(w.packed_b))
    assert torch.equal(mnb.mnb_matmul_experts(A, w, t), want)
    with pytest.raises(ValueError, match="packed_rows"):
        mnb.mnb_matmul_experts(A, dataclasses.replace(w, E=16, N=32), t)


def test_programmatic_launch_off(dev):
    X, logits, ws = layer_inputs(dev, 3, 8, 2, 256, 192, 32, BF16)
    packed = [w for w, _, _ in ws]
    Y = mnb.mnb_moe(X, logits, *packed, 2)
    mnb.mnb_set_programmatic_launch(False)
    try:
        assert torch.equal(mnb.mnb_moe(X, logits, *packed, 2), Y)
    finally:
        mnb.mnb_set_programmatic_launch(True)


@pytest.mark.parametrize("K", [1, 64, 65, 128, 192, 256, 640, 704])
@pytest.mark.parametrize("N", [16, 520])
def test_few_stages_and_units(dev, N, K):
    """Tensor-core kernel with fewer stages than its rings hold, on pairs of CTAs with no work
    item, one or several: every wait at its end is met (at once, and with no fault recorded)."""
    for M, E in ((6, 1), (12, 2), (700, 60), (30000, 200)):
        run_experts(dev, M, E, 1, N, K, 32, BF16, seed=M + K)
    assert mnb.mnb_fault_status() == 0


def test_no_faults_recorded(dev):
    assert mnb.mnb_fault_status() == 0
