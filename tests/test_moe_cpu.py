"""Refusals of the mixture-of-experts entry points, on the host: every call below is turned
down before it reaches a device (fake device addresses), and workspace sizes are plain host
arithmetic."""
import ctypes

import pytest
import torch

import int4_weight_only_matmulnbits_gb300 as mnb
from int4_weight_only_matmulnbits_gb300 import binding as b

F32, BF16 = b.MNB_F32, b.MNB_BF16
BIG = 2 ** 31


@pytest.fixture(scope="module")
def lib():
    mnb.build_library()
    return mnb.load()


def vp(x):
    return ctypes.c_void_p(x) if x else None


# Fake device addresses, 4 GiB apart: nothing is dereferenced.
A, Y, LOG, WS = (0x7000_0000_0000 + i * (1 << 32) for i in range(4))
EXP, WEI, OFF, ORD = (0x7100_0000_0000 + i * (1 << 32) for i in range(4))


def stack(i=0, *, E=8, N=64, K=128, bs=32, sdt=BF16, zp=False, bias=False, register=True,
          packed_as=None):
    base = 0x7200_0000_0000 + i * (1 << 36)
    s = b.ExpertsC(base, base + (1 << 34), base + (2 << 34) if zp else None,
                   base + (1 << 35) + (1 << 34) + (1 << 33), base + (3 << 34) if bias else None,
                   E, N, K, bs, sdt)
    if register:
        e, n, k = packed_as or (E, N, K)
        h = mnb.mnb_packed_header_make(e * (-(-n // 16) * 16), k, bs,
                                       torch.float32 if sdt == F32 else torch.bfloat16, zp)
        mnb.mnb_packed_register(base, h)
    else:
        mnb.mnb_packed_forget(base)
    return s


def test_public_names():
    """Every call of the package is among the names that it exports."""
    calls = {n for n in dir(mnb) if n.startswith("mnb_")}
    assert calls <= set(mnb.__all__) and all(hasattr(mnb, n) for n in mnb.__all__)


def route(lib, logits=LOG, dt=F32, M=4, E=8, k=2, norm=1, w=WEI, e=EXP, off=OFF, order=ORD,
          ws=WS, ws_bytes=1 << 30):
    return lib.mnb_moe_route(vp(logits), dt, M, E, k, norm, vp(w), vp(e), vp(off), vp(order),
                             vp(ws), ws_bytes, None)


@pytest.mark.parametrize("change,status", [
    (dict(logits=0), b.MNB_ERR_NULL), (dict(w=0), b.MNB_ERR_NULL), (dict(e=0), b.MNB_ERR_NULL),
    (dict(off=0), b.MNB_ERR_NULL), (dict(order=0), b.MNB_ERR_NULL),
    (dict(M=0), b.MNB_ERR_SHAPE), (dict(E=0), b.MNB_ERR_SHAPE), (dict(k=0), b.MNB_ERR_SHAPE),
    (dict(k=9), b.MNB_ERR_SHAPE), (dict(M=BIG // 2, k=2), b.MNB_ERR_SHAPE),
    (dict(M=-1), b.MNB_ERR_SHAPE), (dict(norm=2), b.MNB_ERR_SHAPE),
    (dict(E=1025), b.MNB_ERR_UNSUPPORTED), (dict(E=64, k=33), b.MNB_ERR_UNSUPPORTED),
    (dict(dt=2), b.MNB_ERR_DTYPE), (dict(logits=LOG + 2), b.MNB_ERR_ALIGN),
    (dict(logits=LOG + 1, dt=BF16), b.MNB_ERR_ALIGN), (dict(w=WEI + 2), b.MNB_ERR_ALIGN),
    (dict(e=EXP + 1), b.MNB_ERR_ALIGN), (dict(order=ORD + 3), b.MNB_ERR_ALIGN),
    (dict(w=LOG + 4), b.MNB_ERR_ALIAS), (dict(e=WEI + 28), b.MNB_ERR_ALIAS),
    (dict(order=OFF + 32), b.MNB_ERR_ALIAS)])
def test_route_refusals(lib, change, status):
    assert route(lib, **change) == status


def experts(lib, a=A, per_slot=0, w=None, e=EXP, M=4, k=2, y=Y, dt=BF16, ws=WS, ws_bytes=1 << 40):
    w = w if w is not None else stack()
    return lib.mnb_matmul_experts(vp(a), per_slot, w, vp(e), M, k, vp(y), dt, vp(ws), ws_bytes,
                                  None)


@pytest.mark.parametrize("change,status", [
    (dict(a=0), b.MNB_ERR_NULL), (dict(e=0), b.MNB_ERR_NULL), (dict(y=0), b.MNB_ERR_NULL),
    (dict(M=0), b.MNB_ERR_SHAPE), (dict(k=0), b.MNB_ERR_SHAPE),
    (dict(M=BIG // 4, k=4), b.MNB_ERR_SHAPE), (dict(per_slot=2), b.MNB_ERR_SHAPE),
    (dict(dt=5), b.MNB_ERR_DTYPE), (dict(a=A + 1), b.MNB_ERR_ALIGN),
    (dict(y=Y + 2, dt=F32), b.MNB_ERR_ALIGN), (dict(e=EXP + 2), b.MNB_ERR_ALIGN),
    (dict(y=A + 64), b.MNB_ERR_ALIAS), (dict(y=EXP + 16), b.MNB_ERR_ALIAS)])
def test_experts_refusals(lib, change, status):
    assert experts(lib, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(E=0), b.MNB_ERR_SHAPE), (dict(N=0), b.MNB_ERR_SHAPE), (dict(K=0), b.MNB_ERR_SHAPE),
    (dict(E=1025), b.MNB_ERR_UNSUPPORTED), (dict(E=1000, N=BIG - 1), b.MNB_ERR_SHAPE),
    (dict(bs=24), b.MNB_ERR_BLOCKSIZE), (dict(bs=512), b.MNB_ERR_BLOCKSIZE),
    (dict(sdt=7), b.MNB_ERR_DTYPE)])
def test_stack_refusals(lib, change, status):
    w = stack(register=False, **change)
    assert experts(lib, w=w) == status
    assert lib.mnb_matmul_experts_workspace_size(4, 2, w, BF16, 0) == 0


def test_stack_pointers(lib):
    for field in ("packed_b", "packed_scales", "packed_rows"):
        w = stack()
        setattr(w, field, None)
        assert experts(lib, w=w) == b.MNB_ERR_NULL
        w = stack()
        setattr(w, field, getattr(w, field) + 8)
        assert experts(lib, w=w) == b.MNB_ERR_ALIGN
    w = stack(zp=True, bias=True)
    w.packed_zp += 8
    assert experts(lib, w=w) == b.MNB_ERR_ALIGN
    w = stack(zp=True, bias=True)
    w.bias += 2
    assert experts(lib, w=w) == b.MNB_ERR_ALIGN
    w = stack()
    assert experts(lib, w=w, y=w.packed_b + 64) == b.MNB_ERR_ALIAS
    assert experts(lib, w=w, y=w.packed_scales + 64) == b.MNB_ERR_ALIAS
    assert experts(lib, w=w, y=w.packed_rows + 64) == b.MNB_ERR_ALIAS


def test_stack_headers(lib):
    """A stack the library did not pack, packed for another size, or with other zero points."""
    assert experts(lib, w=stack(register=False)) == b.MNB_ERR_LAYOUT
    assert experts(lib, w=stack(packed_as=(8, 80, 128))) == b.MNB_ERR_LAYOUT
    assert experts(lib, w=stack(packed_as=(7, 64, 128))) == b.MNB_ERR_LAYOUT
    assert experts(lib, w=stack(packed_as=(8, 64, 64))) == b.MNB_ERR_LAYOUT
    w = stack()
    w.packed_zp = w.packed_b + (2 << 34)
    assert experts(lib, w=w) == b.MNB_ERR_LAYOUT
    assert b"zero points" in lib.mnb_last_error_string()


def test_binding_refuses_a_wrong_division():
    """8 experts of 64 rows described as 16 of 32 or 4 of 128: the same rows in all."""
    buf = torch.zeros(512, dtype=torch.uint8)
    rows = torch.zeros(8 * 64 + 8)
    b._experts_struct(mnb.PackedExperts(buf, buf, None, rows, 8, 64, 128, 32, torch.bfloat16),
                      None, buf.device)
    for E, N in ((16, 32), (4, 128), (8, 80), (9, 64)):
        w = mnb.PackedExperts(buf, buf, None, rows, E, N, 128, 32, torch.bfloat16)
        with pytest.raises(ValueError, match="packed_rows"):
            b._experts_struct(w, None, buf.device)
    w = mnb.PackedExperts(buf, buf, None, rows.double(), 8, 64, 128, 32, torch.bfloat16)
    with pytest.raises(ValueError, match="packed_rows"):
        b._experts_struct(w, None, buf.device)


def moe(lib, x=A, logits=LOG, ldt=F32, M=4, k=2, norm=1, gate=None, up=None, down=None, y=Y,
        dt=BF16, ws=WS, ws_bytes=1 << 40):
    gate = gate if gate is not None else stack(0)
    up = up if up is not None else stack(1)
    down = down if down is not None else stack(2, N=128, K=64)
    return lib.mnb_moe(vp(x), vp(logits), ldt, M, k, norm, gate, up, down, vp(y), dt, vp(ws),
                       ws_bytes, None)


@pytest.mark.parametrize("change,status", [
    (dict(x=0), b.MNB_ERR_NULL), (dict(logits=0), b.MNB_ERR_NULL), (dict(y=0), b.MNB_ERR_NULL),
    (dict(ws=0), b.MNB_ERR_NULL), (dict(ws=WS + 16), b.MNB_ERR_ALIGN),
    (dict(ws_bytes=0), b.MNB_ERR_SHAPE), (dict(ws=Y), b.MNB_ERR_ALIAS),
    (dict(ws=LOG), b.MNB_ERR_ALIAS), (dict(M=0), b.MNB_ERR_SHAPE), (dict(k=0), b.MNB_ERR_SHAPE),
    (dict(k=9), b.MNB_ERR_SHAPE), (dict(norm=-1), b.MNB_ERR_SHAPE),
    (dict(ldt=9), b.MNB_ERR_DTYPE), (dict(dt=9), b.MNB_ERR_DTYPE), (dict(y=A), b.MNB_ERR_ALIAS),
    (dict(x=A + 1), b.MNB_ERR_ALIGN), (dict(logits=LOG + 2), b.MNB_ERR_ALIGN)])
def test_layer_refusals(lib, change, status):
    assert moe(lib, **change) == status


def test_layer_stacks_must_fit(lib):
    for bad in (dict(gate=stack(0, N=80)), dict(gate=stack(0, K=256)), dict(gate=stack(0, E=7)),
                dict(up=stack(1, bs=64)), dict(up=stack(1, sdt=F32)), dict(up=stack(1, zp=True)),
                dict(down=stack(2, N=64, K=64)), dict(down=stack(2, N=128, K=128)),
                dict(down=stack(2, N=128, K=64, E=9))):
        assert moe(lib, **bad) == b.MNB_ERR_SHAPE, bad
        assert b"fit together" in lib.mnb_last_error_string()
    assert moe(lib, up=stack(1, register=False)) == b.MNB_ERR_LAYOUT
    assert moe(lib, down=stack(2, N=128, K=64, packed_as=(8, 112, 64))) == b.MNB_ERR_LAYOUT


def prepack(lib, B=A, s=LOG, z=0, E=4, N=20, K=100, bs=32, dt=BF16, pb=EXP, ps=WEI, pz=0, pr=Y):
    return lib.mnb_prepack_experts(vp(B), vp(s), vp(z), E, N, K, bs, dt, vp(pb), vp(ps), vp(pz),
                                   vp(pr), None)


@pytest.mark.parametrize("change,status", [
    (dict(B=0), b.MNB_ERR_NULL), (dict(s=0), b.MNB_ERR_NULL), (dict(pb=0), b.MNB_ERR_NULL),
    (dict(ps=0), b.MNB_ERR_NULL), (dict(z=OFF), b.MNB_ERR_NULL), (dict(E=0), b.MNB_ERR_SHAPE),
    (dict(N=0), b.MNB_ERR_SHAPE), (dict(K=0), b.MNB_ERR_SHAPE),
    (dict(E=BIG - 1, N=16), b.MNB_ERR_SHAPE), (dict(bs=8), b.MNB_ERR_BLOCKSIZE),
    (dict(dt=3), b.MNB_ERR_DTYPE), (dict(pb=EXP + 4), b.MNB_ERR_ALIGN),
    (dict(ps=WEI + 8), b.MNB_ERR_ALIGN), (dict(s=LOG + 1), b.MNB_ERR_ALIGN),
    (dict(z=OFF, pz=ORD + 8), b.MNB_ERR_ALIGN), (dict(pb=A), b.MNB_ERR_ALIAS),
    (dict(ps=EXP + 256), b.MNB_ERR_ALIAS), (dict(pr=0), b.MNB_ERR_NULL),
    (dict(pr=Y + 8), b.MNB_ERR_ALIGN), (dict(pr=WEI + 16), b.MNB_ERR_ALIAS)])
def test_prepack_experts_refusals(lib, change, status):
    assert prepack(lib, **change) == status


def test_valid_calls_reach_the_device_check(lib):
    """The base calls are turned down only for want of a device."""
    if torch.cuda.is_available():
        pytest.skip("a device is present: the fake addresses must not reach it")
    want = (b.MNB_ERR_CUDA, b.MNB_ERR_DEVICE)
    assert route(lib) in want
    assert experts(lib) in want
    assert moe(lib) in want
    assert prepack(lib) in want


def test_workspace_sizes(lib):
    """Zero for refused arguments, otherwise what a call with that many bytes accepts."""
    g, u, d = stack(0), stack(1), stack(2, N=128, K=64)
    assert lib.mnb_moe_workspace_size(0, 2, g, u, d, BF16) == 0
    assert lib.mnb_moe_workspace_size(4, 9, g, u, d, BF16) == 0
    assert lib.mnb_moe_workspace_size(4, 2, g, u, d, 4) == 0
    assert lib.mnb_moe_workspace_size(4, 2, g, u, stack(2), BF16) == 0
    assert lib.mnb_moe_route_workspace_size(4, 2000, 2) == 0
    for M in (1, 40, 4000, 200000):
        n = lib.mnb_moe_workspace_size(M, 2, g, u, d, BF16)
        assert n > 0 and moe(lib, M=M, ws_bytes=n - 1) == b.MNB_ERR_SHAPE


def test_binding_refusals(lib):
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    w = mnb.PackedExperts(x, x, None, x, 8, 64, 128, 32, torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        mnb.mnb_moe_route(torch.zeros(4, 8), 2)
    with pytest.raises(ValueError, match=r"\[M, E\]"):
        mnb.mnb_moe_route(torch.zeros(8), 2)
    with pytest.raises(ValueError, match="CUDA"):
        mnb.mnb_matmul_experts(x, w, torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        mnb.mnb_moe(x, torch.zeros(4, 8), w, w, w, 2)
    with pytest.raises(ValueError, match="CUDA"):
        mnb.mnb_prepack_experts(torch.zeros(8, 64, 4, 16, dtype=torch.uint8),
                                torch.zeros(8, 64, 4), None, 64, 128, 32)
