"""The mixture-of-experts operators written out in 64 bits, with the bounds GPU results are
held to. Plain torch float64 on whatever device the inputs are on; shares no code with the
library.

Bounds, element by element. u32 = 2^-24 is half a step of fp32; a sum of n products formed in
fp32 in any order, on tensor cores that may truncate instead of rounding (a whole step, 2^-23),
is within n 2^-23 of the sum of the terms' magnitudes (mag), and applying a block's scale costs
one more rounding per block, at most n of them. On top of that come the roundings the kernels
choose:
  * fp32 activations: weights and activations enter exactly up to 2^-22 of each (the parts of a
    split), so a product is within (2 n + 16) 2^-23 mag + 2^-22 mag;
  * bf16 activations: a weight may be rounded to fp16 (2^-11) and so may a hidden value
    (2^-11); a result is rounded to bf16 (2^-8). fp16 activations (for fp32 ones, the parts
    they are split into) are scaled by a power of two so that a bound of the row (its largest
    magnitude; for a hidden row, at most the product of the bounds of its gate and up sums, which
    is what is allowed here) lies in 2^14 .. 2^15: they are exact down to 2^-14 and within 2^-25 below that, at most
    FLOOR = 2^-39 of the row's bound. The offset of the codes
    may be taken off a block as a whole: codes of 1024 + r q carry an offset of 1024 + r z (r is
    1 or 16, divided out again at the end), and (1024 + r z) s / r times the sum of a block's
    activations comes off. That sum has at most 64 terms; it and the products it comes off are
    each within 64 2^-24 of (1024 + r z) s / r times the activations' magnitudes, at most
    OFFSET = 2 * 64 * 1039 * 2^-24 of the sum of |a| s in all (r = 1, z = 15); or z s may be
    rounded to fp16 before it comes off a code, at most 15 2^-12 s for each |a|, which is less.
    An fp16 weight's row is scaled so that its largest scale lies in 2^-10 .. 2^-9: a weight
    below 2^-14 there is within 2^-25, at most ROW = 2^-15 of the row's largest scale. The layer's
    down sums may leave as fp16 before they are added (2^-11), scaled by a bound of theirs: at
    most 2^-25 of 2^e / 2^15, where 2^e is at most four times twice the bound 15 s K' times the
    hidden row's largest value (K' = K rounded up to 64) or the bias.
"""
import torch

U_W = {torch.float32: 2.0 ** -22, torch.bfloat16: 2.0 ** -11}
U_H = {torch.float32: 2.0 ** -22, torch.bfloat16: 2.0 ** -11}
U_OUT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
FLOOR = {torch.float32: 2.0 ** -39, torch.bfloat16: 2.0 ** -39}
OFFSET = {torch.float32: 0.0, torch.bfloat16: 2 * 64 * 1039 * 2.0 ** -24}
ROW = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -15}
TINY = 1e-30


class Stack:
    """Weights [E, N, K] and their scales, spread over K, in float64."""

    def __init__(self, W, S):
        self.W, self.S = W, S


def sum_u(n):
    return (2 * n + 16) * 2.0 ** -23


def dequant(B, s, z, K):
    """The Stack of a MatMulNBits storage."""
    E, N, nb, half = B.shape
    i = torch.arange(K, device=B.device)
    b = i // (2 * half)
    byte = B.reshape(E, N, -1)[:, :, i // 2].long()
    q = (byte >> (4 * (i % 2))) & 15
    zp = 8 if z is None else (z.long()[:, :, b // 2] >> (4 * (b % 2))) & 15
    S = s.double()[:, :, b]
    return Stack((q - zp).double() * S, S)


def route(logits, k, normalize):
    """(weights [M, k] float64, experts [M, k], offsets [E + 1], order [M * k]), row by row."""
    M, E = logits.shape
    rows = logits.double().cpu().tolist()
    weights = torch.zeros(M, k, dtype=torch.float64)
    experts = torch.full((M, k), -1, dtype=torch.int64)
    inf = float("inf")
    for m, row in enumerate(rows):
        left = {e: v for e, v in enumerate(row) if v == v and v != -inf}
        if not left:
            continue
        top = max(left.values())
        p = {e: 1.0 if v == top else float(torch.exp(torch.tensor(v - top, dtype=torch.float64)))
             for e, v in left.items()}
        pick = sorted(left, key=lambda e: (-left[e], e))[:k]
        total = sum(p[e] for e in pick) if normalize else sum(p.values())
        for j, e in enumerate(pick):
            experts[m, j] = e
            weights[m, j] = p[e] / total
    offsets, order = lists(experts, E)
    return weights, experts, offsets, order


def lists(experts, E):
    flat = experts.flatten().tolist()
    order, offsets = [], [0]
    for e in range(E):
        order += [p for p, v in enumerate(flat) if v == e]
        offsets.append(len(order))
    order += [p for p, v in enumerate(flat) if not 0 <= v < E]
    return torch.tensor(offsets), torch.tensor(order)


def products(A, W, experts, bias, dtype, cap=None):
    """(Y [M, k, N] float64, bound without the output's rounding) for A [M, k, K] float64.
    cap [M, k]: the bound of each row (default: its largest magnitude)."""
    cap = A.abs().amax(2) if cap is None else cap
    W, S = W.W, W.S
    M, k, K = A.shape
    Y = torch.zeros(M, k, W.shape[1], dtype=torch.float64, device=A.device)
    err = torch.zeros_like(Y)
    for e in range(W.shape[0]):
        m, j = torch.nonzero(experts == e, as_tuple=True)
        if len(m):
            a = A[m, j]
            y = a @ W[e].T
            mag = a.abs() @ W[e].abs().T
            if bias is not None:
                y = y + bias[e].double()
                mag = mag + bias[e].double().abs()
            Y[m, j] = y
            low = FLOOR[dtype] * cap[m, j].unsqueeze(1) * W[e].abs().sum(1)
            off = OFFSET[dtype] * (a.abs() @ S[e].abs().T)
            row = ROW[dtype] * a.abs().sum(1, keepdim=True) * S[e].abs().amax(1)
            err[m, j] = (sum_u(K) + U_W[dtype]) * mag + low + off + row
    return Y, err


def layer(X, weights, experts, Wg, Wu, Wd, bg, bu, bd, dtype):
    """(Y [M, H] float64, bound) of the whole layer for the given choices."""
    M, k = experts.shape
    x = X.double().unsqueeze(1).expand(M, k, X.shape[1])
    g, eg = products(x, Wg, experts, bg, dtype)
    u, eu = products(x, Wu, experts, bu, dtype)
    silu = g * torch.sigmoid(g)
    h = silu * u
    # |d silu| <= 1.1; the product, exp and division in fp32 cost a few roundings.
    eh = 1.1 * eg * (u.abs() + eu) + (silu.abs() + 1.1 * eg) * eu
    eh = eh + (U_H[dtype] + 2.0 ** -20) * (h.abs() + eh)
    # Bounds of the hidden rows: 15 times the largest scale times the row's 1-norm, plus the
    # bias, for gate and for up; each is rounded up to a power of two (a factor of 2).
    cap = torch.zeros(M, k, dtype=torch.float64, device=X.device)
    for e in range(Wg.W.shape[0]):
        m, j = torch.nonzero(experts == e, as_tuple=True)
        one = lambda W, b: 2 * (16 * W.S[e].abs().max() * x[m, j].abs().sum(1)  # noqa: E731
                                + (0 if b is None else b[e].double().abs().max()))
        cap[m, j] = one(Wg, bg) * one(Wu, bu)
    y, ey = products(h, Wd, experts, bd, dtype, cap)
    top = (h.abs() + eh).amax(2)
    Wabs = Wd.W.abs()
    for e in range(Wabs.shape[0]):
        m, j = torch.nonzero(experts == e, as_tuple=True)
        if len(m):
            ey[m, j] += eh[m, j] @ Wabs[e].T * 1.01
            if dtype == torch.bfloat16:
                most = 8 * (16 * Wd.S[e].abs().max() * (Wabs.shape[2] + 63) * top[m, j]
                            + (0 if bd is None else bd[e].double().abs().max()))
                ey[m, j] += 2.0 ** -11 * (y[m, j].abs() + ey[m, j]) + 2.0 ** -40 * most.unsqueeze(1)
    w = weights.to(y.device).unsqueeze(2)
    Y = (w * y).sum(1)
    err = (w * ey).sum(1) + (2.0 ** -20 + k * 2.0 ** -23) * (w * y.abs()).sum(1)
    return Y, err


def check(got, ref, err, what=""):
    bound = err + U_OUT[got.dtype] * (ref.abs() + err) + TINY
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    ratio = ((got - ref).abs() / bound)
    worst = float(ratio.max()) if ratio.numel() else 0.0
    assert worst <= 1, f"{what}: max err/bound {worst:.3g}"
    return worst
