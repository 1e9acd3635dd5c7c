"""The attention block's operators written out in 64 bits on the CPU, and how far the kernels may
be off: counted from their roundings."""
import math

import torch

F32_U, BF16_U = 2.0 ** -24, 2.0 ** -8  # half a step, relative


def unit(dtype):
    return F32_U if dtype == torch.float32 else BF16_U


def frequencies(rot, base, factor=1.0, original=0.0, low=1.0, high=32.0):
    out = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        r = 0.0
        if original > 0:
            r = (original * f / (2 * math.pi) - low) / (high - low)
            r = max(0.0, min(1.0, r))
        out.append((1 - r) * f / factor + r * f)
    return out


def norm_rotate(x, gamma, eps, cos, sin, positions, interleaved):
    """x [T, H, D]; returns the result and the magnitude that its roundings are relative to."""
    x = x.double()
    if gamma is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gamma.double()
    y, mag = x.clone(), x.abs()
    if cos is not None:
        n, half = cos.shape
        for t, p in enumerate(positions.tolist()):
            if not 0 <= p < n:
                y[t], mag[t] = 0, 0
                continue
            for i in range(half):
                a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
                c, s = float(cos[p, i]), float(sin[p, i])
                xa, xb = x[t, :, a], x[t, :, b]
                y[t, :, a], y[t, :, b] = xa * c - xb * s, xb * c + xa * s
                mag[t, :, a] = (xa * c).abs() + (xb * s).abs()
                mag[t, :, b] = (xb * c).abs() + (xa * s).abs()
    return y, mag


def norm_rotate_bound(y, mag, D, dtype, normed):
    """Sum of D squares in fp32 (D roundings, halved by the root), the root, three products, the
    rotation's three roundings; then one rounding of the result."""
    steps = (D / 2 + 8 if normed else 0) + 4
    return steps * F32_U * mag + unit(dtype) * y.abs() * (1 + 1e-6) + 1e-30


def places(starts, lengths, table, page_size, pages, T):
    """(row, position, page or None, place) of each row that belongs to a sequence."""
    out = []
    for b, L in enumerate(lengths):
        for t in range(starts[b], min(starts[b + 1], T)):
            p = L - (starts[b + 1] - t)
            page = None
            if 0 <= p < table.shape[1] * page_size:
                g = int(table[b, p // page_size])
                page = g if 0 <= g < pages else None
            out.append((t, p, page, p % page_size))
    return out


def attend(q, k, v, starts, lengths, table, scale, window=0):
    """q [T, Hq, D], k and v [pages, H, page_size, D]; (result, bound) [T, Hq, D], rows of no
    sequence NaN. bf16: a weight's rounding for the product with the values, 2^-8 of each term.
    Scores: D + 8 additions in fp32 (2^-23 each: the tensor cores may cut off) of terms of their
    magnitude, fp32 factors from their parts to 2^-22; the difference from the maximum, its scale,
    the exponential to 2^-21. A weight's relative error enters sum and product: twice."""
    T, Hq, D = q.shape
    pages, H, ps, _ = k.shape
    G = Hq // H
    out = torch.full((T, Hq, D), float("nan"), dtype=torch.float64)
    bound = torch.zeros_like(out)
    f32 = q.dtype == torch.float32
    for b, L in enumerate(lengths):
        t0, t1 = starts[b], starts[b + 1]
        for t in range(t0, t1):
            p = L - (t1 - t)
            js = [j for j in range(max(0, p - window + 1 if window else 0),
                                   min(p + 1, table.shape[1] * ps))
                  if 0 <= int(table[b, j // ps]) < pages]
            if not js:
                out[t] = 0
                continue
            j = torch.tensor(js)
            g = table[b].long()[j // ps]
            keys, values = (x[g, :, j % ps].double() for x in (k, v))  # [n, H, D]
            qt = q[t].double().view(H, G, D)
            s = torch.einsum("hgd,nhd->hgn", qt, keys) * scale
            mag = torch.einsum("hgd,nhd->hgn", qt.abs(), keys.abs()) * abs(scale)
            w = torch.softmax(s, -1)
            o = torch.einsum("hgn,nhd->hgd", w, values)
            spread = torch.einsum("hgn,nhd->hgd", w, values.abs())
            ds = ((D + 8) * 2.0 ** -23 + (2.0 ** -22 if f32 else 0)) * mag.amax(-1)
            # w x with x = (maximum - score): a relative error of the scaled difference.
            dw = ds + 2.0 ** -21 + 3 * F32_U
            rel = 2 * dw + (2.0 ** -22 if f32 else BF16_U) + (len(js) + 16) * 2.0 ** -23
            out[t] = o.reshape(Hq, D)
            bound[t] = (rel[..., None] * (spread + o.abs())).reshape(Hq, D)
    bound += unit(q.dtype) * (out.abs() + bound).nan_to_num() + 1e-30
    return out, bound
