"""Plain forms, in 64 bits, of the operators on a paged cache of e4m3 codes with block scales, and the bounds that
the kernels' roundings give."""
import math

import torch

F8 = torch.float8_e4m3fn


def to_e4m3(x):
    """x rounded to the nearest e4m3 number (ties to even), as float64; not finite, or above 448 after rounding: NaN."""
    x = x.double()
    a = x.abs()
    e = torch.floor(torch.log2(torch.where(a > 0, a, 1.0)))
    e = torch.where(torch.ldexp(torch.ones_like(a), e + 1) <= a, e + 1, torch.where(torch.ldexp(torch.ones_like(a), e) > a, e - 1, e))
    step = torch.ldexp(torch.ones_like(a), e.clamp(min=-6) - 3)
    y = torch.round(a / step) * step  # torch.round: halves to even
    return torch.where(y <= 448, torch.copysign(y, x), math.nan)


def scale_for(amax):
    """The smallest 2^e, e in [-126, 120], with amax <= 448 * 2^e."""
    for e in range(-126, 121):
        if amax <= 448 * 2.0 ** e:
            return 2.0 ** e
    raise AssertionError(amax)


def rotate(x, positions, inv_freq, interleaved=False, amplitude=1.0):
    """x [t, heads, d] float64 turned by positions [t]; with it, how far 32 bits may be off: cosine and sine 2 ulp
    (2^-22), the amplitude and three operations half a step each (2^-24), all relative to |a| + |b|."""
    x = x.double()
    off = torch.zeros_like(x)
    if inv_freq is None:
        return x, off
    rot = 2 * inv_freq.numel()
    t = positions.double()[:, None, None] * inv_freq.double()
    c, s = torch.cos(t), torch.sin(t)
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    na, nb = amplitude * (a * c - b * s), amplitude * (a * s + b * c)
    slack = (2.0 ** -22 + 4 * 2.0 ** -24) * abs(amplitude) * (a.abs() + b.abs())
    y = x.clone()
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = na, nb
        off[..., 0:rot:2] = off[..., 1:rot:2] = slack
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = na, nb
        off[..., :rot // 2] = off[..., rot // 2:rot] = slack
    return y, off


def append(x, codes, scale, slots, block):
    """One side of the append: x [T, H_kv, d] (already turned) into codes [pages, page, H_kv, d] (float64 values of
    the codes) and scale [pages, H_kv, page / block] (float64), both changed in place."""
    page = codes.shape[1]
    runs, t = [], 0
    slots = [s if 0 <= s < codes.shape[0] * page else -1 for s in slots]
    while t < len(slots):
        n = 1
        if slots[t] >= 0:
            while t + n < len(slots) and slots[t + n] == slots[t] + n and slots[t + n] % block:
                n += 1
            runs.append((t, n))
        t += n
    for t, n in runs:
        p, row, b = slots[t] // page, slots[t] % page, slots[t] % page // block
        held = row % block
        for h in range(codes.shape[2]):
            top = x[t:t + n, h].abs()
            now = scale_for(torch.where(torch.isfinite(top), top, 0.0).max().item())
            if held:
                before = scale[p, h, b].item()
                now = max(now, before)
                if now > before:
                    codes[p, row - held:row, h] = to_e4m3(codes[p, row - held:row, h] * (before / now))
            codes[p, row:row + n, h] = to_e4m3(x[t:t + n, h] / now)
            scale[p, h, b] = now


def values(codes, scale, table_row, n):
    """The first n rows of a request as float64 [n, H_kv, d]."""
    page = codes.shape[1]
    block = page // scale.shape[2]
    ids = [int(i) for i in table_row[:-(-n // page)]]
    x = torch.stack([codes[i].double() for i in ids]) if ids else torch.zeros((0,) + codes.shape[1:], dtype=torch.float64)
    s = torch.stack([scale[i].double() for i in ids]) if ids else torch.zeros((0,) + scale.shape[1:], dtype=torch.float64)
    return x.flatten(0, 1)[:n] * s.transpose(1, 2).repeat_interleave(block, 1).flatten(0, 1)[:n, :, None]


def attend(q, k_codes, v_codes, k_scale, v_scale, table, lens, cu, scale, causal):
    """q [T, H, d]; returns (o, lse, bound_o, bound_lse), float64; rows of no request NaN.

    The bounds follow from the roundings.  A query element is two e4m3 numbers over a power of two of its head
    vector, off by at most 2^-22 of the vector's largest element; each product is exact, and d of them summed in
    32 bits, truncating, are off by at most d 2^-23 of the sum of magnitudes; the two halves of the score, its scale and its
    base-2 exponent add four roundings (2^-22 of its magnitude): `off` in all, which moves ln p by as much, in
    numerator and denominator.  A probability times its value's scale is rounded to fp16 (2^-11) and cut into three e4m3 numbers
    that hold it, but for what lies 2^-24 below the row's largest; exponentials and sums in 32 bits add less than 2^-18
    relative; O is rounded to bf16 (2^-8)."""
    T, H, d = q.shape
    H_kv = k_codes.shape[2]
    G = H // H_kv
    q = q.double()
    o, bo = (torch.full((T, H, d), math.nan, dtype=torch.float64) for _ in "ab")
    lse, bl = (torch.full((T, H), math.nan, dtype=torch.float64) for _ in "ab")
    cu = list(range(len(lens) + 1)) if cu is None else cu
    for r, n in enumerate(lens):
        k, v = values(k_codes, k_scale, table[r], n), values(v_codes, v_scale, table[r], n)
        vs = values(torch.ones_like(v_codes, dtype=torch.float64), v_scale, table[r], n)[:, :, 0]
        for t in range(cu[r], cu[r + 1]):
            seen = n - (cu[r + 1] - t) + 1 if causal else n
            if seen <= 0:
                o[t], bo[t], lse[t], bl[t] = 0.0, 0.0, -math.inf, 0.0
                continue
            for h in range(H_kv):
                rows = slice(h * G, (h + 1) * G)
                x, y, w = k[:seen, h], v[:seen, h], vs[:seen, h]
                s = scale * (q[t, rows] @ x.T)
                m = s.amax(-1, keepdim=True)
                p = torch.exp(s - m)
                total = p.sum(-1, keepdim=True)
                lse[t, rows] = (m + torch.log(total))[:, 0]
                p = p / total
                o[t, rows] = p @ y
                size = q[t, rows].abs()
                off = scale * (d * 2.0 ** -23 * (size @ x.abs().T) + 2.0 ** -22 * size.amax(-1, keepdim=True) * x.abs().sum(-1))
                off = (off + 2.0 ** -22 * s.abs()).amax(-1, keepdim=True)
                spread = p @ y.abs()
                floor = 2.0 ** -24 * (p * w).amax(-1, keepdim=True) * (y.abs() / w[:, None]).sum(0)
                bo[t, rows] = 2.0 ** -8 * (o[t, rows].abs() + spread * 2.0 ** -8) + (2.0 ** -11 + 2.0 ** -18 + 2 * off) * spread + floor + 1e-30
                bl[t, rows] = (off + 2.0 ** -18 * (1.0 + lse[t, rows].abs()[:, None]))[:, 0]
    return o, lse, bo, bl
