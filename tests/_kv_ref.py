"""Plain numpy forms of the operators around the paged cache, from their definitions, in 64 bits (the
quantised codes and scores of page selection in the fp32 steps that define them)."""
import math

import numpy as np


def rope(x, positions, inv_freq, rot, interleaved=False, inverse=False, amplitude=1.0):
    """x [..., n, h, d] float64, positions [n] (broadcast against x[..., n]); returns float64."""
    x = np.asarray(x, dtype=np.float64)
    t = np.asarray(positions, dtype=np.longdouble)[..., None] * np.asarray(inv_freq, dtype=np.longdouble)
    c, s = np.cos(t).astype(np.float64)[..., None, :], np.sin(t).astype(np.float64)[..., None, :]
    s = -s if inverse else s
    y = x.copy()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = amplitude * (a * c - b * s), amplitude * (a * s + b * c)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = amplitude * (a * c - b * s), amplitude * (a * s + b * c)
    return y


def plan(ctx, new, table, free, count, page, total):
    """Lists in, (cu, seq_lens, positions, slots, table, left) out."""
    table = [list(row) for row in table]
    cu, lens, pos, slots = [0], [], [], []
    for r, (c, n) in enumerate(zip(ctx, new)):
        for p in range(c, c + n):
            if p % page == 0:
                count -= 1
                table[r][p // page] = free[count]
            pos.append(p)
            slots.append(table[r][p // page] * page + p % page)
        cu.append(cu[-1] + n)
        lens.append(c + n)
    pad = total - cu[-1]
    return cu, lens, pos + [0] * pad, slots + [-1] * pad, table, count


def sketch(keys):
    """keys [rows, H_kv, d] of one page -> (codes int8 [H_kv, 2 d], amp fp32 [H_kv])."""
    k = np.asarray(keys, dtype=np.float32)
    hi, lo = k.max(0), k.min(0)
    amp = np.maximum(np.abs(hi), np.abs(lo)).max(-1)
    code = np.zeros(hi.shape[:1] + (2 * hi.shape[1],), dtype=np.int8)
    for h in range(k.shape[1]):
        if not np.isfinite(k[:, h]).all():
            amp[h] = np.inf
        elif amp[h] > 0:
            both = np.concatenate([hi[h], lo[h]])
            code[h] = np.rint((both / amp[h]).astype(np.float32) * np.float32(127)).astype(np.int8)
    return code, amp


def scores(q, codes, amp):
    """q [G, d] fp32 of one group, codes [n, 2 d], amp [n] -> fp32 [n]."""
    d = q.shape[1]
    best = None
    for x in np.asarray(q, dtype=np.float32):
        top = np.abs(x).max()
        if not np.isfinite(x).all():
            value = np.full(len(codes), np.inf, dtype=np.float32)
        else:
            c = np.rint(x / top * np.float32(127)).astype(np.int64) if top > 0 else np.zeros(d, dtype=np.int64)
            dots = codes[:, :d].astype(np.int64) @ np.maximum(c, 0) + codes[:, d:].astype(np.int64) @ np.minimum(c, 0)
            value = top * dots.astype(np.float32)
        best = value if best is None else np.maximum(best, value)
    with np.errstate(invalid="ignore"):
        s = best * np.asarray(amp, dtype=np.float32)
    return np.where(np.isnan(s) | np.isinf(amp), np.float32(np.inf), s)


def select(q, codes, amp, table, lens, cu, page, budget, first, last):
    """q [T, H, d]; returns (tables [T, H_kv, budget], sel_lens [T])."""
    T, H, _ = q.shape
    H_kv = codes.shape[1]
    G = H // H_kv
    tables = np.full((T, H_kv, budget), -1, dtype=np.int32)
    sel = np.zeros(T, dtype=np.int32)
    cu = list(range(len(lens) + 1)) if cu is None else cu
    for r in range(len(lens)):
        for t in range(cu[r], cu[r + 1]):
            pos = lens[r] - (cu[r + 1] - t)
            if pos < 0:
                continue
            n = pos // page + 1
            sel[t] = (min(n, budget) - 1) * page + pos % page + 1
            for h in range(H_kv):
                ids = np.asarray(table[r][:n])
                chosen = list(range(n))
                if n > budget:
                    s = scores(q[t, h * G:(h + 1) * G], codes[ids, h], amp[ids, h])
                    always = set(range(first)) | set(range(n - last, n))
                    rest = sorted((p for p in range(n) if p not in always), key=lambda p: (-s[p], p))
                    chosen = sorted(always | set(rest[:budget - first - last]))
                tables[t, h, :len(chosen)] = ids[chosen]
    return tables, sel


def attend(q, k_cache, v_cache, tables, sel, scale):
    """Attention over the chosen pages; returns (o, lse, bound_o, bound_lse).

    The bounds follow from the kernel's roundings: P enters the second product in bf16 (half a step,
    2^-8 relative to each p) and O is rounded to bf16 (2^-8 of |o|); scores are fp32 sums of d exact
    products, off by at most d 2^-24 sum |q k|, which moves ln p by scale times that, twice (numerator and
    denominator); fp32 sums and exponentials add below 2^-19 relative."""
    T, H, d = q.shape
    H_kv = tables.shape[1]
    G = H // H_kv
    q = np.asarray(q, dtype=np.float64)
    o, lse = np.zeros((T, H, d)), np.full((T, H), -np.inf)
    bo, bl = np.zeros((T, H, d)), np.zeros((T, H))
    for t in range(T):
        if sel[t] == 0:
            continue
        for h in range(H_kv):
            ids = tables[t, h][tables[t, h] >= 0]
            k = np.asarray(k_cache[ids][:, :, h], dtype=np.float64).reshape(-1, d)[:sel[t]]
            v = np.asarray(v_cache[ids][:, :, h], dtype=np.float64).reshape(-1, d)[:sel[t]]
            for g in range(h * G, (h + 1) * G):
                s = scale * (k @ q[t, g])
                m = s.max()
                p = np.exp(s - m)
                lse[t, g] = m + math.log(p.sum())
                p /= p.sum()
                o[t, g] = p @ v
                off = scale * d * 2.0 ** -24 * (np.abs(k) @ np.abs(q[t, g])).max()
                spread = p @ np.abs(v)
                bo[t, g] = 2.0 ** -8 * (spread + np.abs(o[t, g])) + (2 * off + 2.0 ** -18) * spread + 1e-6
                bl[t, g] = off + 2.0 ** -19 * max(1.0, abs(lse[t, g])) + 2.0 ** -19
    return o, lse, bo, bl
