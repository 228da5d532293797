"""Plain 64-bit references of the paged NVFP4 key/value cache: page bookkeeping
by the documented rules, one step after another, and attention over dequantized
values with the bound of the kernels' roundings."""
import math

import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def e4m3(b):
    """Values of E4M3 bytes (finite ones)."""
    b = b.astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    return np.where(b & 0x80, -v, v)


def dequantize(codes, scales, gscale):
    """float64 values [..., d] of codes [..., d / 2] and scales [..., d / 16]."""
    n = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1)
    v = GRID[n & 7] * np.where(n & 8, -1.0, 1.0)
    return v * np.repeat(e4m3(scales), 16, -1) * float(np.float32(gscale))


def pages_update(held, target, table, free, count, page_size, slot_capacity, max_pages):
    """(status, table, free, count, lens, q_starts, slots) by the rules of include/fh.h."""
    table, free = table.copy(), free.copy()
    held, target = [int(x) for x in held], [int(x) for x in target]
    n = len(held)
    slots = np.full(slot_capacity, -1, np.int64)
    fail = (table.copy(), free.copy(), count, np.array(held), np.zeros(n + 1, np.int64), slots)

    def pages(x):
        return -(-x // page_size)
    status = 0
    new = need = give = 0
    for h, t in zip(held, target):
        if h < 0 or t < 0:
            status |= 4
            continue
        if max(pages(h), pages(t)) > max_pages:
            status |= 2
        need += max(0, pages(t) - pages(h))
        give += max(0, pages(h) - pages(t))
        new += max(0, t - h)
    if count < 0 or count + give > len(free):
        status |= 8
    if need > count + give:
        status |= 1
    if new > slot_capacity:
        status |= 16
    if status:
        return (status, *fail)
    for b in range(n):
        for j in range(pages(target[b]), pages(held[b])):
            free[count] = table[b, j]
            count += 1
    top = count
    for b in range(n):
        for j in range(pages(held[b]), pages(target[b])):
            top -= 1
            table[b, j] = free[top]
    starts = [0]
    for b in range(n):
        for i in range(held[b], target[b]):
            page = int(table[b, i // page_size])
            slots[starts[-1] + i - held[b]] = page * page_size + i % page_size if page >= 0 else -1
        starts.append(starts[-1] + max(0, target[b] - held[b]))
    return 0, table, free, top, np.array(target), np.array(starts), slots


def attention(q, k_of, v_of, lens, q_starts, sm_scale, causal, window, there=None):
    """float64 (out, lse, tol_out, tol_lse) of q [T, Hq, d]; k_of(b), v_of(b): [len, Hk, d] of request b's tokens;
    there(b): which of them can be seen at all.  Rows of no request are NaN.

    The bounds.  Scores: q is exact in FP16 up to a power of two, code * scale is exact, and a sum of d products in
    FP32 (a truncating adder included) is off by at most d 2^-23 of the sum of magnitudes; the scaling rounds three
    times more.  With ds that error in the largest score (natural units), a weight is off by the factor e^ds, ex2's
    2^-22 and the 2^-23 |s| of its argument's rounding.  P is rounded to FP16: 2^-11 relative, and at most 2^-25 in
    units in which the largest weight is at least 2^6.  n weighted sums in FP32: n 2^-23 of the sum of magnitudes.
    The result is rounded to BF16: 2^-8."""
    T, Hq, d = q.shape
    out = np.full((T, Hq, d), np.nan)
    lse = np.full((T, Hq), np.nan)
    tol = np.full((T, Hq, d), np.nan)
    tol_l = np.full((T, Hq), np.nan)
    for b in range(len(lens)):
        r0, r1 = int(q_starts[b]), int(q_starts[b + 1])
        L = int(lens[b])
        if r1 <= r0:
            continue
        k, v = k_of(b), v_of(b)
        G = Hq // k.shape[1]
        ok = np.ones(L, bool) if there is None else there(b)
        for i in range(r1 - r0):
            pos = L - (r1 - r0) + i
            j = np.arange(L)
            see = ok & ((j <= pos) if causal else True) & ((j > pos - window) if window else True)
            for h in range(Hq):
                ks, vs = k[see, h // G], v[see, h // G]
                n = ks.shape[0]
                if n == 0:
                    out[r0 + i, h], lse[r0 + i, h], tol[r0 + i, h], tol_l[r0 + i, h] = 0, -math.inf, 0, 0
                    continue
                s = sm_scale * (ks @ q[r0 + i, h])
                mag = abs(sm_scale) * (np.abs(ks) @ np.abs(q[r0 + i, h]))
                m = s.max()
                w = np.exp(s - m)
                total = w.sum()
                p = w / total
                out[r0 + i, h] = p @ vs
                lse[r0 + i, h] = m + math.log(total)
                ds = (d + 4) * 2.0 ** -23 * mag.max() + 2.0 ** -23 * np.abs(s).max()
                rel = 2 * (math.expm1(ds) + 2.0 ** -21 + 2.0 ** -22 * (np.abs(s).max() + abs(m)) + n * 2.0 ** -23)
                av = p @ np.abs(vs)
                tol[r0 + i, h] = (2.0 ** -8 * np.abs(out[r0 + i, h]) + 1.01 * av * (2.0 ** -11 + rel)
                                  + n * 2.0 ** -31 * np.abs(vs).max() + 1e-38)
                tol_l[r0 + i, h] = rel + 2.0 ** -21 * (1 + abs(lse[r0 + i, h]))
    return out, lse, tol, tol_l
