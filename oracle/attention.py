"""Plain forms, in 64 bits, of the rotary positions, the 8-bit paged cache and
the attention over it.  numpy only; shares no code with the GPU path.

bf16 arrays come as uint16 patterns, E4M3 codes as uint8.
"""
from __future__ import annotations

import math

import numpy as np

E_MIN, E_MAX = -40, 119


def bf16_values(a):
    with np.errstate(invalid="ignore"):                    # signalling NaN patterns
        return (np.asarray(a, dtype=np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def bf16_patterns(v):
    """float64 -> nearest-even bf16 patterns (through float32, whose rounding cannot move a
    bf16 rounding of the values used here: sums of a few bf16 products)."""
    u = np.asarray(v, dtype=np.float32).view(np.uint32)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(v), np.uint16(0x7FC0), r)


def e4m3_table():
    """Value of every E4M3 code (bias 7, no infinities, S.1111.111 = NaN)."""
    v = np.empty(256)
    for c in range(256):
        s, e, m = -1.0 if c & 0x80 else 1.0, (c >> 3) & 15, c & 7
        v[c] = s * (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        if c & 0x7F == 0x7F:
            v[c] = math.nan
    return v


TABLE = e4m3_table()
_MAGS = TABLE[:127]                                       # ascending: 0 .. 448
_MIDS = (_MAGS[1:] + _MAGS[:-1]) / 2


def e4m3_encode(v):
    """Nearest code, ties to the even code, saturating; NaN and infinities give 0x7F."""
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(np.where(np.isfinite(v), v, 0.0))
    lo = np.searchsorted(_MIDS, a, side="left")           # a <= mid stays below: ties go down ...
    tie = (lo < len(_MIDS)) & (a == _MIDS[np.minimum(lo, len(_MIDS) - 1)])
    code = np.where(tie & (lo % 2 == 1), lo + 1, lo).astype(np.uint8)   # ... unless the lower code is odd
    code = code | (np.signbit(v).astype(np.uint8) << 7)
    return np.where(np.isfinite(v), code, np.uint8(0x7F)).astype(np.uint8)


def rope(x, positions, freqs, dims, layout, inverse=False):
    """x [tokens, heads, dim] float64, unrounded result; and the pairs' |a| + |b| for error bounds."""
    y, mag = x.copy(), np.abs(x)
    start = f = 0
    for axis, d in enumerate(dims):
        phi = positions[:, axis, None].astype(np.float64) * freqs[None, f:f + d // 2]
        c, s = np.cos(phi)[:, None], np.sin(phi)[:, None] * (-1 if inverse else 1)
        i = np.arange(d // 2)
        lo = start + (2 * i if layout == "interleaved" else i)
        hi = lo + (1 if layout == "interleaved" else d // 2)
        a, b = x[:, :, lo], x[:, :, hi]
        y[:, :, lo], y[:, :, hi] = a * c - b * s, a * s + b * c
        mag[:, :, lo] = mag[:, :, hi] = np.abs(a) + np.abs(b)
        start, f = start + d, f + d // 2
    return y, mag


def block_scale(amax):
    """2^e, the smallest e in [E_MIN, E_MAX] with amax <= 448 * 2^e."""
    e = E_MIN
    while e < E_MAX and amax > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def cache_write(codes, scale, x, table, held, cu):
    """codes [pages, heads, page, dim] and scale [pages, heads] updated in place from x [tokens, heads, dim] float64."""
    heads, page = codes.shape[1:3]
    for b in range(len(held)):
        n = int(cu[b + 1] - cu[b])
        if n == 0:
            continue
        for blk in range(int(held[b]) // page, (int(held[b]) + n - 1) // page + 1):
            p = table[b, blk]
            lo, hi = max(blk * page, int(held[b])), min((blk + 1) * page, int(held[b]) + n)
            old = lo - blk * page
            for h in range(heads):
                new = x[cu[b] + lo - held[b]:cu[b] + hi - held[b], h]
                fine = np.abs(new[np.isfinite(new)])
                s = block_scale(fine.max() if fine.size else 0.0)
                was = float(scale[p, h])
                if old and was > s:
                    s = was
                if old and s != was:
                    codes[p, h, :old] = e4m3_encode(TABLE[codes[p, h, :old]] * was / s)
                codes[p, h, old:old + hi - lo] = e4m3_encode(new / s)
                scale[p, h] = s


def cache_values(codes, scale):
    """[pages, heads, page, dim] float64."""
    return TABLE[codes] * scale.astype(np.float64)[:, :, None, None]


def gather(values, table, length):
    """[length, heads, dim] of one sequence's row of the page table."""
    page = values.shape[2]
    pos = np.arange(length)
    return values[np.asarray(table)[pos // page], :, pos % page]


def attention(q, k, v, scale, causal=False, window=0, sinks=0, before=0):
    """One sequence: q [n, heads, dim], k, v [L, kv_heads, dim] float64.  The first `sinks` positions stay visible under a
    window; the first `before` keys are a prefix that every query sees, positions counting from its end.  Returns out, lse
    and, for error bounds, the weighted mean of |v|, the largest |s| product sum, and the largest single contribution's share."""
    n, heads, dim = q.shape
    L, kv_heads = k.shape[:2]
    out, mean_abs = np.zeros((n, heads, dim)), np.zeros((n, heads, dim))
    lse = np.full((n, heads), -np.inf)
    prod, top = np.zeros((n, heads)), np.zeros((n, heads))
    pos, j = np.arange(L - before - n, L - before)[:, None], np.arange(-before, L - before)[None]
    see = np.ones((n, L), dtype=bool)
    if causal:
        see &= j <= pos
    if window > 0:
        see &= (j > pos - window) | (j < sinks)
    see |= j < 0
    for h in range(heads):
        kk, vv = k[:, h // (heads // kv_heads)], v[:, h // (heads // kv_heads)]
        for i in range(n):
            at = np.nonzero(see[i])[0]
            if not at.size:
                continue
            with np.errstate(invalid="ignore"):
                s = scale * (kk[at] @ q[i, h])
                m = s.max()
                p = np.exp(s - m)
                out[i, h] = p @ vv[at] / p.sum()
                lse[i, h] = m + np.log(p.sum())
                mean_abs[i, h] = p @ np.abs(vv[at]) / p.sum()
                prod[i, h] = abs(scale) * (np.abs(kk[at]) @ np.abs(q[i, h])).max()
                top[i, h] = np.nanmax(p[:, None] * np.abs(vv[at])) / p.sum() if np.isfinite(m) else np.nan
    return out, lse, mean_abs, prod, top


def norm_rope(x, weight, eps, turn):
    """x [tokens, heads, dim] float64 normed over its channels, times weight, turned by `turn` (a function of rows that
    returns them and a bound on the pairs' sizes).  Unrounded."""
    z = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    return turn(z)


def norm_rope_backward(dy, x, weight, eps, turn_back):
    """Gradients (dx, dweight), and for error bounds the sums of magnitudes that each is made of."""
    g, mag = turn_back(dy)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    hat = x * r
    dx = r * (weight * g - hat * (weight * g * hat).mean(-1, keepdims=True))
    size = r * (np.abs(weight) * mag + np.abs(hat) * (np.abs(weight) * mag * np.abs(hat)).mean(-1, keepdims=True))
    return dx, (g * hat).sum((0, 1)), size, (mag * np.abs(hat)).sum((0, 1))


def kv_tables(held, count, table, free, free_at, page, pages, tokens, most):
    """The batch's tables one token after another.  Returns cu, kv_len, slots, positions, table, free_at, whether anything
    is out of range."""
    table, cu, kv, slots, positions, bad = table.copy(), [0], [], [], [], False
    room, at = table.shape[1], int(free_at)
    for b in range(len(held)):
        h, n = int(held[b]), int(count[b])
        if h < 0 or n < 0 or n > most or h + n >= 2 ** 31 or -(-(h + n) // page) > room:
            h, n, bad = 0, 0, True
        for p in range(-(-h // page), -(-(h + n) // page)):
            ok = 0 <= at < len(free)
            table[b, p] = free[at] if ok and 0 <= free[at] < pages else -1
            at += 1
            bad |= table[b, p] < 0
        for pos in range(h, h + n):
            page_id = int(table[b, pos // page])
            ok = 0 <= page_id < pages
            bad |= not ok
            slots.append(page_id * page + pos % page if ok else -1)
            positions.append(float(pos))
        cu.append(min(cu[-1] + n, 2 ** 31 - 1))
        kv.append(h + n)
    bad |= len(slots) > tokens
    behind = [-1] * (tokens - len(slots))
    taken = min(at - int(free_at), max(0, len(free) - int(free_at)))     # a place before the list is passed like any other
    return cu, kv, (slots + behind)[:tokens], (positions + behind)[:tokens], table, int(free_at) + taken, bad
