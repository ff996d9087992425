"""Oracle of the 4-bit key/value cache: row encoding, cache layout, block tables, attention.

Everything is plain NumPy from the definitions in ``include/kq.h``; encoding and
attention are evaluated in float64.

Pins (``tests/test_oracle_kv.py``): the encoding against exact rational
arithmetic and the q4_0 wire encoder, the layout against a hand-packed page,
block tables against a step-by-step allocator, attention against a scalar
softmax loop and closed forms (uniform weights, one key).
"""

from __future__ import annotations

import numpy as np


def encode(x: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """Rows float32 [..., d] -> codes uint8 [..., d] and float16 scales [..., d / 32].

    NaN counts as 0, magnitudes above 65504 as 65504; the scale is float16 of
    the float32 quotient max|x| / 7, at most 8188; each code is the nearest of
    the sixteen values scale * (c - 8), the lower code at equal distance, and 8
    where the scale is 0.
    """
    x = np.asarray(x, np.float32)
    x = np.where(np.isnan(x), np.float32(0), np.clip(x, np.float32(-65504), np.float32(65504)))
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    amax = np.max(np.abs(b), axis=-1)
    scale = np.minimum(amax / np.float32(7), np.float32(8188)).astype(np.float16)
    grid = scale.astype(np.float64)[..., None, None] * (np.arange(16) - 8)
    dist = np.abs(b.astype(np.float64)[..., None] - grid)
    codes = np.argmin(dist, axis=-1)  # the first minimum: the lower code
    codes = np.where((scale == 0)[..., None], 8, codes)
    return codes.astype(np.uint8).reshape(x.shape), scale


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """float64 values scale * (c - 8)."""
    c = codes.astype(np.float64).reshape(*scales.shape, 32) - 8
    return (c * scales.astype(np.float64)[..., None]).reshape(codes.shape)


def page_bytes(page: int, d: int) -> int:
    return page * (d // 2 + d // 16)


def store(cache: np.ndarray, page: int, slots, codes: np.ndarray, scales: np.ndarray) -> None:
    """Write rows [tokens, heads, d] into cache uint8 [pages, heads, page_bytes]; slots outside it are skipped."""
    pages, heads, _ = cache.shape
    d = codes.shape[-1]
    for t, slot in enumerate(np.asarray(slots).tolist()):
        if not 0 <= slot < pages * page:
            continue
        p, r = divmod(slot, page)
        by = (codes[t, :, 0::2] | (codes[t, :, 1::2] << 4)).astype(np.uint8)
        cache[p, :, r * (d // 2):(r + 1) * (d // 2)] = by
        at = page * (d // 2) + r * (d // 16)
        cache[p, :, at:at + d // 16] = np.ascontiguousarray(scales[t]).view(np.uint8).reshape(heads, -1)


def load(cache: np.ndarray, page: int, d: int, slots) -> np.ndarray:
    """float64 values [len(slots), heads, d] of the rows at the slots (all inside the cache)."""
    slots = np.asarray(slots, np.int64)
    p, r = slots // page, slots % page
    by = cache[:, :, :page * (d // 2)].reshape(cache.shape[0], cache.shape[1], page, d // 2)[p, :, r]
    codes = np.stack((by & 15, by >> 4), axis=-1).reshape(len(slots), cache.shape[1], d)
    sc = np.ascontiguousarray(cache[:, :, page * (d // 2):]).view(np.float16)
    sc = sc.reshape(cache.shape[0], cache.shape[1], page, d // 32)[p, :, r]
    return values(codes, sc)


def block_tables(ctx, new, page, free, head, table, tokens):
    """(table, slots, cu_new, seq_lens, head, status) of one step, requests one after the other."""
    table = [list(map(int, row)) for row in table]
    width = len(table[0]) if table else 0
    free = [int(f) for f in free]
    avail = len(free) - head if 0 <= head <= len(free) else 0
    slots, cu, lens, status, row, asked, taken = [-1] * tokens, [0], [], 0, 0, 0, 0
    for s, (c, n) in enumerate(zip(map(int, ctx), map(int, new))):
        rows = max(n, 0)
        first, row = row, row + rows
        cu.append(min(row, tokens))
        bad = 0
        if c < 0 or n < 0:
            bad = 8
        else:
            held, total = -(-c // page), -(-(c + n) // page)
            if total > width or c + n > 2 ** 31 - 1:
                bad |= 2
            if n > 0 and row > tokens:
                bad |= 4
        if not bad and total > held:
            asked += total - held
            if asked > avail:
                bad = 1
            else:
                table[s][held:total] = free[head + taken:head + asked]
                taken = asked
        status |= bad
        lens.append(0 if bad else c + n)
        for i in range(0 if bad else rows):
            if first + i < tokens:
                pid = table[s][(c + i) // page]
                slot = pid * page + (c + i) % page
                slots[first + i] = slot if pid >= 0 and slot < 2 ** 31 else -1
    return table, slots, cu, lens, head + taken, status


def attention(q, cu, lens, table, k_cache, v_cache, page, scale, window=0, detail=False):
    """float64 [tokens, q_heads, d] from q [tokens, q_heads, d]; rows of no request are NaN.

    With ``detail`` also, per row: sum p |v| [tokens, q_heads, d], the largest
    scale * sum |q| |k| over its keys, and its number of keys.
    """
    q = np.asarray(q, np.float64)
    tokens, hq, d = q.shape
    pages, kv = k_cache.shape[:2]
    group = hq // kv
    out = np.full(q.shape, np.nan)
    absv, mag, count = np.zeros(q.shape), np.zeros((tokens, hq)), np.zeros((tokens, hq))
    for s in range(len(lens)):
        a, b = (min(max(int(cu[s + i]), 0), tokens) for i in (0, 1))
        length = min(max(int(lens[s]), 0), len(table[s]) * page)
        out[a:b] = 0
        ids = np.repeat(np.asarray(table[s], np.int64), page)[:length]
        there = (ids >= 0) & (ids < pages)
        slots = np.where(there, ids, 0) * page + np.arange(length) % page
        k, v = (load(c, page, d, slots) for c in (k_cache, v_cache))
        for t in range(a, b):
            p = length - (b - a) + (t - a)
            see = there & (np.arange(length) <= p)
            if window > 0:
                see &= np.arange(length) > p - window
            if not see.any():
                continue
            for h in range(hq):
                ks, vs = k[see, h // group], v[see, h // group]
                w = scale * (ks @ q[t, h])
                w = np.exp(w - w.max())
                w /= w.sum()
                out[t, h] = w @ vs
                if detail:
                    absv[t, h] = w @ np.abs(vs)
                    mag[t, h] = abs(scale) * (np.abs(ks) @ np.abs(q[t, h])).max()
                    count[t, h] = see.sum()
    return (out, absv, mag, count) if detail else out
