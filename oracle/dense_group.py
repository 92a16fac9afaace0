"""The dense cache with one scale per 64 positions and KV head, in float64: the
quantising insert, row by row, and reading rows back.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).  Written from the formulas
of ``include/v4a_dense.h``, one group of one head at a time.
"""
from __future__ import annotations

import numpy as np

from .formats import e4m3_decode, e4m3_encode

PAGE, GROUP = 256, 64
LEAST = 2.0 ** -126


def block_bytes(kv_heads, dim):
    return 2 * kv_heads * PAGE * dim + 2 * kv_heads * (PAGE // GROUP) * 4


def pow2(a):
    """The smallest power of two s with a / s <= 448, at least 2^-126."""
    s = LEAST
    while a > 448.0 * s:
        s *= 2.0
    return s


def _codes_at(kv_heads, dim, which, head, row):
    return ((which * kv_heads + head) * PAGE + row) * dim


def _scale_at(kv_heads, dim, which, head, row):
    return 2 * kv_heads * PAGE * dim + 4 * ((which * kv_heads + head) * (PAGE // GROUP) + row // GROUP)


def read_scale(blk, kv_heads, dim, which, head, row):
    o = _scale_at(kv_heads, dim, which, head, row)
    return float(blk[o:o + 4].copy().view(np.float32)[0])


def read_row(pool, kv_heads, dim, block, which, head, row):
    o = _codes_at(kv_heads, dim, which, head, row)
    return e4m3_decode(pool[block][o:o + dim]) * read_scale(pool[block], kv_heads, dim, which, head, row)


def insert(pool, kv_heads, dim, slots, rows):
    """Writes one call's tokens into uint8 pool [blocks][bytes]; rows = (keys, values), each [T][kv_heads][dim] float64."""
    groups: dict[int, list[int]] = {}
    for t, s in enumerate(slots):
        if s >= 0:
            groups.setdefault(s // GROUP, []).append(t)
    for g, tokens in groups.items():
        blk = pool[g * GROUP // PAGE]
        first = g * GROUP % PAGE
        written = {slots[t] % PAGE for t in tokens}
        anew = first in written
        for which in (0, 1):
            for h in range(kv_heads):
                x = np.stack([rows[which][t, h] for t in tokens])
                finite = np.abs(x[np.isfinite(x)])
                old = LEAST if anew else max(LEAST, read_scale(blk, kv_heads, dim, which, h, first))
                new = max(old, pow2(finite.max() if finite.size else 0.0))
                if new > old and not anew:
                    for r in range(first, first + GROUP):
                        if r not in written:
                            o = _codes_at(kv_heads, dim, which, h, r)
                            blk[o:o + dim] = e4m3_encode(e4m3_decode(blk[o:o + dim]) * (old / new))
                for t, row in zip(tokens, x):
                    o = _codes_at(kv_heads, dim, which, h, slots[t] % PAGE)
                    blk[o:o + dim] = e4m3_encode(row / new)
                o = _scale_at(kv_heads, dim, which, h, first)
                blk[o:o + 4] = np.array([new], np.float32).view(np.uint8)


def prompt_visible(n, keys, i, causal, window, sinks):
    """Keys that query i of n sees among `keys` of its sequence."""
    if not causal:
        return list(range(keys))
    m = keys - n + i
    return [j for j in range(min(m, keys - 1) + 1) if window == 0 or j > m - window or j < sinks]

