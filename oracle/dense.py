"""Dense paged layers in float64: the step plan, the norm + rotation + insert,
and attention over every cached token.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).  Written from the formulas
of ``include/v4a_dense.h``: sequential bookkeeping for the plan, one token at
a time for the rest.
"""
from __future__ import annotations

import math
from collections import deque

import numpy as np

from .formats import bf16_decode, e4m3_decode

PAGE = 256


# ---- the step plan --------------------------------------------------------------

def step_plan(cached, fresh, tables, ring, first, count, max_tokens):
    """Sequential books: `tables` [L][B][cols] and `ring` are changed in place.
    Returns (seq_ids, positions, slots [L][T], token_starts, first, count)."""
    L, cap = len(tables), len(ring)
    free = deque(ring[(first + i) % cap] for i in range(count))
    taken = 0
    given = []
    seq_ids, positions, slots, starts = [], [], [[] for _ in range(L)], [0]
    for b, (c, f) in enumerate(zip(cached, fresh)):
        held = -(-c // PAGE)
        if f < 0:
            for k in range(held):
                for t in range(L):
                    given.append(tables[t][b][k])
        for p in range(c, c + max(f, 0)):
            if p // PAGE >= held:
                for t in range(L):
                    tables[t][b][held] = free.popleft()
                held += 1
                taken += 1
            seq_ids.append(b)
            positions.append(p)
            for t in range(L):
                slots[t].append(int(tables[t][b][p // PAGE]) * PAGE + p % PAGE)
        starts.append(len(seq_ids))
    for i, page in enumerate(given):
        ring[(first + count + i) % cap] = page
    pad = max_tokens - len(seq_ids)
    return (seq_ids + [-1] * pad, positions + [-1] * pad, [s + [-1] * pad for s in slots], starts,
            (first + taken * L) % cap, count - taken * L + len(given))


# ---- the rotation and the norm -----------------------------------------------------

def frequencies(dims, theta=10000.0, scaling="plain", factor=1.0, original=0.0, beta_fast=32.0, beta_slow=1.0, table=None):
    f = np.array([theta ** (-2.0 * j / dims) for j in range(dims // 2)]) if table is None else np.asarray(table, np.float64)
    if scaling == "linear":
        return f / factor
    if scaling == "yarn":
        turns = original * f / (2 * math.pi)
        g = np.clip((turns - beta_slow) / (beta_fast - beta_slow), 0.0, 1.0)
        return f * g + f / factor * (1.0 - g)
    return f


def rotate(x, pos, freq, first=0, half=False, magnitude=1.0):
    """x [..., dim] at one position."""
    y = np.array(x, np.float64, copy=True)
    for j, f in enumerate(freq):
        a, b = (first + j, first + len(freq) + j) if half else (first + 2 * j, first + 2 * j + 1)
        # the angle's fraction of a turn, so that far positions keep their digits
        ang = 2 * math.pi * math.fmod(float(pos) * float(f) / (2 * math.pi), 1.0)
        c, s = math.cos(ang) * magnitude, math.sin(ang) * magnitude
        u, v = np.asarray(x[..., a], np.float64), np.asarray(x[..., b], np.float64)
        y[..., a] = u * c - v * s
        y[..., b] = u * s + v * c
    return y


def rms_norm(x, gamma, eps):
    x = np.asarray(x, np.float64)
    if gamma is None:
        return x
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * gamma


# ---- the cache -----------------------------------------------------------------------

def block_bytes(kv_heads, dim, fp8):
    return 2 * kv_heads * PAGE * (dim + 4 if fp8 else 2 * dim)


def read_row(pool, kv_heads, dim, fp8, block, which, head, at):
    """One stored row (which: 0 key, 1 value) of uint8 pool [blocks][bytes], in float64."""
    plane = which * kv_heads + head
    blk = pool[block]
    if not fp8:
        o = (plane * PAGE + at) * dim * 2
        return bf16_decode(blk[o:o + 2 * dim].copy().view(np.uint16))
    codes, scale = raw_row(pool, kv_heads, dim, block, which, head, at)
    return e4m3_decode(codes) * float(scale)


def raw_row(pool, kv_heads, dim, block, which, head, at):
    """(codes, scale) of one fp8 row."""
    row = (which * kv_heads + head) * PAGE + at
    o = 2 * kv_heads * PAGE * dim + 4 * row
    return pool[block][row * dim:(row + 1) * dim].copy(), pool[block][o:o + 4].copy().view(np.float32)[0]


# ---- attention -------------------------------------------------------------------------

def visible(m, window, sinks):
    """Positions that a query at position m sees."""
    return [j for j in range(m + 1) if window == 0 or j > m - window or j < sinks]


def attention(q, keys, values, scale):
    """q [G][D], keys and values [N][D] -> (o, lse, sum p|v|, max sum |q||k| scale); N = 0 gives 0 and -inf."""
    if len(keys) == 0:
        z = np.zeros(q.shape)
        return z, np.full(q.shape[0], -np.inf), z, np.zeros(q.shape[0])
    z = scale * (q @ keys.T)
    top = z.max(axis=1, keepdims=True)
    p = np.exp(z - top)
    total = p.sum(axis=1, keepdims=True)
    p = p / total
    return p @ values, (top + np.log(total))[:, 0], p @ np.abs(values), scale * (np.abs(q) @ np.abs(keys).T).max(axis=1)
