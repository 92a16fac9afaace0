"""Dense caches with one scale per 64 positions and KV head, and whole prompts
over packed rows, on the GPU against the fp64 oracle: the quantising insert
(codes and scales byte for byte from the packed rows), the read back (exact),
attention over the cache, prompt attention, and a run of them together.

Tolerances count roundings, as in test_gpu_dense.py: an output bf16 rounding is
off by at most 2^-8 of the value, a probability rounded to bf16 by 2^-8 of
itself (prompts), one rounded to f16 by 2^-11 (caches; those below 2^-25 of the
largest by 2^-36 of it); a logit's dot product of D terms is off by (D + 8)
2^-24 of the largest sum |q||k| (as a relative error of p, twice: in p and in
the sum); the sums over N keys by (N + 32) 2^-24.  Chunks over a cache take a
query as two e4m3 numbers after a power of two that brings the row's largest
element into [2^7, 2^8): a bf16 x of exponent e is a multiple of 2^(e - 7), the
nearest e4m3 (half a step: 2^(e - 4)) leaves at most 8 such units, which four bits
hold, so the sum is x unless the rest falls below e4m3's least step 2^-9: then it
is off by half of that, 2^-10 <= 2^-17 of the largest element.  A logit is off by
at most 2^-17 of that element times the largest sum |k|, times the scale.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from oracle import dense as OD
from oracle import dense_group as OG
from oracle import formats as F
from tests.test_gpu_dense import Layer, _attend, _runs

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32 = dict(dtype=torch.int32, device=DEV)


def _dense():
    from compressed_sparse_long_c4a_gb300 import dense
    return dense


def _f64(t):
    return t.double().cpu().numpy()


# --------------------------------------------------------------------------
# The insert
# --------------------------------------------------------------------------

def _same_cache(pool, want, K, dim):
    got, n = pool.cpu().numpy(), OG.block_bytes(K, dim)
    bad = np.argwhere(got != want)
    assert not len(bad), (bad[:5].tolist(), [int(got[tuple(b)]) for b in bad[:5]], [int(want[tuple(b)]) for b in bad[:5]], n)


def _insert_case(dim, H, K, runs, seed, extra=48, std=2.0, blocks=None):
    """Sequences of (first position, tokens) with blocks of their own."""
    g = torch.Generator().manual_seed(seed)
    T = sum(n for _, n in runs)
    cols = max(-(-(c + n) // 256) for c, n in runs)
    blocks = len(runs) * cols + 2 if blocks is None else blocks
    table = torch.randperm(blocks, generator=g)[:len(runs) * cols].view(len(runs), cols)
    pos = [p for c, n in runs for p in range(c, c + n)]
    slots = [int(table[b, p // 256]) * 256 + p % 256 for b, (c, n) in enumerate(runs) for p in range(c, c + n)]
    x = (torch.randn((T, (H + 2 * K) * dim + 8), generator=g) * std).to(torch.bfloat16).to(DEV)      # odd token stride
    q, k, v = (x[:, a * dim:b * dim].unflatten(1, (b - a, dim)) for a, b in ((0, H), (H, H + K), (H + K, H + 2 * K)))
    pool = torch.zeros((blocks, OG.block_bytes(K, dim) + extra), dtype=torch.uint8)
    # codes of earlier steps, and their scales
    body = 2 * K * 256 * dim
    pool[:, :body] = (torch.randn((blocks, body), generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    pool[:, body:body + 32 * K] = torch.exp2(torch.randint(-10, -5, (blocks, 8 * K), generator=g).float()).view(torch.uint8)
    return T, pos, slots, q, k, v, pool.to(DEV), g


@pytest.mark.parametrize("dim,H,K,runs", [
    (64, 4, 2, ((0, 1),)), (64, 4, 4, ((63, 2), (64, 1), (5, 7))), (128, 16, 4, ((1000, 1),) * 9), (128, 6, 2, ((30, 300), (0, 64), (255, 1), (256, 1))),
    (192, 3, 1, ((100, 129),)), (256, 8, 1, ((1, 70), (0, 3))), (256, 2, 2, ((127, 258),)), (64, 0, 2, ((17, 200),)),
    (128, 8, 8, ((3, 1100), (0, 70), (40, 1))), (64, 64, 8, ((191, 66),))])
def test_insert(dim, H, K, runs):
    """Queries and keys as a bf16 cache's insert leaves them; the cache as the oracle quantises those rows; nothing else changed."""
    D = _dense()
    T, pos, slots, q, k, v, pool, g = _insert_case(dim, H, K, runs, dim + H + len(runs))
    if T > 5:
        slots[3] = -1                                     # a padded row inside a group
    gam = (1 + 0.1 * torch.randn(dim, generator=g)).to(DEV)
    rope = D.Rope(dim // 2 // 16 * 16, layout=1)
    pos_t, slot_t = torch.tensor(pos, **I32), torch.tensor(slots, dtype=torch.int64, device=DEV)
    want = pool.cpu().numpy().copy()
    q_out = torch.full((T, H, dim), 7.0, dtype=torch.bfloat16, device=DEV)
    k_out = torch.full((T, K, dim), 7.0, dtype=torch.bfloat16, device=DEV)
    op = D.DenseInsert(D.DenseCache(pool, None, K, dim, D.KV_FP8_GROUP), H, rope, gam, gam)
    op.run(q if H else None, k, v, q_out if H else None, pos_t, slot_t, k_out=k_out)
    torch.cuda.synchronize()
    assert int(op.status.item()) == 0
    # the rows: those of a bf16 cache
    bf = torch.zeros((pool.shape[0], D.block_bytes(K, dim, D.KV_BF16)), dtype=torch.uint8, device=DEV)
    q2 = torch.full_like(q_out, 7.0)
    D.DenseInsert(D.DenseCache(bf, None, K, dim), H, rope, gam, gam).run(q if H else None, k, v, q2 if H else None, pos_t, slot_t)
    assert torch.equal(q_out, q2)
    rows = bf.view(torch.bfloat16).view(pool.shape[0], 2, K, 256, dim)
    for t, s in enumerate(slots):
        assert torch.equal(k_out[t], rows[s // 256, 0, :, s % 256] if s >= 0 else torch.full_like(k_out[t], 7.0))
    OG.insert(want, K, dim, slots, (_f64(k_out), _f64(v)))
    _same_cache(pool, want, K, dim)


def test_insert_step_by_step_grows_scales():
    """Single tokens of growing and shrinking size fill a group; each step as the oracle does it, and a long call begins the group anew."""
    D = _dense()
    K, dim = 2, 64
    g = torch.Generator().manual_seed(1)
    pool = torch.full((3, OG.block_bytes(K, dim)), 0x7f, dtype=torch.uint8, device=DEV)      # NaN codes, scales of no step
    want = pool.cpu().numpy().copy()
    op = D.DenseInsert(D.DenseCache(pool, None, K, dim, D.KV_FP8_GROUP), 0, None)
    for p in list(range(70)) + [5, 0, 64]:
        x = (torch.randn((1, 2 * K, dim), generator=g) * 2.0 ** (p % 23 - 8)).to(torch.bfloat16).to(DEV)
        k_out = torch.empty((1, K, dim), dtype=torch.bfloat16, device=DEV)
        op.run(None, x[:, :K], x[:, K:], None, torch.tensor([p], **I32), torch.tensor([256 + p], device=DEV), k_out=k_out)
        assert torch.equal(k_out, x[:, :K])
        OG.insert(want, K, dim, [256 + p], (_f64(k_out), _f64(x[:, K:])))
        _same_cache(pool, want, K, dim)
    assert int(op.status.item()) == 0


def test_insert_of_special_values():
    """Zeros, one tiny row, the boundary 448 s, infinities and NaN: they stay in their rows and out of the scale."""
    D = _dense()
    K, dim = 1, 128
    x = torch.zeros((6, 2 * K, dim), dtype=torch.bfloat16)
    x[0, :, 3] = 2.0 ** -120
    x[1, :, 0], x[1, :, 1] = math.inf, -math.inf
    x[2, :, 9] = math.nan
    x[3, 0, 5], x[3, 1, 5] = 448.0, 450.0            # scales 1 and 2
    x[4] = -1.0
    for rows in ([0], [5], [1], [2], [3], [0, 3, 4], [1, 2], [0, 1, 2, 3, 4, 5]):
        y = x[rows].to(DEV)
        pool = torch.zeros((1, OG.block_bytes(K, dim)), dtype=torch.uint8, device=DEV)
        want = pool.cpu().numpy().copy()
        slots = list(range(60, 60 + len(rows)))      # over a group's end
        op = D.DenseInsert(D.DenseCache(pool, None, K, dim, D.KV_FP8_GROUP), 0, None)
        op.run(None, y[:, :K], y[:, K:], None, torch.arange(len(rows), **I32), torch.tensor(slots, device=DEV), k_out=y[:, :K])      # in place
        OG.insert(want, K, dim, slots, (_f64(x[rows][:, :K]), _f64(x[rows][:, K:])))
        _same_cache(pool, want, K, dim)


def test_insert_reports_and_skips():
    D = _dense()
    for slots, pos, bit in (([0, -2, 3], [0, 1, 2], 1), ([0, 512, 3], [0, 1, 2], 1), ([0, 1, 3], [0, -1, 2], 2), ([-1, -1, -1], [0, 1, 2], 0)):
        pool = torch.zeros((2, OG.block_bytes(1, 64)), dtype=torch.uint8, device=DEV)
        x = torch.ones((3, 1, 64), dtype=torch.bfloat16, device=DEV)
        k_out = torch.full_like(x, 7.0)
        op = D.DenseInsert(D.DenseCache(pool, None, 1, 64, D.KV_FP8_GROUP), 0, None)
        op.run(None, x, x, None, torch.tensor(pos, **I32), torch.tensor(slots, device=DEV), k_out=k_out)
        torch.cuda.synchronize()
        assert int(op.status.item()) == bit
        keep = [s if 0 <= s < 512 and p >= 0 else -1 for s, p in zip(slots, pos)]
        assert (k_out[:, 0, 0] == 1).tolist() == [s >= 0 for s in keep]
        want = np.zeros((2, OG.block_bytes(1, 64)), np.uint8)
        OG.insert(want, 1, 64, keep, (np.ones((3, 1, 64)),) * 2)
        _same_cache(pool, want, 1, 64)


@pytest.mark.parametrize("dim,H,K,T", [(64, 4, 1, 3001), (128, 2, 1, 2500), (256, 1, 1, 2600), (192, 4, 2, 1500), (128, 32, 8, 700)])
@pytest.mark.parametrize("fp8", [False, True])
def test_insert_rows_of_other_formats(dim, H, K, T, fp8):
    """With rows asked for, bf16 and fp8 caches and the queries hold what they hold without; the rows are the bf16 cache's."""
    D = _dense()
    fmt = D.KV_FP8_TOKEN if fp8 else D.KV_BF16
    g = torch.Generator(device=DEV).manual_seed(dim + H)
    x = torch.randn((T, (H + 2 * K) * dim), generator=g, device=DEV).to(torch.bfloat16)
    q, k, v = (x[:, a * dim:b * dim].unflatten(1, (b - a, dim)) for a, b in ((0, H), (H, H + K), (H + K, H + 2 * K)))
    gam = torch.rand(dim, generator=g, device=DEV) + 0.5
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device=DEV, dtype=torch.int32)
    slots = torch.randperm(8192, generator=g, device=DEV)[:T].contiguous()
    slots[::97] = -1
    got = []
    for f, rows in ((fmt, False), (fmt, True), (D.KV_BF16, False)):
        pool = torch.zeros((32, D.block_bytes(K, dim, f)), dtype=torch.uint8, device=DEV)
        qo, ko = torch.full((T, H, dim), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((T, K, dim + 8), 7.0, dtype=torch.bfloat16, device=DEV)
        ko = ko.view(T, -1)[:, :K * dim].unflatten(1, (K, dim))
        op = D.DenseInsert(D.DenseCache(pool, None, K, dim, f), H, D.Rope(64, layout=1), gam, gam)
        op.run(q, k, v, qo, pos, slots, k_out=ko if rows else None)
        got.append((pool, qo, ko))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    live = slots >= 0
    rows = got[2][0].view(torch.bfloat16).view(32, 2, K, 256, dim)[slots[live] // 256, 0, :, slots[live] % 256]
    assert torch.equal(got[1][2][live], rows) and (got[1][2][~live] == 7.0).all()


# --------------------------------------------------------------------------
# The read back
# --------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["bf16", "token", "group"])
@pytest.mark.parametrize("dim,K,runs", [
    (64, 1, ((0, 1),)), (128, 4, ((0, 1000),)), (128, 2, ((5, 300), (0, 0), (255, 2), (64, 64))), (192, 3, ((250, 20), (0, 513))),
    (256, 2, ((700, 65), (0, 1), (3, 0))), (64, 8, ((0, 40),) * 300)])
def test_read(fmt, dim, K, runs):
    D = _dense()
    f = {"bf16": D.KV_BF16, "token": D.KV_FP8_TOKEN, "group": D.KV_FP8_GROUP}[fmt]
    g = torch.Generator().manual_seed(dim + K + len(runs))
    cols = max(-(-(c + n) // 256) for c, n in runs) + 1
    blocks = len(runs) * cols + 1
    table = torch.randperm(blocks, generator=g)[:len(runs) * cols].view(len(runs), cols).to(torch.int32)
    body = 2 * K * 256 * dim
    pool = torch.zeros((blocks, D.block_bytes(K, dim, f) + 16), dtype=torch.uint8)
    x = torch.randn((blocks, body), generator=g)
    if fmt == "bf16":
        pool[:, :2 * body] = x.to(torch.bfloat16).view(torch.uint8)
    else:
        pool[:, :body] = (x * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        n = 2 * K * 256 if fmt == "token" else 8 * K
        scales = (torch.rand((blocks, n), generator=g) + 0.5) / 100 if fmt == "token" else torch.exp2(torch.randint(-12, 5, (blocks, n), generator=g).float())
        pool[:, body:body + 4 * n] = scales.view(torch.uint8)
    starts = [2]                                          # rows before the first sequence and behind the last one
    for _, n in runs:
        starts.append(starts[-1] + n)
    N = starts[-1] + 3
    rows = torch.full((N, 2 * K * dim + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    k, v = rows[:, :K * dim].unflatten(1, (K, dim)), rows[:, K * dim:2 * K * dim].unflatten(1, (K, dim))
    op = D.DenseRead(D.DenseCache(pool.to(DEV), table.to(DEV), K, dim, f))
    op.run(torch.tensor(starts, **I32), k, v, first=torch.tensor([c for c, _ in runs], **I32))
    torch.cuda.synchronize()
    assert int(op.status.item()) == 0
    want = np.full((2, N, K, dim), 7.0)
    host = pool.numpy()
    at = [(starts[b] + i, b, c + i) for b, (c, n) in enumerate(runs) for i in range(n) if n < 100 or i % 37 == 0 or i > n - 3]
    for r, b, p in at:
        for w in (0, 1):
            for h in range(K):
                blk = int(table[b, p // 256])
                x = OG.read_row(host, K, dim, blk, w, h, p % 256) if fmt == "group" else OD.read_row(host, K, dim, fmt == "token", blk, w, h, p % 256)
                want[w, r, h] = F.bf16_decode(F.bf16_encode(x.astype(np.float32) if fmt == "token" else x))
    look = [r for r, _, _ in at] + [0, 1, N - 3, N - 2, N - 1]
    for w, t in ((0, k), (1, v)):
        got = _f64(t)[look]
        if fmt == "token":       # the product is rounded to fp32 and then to bf16
            assert (np.abs(got - want[w][look]) <= 2.0 ** -7 * np.abs(want[w][look])).all()
        else:
            assert np.array_equal(got, want[w][look])
    assert (rows[:, 2 * K * dim:] == 7.0).all()


def test_read_holes_and_bad_positions():
    D = _dense()
    K, dim = 2, 64
    pool = torch.zeros((4, OG.block_bytes(K, dim)), dtype=torch.uint8, device=DEV)
    table = torch.tensor([[0, -1, 1], [9, 2, 3]], **I32)
    cache = D.DenseCache(pool, table, K, dim, D.KV_FP8_GROUP)
    for first, starts, bit, wrote in (([255, 300], [0, 2, 4], 1, [0, 2, 3]), ([0, 10], [0, 2, 4], 1, [0, 1]), ([-1, 256], [0, 2, 4], 2, [1, 2, 3]),
                                      ([767, 256], [0, 2, 4], 2, [0, 2, 3]), (None, [0, 3, 3], 0, [0, 1, 2]), (None, [0, 0, 0], 0, []),
                                      ([0, 256], [1, 2, 90], 0, [1, 2, 3])):
        k, v = (torch.full((4, K, dim), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        op = D.DenseRead(cache)
        op.run(torch.tensor(starts, **I32), k, v, first=None if first is None else torch.tensor(first, **I32))
        torch.cuda.synchronize()
        assert int(op.status.item()) == bit
        for x in (k, v):
            assert [r for r in range(4) if (x[r] == 0).all()] == wrote
            assert [r for r in range(4) if (x[r] == 7.0).all()] == [r for r in range(4) if r not in wrote]


# --------------------------------------------------------------------------
# Attention over the cache
# --------------------------------------------------------------------------

class GroupLayer(Layer):
    """A cache with a scale per group, every held row random, and the oracle's view of it."""

    def __init__(self, lengths, H, K, dim, seed, extra=16, cols=None, q_std=1.0, hidden=None, holes=(), exponents=(-9, -5)):
        D = _dense()
        g = torch.Generator().manual_seed(seed)
        self.H, self.K, self.dim, self.fp8, self.lengths = H, K, dim, True, lengths
        held = [-(-n // 256) for n in lengths]
        cols = max(held + [1]) if cols is None else cols
        blocks = sum(held) + 3
        ids = torch.randperm(blocks, generator=g)
        self.table = np.full((len(lengths), cols), -1, np.int32)
        at = 0
        for b, n in enumerate(held):
            self.table[b, :n] = ids[at:at + n]
            at += n
        body = 2 * K * 256 * dim
        pool = torch.zeros((blocks, OG.block_bytes(K, dim) + extra), dtype=torch.uint8)
        pool[:, :body] = (torch.randn((blocks, body), generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        pool[:, body:body + 32 * K] = torch.exp2(torch.randint(*exponents, (blocks, 8 * K), generator=g).float()).view(torch.uint8)
        self.host = pool.numpy().copy()
        if hidden is not None:          # rows that no query sees hold NaN, and groups of such rows NaN scales
            for b, n in enumerate(lengths):
                for p in range(held[b] * 256):
                    if hidden(b, p):
                        blk = pool[int(self.table[b, p // 256])]
                        whole = all(hidden(b, j) for j in range(p // 64 * 64, p // 64 * 64 + 64))
                        for plane in range(2 * K):
                            row = plane * 256 + p % 256
                            blk[row * dim:(row + 1) * dim] = 0x7f
                            if whole:
                                o = body + 4 * (row // 64)
                                blk[o:o + 4] = torch.tensor([math.nan]).view(torch.uint8)
        for b, n in holes:
            self.table[b, n] = -1
        self.pool = pool.to(DEV)
        self.bt = torch.from_numpy(self.table).to(DEV)
        self.cache = D.DenseCache(self.pool, self.bt, K, dim, D.KV_FP8_GROUP)
        self.gen, self.q_std = g, q_std
        self._rows = {}

    def rows(self, b, which, h, n):
        key = (b, which, h)
        if key not in self._rows or len(self._rows[key]) < n:
            out = np.full((n, self.dim), np.nan)
            for p in range(n):
                blk = self.table[b, p // 256]
                if blk >= 0:
                    out[p] = OG.read_row(self.host, self.K, self.dim, blk, which, h, p % 256)
            self._rows[key] = out
        return self._rows[key][:n]

    def check(self, q, out, lse, positions, starts, window, sinks, scale, tokens=None):
        for b in range(len(starts) - 1):
            for t in range(starts[b], starts[b + 1]):
                if tokens is None or t in tokens:
                    m = positions[t]
                    seen = [j for j in OD.visible(m, window, sinks) if self.table[b, j // 256] >= 0]
                    _check_token(q[t], out[t], lse[t], lambda w, h: self.rows(b, w, h, m + 1)[seen], self.K, scale, 2.0 ** -11, (b, t), 2.0 ** -17)


def _check_token(q, out, lse, rows, K, scale, p_step, where, q_step=0.0):
    """One token's heads against the oracle; p_step: half a step of a probability."""
    q, got, got_l = _f64(q), _f64(out), _f64(lse)
    G, dim = q.shape[0] // K, q.shape[1]
    for h in range(K):
        k, v = rows(0, h), rows(1, h)
        o, l, av, amp = OD.attention(q[h * G:(h + 1) * G], k, v, scale)
        dz = (dim + 8) * 2.0 ** -24 * amp[:, None]
        if len(k):
            dz = dz + q_step * scale * np.abs(q[h * G:(h + 1) * G]).max(1, keepdims=True) * np.abs(k).sum(1).max()
        n = (len(k) + 32) * 2.0 ** -24
        small = len(k) * 2.0 ** -34 * np.abs(v).max() if len(k) else 0.0      # (weights that f16 holds as subnormals)
        tol = (p_step + 2 * dz + 2 * n) * av + 2.0 ** -8 * np.abs(o) + small + 1e-30
        err = np.abs(got[h * G:(h + 1) * G] - o)
        assert (err <= tol).all(), (where, h, float((err / tol).max()))
        if len(k) == 0:
            assert (got_l[h * G:(h + 1) * G] == -np.inf).all()
        else:
            assert (np.abs(got_l[h * G:(h + 1) * G] - l) <= dz[:, 0] + n + 2.0 ** -22 * np.abs(l) + 2.0 ** -20).all(), (where, h)


@pytest.mark.parametrize("lengths,H,K,dim,window,sinks", [
    ((1,), 1, 1, 64, 0, 0), ((1, 2, 64, 65, 128), 4, 4, 64, 0, 0), ((256, 257, 1000, 3), 8, 2, 128, 0, 0), ((700, 31), 16, 2, 128, 0, 0),
    ((1025,), 16, 4, 128, 0, 0), ((300, 5), 3, 1, 192, 0, 0), ((300, 77), 24, 2, 192, 0, 0), ((513, 90), 16, 1, 256, 0, 0),
    ((600, 40), 7, 1, 128, 0, 0), ((400, 1), 64, 1, 128, 0, 0), ((900, 130, 60, 1), 8, 2, 64, 100, 4), ((900, 130, 60, 1), 16, 1, 128, 64, 70),
    ((2000, 515), 8, 1, 128, 1, 0), ((2000, 515), 8, 1, 256, 300, 1), ((777,) * 40, 8, 4, 64, 0, 0), ((2000, 515), 4, 2, 64, 1000, 1500)])
def test_decode(lengths, H, K, dim, window, sinks):
    """One new token per sequence; every row that the query does not see holds NaN."""
    def hidden(b, p):
        m = lengths[b] - 1
        return p > m or (window and p <= m - window and p >= sinks)
    layer = GroupLayer(lengths, H, K, dim, seed=len(lengths) + H, hidden=hidden)
    _attend(layer, [n - 1 for n in lengths], list(range(len(lengths) + 1)), window, sinks, pad=3)


@pytest.mark.parametrize("new", [1, 90])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_peaked_flat_and_uneven(dim, new):
    """Large logits, equal ones, and scales from 2^-60 to 2^20 side by side."""
    pos, starts = _runs((900 - new, 400 - new), (new, new))
    for kw in (dict(q_std=20.0), dict(q_std=0.0), dict(exponents=(-60, 20), q_std=2.0 ** -16)):
        layer = GroupLayer((900, 400), 8, 2, dim, seed=3, **kw)
        _attend(layer, pos, starts, tokens={0, new // 2, new - 1, new, 2 * new - 1})


def test_decode_missing_blocks():
    layer = GroupLayer((700, 200, 600), 8, 2, 64, seed=7, holes=[(0, 1), (1, 0), (2, 2)])
    op, q, out, lse = _attend(layer, [699, 199, 599], [0, 1, 2, 3], check=False)
    assert int(op.status.item()) == 1
    layer.check(q, out, lse, [699, 199, 599], [0, 1, 2, 3], 0, 0, op.args.softmax_scale)


CHUNKS = [
    # cached, new, H, K, dim, window, sinks
    ((0,), (5,), 4, 4, 64, 0, 0), ((0, 300), (130, 7), 8, 2, 128, 0, 0), ((10, 0, 250), (3, 1, 20), 8, 1, 128, 0, 0),
    ((500,), (200,), 6, 2, 128, 0, 0), ((0, 700), (300, 129), 4, 1, 64, 100, 4), ((900,), (257,), 16, 2, 128, 64, 130),
    ((30,), (100,), 4, 2, 192, 0, 0), ((30,), (60,), 4, 2, 256, 50, 3), ((0, 90), (65, 64), 2, 2, 64, 30, 2),
    ((400,), (150,), 32, 2, 128, 0, 0), ((0,), (513,), 5, 1, 128, 0, 0), ((255, 256, 511), (2, 256, 130), 8, 8, 64, 0, 0),
    ((0,), (300,), 128, 1, 64, 0, 0), ((0, 0, 0), (1, 260, 2), 64, 4, 128, 1, 0), ((1500, 20), (140, 200), 4, 1, 256, 1300, 0),
    ((2000,), (90,), 4, 2, 64, 1025, 300), ((3000,), (40,), 24, 2, 192, 0, 0),
]


@pytest.mark.parametrize("cached,new,H,K,dim,window,sinks", CHUNKS)
def test_chunks(cached, new, H, K, dim, window, sinks):
    """Chunked prefill and ragged mixes; rows no query of the call sees hold NaN."""
    def hidden(b, p):
        return p >= cached[b] + new[b] or (window and p <= cached[b] - window and p >= sinks)
    layer = GroupLayer([c + n for c, n in zip(cached, new)], H, K, dim, seed=sum(new), hidden=hidden)
    pos, starts = _runs(cached, new)
    some = {t for b in range(len(new)) for t in range(starts[b], starts[b + 1]) if t - starts[b] < 3 or t % 37 == 0 or t > starts[b + 1] - 3}
    _attend(layer, pos, starts, window, sinks, pad=2, tokens=some)


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_chunk_missing_blocks(dim):
    layer = GroupLayer((700, 400), 8, 2, dim, seed=9, holes=[(0, 1), (1, 0)])
    pos, starts = _runs((600, 100), (100, 300))
    op, q, out, lse = _attend(layer, pos, starts, check=False)
    assert int(op.status.item()) == 1
    layer.check(q, out, lse, pos, starts, 0, 0, op.args.softmax_scale, tokens={0, 50, 99, 100, 150, 260, 399})


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_mixed_batches(dim):
    """Decoding sequences beside chunks, more sequences than an even split takes among them."""
    for runs in ([(900, 1), (200, 150), (40, 3), (0, 300), (7, 0)], [(60, 1)] * 550 + [(200, 120)]):
        layer = GroupLayer([c + n for c, n in runs], 8, 2, dim, seed=len(runs))
        pos, starts = _runs(*zip(*runs))
        T = starts[-1]
        _attend(layer, pos, starts, tokens={0, 1, 75, 151, 152, 153, T // 2, T - 150, T - 2, T - 1})


def test_pages_past_four_gigabytes():
    """A page whose offset passes 32 bits."""
    D = _dense()
    K, dim = 8, 256
    bytes_ = OG.block_bytes(K, dim)
    n = (1 << 32) // bytes_ + 3
    pool = torch.zeros((n, bytes_), dtype=torch.uint8, device=DEV)
    host = torch.zeros((1, bytes_), dtype=torch.uint8)
    g = torch.Generator().manual_seed(4)
    body = 2 * K * 256 * dim
    host[:, :body] = (torch.randn((1, body), generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    host[:, body:] = torch.full((1, 8 * K), 2.0 ** -7).view(torch.uint8)
    pool[n - 1] = host[0].to(DEV)
    table = torch.tensor([[n - 1]], **I32)
    cache = D.DenseCache(pool, table, K, dim, D.KV_FP8_GROUP)
    small = D.DenseCache(host.to(DEV), torch.tensor([[0]], **I32), K, dim, D.KV_FP8_GROUP)
    q = torch.randn((200, 8, dim), generator=g).to(torch.bfloat16).to(DEV)
    for new in (1, 200):
        outs = []
        for c in (cache, small):
            out = torch.empty((new, 8, dim), dtype=torch.bfloat16, device=DEV)
            D.DenseAttention(c, 8, new, new).run(q[:new], out, torch.arange(200 - new, 200, **I32), torch.tensor([0, new], **I32))
            outs.append(out)
        assert torch.equal(*outs)
    rows = [[torch.empty((200, K, dim), dtype=torch.bfloat16, device=DEV) for _ in range(2)] for _ in range(2)]
    for c, (k, v) in zip((cache, small), rows):
        D.DenseRead(c).run(torch.tensor([0, 200], **I32), k, v)
    assert all(torch.equal(a, b) for a, b in zip(*rows)) and rows[0][0].abs().sum() > 0
    x = torch.randn((3, 2 * K, dim), generator=g).to(torch.bfloat16).to(DEV)
    slots = torch.tensor([254, 255, 0], device=DEV)
    for c, at in ((cache, (n - 1) * 256), (small, 0)):
        k_out = torch.empty((3, K, dim), dtype=torch.bfloat16, device=DEV)
        D.DenseInsert(c, 0, None).run(None, x[:, :K], x[:, K:], None, torch.arange(3, **I32), at + slots, k_out=k_out)
    assert torch.equal(pool[n - 1], small.pool[0])


# --------------------------------------------------------------------------
# Whole prompts
# --------------------------------------------------------------------------

PROMPTS = [
    # (prefix keys, queries) of each sequence, H, K, dim, causal, window, sinks
    (((0, 1),), 1, 1, 64, True, 0, 0), (((0, 1), (0, 2), (0, 63), (0, 64), (0, 65)), 4, 4, 64, True, 0, 0),
    (((0, 300), (0, 1), (0, 129)), 8, 2, 128, True, 0, 0), (((100, 40), (0, 0), (7, 500)), 6, 2, 128, True, 0, 0),
    (((0, 257), (64, 64)), 16, 1, 128, True, 0, 0), (((0, 200), (30, 77)), 4, 2, 192, True, 0, 0), (((0, 200), (300, 5)), 3, 1, 256, True, 0, 0),
    (((0, 100), (3, 300)), 8, 2, 64, False, 0, 0), (((0, 130), (200, 1), (0, 64)), 4, 4, 128, False, 0, 0), (((5, 70),), 2, 2, 256, False, 0, 0),
    (((0, 400), (0, 90)), 8, 2, 128, True, 100, 4), (((700, 100),), 4, 1, 64, True, 64, 130), (((0, 300), (500, 200)), 4, 2, 256, True, 50, 3),
    (((0, 500),), 64, 4, 64, True, 1, 0), (((0, 20),) * 700, 4, 2, 128, True, 0, 0), (((0, 1500), (2000, 30)), 5, 1, 128, True, 0, 0),
    (((-5, 20), (-300, 300), (0, 70)), 4, 2, 128, True, 0, 0), (((-5, 20), (-3, 3), (-200, 260)), 4, 2, 64, False, 0, 0),
    (((-100, 400), (10, 10)), 8, 1, 192, True, 30, 2),
]


def _prompt(runs, H, K, dim, seed, pad=2, std=1.0):
    """Packed queries and keys with odd strides; prefix < 0: fewer keys than queries."""
    g = torch.Generator().manual_seed(seed)
    starts, kv = [0], [1]                                # a key row in front that no sequence has
    for c, n in runs:
        starts.append(starts[-1] + n)
        kv.append(kv[-1] + c + n)
    T, N = starts[-1] + pad, kv[-1] + 2
    x = (torch.randn((T, H * dim + 8), generator=g) * std).to(torch.bfloat16)
    y = torch.randn((N, 2 * K * dim + 24), generator=g).to(torch.bfloat16)
    y[0] = y[kv[-1]:] = math.nan                         # rows of no sequence
    x, y = x.to(DEV), y.to(DEV)
    return (starts, kv, x[:, :H * dim].unflatten(1, (H, dim)), y[:, :K * dim].unflatten(1, (K, dim)),
            y[:, K * dim + 8:2 * K * dim + 8].unflatten(1, (K, dim)))


def _run_prompt(starts, kv, q, k, v, **kw):
    D = _dense()
    T, H, dim = q.shape
    op = D.PromptAttention(H, k.shape[1], dim, len(starts) - 1, T, max(max(b - a for a, b in zip(starts, starts[1:])), 1), **kw)
    out, lse = torch.full((T, H, dim), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((T, H), 7.0, device=DEV)
    op.run(q, k, v, out, torch.tensor(starts, **I32), None if kv is None else torch.tensor(kv, **I32), lse=lse)
    torch.cuda.synchronize()
    return op, out, lse


def _check_prompt(starts, kv, q, k, v, out, lse, causal, window, sinks, scale, tokens=None):
    kh, vh = _f64(k), _f64(v)
    for b in range(len(starts) - 1):
        n, keys = starts[b + 1] - starts[b], kv[b + 1] - kv[b]
        for i in range(n):
            if tokens is not None and starts[b] + i not in tokens:
                continue
            at = [kv[b] + j for j in OG.prompt_visible(n, keys, i, causal, window, sinks)]
            t = starts[b] + i
            _check_token(q[t], out[t], lse[t], lambda w, h: (vh if w else kh)[at, h], k.shape[1], scale, 2.0 ** -8, (b, i))


def _some(starts):
    return {t for a, b in zip(starts, starts[1:]) for t in range(a, b) if t - a < 2 or t % 41 == 0 or t >= b - 2}


@pytest.mark.parametrize("runs,H,K,dim,causal,window,sinks", PROMPTS)
def test_prompts(runs, H, K, dim, causal, window, sinks):
    """Rows of other sequences and of none hold anything; rows behind the last query are left."""
    starts, kv, q, k, v = _prompt(runs, H, K, dim, seed=len(runs) + H)
    op, out, lse = _run_prompt(starts, kv, q, k, v, causal=causal, window=window, sinks=sinks)
    assert int(op.status.item()) == 0
    tokens = _some(starts)
    if len(tokens) > 200:
        tokens = set(sorted(tokens)[::len(tokens) // 150])
    _check_prompt(starts, kv, q, k, v, out, lse, causal, window, sinks, op.args.softmax_scale, tokens)
    assert (out[starts[-1]:] == 7.0).all() and (lse[starts[-1]:] == 7.0).all()


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_prompts_never_see_other_sequences(dim):
    """NaN and infinities in one sequence's keys and values reach that sequence alone."""
    starts, kv, q, k, v = _prompt(((0, 70), (3, 100), (0, 190)), 4, 2, dim, seed=5)
    _, want, want_l = _run_prompt(starts, kv, q, k, v)
    k[kv[1]:kv[2]] = math.nan
    v[kv[1]:kv[2]] = math.inf
    _, out, lse = _run_prompt(starts, kv, q, k, v)
    for a, b in ((0, 1), (2, 3)):
        assert torch.equal(out[starts[a]:starts[b]], want[starts[a]:starts[b]]) and torch.equal(lse[starts[a]:starts[b]], want_l[starts[a]:starts[b]])
    assert not out[starts[1]:starts[2]].isfinite().any()


@pytest.mark.parametrize("dim,std", [(128, 20.0), (64, 0.0), (256, 20.0)])
def test_prompts_peaked_and_flat(dim, std):
    starts, kv, q, k, v = _prompt(((0, 700), (9, 200)), 8, 2, dim, seed=6, std=std)
    op, out, lse = _run_prompt(starts, kv, q, k, v, scale=0.7)
    _check_prompt(starts, kv, q, k, v, out, lse, True, 0, 0, op.args.softmax_scale, {0, 300, 699, 700, 750, 899})


def test_prompts_without_kv_starts_and_keys():
    """kv_starts None: the queries' own rows; no keys at all: zeros and -inf."""
    starts, _, q, k, v = _prompt(((0, 70), (0, 33)), 4, 2, 64, seed=8, pad=0)
    k, v = k[1:104], v[1:104]
    op, out, lse = _run_prompt(starts, None, q, k, v)
    _check_prompt(starts, starts, q, k, v, out, lse, True, 0, 0, op.args.softmax_scale)
    for causal in (True, False):
        op, out, lse = _run_prompt(starts, [0, 0, 0], q, k[:0], v[:0], causal=causal)
        assert int(op.status.item()) == 0 and (out == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("starts,kv,bad,left", [
    ([0, 1, 0, 3], [0, 1, 2, 3], {1, 2}, [1, 2]), ([0, 1, 3, 9], [0, 1, 3, 3], {2}, []), ([0, 1, 2, 3], [0, 2, 1, 3], {1}, [1]),
    ([0, 1, 2, 3], [0, 1, 2, 99], {2}, [2]), ([0, 1, 2, 3], [-1, 1, 2, 3], {0}, [0]), ([0, 0, 3, 3], [0, 1, 2, 3], {1}, [0, 1, 2])])
def test_inconsistent_prompts_are_reported_and_left(starts, kv, bad, left):
    _, _, q, k, v = _prompt(((0, 3), (0, 3)), 4, 2, 64, seed=9, pad=0)
    q, k, v = q[:3], k[1:7], v[1:7]
    op = _dense().PromptAttention(4, 2, 64, 3, 3, 2)
    out, lse = torch.full((3, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((3, 4), 7.0, device=DEV)
    op.run(q, k, v, out, torch.tensor(starts, **I32), torch.tensor(kv, **I32), lse=lse)
    torch.cuda.synchronize()
    assert int(op.status.item()) == 2
    assert (out[left] == 7.0).all() and (lse[left] == 7.0).all()
    for b in {0, 1, 2} - bad:
        s = [starts[b]] * (b + 1) + [starts[b + 1]] * (3 - b)
        c = [kv[b]] * (b + 1) + [kv[b + 1]] * (3 - b)
        _check_prompt(s, c, q, k, v, out, lse, True, 0, 0, op.args.softmax_scale)


def test_prompts_share_keys():
    """Two sequences over the same keys."""
    starts, kv, q, k, v = _prompt(((0, 90),), 4, 2, 128, seed=10, pad=90)
    two = torch.cat([q[:90], q[:90]])
    D = _dense()
    op = D.PromptAttention(4, 2, 128, 3, 180, 90)
    out, lse = torch.empty((180, 4, 128), dtype=torch.bfloat16, device=DEV), torch.empty((180, 4), device=DEV)
    # kv_starts of neighbours are one array: between the two lies a sequence without queries, whose entries mean nothing
    op.run(two, k, v, out, torch.tensor([0, 90, 90, 180], **I32), torch.tensor([kv[0], kv[1], kv[0], kv[1]], **I32), lse=lse)
    assert int(op.status.item()) == 0
    for s in (slice(0, 90), slice(90, 180)):
        _check_prompt([0, 90], kv, two[s], k, v, out[s], lse[s], True, 0, 0, op.args.softmax_scale)


# --------------------------------------------------------------------------
# Together
# --------------------------------------------------------------------------

def test_same_call_same_bytes_on_any_stream():
    """Repeated, on two streams at once, and captured into a graph whose inputs change."""
    D = _dense()
    starts, kv, q, k, v = _prompt(((0, 700), (100, 300), (0, 64)), 8, 2, 128, seed=11, pad=0)
    st, kt = torch.tensor(starts, **I32), torch.tensor(kv, **I32)
    ops = [D.PromptAttention(8, 2, 128, 3, q.shape[0], 700) for _ in range(2)]
    outs = [torch.empty((q.shape[0], 8, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    ops[0].run(q, k, v, outs[0], st, kt)
    torch.cuda.synchronize()
    want = outs[0].clone()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for i in range(2):
            ops[i].run(q, k, v, outs[i], st, kt, stream=streams[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops[0].run(q, k, v, outs[0], st, kt)
    q.mul_(2)
    ops[1].run(q, k, v, outs[1], st, kt)
    outs[0].zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and not torch.equal(outs[0], want)


@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 4)])
@pytest.mark.parametrize("graph", [False, True])
def test_steps_of_a_small_server(graph, window, sinks):
    """Plan -> insert -> attention over the cache and, for the sequences that begin, over the packed rows: a cached
    start read back in front of the fresh keys gives what those rows give; every step against the oracle."""
    D = _dense()
    H, K, dim, B, T, pages = 8, 2, 128, 4, 330, 24
    gen = torch.Generator().manual_seed(5)
    table = torch.full((1, B, 6), -1, **I32)
    ring = torch.randperm(pages, generator=gen).to(torch.int32).to(DEV)
    free, cached, fresh = torch.tensor([0, pages], **I32), torch.zeros(B, **I32), torch.zeros(B, **I32)
    plan = D.StepPlan(table, ring, T)
    pool = torch.full((pages, OG.block_bytes(K, dim)), 0xff, dtype=torch.uint8, device=DEV)         # NaN everywhere
    cache = D.DenseCache(pool, table[0], K, dim, D.KV_FP8_GROUP)
    gam = torch.rand(dim, generator=gen).to(DEV) + 0.5
    ins = D.DenseInsert(cache, H, D.Rope(dim, layout=1), gam, gam)
    att, read = D.DenseAttention(cache, H, T, 300, window, sinks), D.DenseRead(cache)
    pro = D.PromptAttention(H, K, dim, B, T, 300, window=window, sinks=sinks)
    x = torch.zeros((T, (H + 2 * K) * dim), dtype=torch.bfloat16, device=DEV)
    q, k, v = (x[:, a * dim:b * dim].unflatten(1, (b - a, dim)) for a, b in ((0, H), (H, H + K), (H + K, H + 2 * K)))
    qr, out, pout = (torch.zeros((T, H, dim), dtype=torch.bfloat16, device=DEV) for _ in range(3))
    kr = torch.zeros((T, K, dim), dtype=torch.bfloat16, device=DEV)
    lse, plse = torch.zeros((T, H), device=DEV), torch.zeros((T, H), device=DEV)
    rows, row_starts = [torch.zeros((900, K, dim), dtype=torch.bfloat16, device=DEV) for _ in range(2)], torch.zeros(B + 1, **I32)

    def step():
        plan.run(cached, fresh, free)
        ins.run(q, k, v, qr, plan.positions, plan.slots[0], k_out=kr)
        att.run(qr, out, plan.positions, plan.token_starts, lse)
        read.run(row_starts, *rows)
        pro.run(qr, *rows, pout, plan.token_starts, row_starts, lse=plse)

    g = None
    if graph:
        step()                              # nothing to do: every sequence rests
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
    lengths, want = [0] * B, pool.cpu().numpy().copy()
    host_tables, host_ring, state = table.cpu().numpy().copy(), ring.cpu().numpy().copy(), (0, pages)
    for news in ([250, 0, 3, 1], [1, 7, 300, 1], [1, 1, 0, 1], [-1, 1, 1, 1], [20, -1, 1, 1], [1, 255, 1, -1]):
        x.copy_((torch.randn(x.shape, generator=gen) * 1.5).to(torch.bfloat16))
        cached.copy_(torch.tensor(lengths, **I32))
        fresh.copy_(torch.tensor(news, **I32))
        ends = [c + n if n > 0 else 0 for c, n in zip(lengths, news)]
        row_starts.copy_(torch.tensor(np.cumsum([0] + ends), **I32))
        out.fill_(7.0), pout.fill_(7.0)
        g.replay() if graph else step()
        torch.cuda.synchronize()
        _, pos, slots, starts, *state = OD.step_plan(lengths, news, host_tables, host_ring, *state, T)
        n = starts[-1]
        OG.insert(want, K, dim, slots[0], (_f64(kr), _f64(v)))
        _same_cache(pool, want, K, dim)
        some = {t for t in range(n) if t < 4 or t % 41 == 0 or t >= n - 4 or t in starts}
        view = GroupLayer.__new__(GroupLayer)
        view.K, view.dim, view._rows, view.host, view.table = K, dim, {}, want.copy(), host_tables[0]
        view.check(qr, out, lse, pos, starts, window, sinks, 1 / math.sqrt(dim), tokens=some)
        _check_prompt(starts, np.cumsum([0] + ends).tolist(), qr, *rows, pout, plse, True, window, sinks, 1 / math.sqrt(dim), some)
        for r, t in ((0, ends[0]),):
            for p in range(0, t, 29):
                assert np.array_equal(_f64(rows[1][p, 1]), OG.read_row(want, K, dim, host_tables[0][0, p // 256], 1, 1, p % 256))
        assert (out[n:] == 7.0).all() and (pout[n:] == 7.0).all()
        lengths = [0 if f < 0 else c + f for c, f in zip(lengths, news)]
    assert all(int(o.status.item()) == 0 for o in (plan, ins, att, read, pro))
