"""Dense-layer operators on the GPU against the fp64 oracle: the step plan
(exact), norm + rotation + insert, attention, and a run of the three together
(eager and as one captured graph over a padded batch).

Tolerances count roundings: a bf16 rounding is off by at most 2^-8 of the
value, an e4m3 code by 2^-4 of it (2^-10 of the scale below the normals), an
fp32 operation by 2^-24.  Attention: each probability is rounded to bf16
(2^-8 of sum p|v|) and the output once more; a logit's dot product of D terms
is off by (D + 8) 2^-24 of the largest sum |q||k| (as a relative error of p,
twice: in p and in the sum); the sums over N keys by (N + 32) 2^-24.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from oracle import dense as OD
from oracle import formats as F

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _dense():
    from compressed_sparse_long_c4a_gb300 import dense
    return dense


# --------------------------------------------------------------------------
# The step plan
# --------------------------------------------------------------------------

def _plan_case(rng, B, L, cached_hi, new_hi, ended, pad, spare=11):
    cached = [int(rng.integers(0, cached_hi + 1)) for _ in range(B)]
    fresh = [int(rng.integers(0, new_hi + 1)) for _ in range(B)]
    fresh = [-1 if rng.random() < ended else f for f in fresh]
    held = [-(-c // 256) for c in cached]
    need = sum(-(-(c + f) // 256) - h for c, f, h in zip(cached, fresh, held) if f > 0) * L
    cols = max(max(-(-(c + max(f, 0)) // 256) for c, f in zip(cached, fresh)), 1) if B else 1
    total = sum(held) * L + need + spare
    ids = rng.permutation(total)
    tables = np.full((L, B, cols), -1, np.int32)
    at = 0
    for l in range(L):
        for b in range(B):
            tables[l, b, :held[b]] = ids[at:at + held[b]]
            at += held[b]
    first = int(rng.integers(0, total))
    ring = np.full(total, -1, np.int32)
    count = total - at
    ring[(first + np.arange(count)) % total] = ids[at:]
    return cached, fresh, tables, ring, first, count, sum(max(f, 0) for f in fresh) + pad


def _run_plan(cached, fresh, tables, ring, first, count, T, same_free=True):
    D = _dense()
    plan = D.StepPlan(torch.from_numpy(tables).to(DEV), torch.from_numpy(ring).to(DEV), T)
    i32 = dict(dtype=torch.int32, device=DEV)
    free = torch.tensor([first, count], **i32)
    out = free if same_free else torch.zeros(2, **i32)
    plan.run(torch.tensor(cached, **i32), torch.tensor(fresh, **i32), free, out)
    torch.cuda.synchronize()
    return plan, out


@pytest.mark.parametrize("B,L,cached_hi,new_hi,ended,pad", [
    (1, 1, 0, 1, 0.0, 0), (1, 1, 1000, 0, 0.0, 3), (3, 2, 300, 1, 0.0, 0), (64, 61, 5000, 1, 0.0, 0), (64, 5, 5000, 1, 0.3, 64),
    (7, 3, 600, 700, 0.2, 5), (33, 4, 0, 257, 0.0, 1), (1025, 2, 600, 3, 0.1, 7), (2049, 1, 300, 1, 0.5, 0), (1, 3, 512, 20000, 0.0, 0),
    (8192, 1, 700, 2, 0.05, 100), (5, 2, 900, 900, 1.0, 4)])
def test_step_plan(B, L, cached_hi, new_hi, ended, pad):
    case = _plan_case(np.random.default_rng(B * 100 + L), B, L, cached_hi, new_hi, ended, pad)
    cached, fresh, tables, ring, first, count, T = case
    plan, free = _run_plan(cached, fresh, tables.copy(), ring.copy(), first, count, T, same_free=L % 2 == 0)
    sid, pos, slots, starts, first2, count2 = OD.step_plan(cached, fresh, tables, ring, first, count, T)
    assert int(plan.status.item()) == 0
    assert plan.seq_ids.tolist() == sid and plan.positions.tolist() == pos and plan.token_starts.tolist() == starts
    assert np.array_equal(plan.slots.cpu().numpy(), np.array(slots).reshape(L, T))
    assert np.array_equal(plan.block_table.cpu().numpy(), tables) and np.array_equal(plan.free_ring.cpu().numpy(), ring)
    assert free.tolist() == [first2, count2]


def test_step_plan_of_no_sequences():
    plan, free = _run_plan([], [], np.zeros((2, 0, 3), np.int32), np.arange(4, dtype=np.int32), 1, 2, 5)
    assert plan.seq_ids.tolist() == [-1] * 5 and plan.token_starts.tolist() == [0] and free.tolist() == [1, 2]
    plan, _ = _run_plan([5], [0], np.full((1, 1, 1), 0, np.int32), np.arange(4, dtype=np.int32), 1, 2, 0)
    assert plan.token_starts.tolist() == [0, 0] and int(plan.status.item()) == 0


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("change,bit", [
    (dict(cached=(0, -1)), 2), (dict(fresh=(1, -2)), 2), (dict(fresh=(0, 2000)), 2), (dict(cached=(1, 256 * 3)), 2),
    (dict(count=3), 16), (dict(count=3, T=58), 2), (dict(T=2), 2), (dict(first=-1), 2), (dict(first=40), 2), (dict(count=41), 2), (dict(count=-1), 2),
    (dict(count=39, fresh=(0, -1)), 2)])
def test_step_plan_all_or_nothing(change, bit, wide):
    """A step that cannot be done changes nothing and leaves nothing to do."""
    cached, fresh, first, count, T = [200, 300], [57, 1], 35, 20, 58 + (40000 if wide else 0)
    tables = np.full((2, 2, 3), -1, np.int32)
    tables[:, 0, 0], tables[:, 1, :2] = [20, 21], [[22, 23], [24, 25]]
    ring = np.arange(40, dtype=np.int32)
    if "cached" in change: cached[change["cached"][0]] = change["cached"][1]
    if "fresh" in change: fresh[change["fresh"][0]] = change["fresh"][1]
    first, count, T = change.get("first", first), change.get("count", count), change.get("T", T)
    if count == 3:                           # a second new block: two in each of two tables
        fresh[1], T = 300, change.get("T", T + 300)
    plan, free = _run_plan(cached, fresh, tables.copy(), ring.copy(), first, count, T, same_free=False)
    assert int(plan.status.item()) == bit
    assert (plan.seq_ids == -1).all() and (plan.positions == -1).all() and (plan.slots == -1).all()
    assert plan.token_starts.tolist() == [0, 0, 0] and free.tolist() == [first, count]
    assert np.array_equal(plan.block_table.cpu().numpy(), tables) and np.array_equal(plan.free_ring.cpu().numpy(), ring)


def test_step_plan_bad_page_ids():
    """A held page outside the pool gives slot -1 and the status bit, for its tokens only."""
    tables = np.array([[[3], [99]]], np.int32)
    plan, _ = _run_plan([10, 10], [2, 2], tables, np.arange(8, dtype=np.int32), 0, 2, 4)
    assert plan.slots[0].tolist() == [3 * 256 + 10, 3 * 256 + 11, -1, -1] and int(plan.status.item()) == 1


# --------------------------------------------------------------------------
# Norm + rotation + insert
# --------------------------------------------------------------------------

def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


ROPES = {
    "none": (None, {}),
    "inter": (dict(dims=64, layout=0), dict(dims=64)),
    "inter_tail": (dict(dims=32, first=32, layout=0, theta=500.0), dict(dims=32, theta=500.0)),
    "half": (dict(dims=64, layout=1), dict(dims=64)),
    "half_mid": (dict(dims=16, first=24, layout=1), dict(dims=16)),
    "half48": (dict(dims=48, first=8, layout=1), dict(dims=48)),
    "linear": (dict(dims=64, layout=1, scaling=1, factor=8.0), dict(dims=64, scaling="linear", factor=8.0)),
    "yarn": (dict(dims=64, layout=0, scaling=2, factor=16.0, original=4096.0, magnitude=1.277),
             dict(dims=64, scaling="yarn", factor=16.0, original=4096.0)),
    "table": (dict(dims=16, layout=1, scaling=3, table=[3.1, 1.0, 0.5, 0.2, 0.1, 1e-3, 1e-5, 0.0]),
              dict(dims=16, table=[3.1, 1.0, 0.5, 0.2, 0.1, 1e-3, 1e-5, 0.0])),
}


def _check_insert(q_out, q, k, v, qg, kg, pool, positions, slots, H, K, dim, fp8, rope, eps=1e-6):
    """Every token with a slot against the oracle."""
    spec, of = ROPES[rope]
    freq = OD.frequencies(**of) if spec else np.zeros(0)
    kw = dict(first=spec.get("first", 0), half=spec.get("layout") == 1, magnitude=spec.get("magnitude", 1.0)) if spec else {}
    pool = pool.cpu().numpy()
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    q, k, v, got_q = f64(q), f64(k), f64(v), f64(q_out)
    qg = None if qg is None else f64(qg)
    kg = None if kg is None else f64(kg)
    for t, slot in enumerate(slots):
        if slot < 0:
            continue
        want = OD.rotate(OD.rms_norm(q[t], qg, eps), positions[t], freq, **kw)
        # one bf16 rounding; before it the sum of up to 256 squares and a rotation in fp32: within 2^-16 of the row's largest
        floor = 2.0 ** -16 * np.abs(want).max(-1, keepdims=True)
        assert (np.abs(got_q[t] - want) <= 2.0 ** -8 * np.abs(want) + floor).all(), (t, "q")
        for which, x in ((0, OD.rotate(OD.rms_norm(k[t], kg, eps), positions[t], freq, **kw)), (1, v[t])):
            for h in range(K):
                row = x[h]
                floor = 2.0 ** -16 * np.abs(row).max()
                if not fp8:
                    got = OD.read_row(pool, K, dim, False, slot // 256, which, h, slot % 256)
                    assert (np.abs(got - row) <= 2.0 ** -8 * np.abs(row) + floor).all(), (t, which, h)
                    if which == 1:
                        assert np.array_equal(got, row)
                    continue
                codes, scale = OD.raw_row(pool, K, dim, slot // 256, which, h, slot % 256)
                s = np.abs(row).max() / 448.0 if np.abs(row).max() > 0 else 1.0
                assert abs(float(scale) - s) <= 2.0 ** -16 * s
                got = F.e4m3_decode(codes) * float(scale)
                assert (np.abs(got - row) <= 2.0 ** -4 * np.abs(row) + 2.0 ** -10 * s + floor).all(), (t, which, h)


@pytest.mark.parametrize("dim,H,K,fp8,rope,norm,T", [
    (64, 4, 2, False, "inter", True, 5), (64, 4, 4, True, "half", True, 5), (128, 16, 4, False, "half", True, 1),
    (128, 6, 2, True, "inter_tail", True, 9), (192, 3, 1, False, "half48", True, 4), (192, 3, 3, True, "yarn", True, 4),
    (256, 8, 1, False, "yarn", True, 3), (256, 2, 2, True, "half_mid", False, 3), (64, 64, 8, False, "linear", True, 17),
    (128, 128, 1, False, "table", False, 2), (128, 5, 5, True, "none", True, 7), (64, 0, 2, False, "inter", True, 6),
    (64, 8, 8, False, "half", False, 700), (128, 1024, 8, False, "half", True, 1)])
def test_insert(dim, H, K, fp8, rope, norm, T):
    D = _dense()
    g = torch.Generator().manual_seed(dim + H + T)
    x = (torch.randn((T, (H + 2 * K) * dim + 8), generator=g) * 2).to(torch.bfloat16).to(DEV)      # odd token stride
    q, k, v = (x[:, a:b].unflatten(1, (n, dim)) for a, b, n in
               ((0, H * dim, H), (H * dim, (H + K) * dim, K), ((H + K) * dim, (H + 2 * K) * dim, K)))
    v[0, 0] = 0                                       # a row of zeros: scale 1
    qg, kg = ((1 + 0.1 * torch.randn(dim, generator=g)).to(DEV) for _ in range(2)) if norm else (None, None)
    blocks = -(-T // 256) + 2
    stride = OD.block_bytes(K, dim, fp8) + 48         # pages of a wider bucket
    pool = torch.full((blocks, stride), 0x55, dtype=torch.uint8, device=DEV)
    slots = torch.randperm(blocks * 256, generator=g)[:T].tolist()
    positions = torch.randint(0, 1 << 20, (T,), generator=g).tolist()
    positions[0] = 2 ** 31 - 1
    positions[-1] = 0
    if T > 3:
        slots[2] = -1                                 # a padded row
    q_out = torch.full((T, H, dim), 7.0, dtype=torch.bfloat16, device=DEV)
    before = pool.clone()
    op = D.DenseInsert(D.DenseCache(pool, None, K, dim, D.KV_FP8_TOKEN if fp8 else D.KV_BF16), H,
                       D.Rope(**ROPES[rope][0]) if ROPES[rope][0] else None, qg, kg)
    pos_t = torch.tensor(positions, dtype=torch.int32, device=DEV)
    slot_t = torch.tensor(slots, dtype=torch.int64, device=DEV)
    op.run(q if H else None, k, v, q_out if H else None, pos_t, slot_t)
    torch.cuda.synchronize()
    assert int(op.status.item()) == 0
    some = range(T) if T < 50 else range(0, T, 23)
    _check_insert(q_out, q, k, v, qg, kg, pool, positions, [s if t in some else -1 for t, s in enumerate(slots)], H, K, dim, fp8, rope)
    if T > 3:
        assert (q_out[2] == 7.0).all()                # its row is as it was
    # nothing but the tokens' rows (and scales) changed
    after, was = pool.cpu().numpy(), before.cpu().numpy()
    mask = np.zeros(after.shape, bool)
    es = 1 if fp8 else 2
    for s in slots:
        if s >= 0:
            for plane in range(2 * K):
                row = plane * 256 + s % 256
                mask[s // 256, row * dim * es:(row + 1) * dim * es] = True
                if fp8:
                    mask[s // 256, 2 * K * 256 * dim + 4 * row:][:4] = True
    assert np.array_equal(after[~mask], was[~mask])


@pytest.mark.parametrize("dim,H,K", [(64, 4, 1), (64, 1, 1), (128, 2, 1), (128, 4, 2), (256, 1, 1), (192, 1, 1), (64, 0, 2), (128, 64, 8)])
@pytest.mark.parametrize("fp8", [False, True])
def test_insert_of_many_tokens(dim, H, K, fp8):
    """A long call writes what calls of few tokens write, byte for byte (tokens share a CTA when their rows are few)."""
    D = _dense()
    T = 5003
    g = torch.Generator(device=DEV).manual_seed(dim + H)
    x = torch.randn((T, (H + 2 * K) * dim), generator=g, device=DEV).to(torch.bfloat16)
    q, k, v = (x[:, a * dim:b * dim].unflatten(1, (b - a, dim)) for a, b in ((0, H), (H, H + K), (H + K, H + 2 * K)))
    gam = torch.rand(dim, generator=g, device=DEV) + 0.5
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device=DEV, dtype=torch.int32)
    slots = torch.randperm(8192, generator=g, device=DEV)[:T].contiguous()
    slots[::97] = -1
    outs, ops = [], []
    for parts in ([T], [700] * 7 + [T - 4900], [1, T - 2, 1]):
        pool = torch.zeros((32, D.block_bytes(K, dim, D.KV_FP8_TOKEN if fp8 else D.KV_BF16)), dtype=torch.uint8, device=DEV)
        qo = torch.full((T, H, dim), 7.0, dtype=torch.bfloat16, device=DEV)
        op = D.DenseInsert(D.DenseCache(pool, None, K, dim, D.KV_FP8_TOKEN if fp8 else D.KV_BF16), H, D.Rope(64, first=0, layout=1), gam, gam)
        at = 0
        for n in parts:
            s = slice(at, at + n)
            op.run(q[s] if H else None, k[s], v[s], qo[s] if H else None, pos[s], slots[s])
            at += n
        torch.cuda.synchronize()
        assert int(op.status.item()) == 0
        outs.append((pool, qo))
    for pool, qo in outs[1:]:
        assert torch.equal(outs[0][0], pool) and torch.equal(outs[0][1], qo)
    assert (outs[0][1][::97] == 7.0).all()
    bad = slots.clone()
    bad[2500], bad[4000] = 32 * 256, -5
    op.run(q if H else None, k, v, qo if H else None, pos, bad)
    assert int(op.status.item()) == 1


def test_insert_in_place_and_contiguous():
    """q rotated in place equals q rotated into another tensor, byte for byte."""
    D = _dense()
    q = torch.randn((9, 8, 64), device=DEV).to(torch.bfloat16)
    k, v = torch.randn((9, 2, 64), device=DEV).to(torch.bfloat16), torch.randn((9, 2, 64), device=DEV).to(torch.bfloat16)
    pool = torch.zeros((1, OD.block_bytes(2, 64, False)), dtype=torch.uint8, device=DEV)
    op = D.DenseInsert(D.DenseCache(pool, None, 2, 64), 8, D.Rope(64, layout=1), torch.ones(64, device=DEV), None)
    pos, slots = torch.arange(9, dtype=torch.int32, device=DEV), torch.arange(9, device=DEV)
    out = torch.empty_like(q)
    op.run(q, k, v, out, pos, slots)
    op.run(q, k, v, q, pos, slots)
    assert torch.equal(q, out)


def test_insert_reports_and_skips():
    D = _dense()
    pool = torch.zeros((2, OD.block_bytes(1, 64, False)), dtype=torch.uint8, device=DEV)
    x = torch.ones((4, 1, 64), dtype=torch.bfloat16, device=DEV)
    for slots, pos, bit in (([-2, 512, -1, 0], [0, 1, 2, 3], 1), ([5, 6, -1, 0], [-1, 1, -5, 3], 2), ([1 << 40, -(1 << 40), -1, 0], [0, 0, 0, 3], 1)):
        pool.zero_()
        out = torch.zeros_like(x)
        op = D.DenseInsert(D.DenseCache(pool, None, 1, 64), 1, None)
        op.run(x, x, x, out, torch.tensor(pos, dtype=torch.int32, device=DEV), torch.tensor(slots, device=DEV))
        torch.cuda.synchronize()
        assert int(op.status.item()) == bit
        wrote = [s for s, p in zip(slots, pos) if 0 <= s < 512 and p >= 0]
        assert int((pool.view(torch.bfloat16) == 1).sum()) == 2 * 64 * len(wrote)
        assert (out[:, 0, 0] == 1).tolist() == [0 <= s < 512 and p >= 0 for s, p in zip(slots, pos)]


def test_insert_fp8_nan_and_infinity_reach_the_reader():
    """A NaN or an infinity in a key row makes the row's scale one, so attention over it cannot look finite."""
    D = _dense()
    pool = torch.zeros((1, OD.block_bytes(1, 64, True)), dtype=torch.uint8, device=DEV)
    k = torch.ones((3, 1, 64), dtype=torch.bfloat16, device=DEV)
    k[0, 0, 5], k[1, 0, 63] = math.nan, -math.inf
    D.DenseInsert(D.DenseCache(pool, None, 1, 64, D.KV_FP8_TOKEN), 0, None).run(
        None, k, k, None, torch.arange(3, dtype=torch.int32, device=DEV), torch.arange(3, device=DEV))
    for which in (0, 1):
        s = [OD.raw_row(pool.cpu().numpy(), 1, 64, 0, which, 0, i)[1] for i in range(3)]
        assert math.isnan(s[0]) and math.isinf(s[1]) and s[2] == np.float32(1) / np.float32(448)


# --------------------------------------------------------------------------
# Attention
# --------------------------------------------------------------------------

class Layer:
    """A dense cache with every held row random, and the oracle's view of it."""

    def __init__(self, lengths, H, K, dim, fp8, seed, extra=16, cols=None, q_std=1.0, hidden=None, holes=()):
        D = _dense()
        g = torch.Generator().manual_seed(seed)
        self.H, self.K, self.dim, self.fp8, self.lengths = H, K, dim, fp8, lengths
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
        x = torch.randn((blocks, body), generator=g)
        pool = torch.zeros((blocks, OD.block_bytes(K, dim, fp8) + extra), dtype=torch.uint8)
        if fp8:
            pool[:, :body] = (x * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            pool[:, body:body + 8 * K * 256] = ((torch.rand((blocks, 2 * K * 256), generator=g) + 0.5) / 100).view(torch.uint8)
        else:
            pool[:, :2 * body] = x.to(torch.bfloat16).view(torch.uint8)
        self.host = pool.numpy().copy()
        if hidden is not None:          # rows that no query sees hold NaN (and NaN scales)
            for b, n in enumerate(lengths):
                for p in range(held[b] * 256):
                    if hidden(b, p):
                        for plane in range(2 * K):
                            row = plane * 256 + p % 256
                            blk = pool[int(self.table[b, p // 256])]
                            if fp8:
                                blk[row * dim:(row + 1) * dim] = 0x7f
                                blk[body + 4 * row:body + 4 * row + 4] = torch.tensor([math.nan]).view(torch.uint8)
                            else:
                                blk[row * dim * 2:(row + 1) * dim * 2] = torch.full((dim,), math.nan, dtype=torch.bfloat16).view(torch.uint8)
        for b, n in holes:              # blocks taken out of the table
            self.table[b, n] = -1
        self.pool = pool.to(DEV)
        self.bt = torch.from_numpy(self.table).to(DEV)
        self.cache = D.DenseCache(self.pool, self.bt, K, dim, D.KV_FP8_TOKEN if fp8 else D.KV_BF16)
        self.gen, self.q_std = g, q_std
        self._rows = {}

    def rows(self, b, which, h, n):
        """The first n positions' rows (NaN where the block is missing)."""
        key = (b, which, h)
        if key not in self._rows or len(self._rows[key]) < n:
            out = np.full((n, self.dim), np.nan)
            for p in range(n):
                blk = self.table[b, p // 256]
                if blk >= 0:
                    out[p] = OD.read_row(self.host, self.K, self.dim, self.fp8, blk, which, h, p % 256)
            self._rows[key] = out
        return self._rows[key][:n]

    def query(self, T):
        return (torch.randn((T, self.H, self.dim), generator=self.gen) * self.q_std).to(torch.bfloat16).to(DEV)

    def check(self, q, out, lse, positions, starts, window, sinks, scale, tokens=None):
        q, got, got_l = q.double().cpu().numpy(), out.double().cpu().numpy(), lse.double().cpu().numpy()
        G = self.H // self.K
        for b in range(len(starts) - 1):
            for t in range(starts[b], starts[b + 1]):
                if tokens is not None and t not in tokens:
                    continue
                m = positions[t]
                seen = [j for j in OD.visible(m, window, sinks) if self.table[b, j // 256] >= 0]
                for h in range(self.K):
                    k, v = self.rows(b, 0, h, m + 1)[seen], self.rows(b, 1, h, m + 1)[seen]
                    o, l, av, amp = OD.attention(q[t, h * G:(h + 1) * G], k, v, scale)
                    dz = (self.dim + 8) * 2.0 ** -24 * amp[:, None]
                    n = (len(seen) + 32) * 2.0 ** -24
                    tol = (2.0 ** -8 + 2 * dz + 2 * n) * av + 2.0 ** -8 * np.abs(o) + 1e-30
                    err = np.abs(got[t, h * G:(h + 1) * G] - o)
                    assert (err <= tol).all(), (b, t, h, float((err / tol).max()))
                    if len(seen) == 0:
                        assert (got_l[t, h * G:(h + 1) * G] == -np.inf).all()
                    else:
                        ltol = dz[:, 0] + n + 2.0 ** -22 * np.abs(l) + 2.0 ** -20
                        assert (np.abs(got_l[t, h * G:(h + 1) * G] - l) <= ltol).all(), (b, t, h)


def _attend(layer, positions, starts, window=0, sinks=0, max_new=None, pad=0, scale=None, tokens=None, check=True):
    D = _dense()
    T = starts[-1] + pad
    max_new = max(max(b - a for a, b in zip(starts, starts[1:])), 1) if max_new is None else max_new
    op = D.DenseAttention(layer.cache, layer.H, T, max_new, window, sinks, scale)
    q = layer.query(T)
    out = torch.full_like(q, 7.0)
    lse = torch.full((T, layer.H), 7.0, device=DEV)
    op.run(q, out, torch.tensor(list(positions) + [-1] * pad, dtype=torch.int32, device=DEV),
           torch.tensor(starts, dtype=torch.int32, device=DEV), lse)
    torch.cuda.synchronize()
    if check:
        assert int(op.status.item()) == 0
        layer.check(q, out, lse, positions, starts, window, sinks, op.args.softmax_scale, tokens)
        if pad:
            assert (out[starts[-1]:] == 7.0).all() and (lse[starts[-1]:] == 7.0).all()
    return op, q, out, lse


def _runs(cached, new):
    pos, starts = [], [0]
    for c, n in zip(cached, new):
        pos += range(c, c + n)
        starts.append(starts[-1] + n)
    return pos, starts


DECODE = [
    # lengths (own token included), H, K, dim, fp8, window, sinks
    ((1,), 1, 1, 64, False, 0, 0), ((1, 2, 64, 65, 128), 4, 4, 64, False, 0, 0), ((256, 257, 1000, 3), 8, 2, 128, False, 0, 0),
    ((700, 31), 16, 2, 128, True, 0, 0), ((1025,), 16, 4, 128, False, 0, 0), ((300, 5), 3, 1, 192, False, 0, 0),
    ((300, 77), 24, 2, 192, True, 0, 0), ((513, 90), 8, 8, 256, False, 0, 0), ((513, 90), 16, 1, 256, True, 0, 0),
    ((600, 40), 7, 1, 128, False, 0, 0), ((600, 40), 11, 1, 64, True, 0, 0), ((400, 1), 64, 1, 128, False, 0, 0),
    ((900, 130, 60, 1), 8, 2, 64, False, 100, 4), ((900, 130, 60, 1), 16, 1, 128, True, 64, 70), ((2000, 515), 8, 1, 128, False, 1, 0),
    ((2000, 515), 8, 1, 256, False, 300, 1), ((2000, 515), 4, 2, 64, True, 1000, 1500), ((777,) * 40, 8, 4, 64, False, 0, 0),
]


@pytest.mark.parametrize("lengths,H,K,dim,fp8,window,sinks", DECODE)
def test_decode(lengths, H, K, dim, fp8, window, sinks):
    """One new token per sequence; every row that the query does not see holds NaN."""
    def hidden(b, p):
        m = lengths[b] - 1
        return p > m or (window and p <= m - window and p >= sinks)
    layer = Layer(lengths, H, K, dim, fp8, seed=len(lengths) + H, hidden=hidden)
    _attend(layer, [n - 1 for n in lengths], list(range(len(lengths) + 1)), window, sinks, pad=3)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_peaked_and_flat(fp8):
    """Large logits (a row that one key wins) and equal ones; a scale of another size."""
    layer = Layer((900, 400), 8, 2, 128, fp8, seed=3, q_std=20.0)
    _attend(layer, [899, 399], [0, 1, 2])
    layer = Layer((900, 400), 8, 2, 128, fp8, seed=4, q_std=0.0)
    _attend(layer, [899, 399], [0, 1, 2])
    layer = Layer((900, 400), 8, 2, 128, fp8, seed=5)
    _attend(layer, [899, 399], [0, 1, 2], scale=1.5)


def test_decode_empty_sequences_and_padding():
    layer = Layer((50, 600, 9, 300), 8, 2, 64, False, seed=6, cols=5)
    _attend(layer, [599, 299], [0, 0, 1, 1, 2], pad=5)


def test_decode_missing_blocks():
    """Positions of a missing block are left out and reported; with every block missing the row is 0 and -inf."""
    layer = Layer((700, 200, 600), 8, 2, 64, False, seed=7, holes=[(0, 1), (1, 0), (2, 2)])
    op, q, out, lse = _attend(layer, [699, 199, 599], [0, 1, 2, 3], check=False)
    assert int(op.status.item()) == 1
    layer.check(q, out, lse, [699, 199, 599], [0, 1, 2, 3], 0, 0, op.args.softmax_scale)
    layer.bt[0, 0] = 1 << 30
    op, q, out, lse = _attend(layer, [699, 199, 599], [0, 1, 2, 3], check=False)
    layer.table[0, 0] = -1
    layer.check(q, out, lse, [699, 199, 599], [0, 1, 2, 3], 0, 0, op.args.softmax_scale)


def test_window_never_reads_blocks_it_gave_back():
    """Blocks between the sinks and the window are gone: no status bit, the same result."""
    layer = Layer((3000,), 8, 2, 64, False, seed=8)
    _, q, out, _ = _attend(layer, [2999], [0, 1], window=300, sinks=4)
    for n in range(1, 10):
        layer.bt[0, n] = -1
    op = _dense().DenseAttention(layer.cache, 8, 1, 1, 300, 4)
    out2 = torch.empty_like(out)
    op.run(q, out2, torch.tensor([2999], dtype=torch.int32, device=DEV), torch.tensor([0, 1], dtype=torch.int32, device=DEV))
    assert torch.equal(out, out2) and int(op.status.item()) == 0


@pytest.mark.parametrize("positions,starts,bad,left", [
    ([5, 9, 20], [0, 1, 3, 3], {1}, [1, 2]),            # not consecutive
    ([-1, 9, 10], [0, 1, 3, 3], {0}, [0]),              # negative
    ([5, 9, 10], [0, 1, 0, 3], {1, 2}, [1, 2]),         # starts go back; three tokens where two are allowed
    ([5, 9, 10], [0, 1, 3, 9], {2}, []),                # past the end
    ([256 * 3, 9, 10], [0, 1, 3, 3], {0}, [0]),         # past the table
])
def test_inconsistent_batches_are_reported_and_left(positions, starts, bad, left):
    layer = Layer((100, 100, 100), 4, 2, 64, False, seed=9, cols=3)
    op = _dense().DenseAttention(layer.cache, 4, 3, 2)
    q = layer.query(3)
    out, lse = torch.full_like(q, 7.0), torch.full((3, 4), 7.0, device=DEV)
    op.run(q, out, torch.tensor(positions, dtype=torch.int32, device=DEV), torch.tensor(starts, dtype=torch.int32, device=DEV), lse)
    torch.cuda.synchronize()
    assert int(op.status.item()) == 2
    assert (out[left] == 7.0).all() and (lse[left] == 7.0).all()
    for b in {0, 1, 2} - bad:
        layer.check(q, out, lse, positions, [starts[b]] * (b + 1) + [starts[b + 1]] * (3 - b), 0, 0, op.args.softmax_scale)


CHUNKS = [
    # cached, new, H, K, dim, fp8, window, sinks
    ((0,), (5,), 4, 4, 64, False, 0, 0), ((0, 300), (130, 7), 8, 2, 128, False, 0, 0), ((10, 0, 250), (3, 1, 20), 8, 1, 128, True, 0, 0),
    ((500,), (200,), 6, 2, 128, False, 0, 0), ((0, 700), (300, 129), 4, 1, 64, False, 100, 4), ((900,), (257,), 16, 2, 128, False, 64, 130),
    ((30,), (100,), 4, 2, 192, False, 0, 0), ((30,), (60,), 4, 2, 256, False, 50, 3), ((0, 90), (65, 64), 2, 2, 64, True, 30, 2),
    ((400,), (150,), 32, 2, 128, True, 0, 0), ((0,), (513,), 5, 1, 128, False, 0, 0), ((255, 256, 511), (2, 256, 130), 8, 8, 64, False, 0, 0),
    ((0,), (300,), 128, 1, 64, False, 0, 0), ((0, 0, 0), (1, 260, 2), 64, 4, 128, False, 1, 0),
    ((1500,), (300,), 8, 2, 128, False, 1100, 3), ((1500, 20), (140, 200), 4, 1, 256, True, 1300, 0), ((2000,), (90,), 4, 2, 64, True, 1025, 300),
]


@pytest.mark.parametrize("cached,new,H,K,dim,fp8,window,sinks", CHUNKS)
def test_chunks(cached, new, H, K, dim, fp8, window, sinks):
    """Chunked prefill and ragged mixes; rows no query of the call sees hold NaN."""
    def hidden(b, p):
        return p >= cached[b] + new[b] or (window and p <= cached[b] - window and p >= sinks)
    layer = Layer([c + n for c, n in zip(cached, new)], H, K, dim, fp8, seed=sum(new), hidden=hidden)
    pos, starts = _runs(cached, new)
    some = None if len(pos) < 40 else {t for b in range(len(new)) for t in
                                       {starts[b], starts[b] + 1, starts[b + 1] - 1, *range(starts[b], starts[b + 1], 17)} if t < starts[b + 1]}
    _attend(layer, pos, starts, window, sinks, pad=2, tokens=some)


MIXED = [
    # (cached, new) per sequence, H, K, dim, fp8, window, sinks, room in max_new
    ([(700, 1), (0, 300), (90, 1), (256, 8), (10, 9), (0, 33)], 8, 2, 128, False, 0, 0, 0),
    ([(700, 1), (0, 300), (90, 1), (256, 16), (10, 17), (0, 33)], 8, 2, 64, True, 0, 0, 0),
    ([(700, 1), (300, 200), (0, 0), (256, 3), (0, 0)], 16, 1, 128, True, 100, 5, 0),
    ([(30, 1), (60, 2), (7, 5)], 8, 8, 128, False, 0, 0, 1000),              # the longest allowed is not there
    ([(300, 70), (60, 64), (7, 65)], 4, 4, 64, False, 40, 0, 2000),
    ([(i % 300, 1) for i in range(60)] + [(100, 700)] + [(i, 2) for i in range(60)], 4, 2, 64, False, 0, 0, 0),
    ([(i % 90, 1 + 40 * (i % 61 == 0)) for i in range(700)], 2, 1, 64, False, 0, 0, 0),   # more sequences than are split evenly
    ([(i % 90, 40 * (i % 61 == 0) + (i % 3 > 0)) for i in range(700)], 2, 1, 64, True, 20, 2, 0),
    ([(i % 50, 1 + i % 120) for i in range(40)], 8, 1, 192, False, 0, 0, 0),
    ([(600, 150), (0, 1), (0, 300), (90, 40)], 8, 2, 256, True, 100, 5, 0),
    ([(600, 150), (0, 9), (0, 300), (90, 5)], 4, 2, 192, False, 64, 70, 100),
    ([(i % 50, 1 + 30 * (i % 5 == 0)) for i in range(600)], 2, 1, 256, False, 0, 0, 0),
]


@pytest.mark.parametrize("runs,H,K,dim,fp8,window,sinks,room", MIXED)
def test_mixed_batches(runs, H, K, dim, fp8, window, sinks, room):
    """Decoding sequences beside chunks, with and without limits far above what the batch brings."""
    cached, new = zip(*runs)
    layer = Layer([c + n for c, n in runs], H, K, dim, fp8, seed=len(runs) + dim)
    pos, starts = _runs(cached, new)
    some = {t for b in range(len(new)) for t in (starts[b], starts[b + 1] - 1, (starts[b] + starts[b + 1]) // 2)
            if starts[b] <= t < starts[b + 1] and (len(new) < 100 or b % 61 == 0 or b % 29 == 0)}
    _attend(layer, pos, starts, window, sinks, max_new=max(new) + room, pad=3, tokens=some)


@pytest.mark.parametrize("B", [41, 601])
@pytest.mark.parametrize("dim", [64, 192])
def test_sequences_that_share_tokens_are_reported(B, dim):
    """Every other sequence claims all tokens: more rows than the call has."""
    layer = Layer((100,) * B, 8, 2, dim, False, seed=2)
    op = _dense().DenseAttention(layer.cache, 8, 100, 100)
    q = layer.query(100)
    buf = torch.full((300, 8, dim), 7.0, device=DEV, dtype=torch.bfloat16)
    op.run(q, buf[100:200], torch.arange(100, dtype=torch.int32, device=DEV), torch.tensor(([0, 100] * B)[:B + 1], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert int(op.status.item()) & 2
    assert (buf[:100] == 7.0).all() and (buf[200:] == 7.0).all()


@pytest.mark.parametrize("cached,new,H,K,dim,fp8", [((9000, 100), (700, 500), 8, 2, 128, False), ((9000, 100), (700, 500), 8, 2, 128, True),
                                                    ((0, 0, 5000), (3000, 1, 64), 4, 1, 64, False), ((20000,), (90,), 8, 2, 64, True),
                                                    ((0,), (6000,), 8, 8, 128, False), ((3000,), (1000,), 4, 2, 192, True),
                                                    ((7000, 300), (900, 257), 4, 2, 256, False), ((5000, 0, 20), (600, 200, 1), 8, 2, 256, True),
                                                    ((100,), (2500,), 3, 1, 192, False)])
def test_long_chunks(cached, new, H, K, dim, fp8):
    """Many steps per CTA, units over several CTAs, ranges over several units; every row against fp64."""
    D = _dense()
    g = torch.Generator(device=DEV).manual_seed(H + dim)
    lengths = [c + n for c, n in zip(cached, new)]
    held = [-(-n // 256) for n in lengths]
    ids = torch.randperm(sum(held) + 2, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lengths), max(held)), -1, dtype=torch.int32, device=DEV)
    for b, n in enumerate(held):
        table[b, :n] = ids[sum(held[:b]):sum(held[:b]) + n]
    body = 2 * K * 256 * dim
    x = torch.randn((len(ids), body), generator=g, device=DEV)
    if fp8:
        sc = (torch.rand((len(ids), 2 * K * 256), generator=g, device=DEV) + 0.5) / 100
        pool = torch.cat([(x * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), sc.view(torch.uint8)], 1)
    else:
        pool = x.to(torch.bfloat16).view(torch.uint8)
    pos, starts = _runs(cached, new)
    T = starts[-1]
    q = torch.randn((T, H, dim), generator=g, device=DEV).mul_(2).to(torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty((T, H), device=DEV)
    op = D.DenseAttention(D.DenseCache(pool, table, K, dim, D.KV_FP8_TOKEN if fp8 else D.KV_BF16), H, T, max(new))
    args = (torch.tensor(pos, dtype=torch.int32, device=DEV), torch.tensor(starts, dtype=torch.int32, device=DEV))
    op.run(q, out, *args, lse)
    torch.cuda.synchronize()
    assert int(op.status.item()) == 0
    G = H // K
    for b, n in enumerate(lengths):
        s, m = slice(starts[b], starts[b + 1]), torch.arange(cached[b], n, device=DEV)
        for h in range(H):
            page = table[b, :held[b]].long()
            if fp8:
                blk = pool[page]
                rows = blk[:, :body].contiguous().view(torch.float8_e4m3fn).view(-1, 2, K, 256, dim)[:, :, h // G].double()
                rows = rows * blk[:, body:body + 8 * K * 256].contiguous().view(torch.float32).view(-1, 2, K, 256, 1)[:, :, h // G].double()
            else:
                rows = pool[page][:, :2 * body].contiguous().view(torch.bfloat16).view(-1, 2, K, 256, dim)[:, :, h // G].double()
            k, v = (rows[:, i].reshape(-1, dim)[:n] for i in (0, 1))
            qd = q[s, h].double()
            z = (qd @ k.T / math.sqrt(dim)).masked_fill_(torch.arange(n, device=DEV) > m[:, None], -math.inf)
            amp = ((qd.abs() @ k.abs().T) / math.sqrt(dim)).amax(-1)
            pr, l = torch.softmax(z, -1), torch.logsumexp(z, -1)
            o, av = pr @ v, pr @ v.abs()
            dz, dn = (dim + 8) * 2.0 ** -24 * amp[:, None], (n + 32) * 2.0 ** -24
            assert ((out[s, h].double() - o).abs() <= (2.0 ** -8 + 2 * dz + 2 * dn) * av + 2.0 ** -8 * o.abs()).all(), (b, h)
            assert ((lse[s, h].double() - l).abs() <= dz[:, 0] + dn + 2.0 ** -22 * l.abs() + 2.0 ** -20).all(), (b, h)
    again, lse2 = torch.empty_like(out), torch.empty_like(lse)      # the same call gives the same bytes, on another stream too
    op.run(q, again, *args, lse2, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("fp8", [False, True])
def test_chunk_missing_blocks_and_nan(fp8):
    """Chunk form: missing blocks are left out and reported; a NaN query row reaches its own output row alone."""
    layer = Layer((900, 300), 8, 2, 128, fp8, seed=12, holes=[(0, 1), (0, 2), (1, 0)])
    pos, starts = _runs((700, 100), (200, 150))
    op, q, out, lse = _attend(layer, pos, starts, check=False)
    assert int(op.status.item()) == 1
    layer.check(q, out, lse, pos, starts, 0, 0, op.args.softmax_scale, tokens=set(range(0, 350, 23)))
    q2, out2, lse2 = q.clone(), torch.empty_like(out), torch.empty_like(lse)
    q2[130, 5, 7] = math.nan
    op.run(q2, out2, torch.tensor(pos, dtype=torch.int32, device=DEV), torch.tensor(starts, dtype=torch.int32, device=DEV), lse2)
    assert out2[130, 5].isnan().all() and lse2[130, 5].isnan()
    out2[130, 5], lse2[130, 5] = out[130, 5], lse[130, 5]
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_many_units_take_the_unsplit_form():
    """More (sequence, row group) units than are split evenly: one CTA each."""
    n = 1100
    layer = Layer([1 + i % 90 for i in range(n)], 2, 1, 64, False, seed=10)
    _attend(layer, [i % 90 for i in range(n)], list(range(n + 1)), tokens=set(range(0, n, 37)))


def test_chunk_equals_single_tokens():
    """A chunk's rows within the tolerance of two bf16 outputs of the same formula: each row alone is in the oracle's
    tolerance; here the decode form and the chunk form of the same tokens agree to two roundings of each."""
    layer = Layer((400,), 8, 2, 128, False, seed=11)
    pos, starts = _runs((270,), (130,))
    op, q, out, lse = _attend(layer, pos, starts, check=False)
    one = torch.empty_like(out)
    dec = _dense().DenseAttention(layer.cache, 8, 1, 1)
    for t, p in enumerate(pos):
        o = torch.empty_like(out[:1])
        dec.run(q[t:t + 1], o, torch.tensor([p], dtype=torch.int32, device=DEV), torch.tensor([0, 1], dtype=torch.int32, device=DEV))
        one[t] = o[0]
    layer.check(q, one, lse, pos, starts, 0, 0, op.args.softmax_scale, tokens=set(range(0, 130, 9)))
    layer.check(q, out, lse, pos, starts, 0, 0, op.args.softmax_scale, tokens=set(range(0, 130, 9)))


def _reference(pool, table, b, m, q, K, dim, fp8, h):
    """fp64 on the GPU for one query head group: (o, lse) over positions 0..m (bf16 or fp8 caches of long tests)."""
    n, body = m + 1, 2 * K * 256 * dim
    page = table[b, :(n + 255) // 256].long()
    if fp8:
        rows = pool[page][:, :body].view(torch.float8_e4m3fn).double().view(-1, 2, K, 256, dim)[:, :, h]
        rows = rows * pool[page][:, body:body + 8 * K * 256].contiguous().view(torch.float32).double().view(-1, 2, K, 256, 1)[:, :, h]
    else:
        rows = pool[page][:, :2 * body].contiguous().view(torch.bfloat16).view(-1, 2, K, 256, dim)[:, :, h].double()
    k, v = (rows[:, i].reshape(-1, dim)[:n] for i in (0, 1))
    z = q.double() @ k.T / math.sqrt(dim)
    p = torch.softmax(z, -1)
    return p @ v, torch.logsumexp(z, -1), p @ v.abs(), (q.double().abs() @ k.abs().T).amax(-1) / math.sqrt(dim)


@pytest.mark.parametrize("lengths,H,K,dim,fp8", [((30000, 20011, 1), 16, 4, 128, False), ((40001, 255), 16, 2, 128, True),
                                                  ((25000,), 4, 4, 64, False), ((9000, 14000), 2, 2, 256, False)])
def test_long_caches(lengths, H, K, dim, fp8):
    """Hundreds of tiles per CTA, ranges over several sequences and KV heads."""
    D = _dense()
    g = torch.Generator(device=DEV).manual_seed(H + dim)
    held = [-(-n // 256) for n in lengths]
    ids = torch.randperm(sum(held) + 2, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lengths), max(held)), -1, dtype=torch.int32, device=DEV)
    for b, n in enumerate(held):
        table[b, :n] = ids[sum(held[:b]):sum(held[:b]) + n]
    body = 2 * K * 256 * dim
    x = torch.randn((len(ids), body), generator=g, device=DEV)
    if fp8:
        sc = (torch.rand((len(ids), 2 * K * 256), generator=g, device=DEV) + 0.5) / 100
        pool = torch.cat([(x * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), sc.view(torch.uint8)], 1)
    else:
        pool = x.to(torch.bfloat16).view(torch.uint8)
    T = len(lengths)
    q = torch.randn((T, H, dim), generator=g, device=DEV).mul_(2).to(torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty((T, H), device=DEV)
    op = D.DenseAttention(D.DenseCache(pool, table, K, dim, D.KV_FP8_TOKEN if fp8 else D.KV_BF16), H, T)
    op.run(q, out, torch.tensor([n - 1 for n in lengths], dtype=torch.int32, device=DEV), torch.arange(T + 1, dtype=torch.int32, device=DEV), lse)
    torch.cuda.synchronize()
    assert int(op.status.item()) == 0
    G = H // K
    for b, n in enumerate(lengths):
        for h in range(K):
            s = slice(h * G, (h + 1) * G)
            o, l, av, amp = _reference(pool, table, b, n - 1, q[b, s], K, dim, fp8, h)
            dz, dn = (dim + 8) * 2.0 ** -24 * amp[:, None], (n + 32) * 2.0 ** -24
            assert ((out[b, s].double() - o).abs() <= (2.0 ** -8 + 2 * dz + 2 * dn) * av + 2.0 ** -8 * o.abs()).all(), (b, h)
            assert ((lse[b, s].double() - l).abs() <= dz[:, 0] + dn + 2.0 ** -22 * l.abs() + 2.0 ** -20).all(), (b, h)


def test_nan_query_gives_nan():
    layer = Layer((300, 90), 8, 2, 64, False, seed=30)
    op = _dense().DenseAttention(layer.cache, 8, 2)
    q = layer.query(2)
    q[0, 3, 5] = math.nan
    out, lse = torch.zeros_like(q), torch.zeros((2, 8), device=DEV)
    op.run(q, out, torch.tensor([299, 89], dtype=torch.int32, device=DEV), torch.arange(3, dtype=torch.int32, device=DEV), lse)
    assert out[0, 3].isnan().all() and lse[0, 3].isnan()
    assert int(out.isnan().sum()) == 64 and int(lse.isnan().sum()) == 1


@pytest.mark.parametrize("new", [1, 100])
def test_huge_windows_and_sinks(new):
    """Limits near the ends of their type: a window longer than the sequence hides nothing, as many sinks show everything."""
    layer = Layer((500,), 8, 2, 64, False, seed=31)
    pos, starts = _runs((500 - new,), (new,))
    q = layer.query(new)
    outs = []
    for window, sinks in ((0, 0), (2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (512, 0), (2 ** 30, 3), (7, 2 ** 31 - 1), (0, 2 ** 31 - 1)):
        op = _dense().DenseAttention(layer.cache, 8, new, new, window, sinks)
        out = torch.empty_like(q)
        op.run(q, out, torch.tensor(pos, dtype=torch.int32, device=DEV), torch.tensor(starts, dtype=torch.int32, device=DEV))
        assert int(op.status.item()) == 0
        outs.append(out)
    for o in outs[:5] + outs[6:]:
        assert torch.equal(outs[0], o)
    lse = torch.empty((new, 8), device=DEV)
    _dense().DenseAttention(layer.cache, 8, new, new, 7, 2 ** 31 - 1).run(q, outs[5], torch.tensor(pos, dtype=torch.int32, device=DEV),
                                                                       torch.tensor(starts, dtype=torch.int32, device=DEV), lse)
    layer.check(q, outs[5], lse, pos, starts, 0, 0, 1 / 8, tokens=set(range(0, new, 13)))


@pytest.mark.parametrize("fp8", [False, True])
def test_pools_past_four_gigabytes(fp8):
    """Insert and attention (decode and a chunk) in blocks whose offsets pass 32 bits."""
    D = _dense()
    H, K, dim = 32, 32, 128
    stride = D.block_bytes(K, dim, D.KV_FP8_TOKEN if fp8 else D.KV_BF16)
    blocks = (5 << 30) // stride
    pool = torch.empty((blocks, stride), dtype=torch.uint8, device=DEV)
    high = [blocks - 1, (1 << 32) // stride + 1, blocks - 2, 1]
    table = torch.tensor([high], dtype=torch.int32, device=DEV)
    cache = D.DenseCache(pool, table, K, dim, D.KV_FP8_TOKEN if fp8 else D.KV_BF16)
    n = 4 * 256 - 30
    g = torch.Generator(device=DEV).manual_seed(3)
    k, v = (torch.randn((n, K, dim), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    ins = D.DenseInsert(cache, 0, None)
    ins.run(None, k, v, None, pos, table[0].long()[(pos // 256).long()] * 256 + pos % 256)
    for new in (1, 90):
        q = torch.randn((new, H, dim), generator=g, device=DEV).to(torch.bfloat16)
        out, lse = torch.empty_like(q), torch.empty((new, H), device=DEV)
        att = D.DenseAttention(cache, H, new, new)
        att.run(q, out, pos[n - new:], torch.tensor([0, new], dtype=torch.int32, device=DEV), lse)
        torch.cuda.synchronize()
        assert int(att.status.item()) == 0 and int(ins.status.item()) == 0
        for t in {0, new - 1}:
            for h in (0, 31):
                o, l, av, amp = _reference(pool, table, 0, n - new + t, q[t, h:h + 1], K, dim, fp8, h)
                dz, dn = (dim + 8) * 2.0 ** -24 * amp[:, None], (n + 32) * 2.0 ** -24
                assert ((out[t, h:h + 1].double() - o).abs() <= (2.0 ** -8 + 2 * dz + 2 * dn) * av + 2.0 ** -8 * o.abs()).all()
                assert ((lse[t, h:h + 1].double() - l).abs() <= dz[:, 0] + dn + 2.0 ** -22 * l.abs() + 2.0 ** -20).all()
    rows = (pool[high[1]][:2 * K * 256 * dim * (1 if fp8 else 2)].view(torch.float8_e4m3fn if fp8 else torch.bfloat16)
            .view(2, K, 256, dim)[0].float())
    if not fp8:
        assert torch.equal(rows.transpose(0, 1), k[256:512].float())


def test_same_call_same_bytes():
    layer = Layer((5000, 100, 2600), 16, 2, 128, False, seed=12)
    op, q, out, lse = _attend(layer, [4999, 99, 2599], [0, 1, 2, 3], tokens={1})
    for _ in range(3):
        o2, l2 = torch.empty_like(out), torch.empty_like(lse)
        op.run(q, o2, torch.tensor([4999, 99, 2599], dtype=torch.int32, device=DEV), torch.tensor([0, 1, 2, 3], dtype=torch.int32, device=DEV), l2)
        assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_two_streams_with_their_own_workspaces():
    """Two calls in flight at once, each with its own handle, give what each gives alone."""
    layers = [Layer((3000 + 500 * i, 700), 8, 2, 128, i == 1, seed=20 + i) for i in range(2)]
    pos = [torch.tensor([n - 1 for n in L.lengths], dtype=torch.int32, device=DEV) for L in layers]
    starts = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    ops = [_dense().DenseAttention(L.cache, 8, 2, 1) for L in layers]
    qs = [L.query(2) for L in layers]
    alone = [torch.empty_like(q) for q in qs]
    for i in range(2):
        ops[i].run(qs[i], alone[i], pos[i], starts)
    torch.cuda.synchronize()
    both = [torch.empty_like(q) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for i in range(2):
            ops[i].run(qs[i], both[i], pos[i], starts, stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(alone[i], both[i])


@pytest.mark.parametrize("dim", [128, 256])
def test_two_streams_of_mixed_batches(dim):
    """Both forms of two calls in flight at once."""
    runs = [[(900, 1), (200, 150), (40, 3), (0, 300)], [(10, 90), (1500, 2), (0, 0), (33, 200)]]
    layers = [Layer([c + n for c, n in r], 8, 2, dim, i == 1, seed=40 + i) for i, r in enumerate(runs)]
    ops, args, alone = [], [], []
    for L, r in zip(layers, runs):
        pos, starts = _runs(*zip(*r))
        op = _dense().DenseAttention(L.cache, 8, len(pos), max(n for _, n in r))
        q = L.query(len(pos))
        out = torch.empty_like(q)
        args.append((q, torch.tensor(pos, dtype=torch.int32, device=DEV), torch.tensor(starts, dtype=torch.int32, device=DEV)))
        op.run(q, out, *args[-1][1:])
        torch.cuda.synchronize()
        ops.append(op)
        alone.append(out)
    both = [torch.empty_like(o) for o in alone]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for i in range(2):
            ops[i].run(args[i][0], both[i], *args[i][1:], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(alone[i], both[i]) and int(ops[i].status.item()) == 0


@pytest.mark.parametrize("dim,fp8", [(64, True), (128, True), (128, False), (256, True)])
def test_mixed_steps_see_what_was_just_inserted(dim, fp8):
    """Insert and attention without a pause: rows beside each other, and the scales in one line with older ones, are
    new at every step; a call after a synchronisation gives the same bytes."""
    D = _dense()
    H, K, steps, chunk = 8, 2, 24, 37
    fmt = D.KV_FP8_TOKEN if fp8 else D.KV_BF16
    g = torch.Generator(device=DEV).manual_seed(dim)
    table = torch.randperm(12, generator=g, device=DEV).to(torch.int32).view(3, 4)
    pool = torch.full((12, D.block_bytes(K, dim, fmt)), 0xff, dtype=torch.uint8, device=DEV)      # NaN everywhere
    cache = D.DenseCache(pool, table, K, dim, fmt)
    T = 2 + chunk
    ins, att = D.DenseInsert(cache, H, D.Rope(dim, layout=1)), D.DenseAttention(cache, H, T, chunk)
    xs = torch.randn((steps, T, H + 2 * K, dim), generator=g, device=DEV).to(torch.bfloat16)
    starts = torch.tensor([0, 1, 1 + chunk, T], dtype=torch.int32, device=DEV)
    pos, slots, qr, out = [], [], torch.empty((steps, T, H, dim), dtype=torch.bfloat16, device=DEV), None
    for s in range(steps):
        p = torch.tensor([s, *range(s * chunk, (s + 1) * chunk), s], dtype=torch.int32, device=DEV)
        b = torch.tensor([0] + [1] * chunk + [2], device=DEV)
        pos.append(p)
        slots.append(table[b, (p // 256).long()].long() * 256 + p % 256)
    out = torch.zeros_like(qr)
    torch.cuda.synchronize()
    for s in range(steps):
        ins.run(xs[s, :, :H], xs[s, :, H:H + K], xs[s, :, H + K:], qr[s], pos[s], slots[s])
        att.run(qr[s], out[s], pos[s], starts)
    torch.cuda.synchronize()
    assert int(ins.status.item()) == 0 and int(att.status.item()) == 0 and bool(out.isfinite().all())
    again = torch.zeros_like(out)
    for s in range(steps):                      # later rows are hidden from earlier steps' queries
        att.run(qr[s], again[s], pos[s], starts)
        torch.cuda.synchronize()
    assert torch.equal(out, again)


# --------------------------------------------------------------------------
# The three together
# --------------------------------------------------------------------------

@pytest.mark.parametrize("fp8,window,sinks", [(False, 0, 0), (True, 0, 0), (False, 90, 4)])
@pytest.mark.parametrize("graph", [False, True])
def test_steps_of_a_small_server(fp8, window, sinks, graph):
    """Plan -> insert -> attention for two layers over several steps of a
    changing batch (starting, chunked, decoding, resting and ending
    sequences), eagerly or as one captured graph over padded arrays; the
    caches' rows and the attention of every step against the oracle."""
    D = _dense()
    H, K, dim, B, L, T = 8, 2, 64, 4, 2, 320
    pages = 24
    rope = dict(dims=64, layout=1)
    gen = torch.Generator().manual_seed(5)
    tables = torch.full((L, B, 6), -1, dtype=torch.int32, device=DEV)
    ring = torch.randperm(pages, generator=gen).to(torch.int32).to(DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    free, cached, fresh = torch.tensor([0, pages], **i32), torch.zeros(B, **i32), torch.zeros(B, **i32)
    plan = D.StepPlan(tables, ring, T)
    pools = [torch.full((pages, OD.block_bytes(K, dim, fp8)), 0xff, dtype=torch.uint8, device=DEV) for _ in range(L)]   # NaN everywhere
    caches = [D.DenseCache(p, tables[l], K, dim, D.KV_FP8_TOKEN if fp8 else D.KV_BF16) for l, p in enumerate(pools)]
    gam = torch.rand(dim, generator=gen).to(DEV) + 0.5
    ins = [D.DenseInsert(c, H, D.Rope(**rope), gam, gam) for c in caches]
    att = [D.DenseAttention(c, H, T, 300, window, sinks) for c in caches]
    x = torch.zeros((L, T, (H + 2 * K) * dim), dtype=torch.bfloat16, device=DEV)
    q, k, v = (x[:, :, a * dim:b * dim].unflatten(2, (b - a, dim)) for a, b in ((0, H), (H, H + K), (H + K, H + 2 * K)))
    qr = torch.zeros((L, T, H, dim), dtype=torch.bfloat16, device=DEV)
    out = torch.zeros((L, T, H, dim), dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros((L, T, H), device=DEV)

    def step():
        plan.run(cached, fresh, free)
        for l in range(L):
            ins[l].run(q[l], k[l], v[l], qr[l], plan.positions, plan.slots[l])
            att[l].run(qr[l], out[l], plan.positions, plan.token_starts, lse[l])

    g = None
    if graph:
        step()                              # nothing to do: every sequence rests
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
    lengths = [0] * B
    host_tables, host_ring, state = tables.cpu().numpy().copy(), ring.cpu().numpy().copy(), (0, pages)
    for news in ([250, 0, 3, 1], [1, 7, 300, 1], [1, 1, 0, 1], [-1, 1, 1, 1], [20, -1, 1, 1], [1, 255, 1, -1]):
        x.copy_((torch.randn(x.shape, generator=gen) * 1.5).to(torch.bfloat16))
        cached.copy_(torch.tensor(lengths, **i32))
        fresh.copy_(torch.tensor(news, **i32))
        out.fill_(7.0)
        g.replay() if graph else step()
        torch.cuda.synchronize()
        sid, pos, slots, starts, *state = OD.step_plan(lengths, news, host_tables, host_ring, *state, T)
        assert plan.positions.tolist() == pos and plan.token_starts.tolist() == starts and free.tolist() == state
        assert np.array_equal(plan.slots.cpu().numpy(), np.array(slots)) and np.array_equal(tables.cpu().numpy(), host_tables)
        n = starts[-1]
        some = [t for t in range(n) if t < 4 or t % 41 == 0 or t >= n - 4 or t in starts]
        for l in range(L):
            ROPES["server"] = (rope, dict(dims=64))
            _check_insert(qr[l], q[l], k[l], v[l], gam, gam, pools[l], pos, [s if t in some else -1 for t, s in enumerate(slots[l])],
                          H, K, dim, fp8, "server")
            view = Layer.__new__(Layer)
            view.H, view.K, view.dim, view.fp8, view._rows = H, K, dim, fp8, {}
            view.host, view.table = pools[l].cpu().numpy(), host_tables[l]
            view.check(qr[l], out[l], lse[l], pos, starts, window, sinks, 1 / math.sqrt(dim), tokens=set(some))
            assert (out[l, n:] == 7.0).all()
        lengths = [0 if f < 0 else c + f for c, f in zip(lengths, news)]
    assert all(int(o.status.item()) == 0 for o in [plan] + ins + att)
