"""Edges of the group-scaled dense caches and of prompt attention on the GPU:
streams, steps without a pause, many sequences, strides past 32 bits, order of
tokens, NaN in single rows.  Tolerances as in test_gpu_group.py."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from oracle import dense_group as OG
from tests.test_gpu_dense import _runs
from tests.test_gpu_group import DEV, I32, GroupLayer, _check_prompt, _dense, _f64, _insert_case, _prompt, _run_prompt, _same_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_mixed_steps_see_what_was_just_inserted(dim):
    """Insert and attention without a pause: rows, codes that a grown scale changed and scales are new at every step; a
    call after a synchronisation gives the same bytes."""
    D = _dense()
    H, K, steps, chunk = 8, 2, 20, 37
    g = torch.Generator(device=DEV).manual_seed(dim)
    table = torch.randperm(12, generator=g, device=DEV).to(torch.int32).view(3, 4)
    pool = torch.full((12, D.block_bytes(K, dim, D.KV_FP8_GROUP)), 0xff, dtype=torch.uint8, device=DEV)      # NaN everywhere
    cache = D.DenseCache(pool, table, K, dim, D.KV_FP8_GROUP)
    T = 2 + chunk
    ins, att = D.DenseInsert(cache, H, D.Rope(dim, layout=1)), D.DenseAttention(cache, H, T, chunk)
    xs = torch.randn((steps, T, H + 2 * K, dim), generator=g, device=DEV)
    xs = (xs * torch.exp2(torch.arange(steps, device=DEV) % 7 - 3.0).view(-1, 1, 1, 1)).to(torch.bfloat16)   # scales grow
    starts = torch.tensor([0, 1, 1 + chunk, T], **I32)
    pos, slots, qr = [], [], torch.empty((steps, T, H, dim), dtype=torch.bfloat16, device=DEV)
    kr = torch.empty((steps, T, K, dim), dtype=torch.bfloat16, device=DEV)
    for s in range(steps):
        p = torch.tensor([s, *range(s * chunk, (s + 1) * chunk), s], **I32)
        b = torch.tensor([0] + [1] * chunk + [2], device=DEV)
        pos.append(p)
        slots.append(table[b, (p // 256).long()].long() * 256 + p % 256)
    out, snaps = torch.zeros_like(qr), []
    torch.cuda.synchronize()
    for s in range(steps):
        ins.run(xs[s, :, :H], xs[s, :, H:H + K], xs[s, :, H + K:], qr[s], pos[s], slots[s], k_out=kr[s])
        att.run(qr[s], out[s], pos[s], starts)
        snaps.append(pool.clone())
    torch.cuda.synchronize()
    assert int(ins.status.item()) == 0 and int(att.status.item()) == 0 and bool(out.isfinite().all())
    again = torch.zeros_like(out)
    want = np.full(tuple(pool.shape), 0xff, np.uint8)
    for s in range(steps):
        pool.copy_(snaps[s])
        torch.cuda.synchronize()
        att.run(qr[s], again[s], pos[s], starts)
        OG.insert(want, K, dim, slots[s].tolist(), (_f64(kr[s]), _f64(xs[s, :, H + K:])))
        assert np.array_equal(want, snaps[s].cpu().numpy()), s
    assert torch.equal(out, again)


@pytest.mark.parametrize("dim", [128, 256])
def test_two_streams_of_mixed_batches(dim):
    """Both forms of two calls in flight at once, beside inserts and reads of another cache."""
    D = _dense()
    runs = [[(900, 1), (200, 150), (40, 3), (0, 300)], [(10, 90), (1500, 2), (0, 0), (33, 200)]]
    layers = [GroupLayer([c + n for c, n in r], 8, 2, dim, seed=40 + i) for i, r in enumerate(runs)]
    ops, args, alone = [], [], []
    for L, r in zip(layers, runs):
        pos, starts = _runs(*zip(*r))
        op = D.DenseAttention(L.cache, 8, len(pos), max(n for _, n in r))
        q = L.query(len(pos))
        out = torch.empty_like(q)
        args.append((q, torch.tensor(pos, **I32), torch.tensor(starts, **I32)))
        op.run(q, out, *args[-1][1:])
        torch.cuda.synchronize()
        ops.append(op)
        alone.append(out)
    third = GroupLayer((500, 300), 8, 2, dim, seed=42)
    x = torch.randn((500, 4, dim), device=DEV).to(torch.bfloat16)
    slots = torch.cat([torch.arange(256, device=DEV) + 256 * int(third.table[0, 0]), torch.arange(244, device=DEV) + 256 * int(third.table[0, 1])])
    ins, read = D.DenseInsert(third.cache, 0, None), D.DenseRead(third.cache)
    ko, rk, rv = (torch.empty((500, 2, dim), dtype=torch.bfloat16, device=DEV) for _ in range(3))
    rs, seq = torch.tensor([0, 500, 500], **I32), torch.arange(500, **I32)
    both = [torch.empty_like(o) for o in alone]
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(20):
        for i in range(2):
            ops[i].run(args[i][0], both[i], *args[i][1:], stream=streams[i])
        ins.run(None, x[:, :2], x[:, 2:], None, seq, slots, stream=streams[2], k_out=ko)
        read.run(rs, rk, rv, stream=streams[2])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(alone[i], both[i]) and int(ops[i].status.item()) == 0
    assert torch.equal(ko, x[:, :2]) and int(ins.status.item()) == 0 and int(read.status.item()) == 0
    for y, got in ((x[:, :2], rk), (x[:, 2:], rv)):      # a code is off by half of its last bit, or of the least step of the group's scale
        err, scale = (got.float() - y.float()).abs(), 2.0 ** -6
        assert (err <= y.float().abs() * 2.0 ** -4 + 2.0 ** -10 * scale).all()


def test_group_tokens_in_any_order():
    """The tokens of several groups, interleaved and backwards within 64 of the call."""
    D = _dense()
    K, dim = 2, 128
    T, pos, slots, q, k, v, pool, g = _insert_case(dim, 2, K, ((0, 20), (70, 20), (200, 24)), seed=3)
    order = torch.randperm(T, generator=g).tolist()
    slots, pos = [slots[i] for i in order], [pos[i] for i in order]
    want = pool.cpu().numpy().copy()
    k_out, q_out = torch.empty((T, K, dim), dtype=torch.bfloat16, device=DEV), torch.empty((T, 2, dim), dtype=torch.bfloat16, device=DEV)
    op = D.DenseInsert(D.DenseCache(pool, None, K, dim, D.KV_FP8_GROUP), 2, D.Rope(64))
    op.run(q, k, v, q_out, torch.tensor(pos, **I32), torch.tensor(slots, device=DEV), k_out=k_out)
    OG.insert(want, K, dim, slots, (_f64(k_out), _f64(v)))
    _same_cache(pool, want, K, dim)


def test_insert_of_one_projection_in_place():
    """Queries and keys rotated where they are; the same cache and rows."""
    D = _dense()
    H, K, dim = 6, 2, 64
    got = []
    for in_place in (False, True):
        T, pos, slots, q, k, v, pool, g = _insert_case(dim, H, K, ((40, 1500), (3, 2)), seed=4)
        q_out = q if in_place else torch.empty((T, H, dim), dtype=torch.bfloat16, device=DEV)
        k_out = k if in_place else torch.empty((T, K, dim), dtype=torch.bfloat16, device=DEV)
        op = D.DenseInsert(D.DenseCache(pool, None, K, dim, D.KV_FP8_GROUP), H, D.Rope(64, layout=1))
        op.run(q, k, v, q_out, torch.tensor(pos, **I32), torch.tensor(slots, device=DEV), k_out=k_out)
        torch.cuda.synchronize()
        got.append((q_out.clone(), k_out.clone(), pool.clone(), v.clone()))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_handles_on_other_streams():
    """First calls on a stream that is not the constructing one; handles dropped with calls queued."""
    D = _dense()
    layer = GroupLayer((700,), 8, 2, 128, seed=6)
    q = layer.query(200)
    pos, st = torch.arange(500, 700, **I32), torch.tensor([0, 200], **I32)
    rows = [torch.empty((700, 2, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    want, out, pout = (torch.zeros_like(q) for _ in range(3))
    lse = torch.zeros((200, 8), device=DEV)
    D.DenseAttention(layer.cache, 8, 200, 200).run(q, want, pos, st)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    rs, kv = torch.tensor([0, 700], **I32), torch.tensor([0, 700], **I32)
    torch.cuda.synchronize()
    for _ in range(5):
        D.DenseAttention(layer.cache, 8, 200, 200).run(q, out, pos, st, stream=s)
        D.DenseRead(layer.cache).run(rs, *rows, stream=s)
        D.PromptAttention(8, 2, 128, 1, 200, 200).run(q, *rows, pout, st, kv, lse=lse, stream=s)
        junk = [torch.full((1 << 20,), 0xff, dtype=torch.uint8, device=DEV) for _ in range(8)]
    torch.cuda.synchronize()
    del junk
    assert torch.equal(out, want)
    _check_prompt([0, 200], [0, 700], q, *rows, pout, lse, True, 0, 0, 1 / math.sqrt(128), {0, 99, 199})


@pytest.mark.parametrize("B", [900, 1100])
def test_prompts_of_many_sequences(B):
    """Many sequences, some of them empty."""
    g = torch.Generator().manual_seed(B)
    runs = [(int(c), int(n)) for c, n in zip(torch.randint(0, 40, (B,), generator=g), torch.randint(0, 90, (B,), generator=g))]
    starts, kv, q, k, v = _prompt(runs, 4, 2, 64, seed=B)
    op, out, lse = _run_prompt(starts, kv, q, k, v)
    assert int(op.status.item()) == 0
    _check_prompt(starts, kv, q, k, v, out, lse, True, 0, 0, op.args.softmax_scale, set(range(0, starts[-1], 397)))
    assert (out[starts[-1]:] == 7.0).all()


@pytest.mark.parametrize("B,H,K,window,long", [
    (4096, 2, 1, 0, 900),          # the most sequences that are dealt out, lengths of several tiles each
    (4097, 2, 1, 0, 900),
    (1000, 64, 64, 0, 0),          # more units a CTA than its list in shared memory holds
    (300, 16, 2, 0, 5000), (40, 16, 2, 700, 6000), (40, 12, 4, 0, 3000),
])
@pytest.mark.parametrize("causal", [True, False])
def test_dealt_units_of_ragged_batches(B, H, K, window, long, causal):
    """Every row is written once and by its own unit, whatever the order in which units are dealt out."""
    if window and not causal:
        pytest.skip("a window is causal")
    g = torch.Generator().manual_seed(B + H)
    few = 4 if B > 900 else 60
    runs = [[int(c), int(n)] for c, n in zip(torch.randint(-2, 40, (B,), generator=g), torch.randint(0, few, (B,), generator=g))]
    runs = [[max(c, -n), n] for c, n in runs]
    if long:                       # some long ones among them: all queries, a prefix, both
        runs[B // 3], runs[B // 2], runs[-1] = [0, long // 3], [long, 3], [long // 2, long // 2]
    starts, kv, q, k, v = _prompt(runs, H, K, 64, seed=B)
    op, out, lse = _run_prompt(starts, kv, q, k, v, causal=causal, window=window, sinks=window // 9)
    assert int(op.status.item()) == 0 and (out[starts[-1]:] == 7.0).all() and (lse[starts[-1]:] == 7.0).all()
    assert not (lse[:starts[-1]] == 7.0).any() and out[:starts[-1]].isfinite().all()
    tokens = set(range(0, starts[-1], max(1, starts[-1] * H // 4000)))
    _check_prompt(starts, kv, q, k, v, out, lse, causal, window, window // 9, op.args.softmax_scale, tokens)
    again = _run_prompt(starts, kv, q, k, v, causal=causal, window=window, sinks=window // 9)
    assert torch.equal(out, again[1]) and torch.equal(lse, again[2])


@pytest.mark.parametrize("B", [41, 601, 1101])
@pytest.mark.parametrize("dim", [64, 192])
def test_sequences_that_share_queries_are_reported(B, dim):
    """Entries that go back: more rows than the call has room for; nothing is read or written out of range."""
    D = _dense()
    q = torch.zeros((300, 4, dim), dtype=torch.bfloat16, device=DEV)
    k = torch.zeros((300, 2, dim), dtype=torch.bfloat16, device=DEV)
    starts = torch.tensor([0, 300] * (B // 2) + [0] * (B % 2) + [300], **I32)
    op = D.PromptAttention(4, 2, dim, B, 300, 300)
    op.run(q, k, k, torch.empty_like(q), starts, torch.zeros(B + 1, **I32))
    torch.cuda.synchronize()
    assert int(op.status.item()) & 2


def test_strides_past_four_gigabytes():
    """Rows of queries, keys and values (and of the read back) that lie 64 M elements apart."""
    D = _dense()
    stride, T, dim = (1 << 26) + 8, 40, 128
    big = torch.zeros(T * stride, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator().manual_seed(12)
    view = lambda at, heads: big.as_strided((T, heads, dim), (stride, dim, 1), at)  # noqa: E731
    q, k, v = view(0, 4), view(1024, 2), view(2048, 2)
    for x in (q, k, v):
        x.copy_(torch.randn(x.shape, generator=g).to(torch.bfloat16))
    st = [0, 13, 40]
    op, out, lse = _run_prompt(st, st, q, k, v)
    _check_prompt(st, st, q, k, v, out, lse, True, 0, 0, op.args.softmax_scale)
    q3 = big.as_strided((T, 6, dim), (stride, dim, 1), 0)          # a group of three: rows copied one by one
    op, out, lse = _run_prompt(st, st, q3, k, v)
    _check_prompt(st, st, q3, k, v, out, lse, True, 0, 0, op.args.softmax_scale)
    layer = GroupLayer((40,), 4, 2, dim, seed=13)
    rk, rv = view(4096, 2), view(8192, 2)
    D.DenseRead(layer.cache).run(torch.tensor([0, 40], **I32), rk, rv)
    for t in (0, 33, 39):
        assert np.array_equal(_f64(rk[t, 1]), layer.rows(0, 0, 1, 40)[t]) and np.array_equal(_f64(rv[t, 0]), layer.rows(0, 1, 0, 40)[t])
    pool = torch.zeros((1, OG.block_bytes(2, dim)), dtype=torch.uint8, device=DEV)
    want = pool.cpu().numpy().copy()
    D.DenseInsert(D.DenseCache(pool, None, 2, dim, D.KV_FP8_GROUP), 0, None).run(
        None, k, v, None, torch.arange(T, **I32), torch.arange(T, device=DEV), k_out=rk)
    OG.insert(want, 2, dim, list(range(T)), (_f64(k), _f64(v)))
    _same_cache(pool, want, 2, dim)
    del big
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_nan_query_stays_in_its_row(dim):
    starts, kv, q, k, v = _prompt(((0, 300),), 4, 2, dim, seed=14, pad=0)
    _, want, _ = _run_prompt(starts, kv, q, k, v)
    q[77, 2, 5] = math.nan
    _, out, lse = _run_prompt(starts, kv, q, k, v)
    assert out[77, 2].isnan().all() and lse[77, 2].isnan()
    out[77, 2] = want[77, 2]
    assert torch.equal(out, want)
    layer = GroupLayer((400,), 4, 2, dim, seed=15)
    pos, st = torch.arange(100, 400, **I32), torch.tensor([0, 300], **I32)
    q = layer.query(300)
    outs = []
    for _ in range(2):
        out = torch.empty_like(q)
        _dense().DenseAttention(layer.cache, 4, 300, 300).run(q, out, pos, st)
        outs.append(out)
        q[77, 2, 5] = math.nan
    torch.cuda.synchronize()
    assert outs[1][77, 2].isnan().all()
    outs[1][77, 2] = outs[0][77, 2]
    assert torch.equal(*outs)


@pytest.mark.parametrize("new", [1, 300])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_infinite_query_is_not_made_finite(dim, new):
    """Infinite logits of both signs have no softmax: the row is NaN, the others keep their results."""
    layer = GroupLayer((400,), 4, 2, dim, seed=16)
    pos, st = torch.arange(400 - new, 400, **I32), torch.tensor([0, new], **I32)
    q = layer.query(new)
    at, outs, lses = new // 2, [], []
    for _ in range(2):
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
        _dense().DenseAttention(layer.cache, 4, new, new).run(q, out, pos, st, lse=lse)
        outs.append(out)
        lses.append(lse)
        q[at, 2, 5] = math.inf
    torch.cuda.synchronize()
    assert outs[0].isfinite().all() and outs[1][at, 2].isnan().all() and lses[1][at, 2].isnan()
    for x, y in (outs, lses):
        y[at, 2] = x[at, 2]
        assert torch.equal(x, y)


@pytest.mark.parametrize("form", ["prompt", "chunk"])
@pytest.mark.parametrize("dim", [64, 256])
def test_logits_past_fp32_give_nan(dim, form):
    """Scores of 2^126 with a softmax scale of 8: the row is NaN, never zeros, and the others keep their results."""
    starts, kv, q, k, v = _prompt(((0, 300),), 4, 2, dim, seed=17, pad=0)
    k, v = k[1:301].contiguous(), v[1:301].contiguous()
    k[:, 1, 5] = 2.0 ** 62
    outs = []
    if form == "chunk":
        D = _dense()
        pool = torch.zeros((2, OG.block_bytes(2, dim)), dtype=torch.uint8, device=DEV)
        cache = D.DenseCache(pool, torch.tensor([[0, 1]], **I32), 2, dim, D.KV_FP8_GROUP)
        pos = torch.arange(300, **I32)
        D.DenseInsert(cache, 0, None).run(None, k, v, None, pos, torch.arange(300, device=DEV), k_out=torch.empty_like(k))
    q[:, 2:, 5] = 0
    for _ in range(2):
        if form == "prompt":
            out, lse = _run_prompt(starts, None, q, k, v, scale=8.0)[1:]
        else:
            x = q.contiguous()
            out, lse = torch.empty_like(x), torch.empty(x.shape[:2], device=DEV)
            D.DenseAttention(cache, 4, 300, 300, scale=8.0).run(x, out, pos, torch.tensor([0, 300], **I32), lse=lse)
            torch.cuda.synchronize()
        outs.append((out, lse))
        q[77, 2] = 0
        q[77, 2, 5] = 2.0 ** 64
    assert outs[0][0].isfinite().all() and outs[1][0][77, 2].isnan().all() and outs[1][1][77, 2].isnan()
    for x, y in zip(*outs):
        y[77, 2] = x[77, 2]
        assert torch.equal(x, y)


@pytest.mark.parametrize("new", [1, 60])
def test_nan_code_reaches_the_queries_that_see_it(new):
    """A NaN that was inserted comes out, also where the scale is finite."""
    D = _dense()
    pool = torch.zeros((1, OG.block_bytes(1, 64)), dtype=torch.uint8, device=DEV)
    x = torch.ones((100, 1, 64), dtype=torch.bfloat16, device=DEV)
    x[30, 0, 7] = math.nan
    cache = D.DenseCache(pool, torch.zeros((1, 1), **I32), 1, 64, D.KV_FP8_GROUP)
    D.DenseInsert(cache, 0, None).run(None, x, x, None, torch.arange(100, **I32), torch.arange(100, device=DEV), k_out=torch.empty_like(x))
    q = torch.ones((new, 1, 64), dtype=torch.bfloat16, device=DEV)
    for last, seen in ((100, True), (30, False)):
        out = torch.zeros_like(q)
        n = min(new, last)
        D.DenseAttention(cache, 1, n, n).run(q[:n], out[:n], torch.arange(last - n, last, **I32), torch.tensor([0, n], **I32))
        torch.cuda.synchronize()
        if seen:
            assert out[n - 1].isnan().all()
        else:
            assert bool(out[:n].isfinite().all()) and bool((out[:n] == 1).all())


@pytest.mark.parametrize("grow", [0.02, 0.1, 1.0])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_logits_that_grow_along_the_keys(dim, grow):
    """Later keys' logits pass the earlier ones' by little and by much: the running maximum lags, and is raised."""
    starts, kv, q, k, v = _prompt(((0, 700), (500, 60)), 8, 2, dim, seed=18)
    k.mul_((1 + grow * torch.arange(k.shape[0], device=DEV)).view(-1, 1, 1).to(torch.bfloat16))
    for window, sinks in ((0, 0), (300, 40)):
        op, out, lse = _run_prompt(starts, kv, q, k, v, window=window, sinks=sinks)
        assert int(op.status.item()) == 0
        _check_prompt(starts, kv, q, k, v, out, lse, True, window, sinks, op.args.softmax_scale, set(range(0, starts[-1], 23)))


@pytest.mark.parametrize("H,K,dim", [(128, 1, 64), (256, 2, 128), (96, 1, 128), (1024, 1024, 64), (5, 5, 256)])
def test_prompts_of_odd_head_counts(H, K, dim):
    starts, kv, q, k, v = _prompt(((0, 50), (20, 9), (0, 1)), H, K, dim, seed=H)
    op, out, lse = _run_prompt(starts, kv, q, k, v)
    assert int(op.status.item()) == 0
    _check_prompt(starts, kv, q, k, v, out, lse, True, 0, 0, op.args.softmax_scale, {0, 31, 49, 50, 58, 59} if H < 1000 else {49, 58})
    assert (out[starts[-1]:] == 7.0).all()
