"""The dense-layer entry points refuse bad arguments on the host, before any
device call; the binding refuses tensors that do not fit (no GPU needed)."""
import ctypes as C
import math
import os

import pytest
import torch

from compressed_sparse_long_c4a_gb300 import dense as D
from compressed_sparse_long_c4a_gb300 import pages as P
from compressed_sparse_long_c4a_gb300 import v4a

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(v4a.LIB_PATH):
        from compressed_sparse_long_c4a_gb300 import build
        build.build()
    return D.lib()


def test_block_bytes(lib):
    assert D.block_bytes(8, 128, D.KV_BF16) == 2 * 8 * 256 * 256
    assert D.block_bytes(8, 128, D.KV_FP8_TOKEN) == 2 * 8 * 256 * 132
    for kv, dim, fmt in ((0, 128, 0), (1025, 128, 0), (8, 96, 0), (8, 32, 0), (8, 320, 0), (8, 128, 2), (8, 128, -1)):
        assert D.block_bytes(kv, dim, fmt) == 0


def test_block_is_a_page_kind(lib):
    """A dense cache beside a compressed one in the page allocator: one page per 256-position block and layer."""
    dense, c4a = D.block_bytes(2, 64, D.KV_BF16), 33024
    a = P.PageAllocator([P.block_kind(dense, 3), P.block_kind(c4a, 2)], 2, 8, budget_bytes=100 << 20)
    a.open(0)
    a.reserve(0, 257)
    t = [a.table(0, l)[0, :2].tolist() for l in range(3)]
    assert len({p for row in t for p in row}) == 6 and min(min(r) for r in t) >= 0
    assert {b.page_bytes for b in a.buckets()} == {dense, c4a}


def _plan(**kw):
    f = dict(num_seqs=4, num_tables=2, max_tokens=8, max_blocks=3, cached=0x10, fresh=0x20, block_table=0x30, table_stride=12,
             num_blocks=50, free_ring=0x40, ring_cap=64, free_in=0x50, free_out=0x60, seq_ids=0x70, positions=0x80, slots=0x90,
             token_starts=0xa0, status=None)
    f.update(kw)
    return D.PlanArgs(*[f[n] for n, _ in D.PlanArgs._fields_])


@pytest.mark.parametrize("kw,code", [
    (dict(num_seqs=-1), INVALID), (dict(num_seqs=8193, table_stride=1 << 20), UNSUPPORTED), (dict(num_tables=0), INVALID),
    (dict(num_tables=4097), UNSUPPORTED), (dict(max_tokens=-1), INVALID), (dict(max_blocks=0), INVALID),
    (dict(max_blocks=(1 << 22) + 1, table_stride=1 << 40), UNSUPPORTED), (dict(table_stride=11), INVALID),
    (dict(ring_cap=0), INVALID), (dict(ring_cap=(1 << 30) + 1), UNSUPPORTED), (dict(num_blocks=0), INVALID)])
def test_plan_refuses_shapes(lib, kw, code):
    a = _plan(**kw)
    assert lib.v4a_plan_workspace_size(C.byref(a)) == 0
    assert lib.v4a_step_plan(C.byref(a), 0x1000, 1 << 20, None) == code


@pytest.mark.parametrize("name", ["cached", "fresh", "block_table", "free_ring", "free_in", "free_out", "seq_ids", "positions", "token_starts"])
def test_plan_refuses_null(lib, name):
    a = _plan(**{name: None})
    assert lib.v4a_step_plan(C.byref(a), 0x1000, 1 << 20, None) == INVALID


def test_plan_refuses_workspaces(lib):
    a = _plan()
    need = lib.v4a_plan_workspace_size(C.byref(a))
    assert need > 0
    for ws, n in ((None, need), (0x1000, need - 1), (0x1008, need)):
        assert lib.v4a_step_plan(C.byref(a), ws, n, None) == WORKSPACE
    assert lib.v4a_step_plan(None, 0x1000, need, None) == INVALID


def _cache(**kw):
    f = dict(num_kv_heads=2, dim=128, format=0, pool=0x1000, num_blocks=9, block_bytes=0, block_table=0x2000, max_blocks=4)
    f.update(kw)
    return D.CacheArgs(*[f[n] for n, _ in D.CacheArgs._fields_])


BAD_CACHES = [(dict(num_kv_heads=0), INVALID), (dict(dim=96), UNSUPPORTED), (dict(dim=512), UNSUPPORTED), (dict(format=2), UNSUPPORTED),
              (dict(pool=None), INVALID), (dict(pool=0x1008), INVALID), (dict(num_blocks=0), INVALID),
              (dict(num_blocks=1 << 31), UNSUPPORTED), (dict(block_bytes=2 * 2 * 256 * 256 - 16), INVALID),
              (dict(block_bytes=2 * 2 * 256 * 256 + 8), INVALID)]


def _insert(cache=None, rope=None, **kw):
    f = dict(num_tokens=5, positions=0x10, slots=0x20, num_heads=4, q=0x100, q_stride=512, q_out=0x200, q_out_stride=512, k=0x300,
             k_stride=256, v=0x400, v_stride=256, q_gamma=0x500, k_gamma=0x600, eps=1e-6, rope=(rope or D.Rope(64)).struct(),
             kv=cache or _cache(), status=None)
    f.update(kw)
    return D.InsertArgs(*[f[n] for n, _ in D.InsertArgs._fields_])


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_insert_refuses_caches(lib, kw, code):
    assert lib.v4a_dense_insert(C.byref(_insert(_cache(**kw))), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(num_tokens=-1), INVALID), (dict(num_heads=3), INVALID), (dict(num_heads=-2), INVALID), (dict(num_heads=1026), UNSUPPORTED),
    (dict(positions=None), INVALID), (dict(slots=None), INVALID), (dict(q=None), INVALID), (dict(q_out=None), INVALID),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(q=0x108), INVALID), (dict(q_out=0x208), INVALID), (dict(k=0x308), INVALID),
    (dict(v=0x402), INVALID), (dict(q_gamma=0x504), INVALID), (dict(k_gamma=0x608), INVALID), (dict(q_stride=511), INVALID),
    (dict(q_stride=516), INVALID), (dict(q_out_stride=508), INVALID), (dict(k_stride=255), INVALID), (dict(k_stride=260), INVALID),
    (dict(v_stride=248), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(q_out=0x100, q_out_stride=520), INVALID)])
def test_insert_refuses_arguments(lib, kw, code):
    assert lib.v4a_dense_insert(C.byref(_insert(**kw)), None) == code


@pytest.mark.parametrize("rope", [
    dict(dims=8), dict(dims=-16), dict(dims=272), dict(dims=64, first=4), dict(dims=128, first=8), dict(dims=64, first=-8),
    dict(dims=64, layout=2), dict(dims=64, scaling=4), dict(dims=64, theta=0.0), dict(dims=64, theta=-1.0),
    dict(dims=64, scaling=D.ROPE_LINEAR, factor=0.0), dict(dims=64, scaling=D.ROPE_LINEAR, factor=1e-3),
    dict(dims=64, scaling=D.ROPE_YARN, factor=4.0), dict(dims=64, scaling=D.ROPE_YARN, factor=4.0, original=100.0, beta_fast=1.0),
    dict(dims=64, scaling=D.ROPE_TABLE), dict(dims=16, scaling=D.ROPE_TABLE, table=[4.0] + [1.0] * 7),
    dict(dims=16, scaling=D.ROPE_TABLE, table=[-0.1] + [1.0] * 7), dict(dims=16, scaling=D.ROPE_TABLE, table=[math.nan] + [1.0] * 7),
    dict(dims=64, magnitude=math.inf)])
def test_insert_refuses_rotations(lib, rope):
    assert lib.v4a_dense_insert(C.byref(_insert(rope=D.Rope(**rope))), None) == INVALID


def test_insert_of_no_tokens(lib):
    assert lib.v4a_dense_insert(C.byref(_insert(num_tokens=0, k=None, v=None, q=None, q_out=None, positions=None, slots=None)), None) == 0


def _attn(cache=None, **kw):
    f = dict(num_tokens=5, num_seqs=3, max_new_per_seq=2, positions=0x10, token_starts=0x20, kv=cache or _cache(), num_heads=8, q=0x100,
             softmax_scale=0.1, window=0, sinks=0, out=0x200, lse=None, status=None)
    f.update(kw)
    return D.AttnArgs(*[f[n] for n, _ in D.AttnArgs._fields_])


@pytest.mark.parametrize("kw,code", BAD_CACHES + [(dict(block_table=None), INVALID), (dict(max_blocks=0), INVALID),
                                                  (dict(max_blocks=(1 << 22) + 1), UNSUPPORTED)])
def test_attention_refuses_caches(lib, kw, code):
    assert lib.v4a_dense_attn(C.byref(_attn(_cache(**kw))), 0x1000, 1 << 30, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(num_tokens=-1), INVALID), (dict(num_seqs=-1), INVALID), (dict(max_new_per_seq=0), INVALID), (dict(num_heads=0), INVALID),
    (dict(num_heads=7), INVALID), (dict(num_heads=1026), UNSUPPORTED), (dict(positions=None), INVALID), (dict(token_starts=None), INVALID),
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(q=0x108), INVALID), (dict(out=0x208), INVALID), (dict(out=0x100), INVALID),
    (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(softmax_scale=0.0), INVALID), (dict(softmax_scale=math.nan), INVALID),
    (dict(softmax_scale=math.inf), INVALID), (dict(softmax_scale=3e38), INVALID), (dict(max_new_per_seq=(1 << 22) + 1), UNSUPPORTED),
    (dict(num_heads=1024, max_new_per_seq=1 << 22), UNSUPPORTED)])
def test_attention_refuses_arguments(lib, kw, code):
    assert lib.v4a_dense_attn(C.byref(_attn(**kw)), 0x1000, 1 << 30, None) == code


@pytest.mark.parametrize("num_seqs,num_tokens", [(1 << 22, 1 << 22), (1 << 21, 100 << 21), (1 << 21, 99 << 21)])
def test_attention_refuses_grids_before_any_launch(lib, num_seqs, num_tokens):
    """More (unit, KV head) pairs than a grid holds, in the first, the only and the second launch of the call."""
    a = _attn(_cache(num_kv_heads=1024), num_heads=1024, num_seqs=num_seqs, num_tokens=num_tokens, max_new_per_seq=100)
    assert lib.v4a_dense_attn(C.byref(a), 0x1000, 1 << 40, None) == UNSUPPORTED


def test_attention_refuses_workspaces(lib):
    a = _attn()
    need = lib.v4a_dense_attn_workspace_size(C.byref(a))
    assert need > 0
    for ws, n in ((None, need), (0x1000, need - 1), (0x1004, need)):
        assert lib.v4a_dense_attn(C.byref(a), ws, n, None) == WORKSPACE
    assert lib.v4a_dense_attn_workspace_size(C.byref(_attn(num_heads=7))) == 0
    # nothing to do: no pointer is read, nothing is launched
    assert lib.v4a_dense_attn(C.byref(_attn(num_tokens=0, q=None, out=None)), None, 0, None) == 0
    assert lib.v4a_dense_attn(C.byref(_attn(num_seqs=0, q=None, out=None)), None, 0, None) == 0


def test_binding_refuses_tensors(lib):
    pool = torch.zeros((3, D.block_bytes(2, 64, 0)), dtype=torch.uint8)
    with pytest.raises(ValueError):
        D.DenseCache(pool[:, :-1], None, 2, 64)                     # not contiguous, too small
    with pytest.raises(ValueError):
        D.DenseCache(pool, torch.zeros((2, 3), dtype=torch.int64), 2, 64)
    with pytest.raises(ValueError):
        D.DenseCache(pool, None, 2, 96)
    c = D.DenseCache(pool, None, 2, 64)
    with pytest.raises(ValueError):
        D.DenseAttention(c, 4, 8)                                   # no block table
    with pytest.raises(ValueError):
        D.DenseInsert(c, 4, D.Rope(64), q_gamma=torch.ones(32))
    with pytest.raises(ValueError):
        D.Rope(16, scaling=D.ROPE_TABLE, table=[1.0]).struct()
    op = D.DenseInsert(c, 4, D.Rope(64))
    x = torch.zeros((5, 8, 64), dtype=torch.bfloat16)
    pos, slots = torch.zeros(5, dtype=torch.int32), torch.zeros(5, dtype=torch.int64)
    for q, k in ((x[:, :4].float(), x[:, 4:6]), (x[:, :3], x[:, 4:6]), (x[:4, :4], x[:, 4:6]), (x[:, ::2], x[:, 4:6])):
        with pytest.raises(ValueError):
            op.run(q, k, x[:, 6:], torch.zeros((5, 4, 64), dtype=torch.bfloat16), pos, slots)
    for pos2, slots2 in ((None, slots), (pos, None), (pos.long(), slots), (pos, slots[:4])):
        with pytest.raises(ValueError):
            op.run(x[:, :4], x[:, 4:6], x[:, 6:], torch.zeros((5, 4, 64), dtype=torch.bfloat16), pos2, slots2)
    with pytest.raises(ValueError):
        op.run(x[:, :4], None, x[:, 6:], None, pos, slots)
    with pytest.raises(ValueError):                                # no CPU path
        op.run(x[:, :4], x[:, 4:6], x[:, 6:], torch.zeros((5, 4, 64), dtype=torch.bfloat16), pos, slots)
    with pytest.raises(ValueError):
        D.StepPlan(torch.zeros((1, 2, 3), dtype=torch.int32), torch.zeros(4, dtype=torch.int64), 4)
    plan = D.StepPlan(torch.zeros((1, 2, 3), dtype=torch.int32), torch.zeros(4, dtype=torch.int32), 4)
    two = torch.zeros(2, dtype=torch.int32)
    for args in ((two, two, None), (two, None, two), (two[:1], two, two), (two.long(), two, two), (two, two, two)):
        with pytest.raises(ValueError):
            plan.run(*args)
    att = D.DenseAttention(D.DenseCache(pool, torch.zeros((1, 3), dtype=torch.int32), 2, 64), 4, 8, 8)
    q = torch.zeros((5, 4, 64), dtype=torch.bfloat16)
    for args in ((None, q, pos, two), (q, None, pos, two), (q, q[:4], pos, two), (q, q.clone(), pos, pos), (q, q.clone(), pos, two, q),
                 (torch.zeros((9, 4, 64), dtype=torch.bfloat16), q, pos, two), (q, q.clone(), pos, two)):
        with pytest.raises(ValueError):
            att.run(*args)


def test_yarn_ramp_over_pair_indices_is_a_table(lib):
    """The ramp that is linear in the pair index agrees with ROPE_YARN at both ends and not between; it goes in as a table."""
    from oracle import dense as OD
    dims, theta, factor, original, fast, slow = 128, 1e4, 16.0, 4096.0, 32.0, 1.0
    index = lambda turns: dims * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
    lo, hi = math.floor(index(fast)), math.ceil(index(slow))
    table = []
    for j in range(dims // 2):
        f, keep = theta ** (-2.0 * j / dims), 1 - min(max((j - lo) / (hi - lo), 0.0), 1.0)
        table.append(f * keep + f / factor * (1 - keep))
    yarn = OD.frequencies(dims, theta, "yarn", factor, original, fast, slow)
    assert table[:lo] == pytest.approx(yarn[:lo], rel=1e-14) and table[hi:] == pytest.approx(yarn[hi:], rel=1e-14)
    assert max(abs(t / y - 1) for t, y in zip(table[lo:hi], yarn[lo:hi])) > 0.3
    for rope in (D.Rope(dims, scaling=D.ROPE_TABLE, table=table),
                 D.Rope(dims, scaling=D.ROPE_YARN, factor=factor, original=original, beta_fast=fast, beta_slow=slow)):
        assert lib.v4a_dense_insert(C.byref(_insert(rope=rope, num_tokens=0)), None) == 0


@pytest.mark.parametrize("magnitude,code", [(1e39, INVALID), (-1e300, INVALID), (math.nan, INVALID), (3.4e38, 0), (-1.0, 0), (0.0, 0)])
def test_rotation_magnitude_is_finite_in_fp32(lib, magnitude, code):
    assert lib.v4a_dense_insert(C.byref(_insert(rope=D.Rope(64, magnitude=magnitude), num_tokens=0)), None) == code


def test_binding_takes_one_token_of_any_stride():
    """A single token's rows out of a wide tensor of odd width: its stride means nothing."""
    x = torch.zeros((3, 1001), dtype=torch.bfloat16)
    for tokens, want in ((1, 256), (0, 256), (3, 1001)):
        rows = x.as_strided((tokens, 4, 64), (1001, 64, 1))          # (a view or an unflatten would give one token a stride of its own)
        assert D._rows(rows, "q", x.device, 4, 64, tokens) == want
