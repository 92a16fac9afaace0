"""Refusals of the group-scaled cache's entry points and of prompt attention, on
the host before any device call, and pins of their oracle (no GPU needed)."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

from compressed_sparse_long_c4a_gb300 import dense as D
from oracle import dense as OD
from oracle import dense_group as OG
from oracle import formats as F
from tests.test_dense_host import BAD_CACHES, INVALID, UNSUPPORTED, WORKSPACE, _attn, _cache, _insert, lib  # noqa: F401

GROUP_BYTES = 2 * 2 * 256 * 128 + 64
GROUP_CACHES = [c for c in BAD_CACHES if "block_bytes" not in c[0]] + [(dict(block_bytes=GROUP_BYTES - 16), INVALID), (dict(block_bytes=GROUP_BYTES + 8), INVALID)]


def _group(**kw):
    return _cache(**{"format": 3, **kw})


def test_block_bytes(lib):  # noqa: F811
    assert D.block_bytes(8, 128, D.KV_FP8_GROUP) == 2 * 8 * 256 * 128 + 8 * 32 == OG.block_bytes(8, 128)
    for kv, dim, fmt in ((0, 128, 3), (1025, 128, 3), (8, 96, 3), (8, 128, 4)):
        assert D.block_bytes(kv, dim, fmt) == 0
    assert all(D.block_bytes(k, d, 3) % 16 == 0 for k in (1, 3, 1024) for d in (64, 128, 192, 256))


def test_plain_insert_refuses_groups(lib):  # noqa: F811
    assert lib.v4a_dense_insert(C.byref(_insert(_group())), None) == UNSUPPORTED


@pytest.mark.parametrize("kw,code", GROUP_CACHES)
def test_group_caches_are_checked(lib, kw, code):  # noqa: F811
    assert lib.v4a_dense_insert_rows(C.byref(_insert(_group(**kw))), 0x700, 256, None) == code
    assert lib.v4a_dense_attn(C.byref(_attn(_group(**kw))), 0x1000, 1 << 30, None) == code
    assert lib.v4a_dense_read(C.byref(_read(_group(**kw))), None) == code


@pytest.mark.parametrize("fmt", [0, 1, 3])
@pytest.mark.parametrize("k_out,stride", [(None, 256), (0x708, 256), (0x700, 255), (0x700, 260), (0x700, 248), (0x300, 264)])
def test_insert_rows_refuses_rows(lib, fmt, k_out, stride):  # noqa: F811
    assert lib.v4a_dense_insert_rows(C.byref(_insert(_cache(format=fmt))), k_out, stride, None) == INVALID


@pytest.mark.parametrize("kw,code", [(dict(num_tokens=-1), INVALID), (dict(num_heads=3), INVALID), (dict(v=None), INVALID), (dict(v_stride=248), INVALID),
                                     (dict(slots=None), INVALID), (dict(eps=-1.0), INVALID), (dict(num_heads=1026), UNSUPPORTED)])
def test_insert_rows_refuses_arguments(lib, kw, code):  # noqa: F811
    assert lib.v4a_dense_insert_rows(C.byref(_insert(_group(), **kw)), 0x700, 256, None) == code
    assert lib.v4a_dense_insert_rows(C.byref(_insert(_group(), num_tokens=0)), None, 0, None) == 0


def test_attention_refuses_wide_blocks(lib):  # noqa: F811
    assert lib.v4a_dense_attn(C.byref(_attn(_group(block_bytes=1 << 40))), 0x1000, 1 << 30, None) == UNSUPPORTED


def _read(cache=None, **kw):
    f = dict(num_rows=5, num_seqs=3, row_starts=0x10, first=0x20, kv=cache or _group(), k=0x100, k_stride=256, v=0x200, v_stride=256, status=None)
    f.update(kw)
    return D.ReadArgs(*[f[n] for n, _ in D.ReadArgs._fields_])


@pytest.mark.parametrize("kw,code", [
    (dict(num_rows=-1), INVALID), (dict(num_seqs=-1), INVALID), (dict(row_starts=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(k=0x108), INVALID), (dict(v=0x202), INVALID), (dict(k_stride=248), INVALID), (dict(v_stride=260), INVALID),
    (dict(kv=_group(block_table=None)), INVALID), (dict(kv=_group(max_blocks=0)), INVALID), (dict(kv=_group(max_blocks=(1 << 22) + 1)), UNSUPPORTED),
    (dict(num_rows=0, k=None), 0), (dict(num_seqs=0, k=None), 0)])
def test_read_refuses(lib, kw, code):  # noqa: F811
    assert lib.v4a_dense_read(C.byref(_read(**kw)), None) == code
    assert lib.v4a_dense_read(None, None) == INVALID


def _prompt(**kw):
    f = dict(num_tokens=5, num_kv_tokens=9, num_seqs=3, max_new_per_seq=2, token_starts=0x10, kv_starts=0x20, num_heads=8, num_kv_heads=2, dim=128,
             causal=1, window=0, sinks=0, softmax_scale=0.1, q=0x100, q_stride=1024, k=0x200, k_stride=256, v=0x300, v_stride=256, out=0x400,
             lse=None, status=None)
    f.update(kw)
    return D.PromptArgs(*[f[n] for n, _ in D.PromptArgs._fields_])


@pytest.mark.parametrize("kw,code", [
    (dict(num_tokens=-1), INVALID), (dict(num_kv_tokens=-1), INVALID), (dict(num_seqs=-1), INVALID), (dict(max_new_per_seq=0), INVALID),
    (dict(num_heads=0), INVALID), (dict(num_kv_heads=0), INVALID), (dict(num_heads=7), INVALID), (dict(num_heads=1026), UNSUPPORTED),
    (dict(dim=96), UNSUPPORTED), (dict(dim=512), UNSUPPORTED), (dict(causal=2), INVALID), (dict(causal=-1), INVALID),
    (dict(causal=0, window=5), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(max_new_per_seq=(1 << 22) + 1), UNSUPPORTED),
    (dict(num_kv_tokens=(1 << 30) + 1), UNSUPPORTED), (dict(num_heads=1024, max_new_per_seq=1 << 22), UNSUPPORTED)])
def test_prompt_refuses_shapes(lib, kw, code):  # noqa: F811
    a = _prompt(**kw)
    assert lib.v4a_prompt_attn_workspace_size(C.byref(a)) == 0
    assert lib.v4a_prompt_attn(C.byref(a), 0x1000, 1 << 30, None) == code


@pytest.mark.parametrize("kw", [
    dict(token_starts=None), dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(q=0x108), dict(k=0x208), dict(v=0x302), dict(out=0x408),
    dict(out=0x100), dict(q_stride=1016), dict(q_stride=1028), dict(k_stride=248), dict(v_stride=260), dict(k_stride=1 << 38),
    dict(softmax_scale=0.0), dict(softmax_scale=math.nan), dict(softmax_scale=math.inf), dict(softmax_scale=3e38)])
def test_prompt_refuses_arguments(lib, kw):  # noqa: F811
    assert lib.v4a_prompt_attn(C.byref(_prompt(**kw)), 0x1000, 1 << 30, None) == INVALID


def test_prompt_refuses_workspaces_and_grids(lib):  # noqa: F811
    need = lib.v4a_prompt_attn_workspace_size(C.byref(_prompt()))
    assert need > 0
    for ws, n in ((None, need), (0x1000, need - 1), (0x1004, need)):
        assert lib.v4a_prompt_attn(C.byref(_prompt()), ws, n, None) == WORKSPACE
    assert lib.v4a_prompt_attn(None, 0x1000, need, None) == INVALID
    assert lib.v4a_prompt_attn(C.byref(_prompt(num_tokens=0, q=None, out=None)), None, 0, None) == 0
    assert lib.v4a_prompt_attn(C.byref(_prompt(num_seqs=0, q=None, out=None)), None, 0, None) == 0
    a = _prompt(num_heads=1024, num_kv_heads=1024, num_seqs=1 << 22, num_tokens=1 << 22, q_stride=1 << 17, k_stride=1 << 17, v_stride=1 << 17)
    assert lib.v4a_prompt_attn(C.byref(a), 0x1000, 1 << 40, None) == UNSUPPORTED


def test_binding_refuses(lib):  # noqa: F811
    pool = torch.zeros((3, D.block_bytes(2, 64, 3)), dtype=torch.uint8)
    c = D.DenseCache(pool, torch.zeros((1, 3), dtype=torch.int32), 2, 64, D.KV_FP8_GROUP)
    with pytest.raises(ValueError):
        D.DenseCache(pool[:, :-16].contiguous(), None, 2, 64, D.KV_FP8_GROUP)
    op = D.DenseInsert(c, 4, D.Rope(64))
    x = torch.zeros((5, 8, 64), dtype=torch.bfloat16)
    pos, slots, qo = torch.zeros(5, dtype=torch.int32), torch.zeros(5, dtype=torch.int64), torch.zeros((5, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="k_out"):
        op.run(x[:, :4], x[:, 4:6], x[:, 6:], qo, pos, slots)
    for bad in (qo, qo[:, :2].float(), qo[:4, :2], x[:, ::4]):
        with pytest.raises(ValueError, match="k_out"):
            op.run(x[:, :4], x[:, 4:6], x[:, 6:], qo, pos, slots, k_out=bad)
    with pytest.raises(ValueError):
        D.DenseRead(D.DenseCache(pool, None, 2, 64, D.KV_FP8_GROUP))
    read, two = D.DenseRead(c), torch.zeros(2, dtype=torch.int32)
    k = torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    for args in ((two, k, k[:4]), (two, None, k), (two[:1], k, k), (two.long(), k, k), (None, k, k), (two, k, k, two), (two, k, k.float())):
        with pytest.raises(ValueError):
            read.run(*args)
    for args in ((4, 3, 64, 1, 8, 8), (4, 2, 96, 1, 8, 8), (4, 2, 64, -1, 8, 8), (4, 2, 64, 1, 8, 0)):
        with pytest.raises(ValueError):
            D.PromptAttention(*args, device="cpu")
    with pytest.raises(ValueError):
        D.PromptAttention(4, 2, 64, 1, 8, 8, causal=False, window=3, device="cpu")
    pro = D.PromptAttention(4, 2, 64, 1, 8, 8, device="cpu")
    q = torch.zeros((5, 4, 64), dtype=torch.bfloat16)
    for args in ((None, k, k, q, two), (q, None, k, q, two), (q, k, k[:4], q, two), (q, k, k, q[:4], two), (q, k, k, q, pos), (q, k, k, q, two, pos),
                 (q, k, k, q, two, two, q), (torch.zeros((9, 4, 64), dtype=torch.bfloat16), k, k, q, two), (q, k, k, q.clone(), two)):
        with pytest.raises(ValueError):
            pro.run(*args)


# ---- the oracle, by hand -------------------------------------------------------------

def test_pow2():
    for a, s in ((448.0, 1.0), (449.0, 2.0), (896.0, 2.0), (1.75, 2.0 ** -8), (1.7578125, 2.0 ** -7), (0.0, OG.LEAST), (3e38, 2.0 ** 120), (1e-40, OG.LEAST)):
        assert OG.pow2(a) == s


def test_insert_by_hand():
    """A group of one head: 1.0 at row 0; then 512 at row 1 grows the scale from 2^-8 to 2 and 1.0 becomes code 0.5."""
    pool = np.zeros((1, OG.block_bytes(1, 64)), np.uint8)
    one, big = np.full((1, 1, 64), 1.0), np.full((1, 1, 64), 512.0)
    OG.insert(pool, 1, 64, [0], (one, one))
    assert OG.read_scale(pool[0], 1, 64, 0, 0, 0) == 2.0 ** -8 and (F.e4m3_decode(pool[0][:64]) == 256.0).all()
    OG.insert(pool, 1, 64, [1], (one, big))
    assert (OG.read_row(pool, 1, 64, 0, 1, 0, 0) == 1.0).all() and (OG.read_row(pool, 1, 64, 0, 1, 0, 1) == 512.0).all()
    assert OG.read_scale(pool[0], 1, 64, 1, 0, 1) == 2.0 and OG.read_scale(pool[0], 1, 64, 0, 0, 1) == 2.0 ** -8
    OG.insert(pool, 1, 64, [64, 0], (np.concatenate([big, one]),) * 2)            # row 0 begins the group anew
    assert OG.read_scale(pool[0], 1, 64, 1, 0, 0) == 2.0 ** -8 and OG.read_scale(pool[0], 1, 64, 1, 0, 64) == 2.0


def test_prompt_visibility():
    assert OG.prompt_visible(2, 5, 0, True, 0, 0) == [0, 1, 2, 3] and OG.prompt_visible(2, 5, 1, True, 2, 1) == [0, 3, 4]
    assert OG.prompt_visible(3, 1, 0, True, 0, 0) == [] and OG.prompt_visible(3, 1, 2, True, 0, 0) == [0] and OG.prompt_visible(3, 1, 0, False, 0, 0) == [0]
    for m in range(9):           # a whole prompt's queries see what cached ones do
        assert OG.prompt_visible(9, 9, m, True, 3, 2) == OD.visible(m, 3, 2)
