"""fp8 rows whose largest element is near the smallest fp32 numbers: the
library is built with fast math, which flushes subnormals, so amax / 448 must
not become a zero scale (its row's zeros would be 0 / 0)."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

from oracle import dense as OD
from oracle import formats as F

pytestmark = pytest.mark.gpu
DEV = "cuda"
TINY = 2.0 ** -126          # smallest normal fp32
EDGE = 448 * TINY           # largest elements below it have a subnormal quotient


def _rows(dim):
    """Rows of `dim` bf16 values, each with zeros: one element, several of several sizes, around the edge, subnormal."""
    x = torch.zeros((9, dim), dtype=torch.float64)
    x[0, 3] = 1e-37
    x[1, 0], x[1, 7], x[1, dim - 1] = 1e-36, -3e-37, 2e-38
    x[2, 5] = 1e-40                               # bf16 subnormals
    x[3, :8] = torch.tensor([2.0 ** -133, -2.0 ** -127, 2.0 ** -130, 0, 2.0 ** -128, 0, 0, 2.0 ** -132], dtype=torch.float64)
    x[4, 1] = EDGE * (1 - 2.0 ** -7)              # just below and just above the edge
    x[5, 1] = EDGE * (1 + 2.0 ** -7)
    x[6, 2], x[6, 4] = -EDGE, 2.0 ** -125
    x[7, :4] = torch.tensor([1e-30, 0, -3e-31, 1e-33], dtype=torch.float64)
    return x.to(torch.bfloat16)                   # row 8: zeros


def _check(codes, scale, row, where):
    """The scale is amax / 448, at least the smallest normal number; each element within half a step of its code,
    and of what arithmetic without subnormals loses."""
    amax = np.abs(row).max()
    if amax == 0:
        assert scale == 1.0 and not (codes & 0x7f).any(), where
        return
    assert not ((codes & 0x7f) == 0x7f).any(), where
    if amax < TINY:                               # flushed before the maximum, or not: both are rows of (almost) nothing
        assert scale in (1.0, TINY), where
        scale = TINY if scale == TINY else 0.0
    else:
        want = max(amax / 448, TINY)
        assert abs(scale - want) <= 2.0 ** -22 * want, where
    got = F.e4m3_decode(codes) * scale
    assert (np.abs(got - row) <= 2.0 ** -4 * np.abs(row) + 2.0 ** -10 * scale + TINY).all(), where


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("many", [False, True])
def test_dense_insert_and_attention(dim, many):
    from compressed_sparse_long_c4a_gb300 import dense as D
    x = _rows(dim)
    reps = 300 if many else 1                     # several tokens of few rows share a CTA
    n = len(x) * reps
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    table = torch.randperm(-(-n // 256) + 1, dtype=torch.int32, device=DEV)[None, :-(-n // 256)].contiguous()
    pool = torch.full((table.shape[1] + 1, D.block_bytes(1, dim, D.KV_FP8_TOKEN)), 0xff, dtype=torch.uint8, device=DEV)
    cache = D.DenseCache(pool, table, 1, dim, D.KV_FP8_TOKEN)
    kv = x.repeat(reps, 1)[:, None].to(DEV)
    ins = D.DenseInsert(cache, 0, None)
    ins.run(None, kv, kv, None, pos, table[0].long()[(pos // 256).long()] * 256 + pos % 256)
    torch.cuda.synchronize()
    assert int(ins.status.item()) == 0
    host, rows = pool.cpu().numpy(), x.double().numpy()
    for t in range(n):
        for which in (0, 1):
            codes, scale = OD.raw_row(host, 1, dim, int(table[0, t // 256]), which, 0, t % 256)
            _check(codes, float(scale), rows[t % len(x)], (t, which))
    # every value is within 448 * 2^-100 of zero as attention reads it, in the few-row form and in the form for chunks
    for new in (1, min(n, 200)):
        q = torch.ones((new, 1, dim), dtype=torch.bfloat16, device=DEV)
        out, lse = torch.full_like(q, 7.0), torch.zeros((new, 1), device=DEV)
        D.DenseAttention(cache, 1, new, new).run(q, out, pos[n - new:].contiguous(), torch.tensor([0, new], dtype=torch.int32, device=DEV), lse)
        assert (out.abs() <= 448 * 2.0 ** -100).all()
        # equal logits.  The running maximum carries log2 of the value scale (down to -100), so lse is the sum of two
        # numbers of up to 112 in log2 units: a logarithm to 2^-22 of its value and three roundings to 2^-24 make
        # 112 ln 2 (2^-22 + 3 * 2^-24) < 2^-14.8
        want = torch.log(torch.arange(n - new + 1, n + 1, device=DEV).double())
        assert (lse[:, 0].double() - want).abs().max() <= 2.0 ** -14.8

def test_index_query():
    from compressed_sparse_long_c4a_gb300 import v4a
    x = _rows(128)
    T = len(x)
    q = x[:, None].contiguous().to(DEV)
    codes = torch.empty((T, 1, 128), dtype=torch.uint8, device=DEV)
    scales, w = torch.empty((T, 1), device=DEV), torch.ones((T, 1), device=DEV)
    ids, status = torch.arange(T, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    iq = v4a.IndexQuery(q.data_ptr(), codes.data_ptr(), scales.data_ptr(), w.data_ptr(), w.data_ptr(), 1.0, 1, 128, 0, 10000.0)
    a = v4a.CompressArgs(v4a.Batch(T, ids.data_ptr(), ids.data_ptr(), T, 1), None, None, None, status.data_ptr(), None, C.pointer(iq))
    assert v4a.lib().v4a_compress_insert(C.byref(a), None) == 0
    torch.cuda.synchronize()
    for t in range(T):
        _check(codes[t, 0].cpu().numpy(), float(scales[t, 0]), x[t].double().numpy(), t)


def test_window_key():
    from compressed_sparse_long_c4a_gb300 import v4a
    x = _rows(128)
    T = len(x)
    k = x.contiguous().to(DEV)
    ring = torch.full((T, 4, 128), 0xff, dtype=torch.uint8, device=DEV)
    scales = torch.full((T, 4), math.nan, device=DEV)
    ids, pos = torch.arange(T, dtype=torch.int32, device=DEV), torch.zeros(T, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    win = v4a.Window(k.data_ptr(), 128, 0, 10000.0, F.KV_FP8_TOKEN, ring.data_ptr(), scales.data_ptr(), 4, 4)
    a = v4a.CompressArgs(v4a.Batch(T, ids.data_ptr(), pos.data_ptr(), T, 1), None, None, C.pointer(win), status.data_ptr(), None, None)
    assert v4a.lib().v4a_compress_insert(C.byref(a), None) == 0
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for t in range(T):
        _check(ring[t, 0].cpu().numpy(), float(scales[t, 0]), x[t].double().numpy(), t)


def test_inv_rope_quant():
    from compressed_sparse_long_c4a_gb300 import v4a
    x = _rows(512)
    T = len(x)
    o, pos = x[:, None].contiguous().to(DEV), torch.zeros(T, dtype=torch.int32, device=DEV)
    out, scales = torch.empty((T, 1, 512), dtype=torch.uint8, device=DEV), torch.empty(T, device=DEV)
    a = v4a.OutputArgs(T, pos.data_ptr(), 1, 512, 0, 10000.0, o.data_ptr(), 1, out.data_ptr(), scales.data_ptr())
    assert v4a.lib().v4a_inv_rope_quant(C.byref(a), None) == 0
    torch.cuda.synchronize()
    for t in range(T):
        _check(out[t, 0].cpu().numpy(), float(scales[t]), x[t].double().numpy(), t)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("new", [1, 3, 90])
def test_tiny_queries_and_scales(dim, new, fp8):
    """Queries of 1e-40 to 1e-25, and a softmax scale below the smallest normal number: all logits are (almost) zero, so
    the rows are the visible values' means, whatever the power of two that a query is brought to."""
    from compressed_sparse_long_c4a_gb300 import dense as D

    from .test_gpu_dense import Layer
    layer = Layer((333,), 4, 2, dim, fp8, seed=dim + new)
    sizes = (1e-40, 1e-38, 1e-36, 1e-34, 3e-33, 1e-30, 1e-25)
    q = torch.randn((new, 4, dim), generator=layer.gen) * torch.tensor(sizes).repeat(4 * new // 7 + 1)[:4 * new].view(new, 4, 1)
    q = q.to(torch.bfloat16)
    q[-1, 3] = 0
    pos = torch.arange(333 - new, 333, dtype=torch.int32, device=DEV)
    for scale, queries in ((None, q), (1e-40, q / q.abs().amax(-1, keepdim=True).clamp_min(1e-45)), (1.2e-38, q * 0 + 1), (1e-30, q * 1e20)):
        queries = torch.nan_to_num(queries).to(torch.bfloat16).to(DEV)
        out, lse = torch.full_like(queries, 7.0), torch.full((new, 4), 7.0, device=DEV)
        op = D.DenseAttention(layer.cache, 4, new, new, scale=scale)
        op.run(queries, out, pos, torch.tensor([0, new], dtype=torch.int32, device=DEV), lse)
        torch.cuda.synchronize()
        got, got_l = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for t in {0, new // 2, new - 1}:
            n = 333 - new + t + 1
            for h in range(4):
                v = layer.rows(0, 1, h // 2, n)
                # bf16 caches: every weight is exactly one before the division; fp8: the values' scales, in f16
                tol = ((2.0 ** -11 if fp8 else 2.0 ** -16) + 2 * (n + 32) * 2.0 ** -24) * np.abs(v).mean(0) + 2.0 ** -8 * np.abs(v.mean(0))
                assert (np.abs(got[t, h] - v.mean(0)) <= tol).all(), (scale, t, h)
                assert abs(got_l[t, h] - math.log(n)) <= 2.0 ** -17, (scale, t, h)


def test_norm_without_eps():
    """eps = 0 is allowed: a mean square below the smallest normal number is taken as that number."""
    from compressed_sparse_long_c4a_gb300 import dense as D
    dim = 64
    x = torch.zeros((8, 1, dim), dtype=torch.bfloat16)
    x[0, 0, 3] = 1e-30
    x[1, 0, :] = 1e-21
    x[2, 0, ::2] = -1e-19                         # squares just below 2^-126
    x[3, 0, :40], x[3, 0, 40:] = 2e-19, 1e-19     # some below, some above
    x[4, 0, 5] = 1e-17
    x[5, 0, 5], x[5, 0, 6] = 1e-3, 1e-25
    x[6, 0, 5] = 1e5                              # row 7: zeros
    pool = torch.zeros((1, D.block_bytes(1, dim, 0)), dtype=torch.uint8, device=DEV)
    g = torch.ones(dim, device=DEV)
    op = D.DenseInsert(D.DenseCache(pool, None, 1, dim), 1, None, g, g, eps=0.0)
    q = x.to(DEV)
    out, at = torch.empty_like(q), torch.arange(8, dtype=torch.int32, device=DEV)
    op.run(q, q, q, out, at, at.long())
    torch.cuda.synchronize()
    squares = x.double() ** 2
    mean = squares.mean(-1, keepdim=True)
    want = x.double() / torch.sqrt(mean.clamp_min(TINY))
    got, keys = out.double().cpu(), pool.view(torch.bfloat16).view(2, 256, dim)[0, :8].double().cpu()[:, None]
    # a mean of at least 2^-126 lacks the squares that count as zeros; a smaller one is raised with or without them
    lost = torch.where(squares < TINY, squares, 0.0).mean(-1, keepdim=True)
    rel = 2.0 ** -8 + 2.0 ** -16 + torch.where(mean >= TINY, lost / mean, 0.0)
    assert torch.equal(got, keys) and ((got - want).abs() <= rel * want.abs()).all()
