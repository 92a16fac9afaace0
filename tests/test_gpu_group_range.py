"""Values at the ends of their types' range through the group-scaled dense caches
and whole prompts, on the GPU against the fp64 oracle.  Tolerances as in
test_gpu_group.py, but where a test says otherwise."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from oracle import dense_group as OG
from oracle import formats as F
from tests.test_gpu_dense import _attend, _runs
from tests.test_gpu_group import DEV, I32, GroupLayer, _check_prompt, _check_token, _dense, _f64, _prompt, _run_prompt, _same_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("runs", [((1500, 300),), ((1500, 130), (700, 1), (400, 70))])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("exponent", [-90, 100, 110])
def test_prompts_of_large_and_small_values(dim, exponent, runs):
    """Logits that grow by 2^23 behind the first keys, below what has the maximum raised: the mean of finite values is finite.
    In log2 units the logits are 0 for a sequence's first 256 keys and 23 for the others."""
    starts, kv, q, k, v = _prompt(runs, 4, 2, dim, seed=dim, pad=0)
    q.zero_()
    q[..., 0] = 1.0
    for a, b in zip(kv, kv[1:]):
        k[a:a + 256, :, 0], k[a + 256:b, :, 0] = 0.0, 23.0
        v[a:b] = (v[a:b].sign() * (1 + v[a:b].abs().clamp(max=1)) * 2.0 ** exponent).to(torch.bfloat16)
    op, out, lse = _run_prompt(starts, kv, q, k, v, scale=math.log(2))
    assert int(op.status.item()) == 0 and bool(out.isfinite().all())
    _check_prompt(starts, kv, q, k, v, out, lse, True, 0, 0, op.args.softmax_scale, set(range(0, starts[-1], 29)))


def _line_cache(keys, values, tight=True):
    """One sequence's rows, inserted through the public call; a table as wide as the sequence, or far wider."""
    D = _dense()
    n, K, dim = keys.shape
    blocks = -(-n // 256)
    pool = torch.zeros((blocks, OG.block_bytes(K, dim)), dtype=torch.uint8, device=DEV)
    table = torch.full((1, blocks if tight else 8 * blocks), -1, **I32)
    table[0, :blocks] = torch.arange(blocks, **I32)
    cache = D.DenseCache(pool, table, K, dim, D.KV_FP8_GROUP)
    op = D.DenseInsert(cache, 0, None)
    op.run(None, keys, values, None, torch.arange(n, **I32), torch.arange(n, device=DEV), k_out=torch.empty_like(keys))
    return cache


@pytest.mark.parametrize("values", ["zero", "fresh", "tiny", "some"])
@pytest.mark.parametrize("dim,K,new,n,grow", [
    (64, 1, 1, 20000, 3.5), (64, 1, 40, 20000, 3.5), (192, 1, 50, 20000, 3.5), (256, 1, 100, 20000, 3.5),
    # whole units a CTA: one sum over all keys
    (64, 8, 1200, 20000, 3.5), (128, 8, 1200, 20000, 3.5), (192, 8, 600, 20000, 3.5), (256, 8, 600, 20000, 3.5),
    (64, 1, 1, 140000, 0.0), (128, 1, 40, 140000, 0.0)])
def test_sums_over_groups_of_the_least_scales(dim, K, new, n, grow, values):
    """Groups of zeros (stored with the least scale, or 0 in a pool that was never written) and of the least values that are
    read as they are: out and lse hold over any number of them.  In log2 units the logits are 0 for the first 256 keys and
    `grow` for the others, below what has the maximum raised."""
    D = _dense()
    keys = torch.zeros((n, K, dim), dtype=torch.bfloat16, device=DEV)
    keys[256:, :, 0] = grow
    x = torch.zeros_like(keys)
    if values == "tiny":
        x[:] = 2.0 ** -92                          # its group's scale is 2^-100
    if values == "some":
        x[n - 5000:] = 1.0
    cache = _line_cache(keys, x, tight=K == 8)
    if values == "fresh":
        cache.pool[:, 2 * K * 256 * dim + 16 * K:2 * K * 256 * dim + 32 * K] = 0
    q = torch.zeros((new, 4 * K, dim), dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 1.0
    op = D.DenseAttention(cache, 4 * K, new, new, scale=math.log(2))
    out, lse = torch.empty_like(q), torch.empty((new, 4 * K), device=DEV)
    op.run(q, out, torch.arange(n - new, n, **I32), torch.tensor([0, new], **I32), lse)
    torch.cuda.synchronize()
    assert int(op.status.item()) == 0 and bool(lse.isfinite().all()) and bool(out.isfinite().all())
    kh, vh = _f64(keys[:, 0]), _f64(x[:, 0])
    for t in {0, new // 2, new - 1}:
        m = n - new + t + 1
        _check_token(q[t], out[t], lse[t], lambda w, h: (vh if w else kh)[:m], K, op.args.softmax_scale, 2.0 ** -11, t, 2.0 ** -17)
    if values in ("zero", "fresh"):
        assert not out.any()


@pytest.mark.parametrize("top", [-117, -112])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_codes_of_the_least_values(dim, top):
    """Every bf16 below 2^-116, the ones below 2^-126 among them, in groups of the least scale and of 2^-120: byte for byte."""
    D = _dense()
    bits = torch.arange(0, 11 << 7, dtype=torch.int32)
    bits = torch.cat([bits, bits | 0x8000])
    bits = bits[torch.randperm(len(bits), generator=torch.Generator().manual_seed(dim))]
    n = -(-len(bits) // dim)
    bits = torch.cat([bits, torch.zeros(n * dim - len(bits), dtype=torch.int32)])
    bits = torch.where(bits > 0x7fff, bits - 0x10000, bits).to(torch.int16)
    x = bits.view(torch.bfloat16).view(n, 1, dim).to(DEV)
    x[n // 2, 0, 5] = 2.0 ** top
    pool = torch.zeros((1, OG.block_bytes(1, dim)), dtype=torch.uint8, device=DEV)
    want = pool.cpu().numpy().copy()
    slots = list(range(n))               # one group
    op = D.DenseInsert(D.DenseCache(pool, None, 1, dim, D.KV_FP8_GROUP), 0, None)
    k_out = torch.empty_like(x)
    op.run(None, x, x.flip(0).contiguous(), None, torch.arange(n, **I32), torch.tensor(slots, device=DEV), k_out=k_out)
    assert torch.equal(k_out.view(torch.int16), x.view(torch.int16))
    rows = F.bf16_decode(x.cpu().view(torch.int16).numpy().view(np.uint16))
    OG.insert(want, 1, dim, slots, (rows, rows[::-1]))
    _same_cache(pool, want, 1, dim)


def test_read_rounds_a_row_scaled_product_once():
    """Products of a code and a scale that lie beside a tie of bf16, nearer to it than fp32 resolves: rounded to fp32 first, half
    of them would go to the even neighbour from the wrong side."""
    D = _dense()
    K, dim = 1, 64
    # 1.875 = 15 / 8: with s = S / 2^23, 15 S is beside a tie of bf16, T = (2 i + 1) 2^19 for a product in [2^27, 2^28)
    ties = (2 * torch.arange(128, 256, dtype=torch.int64) + 1) * (1 << 19)
    scales = torch.round(ties.double() / 15).long()
    scales = scales[scales < 1 << 24]
    # scales of nine bits: with codes that are powers of two the product is a tie
    scales = torch.cat([scales, (2 * torch.arange(128, 256, dtype=torch.int64) + 1) << 15])
    assert 200 < len(scales) <= 256
    pool = torch.zeros((1, D.block_bytes(K, dim, D.KV_FP8_TOKEN)), dtype=torch.uint8)
    codes = torch.tensor([1.875, -1.875, 240.0, -30.0, 0.0, -0.0, 448.0, 2.0 ** -9] * 8).to(torch.float8_e4m3fn).view(torch.uint8)
    n = len(scales)
    pool[0, :2 * 256 * dim].view(512, dim)[:] = codes
    for which in (0, 1):           # (the same mantissas at two sizes)
        at = 2 * 256 * dim + which * 1024
        pool[0, at:at + 4 * n] = (scales.double() * 2.0 ** (-30 + 40 * which)).float().view(torch.uint8)
    k, v = (torch.empty((n, K, dim), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    D.DenseRead(D.DenseCache(pool.to(DEV), torch.zeros((1, 1), **I32), K, dim, D.KV_FP8_TOKEN)).run(torch.tensor([0, n], **I32), k, v)
    c = F.e4m3_decode(codes.numpy())
    twice = 0
    for which, got in ((0, k), (1, v)):
        product = c[None] * (scales.double().numpy() * 2.0 ** (-30 + 40 * which))[:, None]        # exact: 28 bits
        want = F.bf16_encode(product)
        twice += int((F.bf16_encode(product.astype(np.float32)) != want).sum())
        assert np.array_equal(got[:, 0].cpu().view(torch.int16).numpy().view(np.uint16), want)
    assert twice > 100             # the inputs do tell one rounding from two


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("new", [1, 60])
def test_nan_scale_is_not_made_finite(dim, new):
    """A group whose key (or value) scale is NaN gives NaN to the queries that see it, and nothing to other sequences."""
    D = _dense()
    g = torch.Generator().manual_seed(dim)
    n, K = 500, 2
    x = torch.randn((2 * n, 2 * K, dim), generator=g).to(torch.bfloat16).to(DEV)
    pool = torch.zeros((4, OG.block_bytes(K, dim)), dtype=torch.uint8, device=DEV)
    cache = D.DenseCache(pool, torch.tensor([[0, 2], [1, 3]], **I32), K, dim, D.KV_FP8_GROUP)
    pos = torch.arange(n, **I32).repeat(2)
    slots = (cache.block_table.long()[torch.arange(2, device=DEV).repeat_interleave(n), pos.long() // 256] * 256 + pos % 256)
    D.DenseInsert(cache, 0, None).run(None, x[:, :K].contiguous(), x[:, K:].contiguous(), None, pos, slots,
                                      k_out=torch.empty((2 * n, K, dim), dtype=torch.bfloat16, device=DEV))
    q = torch.randn((2 * new, 4, dim), generator=g).to(torch.bfloat16).to(DEV)
    at = torch.cat([torch.arange(n - new, n, **I32)] * 2)
    op = D.DenseAttention(cache, 4, 2 * new, new)

    def run():
        out, lse = torch.empty_like(q), torch.empty((2 * new, 4), device=DEV)
        op.run(q, out, at, torch.tensor([0, new, 2 * new], **I32), lse)
        torch.cuda.synchronize()
        return out, lse
    want, want_l = run()
    assert bool(want.isfinite().all())
    body = 2 * K * 256 * dim
    scales = pool[:, body:body + 32 * K].view(torch.float32).view(4, 2, K, 4)      # [block][key, value][head][group]
    for which in (0, 1):
        old = float(scales[0, which, 1, 3])
        scales[0, which, 1, 3] = math.nan          # positions 192..255 of the first sequence, KV head 1
        out, lse = run()
        assert bool(out[:new, 2:].isnan().all()) and (which == 1 or bool(lse[:new, 2:].isnan().all()))      # (lse is of the keys alone)
        assert torch.equal(out[:new, :2], want[:new, :2]) and torch.equal(out[new:], want[new:])
        assert torch.equal(lse[:new, :2], want_l[:new, :2]) and torch.equal(lse[new:], want_l[new:])
        scales[0, which, 1, 3] = old
    assert torch.equal(run()[0], want)


@pytest.mark.parametrize("T,single", [(1025, True), (4097, True), (1025, False), (4096, False), (4097, False)])
@pytest.mark.parametrize("dim,K", [(64, 1), (128, 3)])
def test_insert_around_the_sizes_of_its_forms(dim, K, T, single):
    """Steps of single tokens, each in a group of its own, and one prompt: how many tokens a CTA takes changes nothing."""
    D = _dense()
    g = torch.Generator().manual_seed(T)
    blocks = T if single else T // 256 + 2
    slots = (torch.randperm(T, generator=g) * 256 + torch.randint(0, 256, (T,), generator=g)).tolist() if single else list(range(37, 37 + T))
    body = 2 * K * 256 * dim
    pool = torch.zeros((blocks, OG.block_bytes(K, dim)), dtype=torch.uint8, device=DEV)
    pool[:, body:] = torch.exp2(torch.randint(-10, -5, (blocks, 8 * K), generator=g).float()).view(torch.uint8).to(DEV)
    x = (torch.randn((T, 2 * K, dim), generator=g) * 2).to(torch.bfloat16).to(DEV)
    want = pool.cpu().numpy().copy()
    op = D.DenseInsert(D.DenseCache(pool, None, K, dim, D.KV_FP8_GROUP), 0, None)
    k_out = torch.empty((T, K, dim), dtype=torch.bfloat16, device=DEV)
    op.run(None, x[:, :K], x[:, K:], None, torch.zeros(T, **I32), torch.tensor(slots, device=DEV), k_out=k_out)
    assert int(op.status.item()) == 0
    some = [*range(0, T, 13), T - 1] if single else range(T)
    OG.insert(want, K, dim, [slots[t] for t in some], (_f64(x[some, :K]), _f64(x[some, K:])))
    at = sorted({slots[t] // 256 for t in some})
    _same_cache(pool[at], want[at], K, dim)


@pytest.mark.parametrize("new", [1, 90])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("exponents,q_std", [((86, 95), 2.0 ** -96), ((-99, -92), 2.0 ** 88)])
def test_scales_far_from_one(exponents, q_std, dim, new):
    """Keys and values of sizes up to 2^104 and down to 2^-108, under queries that bring the logits back to ordinary ones."""
    pos, starts = _runs((900 - new, 400 - new), (new, new))
    layer = GroupLayer((900, 400), 8, 2, dim, seed=5, exponents=exponents, q_std=q_std)
    _attend(layer, pos, starts, tokens={0, new // 2, new - 1, new, 2 * new - 1})
