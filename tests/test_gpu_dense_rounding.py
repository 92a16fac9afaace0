"""What each form of the dense attention does to its probabilities: 16 bits
for a few rows over bf16 caches (two bf16 operands), f16 for fp8 caches, one
bf16 for chunks over bf16 caches.

The values come in opposite pairs and the logits are nearly equal, so the
output almost cancels: its own rounding (2^-8 of it) is small beside
sum p|v|, and what is left of the tolerance is the probabilities' rounding.
Half steps of a value: bf16 2^-8, f16 2^-11, and two bf16 operands 2^-16 (the
second holds what the first left, at most 2^-8 of it, to 2^-8)."""
import numpy as np
import pytest
import torch

from oracle import dense as OD

from .test_gpu_dense import DEV, Layer, _dense, _runs

pytestmark = pytest.mark.gpu

BF16_PAIR, F16, BF16 = 2.0 ** -16, 2.0 ** -11, 2.0 ** -8


def _cancelling(lengths, H, K, dim, fp8, seed):
    """A layer whose value rows 2 i and 2 i + 1 are opposite, with queries of small logits."""
    layer = Layer(lengths, H, K, dim, fp8, seed, extra=0, q_std=0.02)
    n, body = layer.host.shape[0], 2 * K * 256 * dim
    host = torch.from_numpy(layer.host)
    if fp8:
        rows = host[:, :body].reshape(n, 2, K, 256, dim)
        rows[:, 1, :, 1::2] = rows[:, 1, :, 0::2] ^ 0x80
        sc = host[:, body:].reshape(n, 2, K, 256, 4)
        sc[:, 1, :, 1::2] = sc[:, 1, :, 0::2]
        host = torch.cat([rows.reshape(n, body), sc.reshape(n, -1)], 1)
    else:
        rows = host.view(torch.int16).reshape(n, 2, K, 256, dim)
        rows[:, 1, :, 1::2] = rows[:, 1, :, 0::2] ^ -0x8000
        host = rows.reshape(n, body).view(torch.uint8)
    layer.host = host.contiguous().numpy()
    layer.pool.copy_(host)
    return layer


def _tolerances(layer, q, b, m, h, p_half, scale):
    """Rows of KV head h of a query at position m of sequence b: fp64 output, lse, and the output's tolerance."""
    G, n, dim = layer.H // layer.K, m + 1, layer.dim
    k, v = layer.rows(b, 0, h, n), layer.rows(b, 1, h, n)
    o, l, av, amp = OD.attention(q[h * G:(h + 1) * G], k, v, scale)
    # a logit's dot product, twice (in p and in the sum); sums, exponentials and logarithms of up to 32 + n steps
    fp32 = 2 * (dim + 8) * 2.0 ** -24 * amp[:, None] + 2 * (n + 32) * 2.0 ** -24
    return o, l, (p_half + fp32) * av + 2.0 ** -8 * np.abs(o)


def _check(layer, q, out, positions, starts, p_half, scale, tokens=None):
    q, got = q.double().cpu().numpy(), out.double().cpu().numpy()
    G = layer.H // layer.K
    for b in range(len(starts) - 1):
        for t in range(starts[b], starts[b + 1]):
            if tokens is not None and t not in tokens:
                continue
            for h in range(layer.K):
                o, _, tol = _tolerances(layer, q[t], b, positions[t], h, p_half, scale)
                err = np.abs(got[t, h * G:(h + 1) * G] - o)
                assert (err <= tol).all(), (b, t, h, float((err / tol).max()))


def _run(layer, positions, starts, max_new, pad=0):
    T = starts[-1] + pad
    op = _dense().DenseAttention(layer.cache, layer.H, T, max_new)
    q = layer.query(T)
    out, lse = torch.full_like(q, 7.0), torch.full((T, layer.H), 7.0, device=DEV)
    op.run(q, out, torch.tensor(list(positions) + [-1] * pad, dtype=torch.int32, device=DEV),
           torch.tensor(starts, dtype=torch.int32, device=DEV), lse)
    torch.cuda.synchronize()
    assert int(op.status.item()) == 0
    return q, out, lse, op.args.softmax_scale


LENGTHS = (2, 3, 4, 6, 7, 8, 10, 16, 24, 33, 64, 100, 257)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,K,dim", [(16, 2, 64), (16, 1, 128), (3, 1, 128), (24, 3, 192), (8, 1, 256)])
def test_few_rows(H, K, dim, fp8):
    layer = _cancelling(LENGTHS, H, K, dim, fp8, seed=H + dim)
    pos, starts = [n - 1 for n in LENGTHS], list(range(len(LENGTHS) + 1))
    q, out, _, scale = _run(layer, pos, starts, 1)
    _check(layer, q, out, pos, starts, F16 if fp8 else BF16_PAIR, scale)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_few_rows_beside_a_chunk(dim, fp8):
    """The decoding sequences of a mixed batch keep their own form's rounding, and several tokens that stay few rows do."""
    new = (1,) * 8 + (2, 120, 3)
    cached = (1, 2, 5, 6, 9, 30, 61, 256, 4, 20, 7)
    layer = _cancelling([c + n for c, n in zip(cached, new)], 4, 1, dim, fp8, seed=dim)
    pos, starts = _runs(cached, new)
    q, out, _, scale = _run(layer, pos, starts, 120, pad=3)
    few = {t for b, n in enumerate(new) if n < 4 for t in range(starts[b], starts[b + 1])}
    _check(layer, q, out, pos, starts, F16 if fp8 else BF16_PAIR, scale, few)
    _check(layer, q, out, pos, starts, F16 if fp8 else BF16, scale, set(range(starts[9], starts[10], 7)))
    assert (out[starts[-1]:] == 7.0).all()


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_fp8_chunks(dim):
    layer = _cancelling((150, 400), 4, 1, dim, True, seed=dim)
    pos, starts = _runs((0, 300), (150, 100))
    q, out, _, scale = _run(layer, pos, starts, 150)
    _check(layer, q, out, pos, starts, F16, scale, set(range(0, 250, 7)) | {1, 2, 3})


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_chunk_and_single_tokens_agree(dim, fp8):
    """The same rows through both forms: as far apart as both forms' tolerances together, outputs and lse."""
    layer = Layer((300,), 8, 2, dim, fp8, seed=dim + 1)
    pos, starts = _runs((170,), (130,))
    q, out, lse, scale = _run(layer, pos, starts, 130)
    one, lse1 = torch.empty_like(out), torch.empty_like(lse)
    dec = _dense().DenseAttention(layer.cache, 8, 1, 1)
    for t, p in enumerate(pos):
        dec.run(q[t:t + 1], one[t:t + 1], torch.tensor([p], dtype=torch.int32, device=DEV),
                torch.tensor([0, 1], dtype=torch.int32, device=DEV), lse1[t:t + 1])
    torch.cuda.synchronize()
    few, many = (F16, F16) if fp8 else (BF16_PAIR, BF16)
    qd, a, b = q.double().cpu().numpy(), out.double().cpu().numpy(), one.double().cpu().numpy()
    la, lb = lse.double().cpu().numpy(), lse1.double().cpu().numpy()
    for t in range(0, 130, 3):
        for h in range(2):
            s = slice(4 * h, 4 * h + 4)
            o, l, tol = _tolerances(layer, qd[t], 0, pos[t], h, few + many, scale)
            assert (np.abs(a[t, s] - b[t, s]) <= 2 * tol).all(), (t, h)
            amp = np.abs(qd[t, s]) @ np.abs(layer.rows(0, 0, h, pos[t] + 1)).T
            ltol = (dim + 8) * 2.0 ** -24 * scale * amp.max(1) + (pos[t] + 33) * 2.0 ** -24 + 2.0 ** -22 * np.abs(l) + 2.0 ** -20
            assert (np.abs(la[t, s] - lb[t, s]) <= 2 * ltol).all(), (t, h)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim", [128, 256])
def test_padding_up_to_the_longest_call_takes_the_chunk_form(dim, fp8):
    """num_tokens = num_seqs * max_new_per_seq says that every sequence brings the most: a shorter one in such a call
    gets the chunk form, its rounding and its own rows only; with one token of room less it gets its own form."""
    H, K = 4, 1
    layer = _cancelling((33,), H, K, dim, fp8, seed=dim)
    for pad, p_half in ((511, F16 if fp8 else BF16), (510, F16 if fp8 else BF16_PAIR)):
        q, out, lse, scale = _run(layer, [32], [0, 1], 512, pad=pad)
        _check(layer, q, out, [32], [0, 1], p_half, scale)
        assert (out[1:] == 7.0).all() and (lse[1:] == 7.0).all()
    layer = _cancelling((33, 600, 90), H, K, dim, fp8, seed=dim + 1)
    pos, starts = _runs((32, 300, 88), (1, 300, 2))
    for room in (0, 1):          # 3 x 300 rows: full, and one below
        q, out, lse, scale = _run(layer, pos, starts, 300, pad=900 - 303 - room)
        some = {0, 1, 2, 150, 300, 301, 302}
        _check(layer, q, out, pos, starts, F16 if fp8 else BF16, scale, some)
        if room:
            _check(layer, q, out, pos, starts, F16 if fp8 else BF16_PAIR, scale, {0, 301, 302})
        assert (out[303:] == 7.0).all() and (lse[303:] == 7.0).all()
