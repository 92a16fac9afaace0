"""Pins the dense-layer oracle (oracle/dense.py) to hand-worked values, library
arithmetic and identities of the formulas."""
import math

import numpy as np
import pytest
import torch

from oracle import dense as OD
from oracle import formats as F


def test_plan_hand_worked():
    """Two tables; sequence 0 ends (2 blocks), 1 grows over a block edge, 2 rests, 3 starts."""
    tables = np.full((2, 4, 3), -1)
    tables[0, 0, :2], tables[1, 0, :2] = [10, 11], [20, 21]
    tables[0, 1, 0], tables[1, 1, 0] = 12, 22
    tables[0, 2, 0], tables[1, 2, 0] = 13, 23
    ring = np.array([1, 2, 3, 4, -1, -1, -1, -1, 0, 9])       # first 8: pages 0, 9, 1, 2, 3, 4
    sid, pos, slots, starts, first, count = OD.step_plan([300, 255, 7, 0], [-1, 3, 0, 1], tables, ring, 8, 6, 6)
    assert sid == [1, 1, 1, 3, -1, -1] and pos == [255, 256, 257, 0, -1, -1] and starts == [0, 0, 3, 3, 4]
    # sequence 1's new block takes pages 0 and 9, sequence 3's pages 1 and 2
    assert slots[0] == [12 * 256 + 255, 0, 1, 1 * 256, -1, -1]
    assert slots[1] == [22 * 256 + 255, 9 * 256, 9 * 256 + 1, 2 * 256, -1, -1]
    assert tables[0, 1].tolist() == [12, 0, -1] and tables[1, 3].tolist() == [2, -1, -1]
    assert (first, count) == (2, 6)                            # 4 taken, 4 given back: (8 + 4) % 10
    assert ring[[4, 5, 6, 7]].tolist() == [10, 20, 11, 21]


def test_rotation_identities():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(3, 64))
    f = OD.frequencies(32)
    for half in (False, True):
        a = OD.rotate(OD.rotate(x, 7, f, 16, half), 1000, f, 16, half)
        np.testing.assert_allclose(a, OD.rotate(x, 1007, f, 16, half), atol=1e-10)      # R_m R_n = R_{m+n}
        np.testing.assert_allclose((a ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-12)
        assert np.array_equal(a[:, :16], x[:, :16]) and np.array_equal(a[:, 48:], x[:, 48:])
    # one layout is the other with the pairs gathered
    perm = np.concatenate([np.arange(0, 64, 2), np.arange(1, 64, 2)])
    f = OD.frequencies(64)
    np.testing.assert_allclose(OD.rotate(x[:, perm], 5, f, 0, True), OD.rotate(x, 5, f, 0, False)[:, perm], atol=1e-14)
    # one pair by hand: position pi / 2 with frequency 1 at theta -> (a, b) -> (-b, a), doubled
    y = OD.rotate(np.array([3.0, 4.0]), 1, np.array([math.pi / 2]), 0, False, 2.0)
    np.testing.assert_allclose(y, [-8.0, 6.0], atol=1e-14)


def test_yarn_frequencies():
    """Short wavelengths keep their frequency, long ones are divided, and the blend is linear in the turns."""
    f = OD.frequencies(128, theta=1e4)
    g = OD.frequencies(128, theta=1e4, scaling="yarn", factor=16.0, original=4096.0, beta_fast=32.0, beta_slow=1.0)
    turns = 4096.0 * f / (2 * math.pi)
    assert np.array_equal(g[turns >= 32], f[turns >= 32]) and (turns >= 32).any()
    np.testing.assert_allclose(g[turns <= 1], f[turns <= 1] / 16, rtol=1e-15)
    mid = (turns > 1) & (turns < 32)
    keep = (g[mid] / f[mid] - 1 / 16) / (1 - 1 / 16)
    np.testing.assert_allclose(keep, (turns[mid] - 1) / 31, rtol=1e-10)


def test_norm_against_torch():
    x = torch.randn(4, 64, dtype=torch.float64)
    g = torch.rand(64, dtype=torch.float64)
    want = torch.nn.functional.rms_norm(x, (64,), g, 1e-6)
    np.testing.assert_allclose(OD.rms_norm(x.numpy(), g.numpy(), 1e-6), want.numpy(), rtol=1e-12)


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (5, 0), (5, 2), (100, 3), (0, 4)])
def test_attention_against_torch(window, sinks):
    torch.manual_seed(1)
    q, k, v = torch.randn(3, 8, dtype=torch.float64), torch.randn(20, 8, dtype=torch.float64), torch.randn(20, 8, dtype=torch.float64)
    for m in (0, 3, 19):
        mask = torch.tensor([j <= m and (window == 0 or j > m - window or j < sinks) for j in range(20)])
        seen = OD.visible(m, window, sinks)
        assert mask.nonzero()[:, 0].tolist() == seen and seen[-1] == m
        want = torch.nn.functional.scaled_dot_product_attention(q[None], k[None], v[None], attn_mask=mask[None, None], scale=0.3)[0]
        o, lse, av, amp = OD.attention(q.numpy(), k.numpy()[seen], v.numpy()[seen], 0.3)
        np.testing.assert_allclose(o, want.numpy(), atol=1e-12)
        z = (0.3 * q @ k.T)[:, mask]
        np.testing.assert_allclose(lse, torch.logsumexp(z, -1).numpy(), atol=1e-12)
        assert (av >= np.abs(o) - 1e-12).all() and (amp >= z.abs().amax(-1).numpy() - 1e-12).all()


def test_attention_of_nothing():
    o, lse, _, _ = OD.attention(np.ones((2, 4)), np.zeros((0, 4)), np.zeros((0, 4)), 1.0)
    assert (o == 0).all() and (lse == -np.inf).all()


def test_rows_of_a_block():
    """Byte positions of a row, its value and its scale in a page of two KV heads."""
    pool = np.zeros((2, OD.block_bytes(2, 64, True)), np.uint8)
    assert pool.shape[1] == 2 * 2 * 256 * 68
    plane = (1 * 2 + 1) * 256 + 5                       # value, head 1, position 5
    pool[1, plane * 64:(plane + 1) * 64] = F.e4m3_encode(np.arange(64.0))
    pool[1, 2 * 2 * 256 * 64 + 4 * plane:][:4] = np.float32(0.5).reshape(1).view(np.uint8)
    got = OD.read_row(pool, 2, 64, True, 1, 1, 1, 5)
    assert got[3] == 1.5 and got[16] == 8.0 and got[33] == 16.0       # 33 rounds to 32 in e4m3
    bf = np.zeros((1, OD.block_bytes(1, 64, False)), np.uint8)
    bf[0, (256 + 7) * 128:(256 + 8) * 128] = F.bf16_encode(np.full(64, 2.5)).view(np.uint8)
    assert (OD.read_row(bf, 1, 64, False, 0, 1, 0, 7) == 2.5).all()
