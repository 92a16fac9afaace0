"""Values at the ends of their types' range through the group-scaled dense caches
and whole prompts, on the GPU against the fp64 oracle.  Tolerances as in
test_gpu_group.py, but where a test says otherwise."""
from __future__ import annotations

import math

import pytest
import torch

from tests.test_gpu_group import _check_prompt, _prompt, _run_prompt

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
