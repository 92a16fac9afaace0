"""Calls of the dense operators that the header allows and that lie at an edge:
tables with holes under chunks, workspaces on the least alignment, other
streams, steps that end long sequences."""
import pytest
import torch

from .test_gpu_dense import DEV, Layer, _attend, _runs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim,H,K", [(64, 8, 2), (128, 8, 2), (192, 4, 2), (256, 4, 1)])
def test_chunks_over_every_other_block(dim, H, K, fp8):
    """A step's missing page is known to the softmax of that step and of no other: present and missing blocks in turn,
    several units a CTA; the hidden blocks' rows may not count."""
    cached, new = (1900, 2500, 30), (150, 100, 230)
    lengths = [c + n for c, n in zip(cached, new)]
    holes = [(b, n) for b, size in enumerate(lengths) for n in range(b % 2, -(-size // 256), 2)]
    layer = Layer(lengths, H, K, dim, fp8, seed=dim, holes=holes)
    pos, starts = _runs(cached, new)
    op, q, out, lse = _attend(layer, pos, starts, check=False)
    assert int(op.status.item()) == 1
    layer.check(q, out, lse, pos, starts, 0, 0, op.args.softmax_scale, tokens=set(range(0, len(pos), 31)) | {149, 150, 479})
    for _ in range(5):
        again, lse2 = torch.empty_like(out), torch.empty_like(lse)
        op.run(q, again, torch.tensor(pos, dtype=torch.int32, device=DEV), torch.tensor(starts, dtype=torch.int32, device=DEV), lse2)
        assert torch.equal(out, again) and torch.equal(lse, lse2)
