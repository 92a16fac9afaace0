"""Calls of the dense operators that the header allows and that lie at an edge:
tables with holes under chunks, workspaces on the least alignment, other
streams, steps that end long sequences."""
import numpy as np
import pytest
import torch

from .test_gpu_dense import DEV, Layer, _attend, _dense, _plan_case, _run_plan, _runs

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


def _shifted(op, by):
    """The handle with its workspace moved to `by` bytes past a 512-byte boundary, among guard bytes."""
    need = op.workspace.numel()
    whole = torch.full((need + 1024,), 0xa5, dtype=torch.uint8, device=DEV)
    at = -whole.data_ptr() % 512 + by
    op._bind(op._where, op._fn, whole[at:at + need])
    return whole, at, need


@pytest.mark.parametrize("dim,fp8", [(64, False), (128, True), (192, False), (256, True)])
def test_workspaces_on_sixteen_bytes(dim, fp8):
    """The least alignment that the host accepts: split decode, a split chunk and a mixed batch give the bytes of an
    aligned workspace and write nothing beside it."""
    runs = [((4000, 1), (900, 1)), ((2500, 300),), ((3000, 1), (1200, 250), (700, 1), (40, 2))]
    for r in runs:
        cached, new = zip(*r)
        layer = Layer([c + n for c, n in r], 8, 2, dim, fp8, seed=dim + len(r))
        pos, starts = _runs(cached, new)
        op, q, out, lse = _attend(layer, pos, starts, tokens={0, len(pos) - 1})
        args = (torch.tensor(pos, dtype=torch.int32, device=DEV), torch.tensor(starts, dtype=torch.int32, device=DEV))
        for by in (16, 48, 496):
            whole, at, need = _shifted(op, by)
            again, lse2 = torch.empty_like(out), torch.empty_like(lse)
            op.run(q, again, *args, lse2)
            torch.cuda.synchronize()
            assert torch.equal(out, again) and torch.equal(lse, lse2) and int(op.status.item()) == 0
            assert (whole[:at] == 0xa5).all() and (whole[at + need:] == 0xa5).all()


def test_plan_workspaces_on_sixteen_bytes():
    case = _plan_case(np.random.default_rng(7), 300, 5, 2000, 4, 0.1, 9)
    cached, fresh, tables, ring, first, count, T = case
    want, _ = _run_plan(cached, fresh, tables.copy(), ring.copy(), first, count, T)
    got = _dense().StepPlan(torch.from_numpy(tables).to(DEV), torch.from_numpy(ring).to(DEV), T)
    whole, at, need = _shifted(got, 16)
    got.run(*(torch.tensor(x, dtype=torch.int32, device=DEV) for x in (cached, fresh, [first, count])))
    torch.cuda.synchronize()
    for name in ("seq_ids", "positions", "slots", "token_starts", "block_table", "free_ring"):
        assert torch.equal(getattr(want, name), getattr(got, name)), name
    assert (whole[:at] == 0xa5).all() and (whole[at + need:] == 0xa5).all()
