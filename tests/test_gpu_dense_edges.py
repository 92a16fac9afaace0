"""Calls of the dense operators that the header allows and that lie at an edge:
tables with holes under chunks, workspaces on the least alignment, other
streams, steps that end long sequences."""
import numpy as np
import pytest
import torch

from oracle import dense as OD

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


def test_plan_on_another_stream_than_its_construction():
    """What the constructor queues (here behind a fifth of a second of other work) comes before a first run elsewhere."""
    _run_plan([10], [1], np.array([[[3]]], np.int32), np.arange(8, dtype=np.int32), 0, 8, 1)      # loads the kernels
    tables = torch.tensor([[[3, -1], [4, -1]]], dtype=torch.int32, device=DEV)
    ring, args = torch.arange(8, dtype=torch.int32, device=DEV), [torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([10, 250], [1, 10], [5, 3])]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)
    plan = _dense().StepPlan(tables, ring, 11)
    plan.run(*args, stream=side)
    torch.cuda.synchronize()
    assert plan.positions.tolist() == [10, *range(250, 260)] and plan.seq_ids.tolist() == [0] + [1] * 10
    assert plan.slots[0].tolist() == [3 * 256 + 10, *(4 * 256 + i for i in range(250, 256)), *(5 * 256 + i for i in range(4))]
    assert plan.token_starts.tolist() == [0, 1, 11] and args[2].tolist() == [6, 2]


def test_insert_and_attention_on_another_stream_than_their_construction():
    """Status words are cleared before the first run, wherever it is."""
    layer = Layer((300, 200), 4, 2, 64, False, seed=2, holes=[(0, 0)])
    q, x = layer.query(2), torch.ones((2, 2, 64), dtype=torch.bfloat16, device=DEV)
    out, pos, starts = torch.empty_like(q), torch.tensor([299, 199], dtype=torch.int32, device=DEV), torch.arange(3, dtype=torch.int32, device=DEV)
    slots = torch.tensor([-2, -1], device=DEV)
    for warm in (True, False):
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        if not warm:
            torch.cuda._sleep(400_000_000)
        att, ins = _dense().DenseAttention(layer.cache, 4, 2), _dense().DenseInsert(layer.cache, 0, None)
        att.run(q, out, pos, starts, stream=side)
        with torch.cuda.stream(side):
            ins.run(None, x, x, None, pos, slots)
        torch.cuda.synchronize()
        assert int(att.status.item()) == 1 and int(ins.status.item()) == 1


def test_handles_dropped_while_their_calls_are_queued():
    """The memory of a dropped handle is not another tensor's before its calls on a side stream are done."""
    layer = Layer((5000, 300), 8, 2, 128, False, seed=3)
    pos, starts = _runs((4999, 170), (1, 130))
    op, q, want, _ = _attend(layer, pos, starts, tokens={0, 1, 130})
    args = (torch.tensor(pos, dtype=torch.int32, device=DEV), torch.tensor(starts, dtype=torch.int32, device=DEV))
    size, side = op.workspace.numel(), torch.cuda.Stream()
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    op = _dense().DenseAttention(layer.cache, 8, len(pos), 130)
    at = op.workspace.data_ptr()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)
    op.run(q, out, *args, stream=side)
    del op
    taken = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in range(4)]
    assert all(t.data_ptr() != at for t in taken)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_first_call_of_a_stream_inside_a_capture():
    """A handle made before the capture may have its first call in it, and is used eagerly on that stream after it."""
    layer = Layer((700, 90), 8, 2, 64, False, seed=4)
    pos, starts = torch.tensor([699, 89], dtype=torch.int32, device=DEV), torch.arange(3, dtype=torch.int32, device=DEV)
    op, q, want, _ = _attend(layer, [699, 89], [0, 1, 2])
    fresh = _dense().DenseAttention(layer.cache, 8, 2)
    out, stream = torch.zeros_like(want), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        fresh.run(q, out, pos, starts)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    torch.cuda.synchronize()
    fresh.run(q, out, pos, starts, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and int(fresh.status.item()) == 0


@pytest.mark.parametrize("B,L,cached_hi,ended,new", [(3, 61, 120000, 0.7, 1), (40, 61, 60000, 0.5, 1), (9, 7, 300000, 1.0, 1), (600, 3, 9000, 0.6, 2),
                                                     (2, 300, 70000, 1.0, 1), (5, 1, 400000, 0.6, 3000)])
def test_steps_that_end_long_sequences(B, L, cached_hi, ended, new):
    """Far more given-back pages than tokens, in steps of few tokens (one CTA) and of more; the ring wraps."""
    case = _plan_case(np.random.default_rng(B * 1000 + L), B, L, cached_hi, new, ended, 1)
    cached, fresh, tables, ring, first, count, T = case
    plan, free = _run_plan(cached, fresh, tables.copy(), ring.copy(), first, count, T)
    sid, pos, slots, starts, first2, count2 = OD.step_plan(cached, fresh, tables, ring, first, count, T)
    assert int(plan.status.item()) == 0 and free.tolist() == [first2, count2]
    assert plan.seq_ids.tolist() == sid and plan.positions.tolist() == pos and plan.token_starts.tolist() == starts
    assert np.array_equal(plan.slots.cpu().numpy(), np.array(slots).reshape(L, T))
    assert np.array_equal(plan.block_table.cpu().numpy(), tables) and np.array_equal(plan.free_ring.cpu().numpy(), ring)


@pytest.mark.parametrize("layers", [1, 2])
def test_window_layers_whose_caller_gives_blocks_back(layers):
    """A window layer's sequence far longer than its pages: between two plans the caller puts blocks that no later
    query sees behind the last free page, and ends the sequence so; the pages serve the next one.  With two layers the
    second keeps every block."""
    D = _dense()
    H, K, dim, window, sinks, cols = 4, 2, 64, 300, 4, 9
    pages = 7 if layers == 1 else 7 + cols
    i32 = dict(dtype=torch.int32, device=DEV)
    tables, ring = torch.full((layers, 1, cols), -1, **i32), torch.randperm(pages, device=DEV).to(torch.int32)
    free, cached, fresh = torch.tensor([3, pages], **i32), torch.zeros(1, **i32), torch.zeros(1, **i32)
    pool = torch.full((pages, OD.block_bytes(K, dim, False)), 0xff, dtype=torch.uint8, device=DEV)
    caches = [D.DenseCache(pool, tables[l], K, dim) for l in range(layers)]
    plan = D.StepPlan(tables, ring, 256)
    ins = [D.DenseInsert(c, 0, None) for c in caches]
    att = [D.DenseAttention(c, H, 256, 256, window if l == 0 else 0, sinks if l == 0 else 0) for l, c in enumerate(caches)]
    g = torch.Generator().manual_seed(1)

    def give_back(l, blocks):
        first, count = free.tolist()
        held = [n for n in blocks if int(tables[l, 0, n]) >= 0]
        for i, n in enumerate(held):
            ring[(first + count + i) % pages] = tables[l, 0, n]
            tables[l, 0, n] = -1
        free[1] += len(held)

    for life in range(2):
        history = torch.zeros((2, 0, K, dim))
        at = 0
        for new in (250, 256, 1, 200, 256, 256, 17, 256, 256, 1, 100, 256):
            kv = torch.randn((2, 256, K, dim), generator=g).to(torch.bfloat16)
            q = torch.randn((256, H, dim), generator=g).to(torch.bfloat16).to(DEV)
            cached.fill_(at)
            fresh.fill_(new)
            plan.run(cached, fresh, free)
            assert int(plan.status.item()) == 0 and plan.token_starts.tolist() == [0, new]
            held = tables[tables >= 0].tolist()
            assert len(set(held)) == len(held) == pages - int(free[1])
            history = torch.cat([history, kv[:, :new].float()], 1)
            for l in range(layers):
                out, lse = torch.empty_like(q), torch.zeros((256, H), device=DEV)
                ins[l].run(None, kv[0].to(DEV), kv[1].to(DEV), None, plan.positions, plan.slots[l])
                att[l].run(q, out, plan.positions, plan.token_starts, lse)
                assert int(ins[l].status.item()) == 0 and int(att[l].status.item()) == 0
                for t in (0, new // 2, new - 1):
                    seen = OD.visible(at + t, *((window, sinks) if l == 0 else (0, 0)))
                    for h in range(K):
                        k, v = (history[i, seen, h].double().numpy() for i in (0, 1))
                        o, _, av, amp = OD.attention(q[t, 2 * h:2 * h + 2].double().cpu().numpy(), k, v, dim ** -0.5)
                        tol = (2.0 ** -8 + 2 * (dim + 8) * 2.0 ** -24 * amp[:, None] + 2 * (len(seen) + 32) * 2.0 ** -24) * av + 2.0 ** -8 * np.abs(o)
                        assert (np.abs(out[t, 2 * h:2 * h + 2].double().cpu().numpy() - o) <= tol).all(), (life, l, at, t)
            at += new
            # a query from `at` on sees j > at - window and j < sinks
            give_back(0, [n for n in range(1, cols) if 256 * n + 255 <= at - window])
        assert at > 2000
        for l in range(layers):
            give_back(l, range(cols))
        assert int(free[1]) == pages and sorted(ring.tolist()) == list(range(pages))


def test_ending_a_row_with_holes_is_reported():
    plan, free = _run_plan([300, 10], [-1, 1], np.array([[[3, -1], [4, -1]]], np.int32), np.arange(8, dtype=np.int32), 6, 2, 1)
    assert int(plan.status.item()) == 1 and free.tolist() == [6, 4] and plan.slots.tolist() == [[4 * 256 + 10]]
    assert plan.free_ring.tolist() == [3, -1, 2, 3, 4, 5, 6, 7]


@pytest.mark.parametrize("fp8", [False, True])
def test_insert_of_two_tokens_with_one_slot(fp8):
    """Pieces of either there, and every other slot and every query as without the clash."""
    D = _dense()
    K, dim, T, fmt = 2, 128, 400, D.KV_FP8_TOKEN if fp8 else D.KV_BF16
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn((T, 4 + 2 * K, dim), generator=g, device=DEV).to(torch.bfloat16)
    pos, slots = torch.arange(T, dtype=torch.int32, device=DEV), torch.arange(T, device=DEV)
    got = []
    for s in (slots, torch.where(slots >= 300, slots - 300, slots)):          # slots 0..99 twice
        pool, qo = torch.zeros((2, D.block_bytes(K, dim, fmt)), dtype=torch.uint8, device=DEV), torch.zeros((T, 4, dim), dtype=torch.bfloat16, device=DEV)
        op = D.DenseInsert(D.DenseCache(pool, None, K, dim, fmt), 4, D.Rope(dim, layout=1))
        op.run(x[:, :4], x[:, 4:4 + K], x[:, 4 + K:], qo, pos, s.contiguous())
        torch.cuda.synchronize()
        assert int(op.status.item()) == 0
        body = pool[:, :2 * K * 256 * dim * (1 if fp8 else 2)].contiguous().view(torch.uint8 if fp8 else torch.int16)
        got.append((qo, body.view(2, 2 * K, 256, dim).transpose(0, 1).reshape(2 * K, 512, dim)))
    (q0, alone), (q1, both) = got
    assert torch.equal(q0, q1) and torch.equal(alone[:, 100:300], both[:, 100:300]) and not both[:, 300:].any()
    assert ((both[:, :100] == alone[:, :100]) | (both[:, :100] == alone[:, 300:400])).all()


@pytest.mark.parametrize("T", [40, 3000])
def test_plan_without_slots_or_status_and_with_wide_tables(T):
    """What only the C entry takes: no slot maps, no status word, tables further apart than they are long."""
    L, B, cols, apart = 3, 9, 5, 77
    rng = np.random.default_rng(T)
    cached, fresh = [int(x) for x in rng.integers(0, 1000, B)], [int(x) for x in rng.integers(0, 5, B)]
    fresh[4] = -1
    whole = torch.full((L, apart), 1000, dtype=torch.int32, device=DEV)
    tables, at = np.full((L, B, cols), -1, np.int32), 0
    for l in range(L):
        for b, c in enumerate(cached):
            tables[l, b, :-(-c // 256)] = np.arange(at, at - (-c // 256))
            at += -(-c // 256)
    whole[:, :B * cols] = torch.from_numpy(tables).to(DEV).view(L, -1)
    ring = np.arange(200, dtype=np.int32) + 300
    plan = _dense().StepPlan(torch.from_numpy(tables).to(DEV), torch.from_numpy(ring).to(DEV), T, num_blocks=500)
    plan.args.block_table, plan.args.table_stride, plan.args.slots, plan.args.status = whole.data_ptr(), apart, None, None
    free = torch.tensor([190, 100], dtype=torch.int32, device=DEV)
    plan.run(torch.tensor(cached, dtype=torch.int32, device=DEV), torch.tensor(fresh, dtype=torch.int32, device=DEV), free)
    torch.cuda.synchronize()
    sid, pos, _, starts, first, count = OD.step_plan(cached, fresh, tables, ring, 190, 100, T)
    assert plan.seq_ids.tolist() == sid and plan.positions.tolist() == pos and plan.token_starts.tolist() == starts
    assert np.array_equal(whole[:, :B * cols].cpu().numpy().reshape(L, B, cols), tables) and (whole[:, B * cols:] == 1000).all()
    assert plan.free_ring.tolist() == ring.tolist() and free.tolist() == [first, count]
    assert (plan.slots == -1).all()


def test_attention_of_default_block_bytes_without_lse_and_status():
    """block_bytes = 0 is the shape's own size; lse and status may be NULL, in both forms."""
    for new in (1, 150):
        layer = Layer((400, 290), 8, 2, 64, False, seed=6, extra=0)
        pos, starts = _runs((400 - new, 290 - new), (new, new))
        op, q, out, _ = _attend(layer, pos, starts, pad=0, tokens={0, len(pos) - 1})
        op.args.kv.block_bytes, op.args.status = 0, None
        again = torch.empty_like(out)
        op.run(q, again, torch.tensor(pos, dtype=torch.int32, device=DEV), torch.tensor(starts, dtype=torch.int32, device=DEV))
        assert torch.equal(out, again)
