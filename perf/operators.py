"""Cases of the dense-layer operators: the step plan (block tables and slot
maps built on the GPU), the query/key norm with the position rotation and the
cache insert, and attention over the dense paged cache (decode and chunked
prefill, with a sliding window and sinks).

A dense layer keeps one key and one value per KV head and token, in pages of
256 positions.  A page holds [KV heads][256][dim] keys, then the values in the
same layout, then (fp8 caches) one fp32 scale per key row and one per value
row.  The block table maps a sequence's n-th 256 positions to a page.

`run` computes an operator in elementary torch operations, or, where `own` is
true, through the framework's entry points.
"""
from __future__ import annotations

import math
import random

import torch

own = False

PAGE = 256          # positions per page
DEVICE = "cuda"


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def listed():
    return [
        # ---- the step plan: block tables, slot maps, positions ----
        # one decode step of 64 sequences in a 61-layer model (a table per layer)
        {"name": "plan_decode_b64", "op": "plan", "seqs": 64, "tables": 61, "cached_lo": 65536, "cached_hi": 131072,
         "new_lo": 1, "new_hi": 1, "ended": 0.0, "pad": 0, "shape_seed": 1},
        # chunked prefill of four sequences, 61 layers
        {"name": "plan_prefill_4x4k", "op": "plan", "seqs": 4, "tables": 61, "cached_lo": 32768, "cached_hi": 32768,
         "new_lo": 4096, "new_hi": 4096, "ended": 0.0, "pad": 0, "shape_seed": 2},
        # a busy server's mixed step: most sequences decode, some bring a chunk, some rest, some end;
        # the step's token arrays are padded for a captured graph
        {"name": "plan_mixed_b1000", "op": "plan", "seqs": 1000, "tables": 30, "cached_lo": 0, "cached_hi": 32768,
         "new_lo": 0, "new_hi": 160, "ended": 0.05, "pad": 1001, "shape_seed": 3},
        # ---- norm + rotation + cache insert ----
        # a decode step of four sequences at 1M positions (latency), half layout stretched for long contexts
        {"name": "insert_decode_b4_1m", "op": "insert", "tokens": 4, "heads": 16, "kv_heads": 4, "dim": 128,
         "fmt": "bf16", "layout": "half", "rope_first": 0, "rope_dims": 128, "scaling": "yarn", "pos_lo": 1048575,
         "norm": True, "fused": True, "shape_seed": 4},
        # an odd chunk into an fp8 cache, 64-wide heads, interleaved rotation of half of the head
        {"name": "insert_chunk_4097_fp8", "op": "insert", "tokens": 4097, "heads": 64, "kv_heads": 8, "dim": 64,
         "fmt": "fp8", "layout": "interleaved", "rope_first": 32, "rope_dims": 32, "scaling": "linear", "pos_lo": 32768,
         "norm": True, "fused": True, "shape_seed": 5},
        # four chunks of 4096 tokens, bf16 cache
        {"name": "insert_prefill_4x4k", "op": "insert", "tokens": 16384, "heads": 64, "kv_heads": 8, "dim": 128,
         "fmt": "bf16", "layout": "half", "rope_first": 0, "rope_dims": 128, "scaling": "none", "pos_lo": 32768,
         "norm": True, "fused": False, "shape_seed": 6},
        # ---- attention over the paged cache ----
        # one sequence, 1k context (latency)
        {"name": "attn_decode_b1_1k", "op": "attn", "seqs": 1, "heads": 16, "kv_heads": 4, "dim": 128, "fmt": "bf16",
         "cached_lo": 1024, "cached_hi": 1024, "new_lo": 1, "new_hi": 1, "window": 0, "sinks": 0, "shape_seed": 7},
        # 32 sequences of 32k to 64k, bf16 cache (bandwidth, ragged lengths)
        {"name": "attn_decode_b32_32k_64k", "op": "attn", "seqs": 32, "heads": 64, "kv_heads": 8, "dim": 128,
         "fmt": "bf16", "cached_lo": 32768, "cached_hi": 65536, "new_lo": 1, "new_hi": 1, "window": 0, "sinks": 0,
         "shape_seed": 8},
        # four sequences at 1M, fp8 cache
        {"name": "attn_decode_b4_1m_fp8", "op": "attn", "seqs": 4, "heads": 16, "kv_heads": 2, "dim": 128,
         "fmt": "fp8", "cached_lo": 1048575, "cached_hi": 1048575, "new_lo": 1, "new_hi": 1, "window": 0, "sinks": 0,
         "shape_seed": 9},
        # 64 sequences of 64k to 128k that see their last 1024 tokens and 4 sinks, 64-wide heads
        {"name": "attn_window_decode_b64", "op": "attn", "seqs": 64, "heads": 64, "kv_heads": 8, "dim": 64,
         "fmt": "bf16", "cached_lo": 65536, "cached_hi": 131072, "new_lo": 1, "new_hi": 1, "window": 1024, "sinks": 4,
         "shape_seed": 10},
        # ragged chunks with a window and sinks
        {"name": "attn_window_prefill_b4", "op": "attn", "seqs": 4, "heads": 32, "kv_heads": 8, "dim": 128,
         "fmt": "bf16", "cached_lo": 0, "cached_hi": 32768, "new_lo": 1000, "new_hi": 2048, "window": 1024, "sinks": 4,
         "shape_seed": 11},
        # the last chunk of a 32k prompt (tensor cores)
        {"name": "attn_prefill_32k", "op": "attn", "seqs": 1, "heads": 32, "kv_heads": 8, "dim": 128, "fmt": "bf16",
         "cached_lo": 28672, "cached_hi": 28672, "new_lo": 4096, "new_hi": 4096, "window": 0, "sinks": 0,
         "shape_seed": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "insert", "attn", "attn"])
    seed = rng.randrange(1 << 30)
    if op == "plan":
        seqs = _log(rng, 1, 1000)
        new_hi = rng.choice([1, _log(rng, 2, max(2, 60000 // seqs))])
        return {"op": "plan", "seqs": seqs, "tables": rng.randint(1, 30), "cached_lo": 0,
                "cached_hi": _log(rng, 100, 100000), "new_lo": rng.choice([0, 1]), "new_hi": new_hi,
                "ended": rng.choice([0.0, 0.1]), "pad": rng.choice([0, _log(rng, 1, 500)]), "shape_seed": seed}
    if op == "insert":
        dim = rng.choice([64, 128, 256])
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 3, 4, 8])
        rope = rng.choice([dim, dim // 2, 16])
        return {"op": "insert", "tokens": _log(rng, 1, 16384 * 80 * 128 // (dim * (heads + 2 * kv)) if dim * (heads + 2 * kv) > 10240 else 16384),
                "heads": heads, "kv_heads": kv, "dim": dim, "fmt": rng.choice(["bf16", "fp8"]),
                "layout": rng.choice(["half", "interleaved"]), "rope_first": rng.choice([0, dim - rope]),
                "rope_dims": rope, "scaling": rng.choice(["none", "linear", "yarn"]),
                "pos_lo": _log(rng, 1, 1 << 20), "norm": rng.random() < 0.8, "fused": rng.random() < 0.5,
                "shape_seed": seed}
    dim = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 3, 4, 8, 16])
    window = rng.choice([0, 0, 128, 1024])
    c = {"op": "attn", "seqs": _log(rng, 1, 64), "heads": kv * group, "kv_heads": kv, "dim": dim,
         "fmt": rng.choice(["bf16", "bf16", "fp8"]), "cached_lo": 0, "new_lo": 1, "new_hi": 1, "window": window,
         "sinks": rng.choice([0, 4]) if window else 0, "shape_seed": seed}
    if rng.random() < 0.6:      # decode; the cache's values are bounded as in the listed cases
        most = min(1 << 20, (1 << 30) // (c["seqs"] * kv * dim))
        c["cached_hi"] = _log(rng, 16, max(17, most))
    else:                       # chunks; the rows x keys are bounded as in the listed cases
        c["seqs"] = _log(rng, 1, 8)
        c["new_hi"] = _log(rng, 2, 2048)
        most = min(32768, (1 << 31) // (c["seqs"] * c["heads"] * c["new_hi"]))
        c["cached_hi"] = _log(rng, 16, max(17, most - c["new_hi"]))
    return c


def _lengths(case):
    """Cached and new tokens of each sequence (new = -1: the sequence ends), from the case alone."""
    r = random.Random(case["shape_seed"])
    n = case["seqs"]
    cached = [r.randint(case["cached_lo"], case["cached_hi"]) for _ in range(n)]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(n)]
    if case["op"] == "plan" and case["new_hi"] > 1 and n > 16:
        new = [v if r.random() < 0.2 else min(1, v) for v in new]       # most sequences decode
    if case.get("ended"):
        new = [-1 if r.random() < case["ended"] else v for v in new]
    return cached, new


def _pages(n):
    return (n + PAGE - 1) // PAGE


# --------------------------------------------------------------------------
# Work
# --------------------------------------------------------------------------

def work(case):
    if case["op"] == "plan":
        cached, new = _lengths(case)
        L, B = case["tables"], case["seqs"]
        T = sum(max(0, v) for v in new) + case["pad"]
        fresh = sum(_pages(c + v) - _pages(c) for c, v in zip(cached, new) if v > 0)
        ended = sum(_pages(c) for c, v in zip(cached, new) if v < 0)
        # lengths in; ids, positions and slots out; a page taken or given back is read once and written once;
        # the page of a token in an earlier block is read once per sequence and table
        return {"bytes": 8 * B + 4 * (B + 1) + T * (8 + 8 * L) + 8 * L * (fresh + ended) + 4 * L * B + 16, "flops": T * L}
    if case["op"] == "insert":
        T, H, K, D = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        out = 2 * D if case["fmt"] == "bf16" else D + 4
        return {"bytes": T * (H * D * 4 + 2 * K * D * 2 + 2 * K * out + 12), "flops": T * (H + K) * D * 8}
    cached, new = _lengths(case)
    H, K, D, W, S = case["heads"], case["kv_heads"], case["dim"], case["window"], case["sinks"]
    row = 2 * (2 * D if case["fmt"] == "bf16" else D + 4)
    keys = pairs = 0
    for c, n in zip(cached, new):
        last = c + n - 1
        lo = max(0, c - W + 1) if W else 0
        keys += last - lo + 1 + min(S, lo)
        if W:
            pairs += sum(min(m + 1, W) + min(S, max(0, m + 1 - W)) for m in range(c, c + n))
        else:
            pairs += n * c + n * (n + 1) // 2
    T = sum(new)
    return {"bytes": keys * K * row + T * H * (4 * D + 4), "flops": 4 * D * H * pairs}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def _gen(seed, n):
    g = torch.Generator(device=DEVICE)
    g.manual_seed((seed * 1_000_003 + n * 7919) & 0x7FFF_FFFF_FFFF)
    return g


def _randn(shape, seed, n, std=1.0, mean=0.0, dtype=torch.float32):
    return torch.randn(shape, generator=_gen(seed, n), device=DEVICE, dtype=torch.float32).mul_(std).add_(mean).to(dtype)


def _block_bytes(case):
    K, D = case["kv_heads"], case["dim"]
    return 4 * K * PAGE * D if case["fmt"] == "bf16" else 2 * K * PAGE * (D + 4)


def _pool(case, blocks, seed):
    """A page pool with every row filled, as by earlier steps."""
    K, D = case["kv_heads"], case["dim"]
    pool = torch.empty((blocks, _block_bytes(case)), dtype=torch.uint8, device=DEVICE)
    g = _gen(seed, 100)
    codes = 2 * K * PAGE * D
    at_once = max(1, (1 << 28) // codes)
    for i in range(0, blocks, at_once):
        n = min(at_once, blocks - i)
        v = torch.randn((n, codes), generator=g, device=DEVICE, dtype=torch.float32)
        if case["fmt"] == "bf16":
            pool[i:i + n] = v.to(torch.bfloat16).view(torch.uint8)
        else:
            pool[i:i + n, :codes] = v.mul_(100).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            s = torch.rand((n, 2 * K * PAGE), generator=g, device=DEVICE).add_(0.5).mul_(0.01)
            pool[i:i + n, codes:] = s.view(torch.uint8)
    return pool


def _frequencies(case):
    """Inverse frequencies (fp64) and the factor on cos and sin."""
    R, theta = case["rope_dims"], 10000.0
    f = theta ** (-torch.arange(0, R, 2, dtype=torch.float64, device=DEVICE) / R)
    if case["scaling"] == "linear":
        return f / 4.0, 1.0
    if case["scaling"] == "yarn":      # long wavelengths are stretched, short ones kept
        turns = 65536.0 * f / (2 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        return f * keep + f / 16.0 * (1.0 - keep), 0.1 * math.log(16.0) + 1.0
    return f, 1.0


def prepare(case, seed):
    s = {"case": case}
    if case["op"] == "plan":
        cached, new = _lengths(case)
        L, B = case["tables"], case["seqs"]
        T = max(1, sum(max(0, v) for v in new) + case["pad"])
        cols = max(1, max(_pages(c + max(0, v)) for c, v in zip(cached, new)))
        held = sum(_pages(c) for c in cached) * L
        fresh = sum(_pages(c + v) - _pages(c) for c, v in zip(cached, new) if v > 0) * L
        total = held + fresh + 37
        order = torch.randperm(total, generator=_gen(seed, 1), device=DEVICE).to(torch.int32)
        table = torch.full((L, B, cols), -1, dtype=torch.int32, device=DEVICE)
        has = torch.tensor([_pages(c) for c in cached], device=DEVICE)
        table[(torch.arange(cols, device=DEVICE)[None] < has[:, None])[None].expand(L, -1, -1)] = order[:held]
        head = (seed * 7919 + 5) % total        # the ring's first free page
        ring = torch.full((total,), -1, dtype=torch.int32, device=DEVICE)
        free = total - held
        ring[(head + torch.arange(free, device=DEVICE)) % total] = order[held:]
        s.update(cached=torch.tensor(cached, dtype=torch.int32, device=DEVICE),
                 fresh=torch.tensor(new, dtype=torch.int32, device=DEVICE), table=table, ring=ring,
                 free_in=torch.tensor([head, free], dtype=torch.int32, device=DEVICE),
                 free_out=torch.zeros(2, dtype=torch.int32, device=DEVICE), tokens=T)
        return s
    if case["op"] == "insert":
        T, H, K, D = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        runs = min(T, 4)                        # sequences of about equal length
        r = torch.arange(T, device=DEVICE)
        seq, first = r * runs // T, torch.tensor([-(-i * T // runs) for i in range(runs)], device=DEVICE)
        start = case["pos_lo"] + torch.randint(0, 1000, (runs,), generator=_gen(seed, 1), device=DEVICE)
        pos = start[seq] + r - first[seq]
        per = _pages(T // runs + 1) + 1
        pages = torch.randperm(runs * per + 3, generator=_gen(seed, 2), device=DEVICE)
        page = pages[seq * per + pos // PAGE - (start // PAGE)[seq]]
        s.update(positions=pos.to(torch.int32), slots=page * PAGE + pos % PAGE,
                 pool=_pool(case, runs * per + 3, seed), q_out=torch.zeros((T, H, D), dtype=torch.bfloat16, device=DEVICE))
        if case["fused"]:                       # one projection's output, split by strides
            x = _randn((T, (H + 2 * K) * D), seed, 3, std=2.0, dtype=torch.bfloat16)
            s.update(q=x[:, :H * D].view(T, H, D), k=x[:, H * D:(H + K) * D].view(T, K, D), v=x[:, (H + K) * D:].view(T, K, D))
        else:
            s.update(q=_randn((T, H, D), seed, 3, std=2.0, dtype=torch.bfloat16),
                     k=_randn((T, K, D), seed, 4, std=2.0, dtype=torch.bfloat16),
                     v=_randn((T, K, D), seed, 5, dtype=torch.bfloat16))
        s["q_gamma"] = _randn((D,), seed, 6, std=0.1, mean=1.0) if case["norm"] else None
        s["k_gamma"] = _randn((D,), seed, 7, std=0.1, mean=1.0) if case["norm"] else None
        s["inv_freq"], s["magnitude"] = _frequencies(case)
        return s
    cached, new = _lengths(case)
    B, H, D, W, S = case["seqs"], case["heads"], case["dim"], case["window"], case["sinks"]
    T = sum(new)
    # pages of the positions that some query sees (a window layer gives the others back)
    table = torch.full((B, max(_pages(c + n) for c, n in zip(cached, new))), -1, dtype=torch.int32)
    at = 0
    for b, (c, n) in enumerate(zip(cached, new)):
        lo = max(0, c - W + 1) // PAGE if W else 0
        cols = sorted(set(range(_pages(S))) | set(range(lo, _pages(c + n)))) if W else range(_pages(c + n))
        cols = [x for x in cols if x < _pages(c + n)]
        table[b, cols] = torch.arange(at, at + len(cols), dtype=torch.int32)
        at += len(cols)
    order = torch.randperm(at + 3, generator=_gen(seed, 1), device=DEVICE).to(torch.int32)
    table = table.to(DEVICE)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s.update(table=torch.where(table < 0, table, order[table.clamp_min(0).long()]).contiguous(),
             pool=_pool(case, at + 3, seed), q=_randn((T, H, D), seed, 3, std=2.0, dtype=torch.bfloat16),
             starts=torch.tensor(starts, dtype=torch.int32, device=DEVICE),
             positions=torch.cat([torch.arange(c, c + n, dtype=torch.int32) for c, n in zip(cached, new)]).to(DEVICE),
             max_new=max(new), max_seen=max(c + n for c, n in zip(cached, new)),
             out=torch.zeros((T, H, D), dtype=torch.bfloat16, device=DEVICE),
             lse=torch.zeros((T, H), dtype=torch.float32, device=DEVICE))
    return s


# --------------------------------------------------------------------------
# The plain forms
# --------------------------------------------------------------------------

def _plan_plain(s):
    cached, fresh, table, ring, T = s["cached"].long(), s["fresh"].long(), s["table"], s["ring"], s["tokens"]
    L, B, cols = table.shape
    cap = ring.numel()
    head, count = s["free_in"][0].long(), s["free_in"][1].long()
    new = fresh.clamp_min(0)
    has = (cached + PAGE - 1) // PAGE
    need = torch.where(new > 0, (cached + new + PAGE - 1) // PAGE - has, 0)
    back = torch.where(fresh < 0, has, 0)
    zero = torch.zeros(1, dtype=torch.long, device=table.device)
    starts = torch.cat([zero, new.cumsum(0)])
    nstart = torch.cat([zero, need.cumsum(0)])
    bstart = torch.cat([zero, back.cumsum(0)])
    layer = torch.arange(L, device=table.device)[:, None]
    rows = torch.arange(B, device=table.device)
    # pages given back go behind the last free page
    b = rows.repeat_interleave(back)
    k = torch.arange(b.numel(), device=table.device)
    at = (head + count + k[None] * L + layer) % cap
    ring[at] = table[layer, b[None], (k - bstart[b])[None]]
    # new pages come from the ring's first free page on
    b = rows.repeat_interleave(need)
    k = torch.arange(b.numel(), device=table.device)
    table[layer, b[None], (has[b] + k - nstart[b])[None]] = ring[(head + k[None] * L + layer) % cap]
    # tokens
    t = torch.arange(T, device=table.device)
    live = t < starts[-1]
    seq = torch.searchsorted(starts[1:].contiguous(), t, right=True).clamp_max(B - 1)
    pos = cached[seq] + t - starts[seq]
    page = table[layer, seq[None], torch.where(live, pos // PAGE, 0)[None]].long()
    slots = torch.where(live[None], page * PAGE + pos[None] % PAGE, -1)
    s["free_out"].copy_(torch.stack([(head + nstart[-1] * L) % cap, count + (bstart[-1] - nstart[-1]) * L]))
    return {"seq_ids": torch.where(live, seq, -1).int(), "positions": torch.where(live, pos, -1).int(), "slots": slots,
            "token_starts": starts.int(), "table": table, "ring": ring, "free": s["free_out"]}


def _rotate(x, case, cos, sin):
    """x [T][heads][dim], cos and sin [T][rotated / 2], in x's type."""
    R, a = case["rope_dims"], case["rope_first"]
    y = x.clone()
    if case["layout"] == "half":
        p, q = x[..., a:a + R // 2], x[..., a + R // 2:a + R]
        y[..., a:a + R // 2] = p * cos[:, None] - q * sin[:, None]
        y[..., a + R // 2:a + R] = p * sin[:, None] + q * cos[:, None]
    else:
        p, q = x[..., a:a + R:2], x[..., a + 1:a + R:2]
        y[..., a:a + R:2] = p * cos[:, None] - q * sin[:, None]
        y[..., a + 1:a + R:2] = p * sin[:, None] + q * cos[:, None]
    return y


def _views(case, pool):
    """Keys and values [page][key, value][KV head][256][dim], and fp8 caches' scales."""
    K, D, n = case["kv_heads"], case["dim"], pool.shape[0]
    if case["fmt"] == "bf16":
        return pool.view(torch.bfloat16).view(n, 2, K, PAGE, D), None
    codes = 2 * K * PAGE * D
    return (pool[:, :codes].view(torch.float8_e4m3fn).unflatten(1, (2, K, PAGE, D)),
            pool[:, codes:].view(torch.float32).unflatten(1, (2, K, PAGE)))


def _insert_plain(s):
    case, slots = s["case"], s["slots"]
    ang = s["positions"].double()[:, None] * s["inv_freq"][None]
    cos, sin = (ang.cos() * s["magnitude"]).float(), (ang.sin() * s["magnitude"]).float()

    def prep(x, gamma):
        x = x.float()
        if gamma is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * gamma
        return _rotate(x, case, cos, sin)

    s["q_out"].copy_(prep(s["q"], s["q_gamma"]))
    rows, scales = _views(case, s["pool"])
    kv = torch.stack([prep(s["k"], s["k_gamma"]), s["v"].float()], 1)       # [T][2][K][D]
    page, at = slots // PAGE, slots % PAGE
    if scales is None:
        rows[page, :, :, at] = kv.to(torch.bfloat16)
        return {"q": s["q_out"], "cache": rows}
    amax = kv.abs().amax(-1)
    sc = torch.where(amax > 0, amax / 448.0, 1.0)
    code = (kv / sc[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    rows.view(torch.uint8)[page, :, :, at] = code.view(torch.uint8)
    scales[page, :, :, at] = sc
    return {"q": s["q_out"], "cache": rows, "scales": scales}


def _seen(case, s, B, keys):
    """Positions [B][keys] that the padded key list holds: the sinks, then the range up to the last query."""
    first = s["positions"][s["starts"][:-1].long()].long()
    W, S = case["window"], case["sinks"]
    lo = (first - W + 1).clamp_min(0) if W else torch.zeros_like(first)
    j = torch.arange(keys, device=first.device)[None]
    n = torch.minimum(lo, torch.tensor(S, device=first.device))[:, None]    # sinks in front of the range
    return torch.where(j < n, j, lo[:, None] + j - n)


def _attn_plain(s, wide=torch.float32):
    case = s["case"]
    B, H, K, D, W, S = (case[n] for n in ("seqs", "heads", "kv_heads", "dim", "window", "sinks"))
    G, starts, pos, n = H // K, s["starts"].long(), s["positions"].long(), s["max_new"]
    keys = min(s["max_seen"], W - 1 + n + S) if W else s["max_seen"]
    count = starts[1:] - starts[:-1]
    i = torch.arange(n, device=pos.device)[None]
    t = (starts[:-1, None] + i).clamp_max(pos.numel() - 1)
    m = pos[starts[:-1]][:, None] + i                                       # [B][n] query positions
    j = _seen(case, s, B, keys)                                             # [B][keys]
    last = (m[:, 0] + count - 1)[:, None]
    page = s["table"][torch.arange(B, device=pos.device)[:, None], torch.minimum(j, last) // PAGE].long()
    rows, scales = _views(case, s["pool"])
    live = ((j <= last) & (page >= 0))
    page, at = page.clamp_min(0), j % PAGE

    def gather(which):      # [B][K][keys][D]
        x = rows.view(torch.uint8)[page, which, :, at].view(rows.dtype).to(wide) if scales is not None else rows[page, which, :, at].to(wide)
        if scales is not None:
            x = x * scales[page, which, :, at].to(wide)[..., None]
        return torch.where(live[..., None, None], x, 0.0).transpose(1, 2)

    q = s["q"][t].to(wide).view(B, n, K, G, D).permute(0, 2, 3, 1, 4).reshape(B, K, G * n, D)
    z = torch.matmul(q, gather(0).transpose(2, 3)).view(B, K, G, n, keys) * (1.0 / math.sqrt(D))
    ok = live[:, None] & (j[:, None] <= m[..., None])                        # [B][n][keys]
    if W:
        ok = ok & ((j[:, None] > m[..., None] - W) | (j[:, None] < S))
    z = z.masked_fill_(~ok[:, None, None], -math.inf)
    mx = z.amax(-1, keepdim=True)
    p = z.sub_(mx).exp_()
    total = p.sum(-1)
    o = torch.matmul(p.view(B, K, G * n, keys), gather(1)).view(B, K, G, n, D) / total[..., None]
    lse = mx[..., 0] + total.log()                                          # [B][K][G][n]
    row = torch.arange(pos.numel(), device=pos.device)
    b = torch.searchsorted(starts[1:].contiguous(), row, right=True)
    at = row - starts[b]
    return o.permute(0, 3, 1, 2, 4)[b, at].reshape(-1, H, D), lse.permute(0, 3, 1, 2)[b, at].reshape(-1, H)


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------

def _handle(s):
    """The framework's object for the operator, kept in the state as a program keeps it."""
    if "handle" in s:
        return s["handle"]
    from compressed_sparse_long_c4a_gb300 import dense
    case = s["case"]
    if case["op"] == "plan":
        h = dense.StepPlan(s["table"], s["ring"], s["tokens"])
    else:
        fmt = dense.KV_BF16 if case["fmt"] == "bf16" else dense.KV_FP8_TOKEN
        cache = dense.DenseCache(s["pool"], s.get("table"), case["kv_heads"], case["dim"], fmt)
        if case["op"] == "insert":
            rope = dense.Rope(dims=case["rope_dims"], first=case["rope_first"], theta=10000.0,
                              layout=dense.ROPE_HALF if case["layout"] == "half" else dense.ROPE_INTERLEAVED,
                              **{"none": {}, "linear": {"scaling": dense.ROPE_LINEAR, "factor": 4.0},
                                 "yarn": {"scaling": dense.ROPE_YARN, "factor": 16.0, "original": 65536.0,
                                          "beta_fast": 32.0, "beta_slow": 1.0, "magnitude": s["magnitude"]}}[case["scaling"]])
            h = dense.DenseInsert(cache, case["heads"], rope, s["q_gamma"], s["k_gamma"], eps=1e-6)
        else:
            h = dense.DenseAttention(cache, case["heads"], s["q"].shape[0], s["max_new"], window=case["window"], sinks=case["sinks"])
    s["handle"] = h
    return h


def run(s):
    case = s["case"]
    if case["op"] == "plan":
        if not own:
            return _plan_plain(s)
        h = _handle(s)
        h.run(s["cached"], s["fresh"], s["free_in"], s["free_out"])
        return {"seq_ids": h.seq_ids, "positions": h.positions, "slots": h.slots, "token_starts": h.token_starts,
                "table": s["table"], "ring": s["ring"], "free": s["free_out"]}
    if case["op"] == "insert":
        if not own:
            return _insert_plain(s)
        _handle(s).run(s["q"], s["k"], s["v"], s["q_out"], s["positions"], s["slots"])
        rows, scales = _views(case, s["pool"])
        return {"q": s["q_out"], "cache": rows} if scales is None else {"q": s["q_out"], "cache": rows, "scales": scales}
    if not own:
        o, lse = _attn_plain(s)
        return {"out": s["out"].copy_(o), "lse": s["lse"].copy_(lse)}
    _handle(s).run(s["q"], s["out"], s["positions"], s["starts"], s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "plan":
        return None                 # whole numbers only
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "insert":
        def norm_rope(x, gamma):
            # each pair as a complex number, turned by e^{i position frequency}
            x = x.to(f64)
            if gamma is not None:
                x = x / (x.square().sum(-1, keepdim=True) / case["dim"] + 1e-6).sqrt() * gamma.to(f64)
            R, a = case["rope_dims"], case["rope_first"]
            part = x[..., a:a + R]
            pairs = part.unflatten(-1, (2, R // 2)).transpose(-1, -2) if case["layout"] == "half" else part.unflatten(-1, (R // 2, 2))
            phase = s["positions"].to(f64)[:, None] * s["inv_freq"][None]
            turned = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.full_like(phase, s["magnitude"]), phase)[:, None]
            pairs = torch.view_as_real(turned)
            part = (pairs.transpose(-1, -2) if case["layout"] == "half" else pairs).flatten(-2)
            return torch.cat([x[..., :a], part, x[..., a + R:]], -1)

        rows, scales = _views(case, s["pool"])
        rows = rows.to(f64)
        k, v = norm_rope(s["k"], s["k_gamma"]), s["v"].to(f64)
        page, at = s["slots"] // PAGE, s["slots"] % PAGE
        out = {"q": norm_rope(s["q"], s["q_gamma"])}
        if scales is not None:
            scales = scales.to(f64)
            for n, x in ((0, k), (1, v)):
                sc = x.abs().amax(-1) / 448.0
                sc = torch.where(sc > 0, sc, torch.ones_like(sc))
                scales[page, n, :, at] = sc
                rows[page, n, :, at] = x / sc[..., None]
            return {**out, "cache": rows, "scales": scales}
        rows[page, 0, :, at] = k
        rows[page, 1, :, at] = v
        return {**out, "cache": rows}

    B, H, K, D, W, S = (case[n] for n in ("seqs", "heads", "kv_heads", "dim", "window", "sinks"))
    rows, scales = _views(case, s["pool"])
    out = torch.zeros((s["q"].shape[0], H, D), dtype=f64, device=DEVICE)
    lse = torch.zeros((s["q"].shape[0], H), dtype=f64, device=DEVICE)
    cached, new = _lengths(case)
    t0 = 0
    for b, (c, n) in enumerate(zip(cached, new)):
        lo = max(0, c - W + 1) if W else 0
        j = torch.cat([torch.arange(min(S, lo), device=DEVICE), torch.arange(lo, c + n, device=DEVICE)])
        page, at = s["table"][b].long()[j // PAGE], j % PAGE
        for h in range(K):
            def values(which):
                if scales is None:
                    return rows[page, which, h, at].to(f64)
                return rows.view(torch.uint8)[page, which, h, at].view(torch.float8_e4m3fn).to(f64) * scales[page, which, h, at].to(f64)[:, None]
            k, v = values(0), values(1)
            per = max(1, (1 << 27) // (j.numel() * (H // K)))      # query tokens at once
            for i in range(0, n, per):
                e = min(n, i + per)
                q = s["q"][t0 + i:t0 + e].view(e - i, K, H // K, D)[:, h].to(f64)
                m = torch.arange(c + i, c + e, device=DEVICE)
                z = (q.reshape(-1, D) @ k.T / math.sqrt(D)).view(e - i, H // K, -1)
                hidden = j[None] > m[:, None]
                if W:
                    hidden |= (j[None] <= m[:, None] - W) & (j[None] >= S)
                z.masked_fill_(hidden[:, None], -math.inf)
                top = z.amax(-1, keepdim=True)
                z = (z - top).exp_()
                total = z.sum(-1)
                o = (z.reshape(-1, j.numel()) @ v).view(e - i, H // K, D) / total[..., None]
                out[t0 + i:t0 + e].view(e - i, K, H // K, D)[:, h] = o
                lse[t0 + i:t0 + e].view(e - i, K, H // K)[:, h] = top[..., 0] + total.log()
        t0 += n
    return {"out": out, "lse": lse}
