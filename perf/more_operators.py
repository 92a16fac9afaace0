"""Cases of the operators around a dense cache whose rows are held in 8 bits with
one scale per 64 positions and KV head, and of attention over whole prompts:
the quantising insert, the read back, attention over that cache (decode and
chunks), and attention over packed rows without a cache.

A page holds 256 positions: [KV heads][256][dim] e4m3 key codes, the value codes
in the same layout, then the fp32 scales of the keys' groups [KV heads][4] and
of the values'.  A group is 64 consecutive positions of one page; its scale is
a power of two.  The block table maps a sequence's n-th 256 positions to a page.

`run` computes an operator in elementary torch operations, or, where `own` is
true, through the framework's entry points.
"""
from __future__ import annotations

import math
import random

import torch

own = False

PAGE = 256          # positions per page
GROUP = 64          # positions per scale
LEAST = 2.0 ** -126
DEVICE = "cuda"


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def listed():
    return [
        # ---- norm + rotation + quantising insert (and the rotated keys as rows) ----
        # a decode step of 64 sequences: every token joins a group that earlier steps began (latency)
        {"name": "insert_decode_b64", "op": "insert", "seqs": 64, "heads": 16, "kv_heads": 4, "dim": 128, "new_lo": 1,
         "new_hi": 1, "pos_lo": 65536, "pos_hi": 131072, "layout": "half", "rope_dims": 128, "norm": True,
         "fused": True, "shape_seed": 1},
        # one odd chunk from an odd position on, 64-wide heads, half of the head rotated
        {"name": "insert_chunk_4097", "op": "insert", "seqs": 1, "heads": 64, "kv_heads": 8, "dim": 64, "new_lo": 4097,
         "new_hi": 4097, "pos_lo": 32771, "pos_hi": 32771, "layout": "interleaved", "rope_dims": 32, "norm": True,
         "fused": True, "shape_seed": 2},
        # four whole chunks
        {"name": "insert_prefill_4x4k", "op": "insert", "seqs": 4, "heads": 64, "kv_heads": 8, "dim": 128, "new_lo": 4096,
         "new_hi": 4096, "pos_lo": 0, "pos_hi": 32768, "layout": "half", "rope_dims": 128, "norm": True,
         "fused": False, "shape_seed": 3},
        # ---- reading the cache back ----
        # the cached start of one short conversation (latency)
        {"name": "read_b1_1k", "op": "read", "seqs": 1, "kv_heads": 4, "dim": 128, "len_lo": 1000, "len_hi": 1000,
         "skip_hi": 0, "shape_seed": 4},
        # the shared prefixes of 32 sequences, in front of their fresh tokens
        {"name": "read_b32_8k", "op": "read", "seqs": 32, "kv_heads": 8, "dim": 128, "len_lo": 1000, "len_hi": 8192,
         "skip_hi": 500, "shape_seed": 5},
        # ---- attention over the cache ----
        # one sequence, 1k context (latency)
        {"name": "attn_decode_b1_1k", "op": "attn", "seqs": 1, "heads": 16, "kv_heads": 4, "dim": 128, "cached_lo": 1024,
         "cached_hi": 1024, "new_lo": 1, "new_hi": 1, "window": 0, "sinks": 0, "shape_seed": 6},
        # 32 sequences of 32k to 64k (bandwidth, ragged lengths)
        {"name": "attn_decode_b32_32k_64k", "op": "attn", "seqs": 32, "heads": 64, "kv_heads": 8, "dim": 128,
         "cached_lo": 32768, "cached_hi": 65536, "new_lo": 1, "new_hi": 1, "window": 0, "sinks": 0, "shape_seed": 7},
        # four sequences at 1M
        {"name": "attn_decode_b4_1m", "op": "attn", "seqs": 4, "heads": 16, "kv_heads": 2, "dim": 128,
         "cached_lo": 1048575, "cached_hi": 1048575, "new_lo": 1, "new_hi": 1, "window": 0, "sinks": 0, "shape_seed": 8},
        # the last chunk of a 32k prompt (tensor cores)
        {"name": "attn_prefill_32k", "op": "attn", "seqs": 1, "heads": 32, "kv_heads": 8, "dim": 128, "cached_lo": 28672,
         "cached_hi": 28672, "new_lo": 4096, "new_hi": 4096, "window": 0, "sinks": 0, "shape_seed": 9},
        # ---- attention over whole prompts ----
        # many short prompts of a chat server (latency, ragged)
        {"name": "prompt_short_b64", "op": "prompt", "seqs": 64, "heads": 16, "kv_heads": 4, "dim": 128, "len_lo": 1,
         "len_hi": 256, "prefix_hi": 0, "window": 0, "sinks": 0, "causal": True, "fused": True, "shape_seed": 10},
        # a window layer, some prompts behind a prefix that was read back, 64-wide heads
        {"name": "prompt_window_b8", "op": "prompt", "seqs": 8, "heads": 64, "kv_heads": 8, "dim": 64, "len_lo": 1000,
         "len_hi": 4096, "prefix_hi": 1000, "window": 1024, "sinks": 4, "causal": True, "fused": False, "shape_seed": 11},
        # one 16k prompt
        {"name": "prompt_16k", "op": "prompt", "seqs": 1, "heads": 32, "kv_heads": 8, "dim": 128, "len_lo": 16384,
         "len_hi": 16384, "prefix_hi": 0, "window": 0, "sinks": 0, "causal": True, "fused": False, "shape_seed": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["insert", "read", "attn", "attn", "prompt", "prompt"])
    seed = rng.randrange(1 << 30)
    dim = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 3, 4, 8])
    window = rng.choice([0, 0, 128, 1024])
    sinks = rng.choice([0, 4]) if window else 0
    if op == "insert":
        most = min(16384, 16384 * 80 * 128 // (kv * (group + 2) * dim))
        seqs = _log(rng, 1, 256)
        return {"op": "insert", "seqs": seqs, "heads": kv * group, "kv_heads": kv, "dim": dim, "new_lo": 1,
                "new_hi": rng.choice([1, _log(rng, 2, max(3, most // seqs))]), "pos_lo": 0, "pos_hi": _log(rng, 1, 1 << 20),
                "layout": rng.choice(["half", "interleaved"]), "rope_dims": rng.choice([dim, dim // 2, 16]),
                "norm": rng.random() < 0.8, "fused": rng.random() < 0.5, "shape_seed": seed}
    if op == "read":
        seqs = _log(rng, 1, 64)
        most = min(16384, (1 << 28) // (seqs * kv * dim))
        return {"op": "read", "seqs": seqs, "kv_heads": kv, "dim": dim, "len_lo": 1, "len_hi": _log(rng, 2, most),
                "skip_hi": rng.choice([0, 700]), "shape_seed": seed}
    if op == "attn":
        c = {"op": "attn", "seqs": _log(rng, 1, 64), "heads": kv * group, "kv_heads": kv, "dim": dim, "cached_lo": 0,
             "new_lo": 1, "new_hi": 1, "window": window, "sinks": sinks, "shape_seed": seed}
        if rng.random() < 0.5:      # decode; the cache's values are bounded as in the listed cases
            c["cached_hi"] = _log(rng, 16, max(17, min(1 << 20, (1 << 30) // (c["seqs"] * kv * dim))))
        else:                       # chunks; the rows x keys are bounded as in the listed cases
            c["seqs"] = _log(rng, 1, 8)
            c["new_hi"] = _log(rng, 2, 2048)
            c["cached_hi"] = _log(rng, 16, max(17, min(32768, (1 << 31) // (c["seqs"] * c["heads"] * c["new_hi"])) - c["new_hi"]))
        return c
    seqs = _log(rng, 1, 64)
    most = int(math.sqrt((1 << 33) / (seqs * kv * group)))      # rows x keys
    return {"op": "prompt", "seqs": seqs, "heads": kv * group, "kv_heads": kv, "dim": dim, "len_lo": 1,
            "len_hi": _log(rng, 2, max(3, min(16384, most))), "prefix_hi": rng.choice([0, 0, 300]), "window": window,
            "sinks": sinks, "causal": window > 0 or rng.random() < 0.8, "fused": rng.random() < 0.5, "shape_seed": seed}


def _lengths(case):
    """Two numbers of each sequence, from the case alone: earlier positions (attn, insert: cached; read: skipped;
    prompt: prefix) and rows of the call."""
    r = random.Random(case["shape_seed"])
    lo, hi, a, b = {"insert": ("pos_lo", "pos_hi", "new_lo", "new_hi"), "attn": ("cached_lo", "cached_hi", "new_lo", "new_hi"),
                    "read": (None, "skip_hi", "len_lo", "len_hi"), "prompt": (None, "prefix_hi", "len_lo", "len_hi")}[case["op"]]
    n = case["seqs"]
    before = [r.randint(case[lo] if lo else 0, case[hi]) for _ in range(n)]
    return before, [r.randint(case[a], case[b]) for _ in range(n)]


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _starts(counts):
    s = [0]
    for n in counts:
        s.append(s[-1] + n)
    return s


# --------------------------------------------------------------------------
# Work
# --------------------------------------------------------------------------

def work(case):
    before, new = _lengths(case)
    K, D = case["kv_heads"], case["dim"]
    T = sum(new)
    groups = sum((c + n - 1) // GROUP - c // GROUP + 1 for c, n in zip(before, new))
    if case["op"] == "insert":
        H = case["heads"]
        # rows in; queries and keys out; codes out; a scale per group; positions and slots
        return {"bytes": T * ((H + 2 * K) * D * 2 + (H + K) * D * 2 + 2 * K * D + 12) + groups * 2 * K * 4, "flops": T * (H + 2 * K) * D * 8}
    if case["op"] == "read":
        return {"bytes": T * 2 * K * D * 3 + groups * 2 * K * 4, "flops": T * 2 * K * D}
    H, W, S = case["heads"], case["window"], case["sinks"]
    keys = pairs = 0
    for c, n in zip(before, new):
        last = c + n - 1
        lo = max(0, c - W + 1) if W else 0
        keys += last - lo + 1 + min(S, lo)
        if W:
            pairs += sum(min(m + 1, W) + min(S, max(0, m + 1 - W)) for m in range(c, c + n))
        elif case["op"] == "prompt" and not case["causal"]:
            pairs += n * (c + n)
        else:
            pairs += n * c + n * (n + 1) // 2
    row = 2 * D * (1 if case["op"] == "attn" else 2)
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


def _pool(case, blocks, seed):
    """A page pool with every row filled, as by earlier steps: values of about one, scales 2^-9 to 2^-7."""
    K, D = case["kv_heads"], case["dim"]
    codes = 2 * K * PAGE * D
    pool = torch.empty((blocks, codes + 2 * K * (PAGE // GROUP) * 4), dtype=torch.uint8, device=DEVICE)
    g = _gen(seed, 100)
    at_once = max(1, (1 << 28) // codes)
    for i in range(0, blocks, at_once):
        n = min(at_once, blocks - i)
        v = torch.randn((n, codes), generator=g, device=DEVICE, dtype=torch.float32)
        pool[i:i + n, :codes] = v.mul_(100).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        e = torch.randint(-9, -6, (n, codes // (GROUP * D)), generator=g, device=DEVICE)
        pool[i:i + n, codes:] = torch.exp2(e.float()).view(torch.uint8)
    return pool


def _table(case, first, last, seed):
    """A random block table with pages for positions [first, last) of each sequence, and the pages' count."""
    cols = max(_pages(e) for e in last)
    table = torch.full((len(first), cols), -1, dtype=torch.int32)
    at = 0
    W, S = case.get("window", 0), case.get("sinks", 0)
    for b, (f, e) in enumerate(zip(first, last)):
        lo = max(0, f - W + 1) // PAGE if W else (f // PAGE if case["op"] in ("insert", "read") else 0)
        held = sorted(x for x in set(range(_pages(S) if W else 0)) | set(range(lo, _pages(e))) if x < _pages(e))
        table[b, held] = torch.arange(at, at + len(held), dtype=torch.int32)
        at += len(held)
    order = torch.randperm(at + 3, generator=_gen(seed, 1), device=DEVICE).to(torch.int32)
    table = table.to(DEVICE)
    return torch.where(table < 0, table, order[table.clamp_min(0).long()]).contiguous(), at + 3


def _positions(before, new):
    return torch.cat([torch.arange(c, c + n, dtype=torch.int32) for c, n in zip(before, new)]).to(DEVICE)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _frequencies(case):
    R = case["rope_dims"]
    return 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=DEVICE) / R)


def prepare(case, seed):
    s = {"case": case}
    before, new = _lengths(case)
    ends = [c + n for c, n in zip(before, new)]
    K, D, T = case["kv_heads"], case["dim"], sum(new)
    if case["op"] != "prompt":
        s["table"], pages = _table(case, before, ends, seed)
        s["pool"] = _pool(case, pages, seed)
    if case["op"] == "insert":
        H = case["heads"]
        s["positions"] = _positions(before, new)
        seq = torch.arange(case["seqs"], device=DEVICE).repeat_interleave(torch.tensor(new, device=DEVICE))
        pos = s["positions"].long()
        s["slots"] = s["table"][seq, pos // PAGE].long() * PAGE + pos % PAGE
        if case["fused"]:                       # one projection's output, split by strides
            x = _randn((T, (H + 2 * K) * D), seed, 3, std=2.0, dtype=torch.bfloat16)
            s.update(q=x[:, :H * D].view(T, H, D), k=x[:, H * D:(H + K) * D].view(T, K, D), v=x[:, (H + K) * D:].view(T, K, D))
        else:
            s.update(q=_randn((T, H, D), seed, 3, std=2.0, dtype=torch.bfloat16),
                     k=_randn((T, K, D), seed, 4, std=2.0, dtype=torch.bfloat16),
                     v=_randn((T, K, D), seed, 5, dtype=torch.bfloat16))
        s["q_gamma"] = _randn((D,), seed, 6, std=0.1, mean=1.0) if case["norm"] else None
        s["k_gamma"] = _randn((D,), seed, 7, std=0.1, mean=1.0) if case["norm"] else None
        s["q_out"] = torch.zeros((T, H, D), dtype=torch.bfloat16, device=DEVICE)
        s["k_out"] = torch.zeros((T, K, D), dtype=torch.bfloat16, device=DEVICE)
        return s
    if case["op"] == "read":
        s.update(starts=_int32(_starts(new)), first=_int32(before),
                 k_out=torch.zeros((T, K, D), dtype=torch.bfloat16, device=DEVICE),
                 v_out=torch.zeros((T, K, D), dtype=torch.bfloat16, device=DEVICE))
        return s
    H = case["heads"]
    s.update(starts=_int32(_starts(new)), out=torch.zeros((T, H, D), dtype=torch.bfloat16, device=DEVICE),
             lse=torch.zeros((T, H), dtype=torch.float32, device=DEVICE), max_new=max(new), max_seen=max(ends))
    if case["op"] == "attn":
        s.update(positions=_positions(before, new), q=_randn((T, H, D), seed, 3, std=2.0, dtype=torch.bfloat16))
        return s
    N = sum(ends)
    s.update(kv_starts=_int32(_starts(ends)), q=_randn((T, H, D), seed, 3, std=2.0, dtype=torch.bfloat16))
    if case["fused"]:                           # keys and values side by side in wider rows
        x = _randn((N, 2 * K * D), seed, 4, dtype=torch.bfloat16)
        s.update(k=x[:, :K * D].view(N, K, D), v=x[:, K * D:].view(N, K, D))
    else:
        s.update(k=_randn((N, K, D), seed, 4, dtype=torch.bfloat16), v=_randn((N, K, D), seed, 5, dtype=torch.bfloat16))
    return s


# --------------------------------------------------------------------------
# The plain forms
# --------------------------------------------------------------------------

def _views(case, pool):
    """Codes [page][key, value][KV head][256][dim] and scales [page][key, value][KV head][4]."""
    K, D = case["kv_heads"], case["dim"]
    codes = 2 * K * PAGE * D
    return (pool[:, :codes].view(torch.float8_e4m3fn).unflatten(1, (2, K, PAGE, D)),
            pool[:, codes:].view(torch.float32).unflatten(1, (2, K, PAGE // GROUP)))


def _rotate(x, case, cos, sin):
    """x [T][heads][dim], cos and sin [T][rotated / 2], in x's type."""
    R = case["rope_dims"]
    y = x.clone()
    if case["layout"] == "half":
        p, q = x[..., :R // 2], x[..., R // 2:R]
        y[..., :R // 2] = p * cos[:, None] - q * sin[:, None]
        y[..., R // 2:R] = p * sin[:, None] + q * cos[:, None]
    else:
        p, q = x[..., :R:2], x[..., 1:R:2]
        y[..., :R:2] = p * cos[:, None] - q * sin[:, None]
        y[..., 1:R:2] = p * sin[:, None] + q * cos[:, None]
    return y


def _power(amax):
    """The smallest power of two s with amax / s <= 448, at least 2^-126."""
    m, e = torch.frexp(amax)                    # amax = m 2^e, m in [0.5, 1)
    e = e - torch.where(m > 0.875, 8, 9)        # 448 = 0.875 * 2^9
    return torch.where(amax > 0, torch.exp2(e.clamp_min(-126).to(amax.dtype)), LEAST)


def _insert_plain(s):
    case, slots = s["case"], s["slots"]
    K, D = case["kv_heads"], case["dim"]
    ang = s["positions"].double()[:, None] * _frequencies(case)[None]
    cos, sin = ang.cos().float(), ang.sin().float()

    def prep(x, gamma):
        x = x.float()
        if gamma is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * gamma
        return _rotate(x, case, cos, sin)

    s["q_out"].copy_(prep(s["q"], s["q_gamma"]))
    s["k_out"].copy_(prep(s["k"], s["k_gamma"]))
    codes, scales = _views(case, s["pool"])
    kv = torch.stack([s["k_out"], s["v"]], 1).float()                       # [T][2][K][D]
    page, row = slots // PAGE, slots % PAGE
    each, back = torch.unique(slots // GROUP, return_inverse=True)          # the groups that the call writes to
    gp, gr = each // (PAGE // GROUP), each % (PAGE // GROUP)
    mag = kv.abs().amax(-1)                                                 # [T][2][K]
    amax = torch.zeros((each.numel(), 2, K), device=DEVICE).scatter_reduce_(0, back[:, None, None].expand(-1, 2, K), mag, "amax")
    written = torch.zeros((each.numel(), GROUP), dtype=torch.bool, device=DEVICE)
    written[back, row % GROUP] = True
    old = torch.where(written[:, :1, None], LEAST, scales[gp, :, :, gr])    # a group begins anew with its first row
    new = torch.maximum(_power(amax), old)
    # rows that stay: their values in the grown scale
    at = gr[:, None] * GROUP + torch.arange(GROUP, device=DEVICE)           # [groups][64] rows of the page
    raw = codes.view(torch.uint8)
    rows = raw[gp[:, None], :, :, at]                                       # [groups][64][2][K][D]
    grown = (rows.view(torch.float8_e4m3fn).float() * (old / new)[:, None, :, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    stay = ~written[:, :, None, None, None] & (new > old)[:, None, :, :, None] & ~written[:, :1, None, None, None]
    raw[gp[:, None], :, :, at] = torch.where(stay, grown, rows)
    code = (kv / new[back][..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    raw[page, :, :, row] = code.view(torch.uint8)
    scales[gp, :, :, gr] = new
    return {"q": s["q_out"], "k": s["k_out"], "cache": codes, "scales": scales}


def _read_plain(s):
    case, starts = s["case"], s["starts"].long()
    r = torch.arange(s["k_out"].shape[0], device=DEVICE)
    b = torch.searchsorted(starts[1:].contiguous(), r, right=True)
    pos = s["first"].long()[b] + r - starts[b]
    page, at = s["table"][b, pos // PAGE].long(), pos % PAGE
    codes, scales = _views(case, s["pool"])
    for which, out in ((0, s["k_out"]), (1, s["v_out"])):
        x = codes.view(torch.uint8)[page, which, :, at].view(torch.float8_e4m3fn).float()
        out.copy_(x * scales[page, which, :, at // GROUP][..., None])
    return {"k": s["k_out"], "v": s["v_out"]}


def _softmax_attention(q, k, v, seen, scale):
    """q [B][K][G][n][D], k and v [B][K][keys][D], seen(i, e) the mask [B][e - i][keys] -> (o, lse) [B][n][K][G]..."""
    B, K, G, n, D = q.shape
    keys = k.shape[2]
    o = torch.empty((B, n, K, G, D), device=DEVICE)
    lse = torch.empty((B, n, K, G), device=DEVICE)
    per = max(1, (1 << 30) // (B * K * G * keys))           # query tokens at once
    for i in range(0, n, per):
        e = min(n, i + per)
        z = torch.matmul(q[:, :, :, i:e].reshape(B, K, G * (e - i), D), k.transpose(2, 3)).view(B, K, G, e - i, keys).mul_(scale)
        z.masked_fill_(~seen(i, e)[:, None, None], -math.inf)
        top = z.amax(-1, keepdim=True)
        p = z.sub_(top.clamp_min(-1e30)).exp_()
        total = p.sum(-1)
        x = torch.matmul(p.view(B, K, G * (e - i), keys), v).view(B, K, G, e - i, D) / total.clamp_min(1e-30)[..., None]
        o[:, i:e] = x.permute(0, 3, 1, 2, 4)
        lse[:, i:e] = (top[..., 0] + total.log()).permute(0, 3, 1, 2)
    return o, lse


def _pack(s, x):
    """Padded rows [B][n]... of each sequence -> the packed ones."""
    starts = s["starts"].long()
    r = torch.arange(s["q"].shape[0], device=DEVICE)
    b = torch.searchsorted(starts[1:].contiguous(), r, right=True)
    return x[b, r - starts[b]].flatten(1, 2)


def _attn_plain(s):
    case = s["case"]
    B, H, K, D, W, S = (case[n] for n in ("seqs", "heads", "kv_heads", "dim", "window", "sinks"))
    G, starts, pos, n = H // K, s["starts"].long(), s["positions"].long(), s["max_new"]
    keys = min(s["max_seen"], W - 1 + n + S) if W else s["max_seen"]
    first, count = pos[starts[:-1]], starts[1:] - starts[:-1]
    t = (starts[:-1, None] + torch.arange(n, device=DEVICE)).clamp_max(pos.numel() - 1)
    lo = (first - W + 1).clamp_min(0) if W else torch.zeros_like(first)
    lead = lo.clamp_max(S)[:, None]                                         # sinks in front of the range
    j = torch.arange(keys, device=DEVICE)[None]
    j = torch.where(j < lead, j, lo[:, None] + j - lead)                    # [B][keys] positions
    last = (first + count - 1)[:, None]
    page = s["table"][torch.arange(B, device=DEVICE)[:, None], torch.minimum(j, last) // PAGE].long()
    live = (j <= last) & (page >= 0)
    page, at = page.clamp_min(0), j % PAGE
    codes, scales = _views(case, s["pool"])

    def gather(which):      # [B][K][keys][D]
        x = codes.view(torch.uint8)[page, which, :, at].view(torch.float8_e4m3fn).float()
        x = x * scales[page, which, :, at // GROUP][..., None]
        return torch.where(live[..., None, None], x, 0.0).transpose(1, 2)

    def seen(i, e):
        m = first[:, None, None] + torch.arange(i, e, device=DEVICE)[None, :, None]
        ok = live[:, None] & (j[:, None] <= m)
        return ok & ((j[:, None] > m - W) | (j[:, None] < S)) if W else ok

    q = s["q"][t].float().view(B, n, K, G, D).permute(0, 2, 3, 1, 4)
    o, lse = _softmax_attention(q, gather(0), gather(1), seen, 1.0 / math.sqrt(D))
    return {"out": s["out"].copy_(_pack(s, o)), "lse": s["lse"].copy_(_pack(s, lse[..., None])[..., 0])}


def _prompt_plain(s):
    case = s["case"]
    H, K, D, W, S = (case[n] for n in ("heads", "kv_heads", "dim", "window", "sinks"))
    G, starts, ks, n, keys = H // K, s["starts"].long(), s["kv_starts"].long(), s["max_new"], s["max_seen"]
    count, have = starts[1:] - starts[:-1], ks[1:] - ks[:-1]
    t = (starts[:-1, None] + torch.arange(n, device=DEVICE)).clamp_max(s["q"].shape[0] - 1)
    j = torch.arange(keys, device=DEVICE)[None]
    at = (ks[:-1, None] + j).clamp_max(s["k"].shape[0] - 1)

    def seen(i, e):
        m = (have - count)[:, None, None] + torch.arange(i, e, device=DEVICE)[None, :, None]
        ok = (j < have[:, None])[:, None].expand(-1, e - i, -1)
        if case["causal"]:
            ok = ok & (j[:, None] <= m)
        return ok & ((j[:, None] > m - W) | (j[:, None] < S)) if W else ok

    q = s["q"][t].float().view(-1, n, K, G, D).permute(0, 2, 3, 1, 4)
    k, v = (x[at].float().transpose(1, 2) for x in (s["k"], s["v"]))
    o, lse = _softmax_attention(q, k, v, seen, 1.0 / math.sqrt(D))
    return {"out": s["out"].copy_(_pack(s, o)), "lse": s["lse"].copy_(_pack(s, lse[..., None])[..., 0])}


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------

def _handle(s):
    """The framework's object for the operator, kept in the state as a program keeps it."""
    if "handle" in s:
        return s["handle"]
    from compressed_sparse_long_c4a_gb300 import dense
    case = s["case"]
    if case["op"] == "prompt":
        h = dense.PromptAttention(case["heads"], case["kv_heads"], case["dim"], case["seqs"], s["q"].shape[0], s["max_new"],
                                  causal=case["causal"], window=case["window"], sinks=case["sinks"], device=s["q"].device)
    else:
        cache = dense.DenseCache(s["pool"], s["table"], case["kv_heads"], case["dim"], dense.KV_FP8_GROUP)
        if case["op"] == "insert":
            rope = dense.Rope(dims=case["rope_dims"], theta=10000.0,
                              layout=dense.ROPE_HALF if case["layout"] == "half" else dense.ROPE_INTERLEAVED)
            h = dense.DenseInsert(cache, case["heads"], rope, s["q_gamma"], s["k_gamma"], eps=1e-6)
        elif case["op"] == "read":
            h = dense.DenseRead(cache)
        else:
            h = dense.DenseAttention(cache, case["heads"], s["q"].shape[0], s["max_new"], window=case["window"], sinks=case["sinks"])
    s["handle"] = h
    return h


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"insert": _insert_plain, "read": _read_plain, "attn": _attn_plain, "prompt": _prompt_plain}[op](s)
    h = _handle(s)
    if op == "insert":
        h.run(s["q"], s["k"], s["v"], s["q_out"], s["positions"], s["slots"], k_out=s["k_out"])
        codes, scales = _views(s["case"], s["pool"])
        return {"q": s["q_out"], "k": s["k_out"], "cache": codes, "scales": scales}
    if op == "read":
        h.run(s["starts"], s["k_out"], s["v_out"], first=s["first"])
        return {"k": s["k_out"], "v": s["v_out"]}
    if op == "attn":
        h.run(s["q"], s["out"], s["positions"], s["starts"], s["lse"])
    else:
        h.run(s["q"], s["k"], s["v"], s["out"], s["starts"], s["kv_starts"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------

def _exact_insert(s, case):
    f64 = torch.float64
    K, D, R = case["kv_heads"], case["dim"], case["rope_dims"]

    def norm_rope(x, gamma):
        # each pair as a complex number, turned by e^{i position frequency}
        x = x.to(f64)
        if gamma is not None:
            x = x / (x.square().sum(-1, keepdim=True) / D + 1e-6).sqrt() * gamma.to(f64)
        part = x[..., :R]
        half = case["layout"] == "half"
        pairs = part.unflatten(-1, (2, R // 2)).transpose(-1, -2) if half else part.unflatten(-1, (R // 2, 2))
        phase = s["positions"].to(f64)[:, None] * 10000.0 ** (-torch.arange(R // 2, device=DEVICE, dtype=f64) * 2 / R)
        turned = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.ones_like(phase), phase)[:, None]
        pairs = torch.view_as_real(turned)
        return torch.cat([(pairs.transpose(-1, -2) if half else pairs).flatten(-2), x[..., R:]], -1)

    k = norm_rope(s["k"], s["k_gamma"])
    codes, scales = _views(case, s["pool"])
    codes, scales = codes.to(f64), scales.to(f64)
    # the cache holds the keys as they are rounded to bf16
    rows = (k.to(torch.bfloat16).to(f64), s["v"].to(f64))
    slots = s["slots"].tolist()
    at = 0
    while at < len(slots):                      # a run of tokens in one group
        g = slots[at] // GROUP
        end = at
        while end < len(slots) and slots[end] // GROUP == g:
            end += 1
        page, r0, r1 = slots[at] // PAGE, slots[at] % PAGE, slots[end - 1] % PAGE + 1
        gr = r0 // GROUP
        for which in (0, 1):
            x = rows[which][at:end].transpose(0, 1)                         # [K][n][D]
            amax = x.abs().amax((1, 2))
            s_new = torch.full_like(amax, LEAST)                            # doubled until the largest value fits
            while (amax > 448.0 * s_new).any():
                s_new = torch.where(amax > 448.0 * s_new, 2.0 * s_new, s_new)
            if r0 % GROUP:
                s_old = scales[page, which, :, gr]
                s_new = torch.maximum(s_new, s_old)
                lo = gr * GROUP
                part = codes[page, which, :, lo:lo + GROUP]
                part *= (s_old / s_new)[:, None, None]
            codes[page, which, :, r0:r1] = x / s_new[:, None, None]
            scales[page, which, :, gr] = s_new
        at = end
    return {"q": norm_rope(s["q"], s["q_gamma"]), "k": k, "cache": codes, "scales": scales}


def exact(case, seed):
    if case["op"] in ("attn", "prompt") and work(case)["flops"] > 6e12:
        return None                             # over 20 seconds in 64 bits
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "insert":
        return _exact_insert(s, case)
    before, new = _lengths(case)
    K, D = case["kv_heads"], case["dim"]

    def cached(b, which, h, j):                 # values of positions j
        codes, scales = _views(case, s["pool"])
        page, at = s["table"][b].long()[j // PAGE], j % PAGE
        return (codes.view(torch.uint8)[page, which, h, at].view(torch.float8_e4m3fn).to(f64)
                * scales[page, which, h, at // GROUP].to(f64)[:, None])

    if case["op"] == "read":
        out = [[], []]
        for b, (c, n) in enumerate(zip(before, new)):
            j = torch.arange(c, c + n, device=DEVICE)
            for which in (0, 1):
                out[which].append(torch.stack([cached(b, which, h, j) for h in range(K)], 1))
        return {"k": torch.cat(out[0]), "v": torch.cat(out[1])}

    H, W, S = case["heads"], case["window"], case["sinks"]
    G = H // K
    out = torch.zeros((sum(new), H, D), dtype=f64, device=DEVICE)
    lse = torch.zeros((sum(new), H), dtype=f64, device=DEVICE)
    t0 = n0 = 0
    for b, (c, n) in enumerate(zip(before, new)):
        lo = max(0, c - W + 1) if W else 0
        j = torch.cat([torch.arange(min(S, lo), device=DEVICE), torch.arange(lo, c + n, device=DEVICE)])
        for h in range(K):
            if case["op"] == "attn":
                k, v = cached(b, 0, h, j), cached(b, 1, h, j)
            else:
                k, v = (x[n0:n0 + c + n, h][j].to(f64) for x in (s["k"], s["v"]))
            per = max(1, (1 << 27) // (j.numel() * G))                      # query tokens at once
            causal = case["op"] == "attn" or case["causal"]
            for i in range(0, n, per):
                e = min(n, i + per)
                near = int((j < c + e).sum()) if causal else j.numel()      # keys that one of them sees
                q = s["q"][t0 + i:t0 + e, h * G:(h + 1) * G].to(f64)
                z = (q.reshape(-1, D) @ k[:near].T / math.sqrt(D)).view(e - i, G, -1)
                if causal:
                    m = torch.arange(c + i, c + e, device=DEVICE)
                    hidden = j[None, :near] > m[:, None]
                    if W:
                        hidden |= (j[None, :near] <= m[:, None] - W) & (j[None, :near] >= S)
                    z.masked_fill_(hidden[:, None], -math.inf)
                top = z.amax(-1, keepdim=True)
                z = (z - top).exp_()
                total = z.sum(-1)
                out[t0 + i:t0 + e, h * G:(h + 1) * G] = (z.reshape(-1, near) @ v[:near]).view(e - i, G, D) / total[..., None]
                lse[t0 + i:t0 + e, h * G:(h + 1) * G] = top[..., 0] + total.log()
        t0 += n
        n0 += c + n
    return {"out": out, "lse": lse}
