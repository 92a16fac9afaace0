"""ctypes binding of the dense-layer operators (v4a_dense.h): the step plan,
norm + rotation + cache insert, attention over the dense paged cache, the read
back of cached rows, and attention of whole prompts over packed rows.

Argument marshalling only: every object checks its tensors, keeps the C
argument struct and the workspace, and calls the library on the current (or
the given) stream of its tensors' device.  There is no CPU or eager fallback.
"""
from __future__ import annotations

import ctypes as C
import math
from dataclasses import dataclass

import torch

from . import v4a
from .v4a import KV_BF16, KV_FP8_TOKEN  # noqa: F401

BLOCK_POSITIONS = 256
ROPE_INTERLEAVED, ROPE_HALF = 0, 1
ROPE_PLAIN, ROPE_LINEAR, ROPE_YARN, ROPE_TABLE = 0, 1, 2, 3
KV_FP8_GROUP = 3           # e4m3 codes with one power-of-two scale per 64 positions and KV head
GROUP_POSITIONS = 64
DEV_OUT_OF_PAGES = 16

_p = C.c_void_p


class PlanArgs(C.Structure):
    _fields_ = [("num_seqs", C.c_int32), ("num_tables", C.c_int32), ("max_tokens", C.c_int32), ("max_blocks", C.c_int32),
                ("cached", _p), ("fresh", _p), ("block_table", _p), ("table_stride", C.c_int64), ("num_blocks", C.c_int64),
                ("free_ring", _p), ("ring_cap", C.c_int32), ("free_in", _p), ("free_out", _p), ("seq_ids", _p),
                ("positions", _p), ("slots", _p), ("token_starts", _p), ("status", _p)]


class CacheArgs(C.Structure):
    _fields_ = [("num_kv_heads", C.c_int32), ("dim", C.c_int32), ("format", C.c_int32), ("pool", _p),
                ("num_blocks", C.c_int64), ("block_bytes", C.c_int64), ("block_table", _p), ("max_blocks", C.c_int32)]


class RopeArgs(C.Structure):
    _fields_ = [("dims", C.c_int32), ("first", C.c_int32), ("layout", C.c_int32), ("scaling", C.c_int32),
                ("theta", C.c_double), ("factor", C.c_double), ("original", C.c_double), ("beta_fast", C.c_double),
                ("beta_slow", C.c_double), ("magnitude", C.c_double), ("inv_freq", C.POINTER(C.c_double))]


class InsertArgs(C.Structure):
    _fields_ = [("num_tokens", C.c_int32), ("positions", _p), ("slots", _p), ("num_heads", C.c_int32), ("q", _p),
                ("q_stride", C.c_int64), ("q_out", _p), ("q_out_stride", C.c_int64), ("k", _p), ("k_stride", C.c_int64),
                ("v", _p), ("v_stride", C.c_int64), ("q_gamma", _p), ("k_gamma", _p), ("eps", C.c_float),
                ("rope", RopeArgs), ("kv", CacheArgs), ("status", _p)]


class AttnArgs(C.Structure):
    _fields_ = [("num_tokens", C.c_int32), ("num_seqs", C.c_int32), ("max_new_per_seq", C.c_int32), ("positions", _p),
                ("token_starts", _p), ("kv", CacheArgs), ("num_heads", C.c_int32), ("q", _p), ("softmax_scale", C.c_float),
                ("window", C.c_int32), ("sinks", C.c_int32), ("out", _p), ("lse", _p), ("status", _p)]


class ReadArgs(C.Structure):
    _fields_ = [("num_rows", C.c_int32), ("num_seqs", C.c_int32), ("row_starts", _p), ("first", _p), ("kv", CacheArgs), ("k", _p),
                ("k_stride", C.c_int64), ("v", _p), ("v_stride", C.c_int64), ("status", _p)]


class PromptArgs(C.Structure):
    _fields_ = [("num_tokens", C.c_int32), ("num_kv_tokens", C.c_int32), ("num_seqs", C.c_int32), ("max_new_per_seq", C.c_int32),
                ("token_starts", _p), ("kv_starts", _p), ("num_heads", C.c_int32), ("num_kv_heads", C.c_int32), ("dim", C.c_int32),
                ("causal", C.c_int32), ("window", C.c_int32), ("sinks", C.c_int32), ("softmax_scale", C.c_float), ("q", _p),
                ("q_stride", C.c_int64), ("k", _p), ("k_stride", C.c_int64), ("v", _p), ("v_stride", C.c_int64), ("out", _p),
                ("lse", _p), ("status", _p)]


_sigs_done = False


def lib() -> C.CDLL:
    """libv4a with the dense operators' signatures set."""
    global _sigs_done
    L = v4a.lib()
    if not _sigs_done:
        L.v4a_plan_workspace_size.argtypes = [C.POINTER(PlanArgs)]
        L.v4a_plan_workspace_size.restype = C.c_size_t
        L.v4a_step_plan.argtypes = [C.POINTER(PlanArgs), _p, C.c_size_t, _p]
        L.v4a_dense_block_bytes.argtypes = [C.c_int32, C.c_int32, C.c_int32]
        L.v4a_dense_block_bytes.restype = C.c_int64
        L.v4a_dense_insert.argtypes = [C.POINTER(InsertArgs), _p]
        L.v4a_dense_insert_rows.argtypes = [C.POINTER(InsertArgs), _p, C.c_int64, _p]
        L.v4a_dense_read.argtypes = [C.POINTER(ReadArgs), _p]
        L.v4a_prompt_attn_workspace_size.argtypes = [C.POINTER(PromptArgs)]
        L.v4a_prompt_attn_workspace_size.restype = C.c_size_t
        L.v4a_prompt_attn.argtypes = [C.POINTER(PromptArgs), _p, C.c_size_t, _p]
        L.v4a_dense_attn_workspace_size.argtypes = [C.POINTER(AttnArgs)]
        L.v4a_dense_attn_workspace_size.restype = C.c_size_t
        L.v4a_dense_attn.argtypes = [C.POINTER(AttnArgs), _p, C.c_size_t, _p]
        _sigs_done = True
    return L


def block_bytes(num_kv_heads: int, dim: int, fmt: int) -> int:
    """Bytes of one 256-position block (the page size of a pages.block_kind); 0 on a bad shape."""
    return int(lib().v4a_dense_block_bytes(num_kv_heads, dim, fmt))


def _want(t, name, dtype, device, shape=None, contiguous=True):
    """Raises ValueError unless t is a tensor of that type, device and shape (None in shape: any)."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name}: want a {dtype} tensor on {device}")
    if shape is not None and (t.dim() != len(shape) or any(w is not None and w != n for w, n in zip(shape, t.shape))):
        raise ValueError(f"{name}: want shape {shape}, got {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t


class _Op:
    """Launches on the tensors' device, whatever the current one is.  A handle
    keeps one argument struct and one workspace: calls that may run at the same
    time (streams, threads, graphs replayed side by side) need handles of their own.

    The handle's own tensors are made on the stream that is current at its
    construction.  Its first call on another stream waits for that, and the
    handle may be dropped while calls are queued; neither holds for a capture:
    construct the handle before it (torch.cuda.graph synchronises when it
    begins) and keep the handle as long as the graph.  The caller's tensors are
    the caller's to order and to keep."""

    def _launch(self, stream):
        """Calls the C entry on the kept argument struct."""
        dev = self.device
        if dev.type != "cuda":
            raise ValueError(f"{self._where}: the tensors are on {dev}")
        if stream is None:
            raw = torch._C._cuda_getCurrentRawStream(dev.index)      # (a stream object takes 2 us)
        elif stream.device != dev:
            raise ValueError(f"{self._where}: the stream is on {stream.device}, the tensors on {dev}")
        else:
            raw = stream.cuda_stream
        if raw not in self._streams:
            self._enter(raw, torch.cuda.current_stream(dev) if stream is None else stream)
        if torch.cuda.current_device() == dev.index:
            rc = self._fn(*self._call, raw)
        else:
            with torch.cuda.device(dev):
                rc = self._fn(*self._call, raw)
        if rc:
            v4a._check(self._where, rc)

    def _enter(self, raw, stream):
        """The first call on a stream: behind the construction, whose memory the stream uses from now on."""
        with torch.cuda.stream(stream):
            if torch.cuda.is_current_stream_capturing():
                return
        if self._made is not None:
            stream.wait_event(self._made)
        for t in self._own:
            t.record_stream(stream)
        self._streams.add(raw)

    def _bind(self, where, fn, workspace=None, outputs=()):
        """The C entry, and the tensors that the handle has made for it."""
        self._where, self._fn, self.workspace = where, fn, workspace
        ws = () if workspace is None else (workspace.data_ptr(), workspace.numel())
        self._call = (C.byref(self.args), *ws)
        self._own = [t for t in (self.status, workspace, *outputs) if t is not None]
        self._streams, self._made = set(), None
        if self.device.type == "cuda":
            with torch.cuda.device(self.device):
                self._streams.add(torch._C._cuda_getCurrentRawStream(self.device.index))
                if not torch.cuda.is_current_stream_capturing():
                    self._made = torch.cuda.Event()
                    self._made.record()


class StepPlan(_Op):
    """v4a_step_plan for block tables [tables][sequences][columns] (int32) and
    a ring of free page ids; owns the step's token arrays (seq_ids, positions,
    slots [tables][max_tokens], token_starts), the status word and the workspace.

    num_blocks: pages of the pool (default: the ring's length).

    A sequence ends with all blocks of its row.  Blocks behind a window are the
    caller's to give back, between two calls and behind the ring's last free
    page, and so is the end of a sequence whose row has such holes.
    """

    def __init__(self, block_table: torch.Tensor, free_ring: torch.Tensor, max_tokens: int, num_blocks: int | None = None):
        dev = self.device = block_table.device
        _want(block_table, "block_table", torch.int32, dev, (None, None, None))
        _want(free_ring, "free_ring", torch.int32, dev, (None,))
        n_tab, n_seq, cols = block_table.shape
        self.block_table, self.free_ring = block_table, free_ring
        self.seq_ids = torch.full((max_tokens,), -1, dtype=torch.int32, device=dev)
        self.positions = torch.full((max_tokens,), -1, dtype=torch.int32, device=dev)
        self.slots = torch.full((n_tab, max_tokens), -1, dtype=torch.int64, device=dev)
        self.token_starts = torch.zeros(n_seq + 1, dtype=torch.int32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.args = PlanArgs(n_seq, n_tab, max_tokens, cols, None, None, block_table.data_ptr(), n_seq * cols,
                             free_ring.numel() if num_blocks is None else num_blocks, free_ring.data_ptr(),
                             free_ring.numel(), None, None, self.seq_ids.data_ptr(), self.positions.data_ptr(),
                             self.slots.data_ptr(), self.token_starts.data_ptr(), self.status.data_ptr())
        need = lib().v4a_plan_workspace_size(C.byref(self.args))
        if need == 0:
            raise ValueError("StepPlan: sizes outside v4a_step_plan's limits")
        self._bind("v4a_step_plan", lib().v4a_step_plan, torch.empty(need, dtype=torch.uint8, device=dev),
                   (self.seq_ids, self.positions, self.slots, self.token_starts))

    def run(self, cached: torch.Tensor, fresh: torch.Tensor, free_in: torch.Tensor, free_out: torch.Tensor | None = None,
            stream=None):
        """cached, fresh: int32 [sequences]; free_in, free_out: int32 [2] (first free, count); free_out defaults to free_in."""
        a, dev = self.args, self.device
        free_out = free_in if free_out is None else free_out
        for n, t, k in (("cached", cached, a.num_seqs), ("fresh", fresh, a.num_seqs), ("free_in", free_in, 2), ("free_out", free_out, 2)):
            if not (isinstance(t, torch.Tensor) and t.dtype is torch.int32 and t.device == dev and t.shape == (k,) and t.is_contiguous()):
                _want(t, n, torch.int32, dev, (k,))
        a.cached, a.fresh, a.free_in, a.free_out = cached.data_ptr(), fresh.data_ptr(), free_in.data_ptr(), free_out.data_ptr()
        self._launch(stream)


@dataclass
class Rope:
    """The position rotation of v4a_rope; table: inverse frequencies (ROPE_TABLE).

    ROPE_YARN blends frequencies by a ramp that is linear in their turns over
    the original context, as the YaRN paper has it.  Many models' own code has
    a ramp linear in the pair index instead: their frequencies are a table."""
    dims: int
    first: int = 0
    layout: int = ROPE_INTERLEAVED
    scaling: int = ROPE_PLAIN
    theta: float = 10000.0
    factor: float = 1.0
    original: float = 0.0
    beta_fast: float = 32.0
    beta_slow: float = 1.0
    magnitude: float = 1.0
    table: list | None = None

    def struct(self) -> RopeArgs:
        tab = None
        if self.table is not None:
            if len(self.table) != self.dims // 2:
                raise ValueError("Rope: the table holds dims / 2 inverse frequencies")
            tab = (C.c_double * len(self.table))(*self.table)
        return RopeArgs(self.dims, self.first, self.layout, self.scaling, self.theta, self.factor, self.original,
                        self.beta_fast, self.beta_slow, self.magnitude, tab)


class DenseCache:
    """A dense paged cache: pool [blocks][block bytes] uint8 (rows may be wider
    than block_bytes(), as pages of a shared bucket are) and a block table
    [sequences][columns] int32 (None where only inserts use the cache)."""

    def __init__(self, pool: torch.Tensor, block_table: torch.Tensor | None, num_kv_heads: int, dim: int, fmt: int = KV_BF16):
        self.device = pool.device
        _want(pool, "pool", torch.uint8, self.device, (None, None))
        need = block_bytes(num_kv_heads, dim, fmt)
        if need == 0 or pool.shape[1] < need:
            raise ValueError(f"DenseCache: a block of this shape takes {need} bytes, the pool's have {pool.shape[1]}")
        if block_table is not None:
            _want(block_table, "block_table", torch.int32, self.device, (None, None))
        self.pool, self.block_table = pool, block_table
        self.num_kv_heads, self.dim, self.fmt = num_kv_heads, dim, fmt

    def struct(self) -> CacheArgs:
        bt = self.block_table
        return CacheArgs(self.num_kv_heads, self.dim, self.fmt, self.pool.data_ptr(), self.pool.shape[0],
                         self.pool.shape[1], None if bt is None else bt.data_ptr(), 0 if bt is None else bt.shape[1])


def _rows(t, name, device, heads, dim, tokens):
    """Token stride of a [tokens][heads][dim] bf16 tensor whose heads are contiguous."""
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.bfloat16 and t.device == device and t.shape == (tokens, heads, dim)):
        _want(t, name, torch.bfloat16, device, (tokens, heads, dim), contiguous=False)
    st = t.stride()
    if st[2] != 1 or st[1] != dim and heads > 1:
        raise ValueError(f"{name}: heads and dims must be contiguous")
    return st[0] if tokens > 1 else heads * dim      # (one token's stride may be anything, and is not used)


class DenseInsert(_Op):
    """v4a_dense_insert into `cache`: the queries' and keys' norm (None gamma:
    none) and rotation, and the keys' and values' insert.  With k_out a run also
    leaves the keys as packed rows (v4a_dense_insert_rows), which a KV_FP8_GROUP
    cache always needs: it holds those rows quantised."""

    def __init__(self, cache: DenseCache, num_heads: int, rope: Rope | None, q_gamma=None, k_gamma=None, eps: float = 1e-6):
        self.cache, self.device = cache, cache.device
        for n, g in (("q_gamma", q_gamma), ("k_gamma", k_gamma)):
            if g is not None:
                _want(g, n, torch.float32, self.device, (cache.dim,))
        self.q_gamma, self.k_gamma = q_gamma, k_gamma
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._rope = (rope or Rope(0)).struct()      # keeps a frequency table alive
        self.args = InsertArgs(0, None, None, num_heads, None, 0, None, 0, None, 0, None, 0,
                               None if q_gamma is None else q_gamma.data_ptr(), None if k_gamma is None else k_gamma.data_ptr(),
                               eps, self._rope, cache.struct(), self.status.data_ptr())
        self._bind("v4a_dense_insert", lib().v4a_dense_insert)
        self._args = self._call[0]
        self._plain = None if cache.fmt == KV_FP8_GROUP else (self._where, self._fn, self._call)
        self._with_rows = "v4a_dense_insert_rows", lib().v4a_dense_insert_rows

    def run(self, q, k, v, q_out, positions: torch.Tensor, slots: torch.Tensor, stream=None, k_out=None):
        """q, q_out [T][heads][dim], k, v, k_out [T][KV heads][dim] bf16 (any
        token stride of a multiple of 8; q and q_out None with num_heads = 0;
        k_out may be k); positions int32 [T], slots int64 [T]."""
        a, c, dev = self.args, self.cache, self.device
        n = k.shape[0] if isinstance(k, torch.Tensor) and k.dim() else 0
        a.num_tokens = n
        if a.num_heads:
            a.q_stride = _rows(q, "q", dev, a.num_heads, c.dim, n)
            a.q_out_stride = _rows(q_out, "q_out", dev, a.num_heads, c.dim, n)
            a.q, a.q_out = q.data_ptr(), q_out.data_ptr()
        a.k_stride = _rows(k, "k", dev, c.num_kv_heads, c.dim, n)
        a.v_stride = _rows(v, "v", dev, c.num_kv_heads, c.dim, n)
        a.k, a.v = k.data_ptr(), v.data_ptr()
        for name, t, dtype in (("positions", positions, torch.int32), ("slots", slots, torch.int64)):
            if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == dev and t.shape == (n,) and t.is_contiguous()):
                _want(t, name, dtype, dev, (n,))
        a.positions, a.slots = positions.data_ptr(), slots.data_ptr()
        if k_out is not None:
            stride = _rows(k_out, "k_out", dev, c.num_kv_heads, c.dim, n)
            self._where, self._fn = self._with_rows
            self._call = (self._args, k_out.data_ptr(), stride)
        elif self._plain is None:
            raise ValueError("DenseInsert: a cache with a scale per group needs k_out")
        else:
            self._where, self._fn, self._call = self._plain
        self._launch(stream)


class DenseRead(_Op):
    """v4a_dense_read from `cache` (its block table's rows are the sequences)."""

    def __init__(self, cache: DenseCache):
        if cache.block_table is None:
            raise ValueError("DenseRead: the cache has no block table")
        self.cache, self.device = cache, cache.device
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.args = ReadArgs(0, cache.block_table.shape[0], None, None, cache.struct(), None, 0, None, 0, self.status.data_ptr())
        self._bind("v4a_dense_read", lib().v4a_dense_read)

    def run(self, row_starts: torch.Tensor, k: torch.Tensor, v: torch.Tensor, first: torch.Tensor | None = None, stream=None):
        """k, v [N][KV heads][dim] bf16 (any row stride of a multiple of 8)
        receive positions first[b] .. of sequence b (None: 0 ..) at rows
        row_starts[b] ..; row_starts int32 [sequences + 1], first int32 [sequences]."""
        a, c, dev = self.args, self.cache, self.device
        n = k.shape[0] if isinstance(k, torch.Tensor) and k.dim() else 0
        a.k_stride = _rows(k, "k", dev, c.num_kv_heads, c.dim, n)
        a.v_stride = _rows(v, "v", dev, c.num_kv_heads, c.dim, n)
        for name, t, shape in (("row_starts", row_starts, (a.num_seqs + 1,)), ("first", first, (a.num_seqs,))):
            if t is None and name == "first":
                continue
            if not (isinstance(t, torch.Tensor) and t.dtype is torch.int32 and t.device == dev and t.shape == shape and t.is_contiguous()):
                _want(t, name, torch.int32, dev, shape)
        a.num_rows, a.k, a.v, a.row_starts = n, k.data_ptr(), v.data_ptr(), row_starts.data_ptr()
        a.first = None if first is None else first.data_ptr()
        self._launch(stream)


class DenseAttention(_Op):
    """v4a_dense_attn over `cache` (its block table's rows are the sequences).

    max_new_per_seq: the most tokens one sequence brings in a call.  A run of
    T >= sequences x max_new_per_seq tokens is taken as one where each brings
    that many, padded or not: shorter sequences then take the chunks' form.
    Chunks over a KV_FP8_GROUP cache are divided as if sequences filled the
    block table's columns: a table far wider than they are costs time.
    window: 0 for every earlier position, else the last `window` ones (own
    included) and the first `sinks`.  scale defaults to 1 / sqrt(dim).
    """

    def __init__(self, cache: DenseCache, num_heads: int, max_tokens: int, max_new_per_seq: int = 1, window: int = 0,
                 sinks: int = 0, scale: float | None = None):
        if cache.block_table is None:
            raise ValueError("DenseAttention: the cache has no block table")
        self.cache, self.device, self.max_tokens = cache, cache.device, max_tokens
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.args = AttnArgs(max_tokens, cache.block_table.shape[0], max_new_per_seq, None, None, cache.struct(), num_heads,
                             None, 1.0 / math.sqrt(cache.dim) if scale is None else scale, window, sinks, None, None,
                             self.status.data_ptr())
        need = lib().v4a_dense_attn_workspace_size(C.byref(self.args))
        if need == 0:
            raise ValueError("DenseAttention: sizes outside v4a_dense_attn's limits")
        self._bind("v4a_dense_attn", lib().v4a_dense_attn, torch.empty(need, dtype=torch.uint8, device=self.device))

    def run(self, q: torch.Tensor, out: torch.Tensor, positions: torch.Tensor, token_starts: torch.Tensor, lse=None, stream=None):
        """q, out [T][heads][dim] bf16, T <= max_tokens; positions int32 [T];
        token_starts int32 [sequences + 1]; lse fp32 [T][heads] or None."""
        a, dev = self.args, self.device
        n = q.shape[0] if isinstance(q, torch.Tensor) and q.dim() else 0
        if n > self.max_tokens:
            raise ValueError(f"q: {n} tokens, at most {self.max_tokens}")
        for name, t, dtype, shape in (("q", q, torch.bfloat16, (n, a.num_heads, self.cache.dim)),
                                      ("out", out, torch.bfloat16, (n, a.num_heads, self.cache.dim)),
                                      ("positions", positions, torch.int32, (n,)),
                                      ("token_starts", token_starts, torch.int32, (a.num_seqs + 1,)),
                                      ("lse", lse, torch.float32, (n, a.num_heads))):
            if t is None and name == "lse":
                continue
            if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == dev and t.shape == shape and t.is_contiguous()):
                _want(t, name, dtype, dev, shape)
        a.num_tokens = n
        a.q, a.out, a.positions, a.token_starts = q.data_ptr(), out.data_ptr(), positions.data_ptr(), token_starts.data_ptr()
        a.lse = None if lse is None else lse.data_ptr()
        self._launch(stream)


class PromptAttention(_Op):
    """v4a_prompt_attn: attention of whole packed prompts over packed keys and
    values, for num_seqs sequences of at most max_new_per_seq queries, max_tokens
    queries in all.  A sequence's queries are its last positions.  causal=False:
    every query sees every key; window, sinks and scale as DenseAttention has them.
    """

    def __init__(self, num_heads: int, num_kv_heads: int, dim: int, num_seqs: int, max_tokens: int, max_new_per_seq: int,
                 causal: bool = True, window: int = 0, sinks: int = 0, scale: float | None = None, device="cuda"):
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device, self.max_tokens = dev, max_tokens
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.args = PromptArgs(max_tokens, 0, num_seqs, max_new_per_seq, None, None, num_heads, num_kv_heads, dim, int(bool(causal)),
                               window, sinks, 1.0 / math.sqrt(dim) if scale is None else scale, None, 0, None, 0, None, 0, None, None,
                               self.status.data_ptr())
        need = lib().v4a_prompt_attn_workspace_size(C.byref(self.args))
        if need == 0:
            raise ValueError("PromptAttention: sizes outside v4a_prompt_attn's limits")
        self._bind("v4a_prompt_attn", lib().v4a_prompt_attn, torch.empty(need, dtype=torch.uint8, device=dev))

    def run(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor, token_starts: torch.Tensor,
            kv_starts: torch.Tensor | None = None, lse=None, stream=None):
        """q [T][heads][dim], k, v [N][KV heads][dim] bf16 (any token stride of a
        multiple of 8), out [T][heads][dim] bf16, T <= max_tokens; token_starts,
        kv_starts int32 [sequences + 1] (None: token_starts); lse fp32 [T][heads] or None."""
        a, dev = self.args, self.device
        n, nk = (x.shape[0] if isinstance(x, torch.Tensor) and x.dim() else 0 for x in (q, k))
        if n > self.max_tokens:
            raise ValueError(f"q: {n} tokens, at most {self.max_tokens}")
        a.q_stride = _rows(q, "q", dev, a.num_heads, a.dim, n)
        a.k_stride = _rows(k, "k", dev, a.num_kv_heads, a.dim, nk)
        a.v_stride = _rows(v, "v", dev, a.num_kv_heads, a.dim, nk)
        for name, t, dtype, shape in (("out", out, torch.bfloat16, (n, a.num_heads, a.dim)),
                                      ("token_starts", token_starts, torch.int32, (a.num_seqs + 1,)),
                                      ("kv_starts", kv_starts, torch.int32, (a.num_seqs + 1,)),
                                      ("lse", lse, torch.float32, (n, a.num_heads))):
            if t is None and name in ("kv_starts", "lse"):
                continue
            if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == dev and t.shape == shape and t.is_contiguous()):
                _want(t, name, dtype, dev, shape)
        a.num_tokens, a.num_kv_tokens = n, nk
        a.q, a.k, a.v, a.out, a.token_starts = q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), token_starts.data_ptr()
        a.kv_starts = None if kv_starts is None else kv_starts.data_ptr()
        a.lse = None if lse is None else lse.data_ptr()
        self._launch(stream)
