// What the dense attention kernels share: the arguments on the device, which
// keys a group of rows sees, and the tiles that cover them.
#pragma once
#include <algorithm>
#include <atomic>

#include "tc_common.cuh"
#include "v4a_dense.h"
#include "v4a_dense_internal.h"

namespace v4a {

struct DenseAttnDev {
  int T, B, H, K, G, max_new, max_blocks, window, sinks;
  int64_t num_blocks, block_bytes;
  const int32_t *positions, *starts, *bt;
  const uint8_t* pool;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  int32_t* status;
  float scale_log2;               // softmax_scale * log2(e): logits in log2 units
};

// Sequences of at most this many rows (tokens x heads of a group) go to the
// form for few rows, which reads the cache once per 16 rows (8 of dim 256), so
// up to twice for bf16 and group-scaled fp8 and four times for fp8; the form for many reads it once
// but converts fp8 codes on the way.  Few / many, 32 + 8 heads
// of 128, us: bf16, 8 sequences at 8k: 32 rows 69 / 62, 64 rows 123 / 64; one
// at 8k: 32 rows 22 / 32, 64 rows 28 / 32; 16 at 1k (dim 64): 24 / 26 and
// 35 / 26; fp8, 8 at 8k: 32 rows 63 / 130, 64 rows 111 / 131, 128 rows 203 / 132;
// dim 256, 8 at 8k: bf16 16 rows 163 / 107, 32 rows 311 / 107, one at 8k 16 rows
// 24 / 33; fp8 32 rows 186 / 187, 64 rows 355 / 186.  These limits are those of
// one sequence, where the second pass costs nothing; with more sequences 9 to
// 16 rows of dim 256 (bf16) would be faster in the form for many.  The limits of
// group-scaled fp8 (its form for many does not convert keys) are those of several
// sequences: 8 at 8k: 32 rows 68 / 82, 64 rows 117 / 82; dim 256: 16 rows 70 / 70, 32
// rows 111 / 72.  One sequence alone would gain from twice as many: at 8k 64 rows 33 /
// 41, 128 rows 45 / 43; dim 256, 32 rows 31 / 43.
constexpr int few_rows(int dim, int format) { return (dim == 256 ? 8 : 16) * (format == V4A_KV_FP8_TOKEN ? 4 : 2); }

// One sequence's tokens of the call: first row, count and first position;
// n = 0 when there are none, the entries are inconsistent (reported) or the
// sequence belongs to the call's other launch.
struct SeqRun { int s0, n, p0; };

// Past the L1 in a launch that does not wait for the writers (SplitDev::late).  Many CTAs that look
// through the same starts want it (1000 decoding sequences beside a chunk of 4096: 849 us, past it 973).
__device__ __forceinline__ int32_t load(const int32_t* x, bool late) { return late ? __ldcg(x) : *x; }

__device__ __forceinline__ SeqRun seq_run(const DenseAttnDev& a, int64_t rows_from, int64_t rows_to, bool late, int b, int32_t* status) {
  const int s0 = load(a.starts + b, late), s1 = load(a.starts + b + 1, late);
  SeqRun r{s0, 0, 0};
  if (s0 == s1 && s0 >= 0 && s1 <= a.T) return r;
  bool ok = s0 >= 0 && s1 > s0 && s1 <= a.T && s1 - s0 <= a.max_new;
  if (ok) {
    const int p0 = load(a.positions + s0, late), p1 = load(a.positions + s1 - 1, late);
    ok = p0 >= 0 && int64_t(p1) == int64_t(p0) + (s1 - s0) - 1 && p1 < int64_t(a.max_blocks) * kBlockPositions;
    r.p0 = p0;
  }
  const int64_t rows = int64_t(s1 - s0) * a.G;
  if (!ok) report(status, V4A_DEV_BAD_BATCH);
  else if (rows >= rows_from && rows <= rows_to) r.n = s1 - s0;
  return r;
}

// The key tiles of kTile positions that rows at positions [m_lo, m_hi] see:
// the tiles of the sinks in front of the window's range, then the range's.
// Tile i of `tiles` starts at position kTile * at(i).
template <int kTile>
struct TileRange {
  int lead, first, tiles;         // tiles of sinks alone, first tile of the range, count
  __device__ __forceinline__ int at(int i) const { return i < lead ? i : first + (i - lead); }
};

template <int kTile>
__device__ __forceinline__ TileRange<kTile> tile_range(const DenseAttnDev& a, int m_lo, int m_hi) {
  TileRange<kTile> r;
  const int lo = a.window ? max(0, m_lo - a.window + 1) : 0;
  r.first = lo / kTile;
  r.lead = a.window ? min((min(a.sinks, lo) + kTile - 1) / kTile, r.first) : 0;
  r.tiles = r.lead + m_hi / kTile - r.first + 1;
  return r;
}

// A positive factor of logits, at least the smallest normal number (flushed to zero, it would make NaNs of hidden keys'
// -inf); a NaN stays one.
__device__ __forceinline__ float logit_factor(float f) {
  float r;
  asm("max.NaN.f32 %0, %1, 0f00800000;" : "=f"(r) : "f"(f));
  return r;
}

// Whether a row at position m sees position j.
__device__ __forceinline__ bool visible(const DenseAttnDev& a, int m, int j) {
  return j <= m && (a.window == 0 || j > m - a.window || j < a.sinks);
}

// Whether every row at positions [m_lo, m_hi] sees all of [j, j + n).
__device__ __forceinline__ bool all_visible(const DenseAttnDev& a, int m_lo, int m_hi, int j, int n) {
  return j + n - 1 <= m_lo && (a.window == 0 || j > m_hi - a.window || j + n <= a.sinks);
}

// ---- units and the line of their tiles ---------------------------------------------
// A unit is up to R consecutive rows (token, head of the group) of one sequence
// and one KV head; its row group `rg` starts at row rg * R of the sequence.
template <int kTile>
struct Unit { int b, row0, rows, s0, m_lo, m_hi; TileRange<kTile> tr; };

// What a unit is kept as: its last row gives the first (a multiple of R); -1: no rows.
struct alignas(16) UnitRef { int b, s0, p0, last; };

template <int R, int kTile>
__device__ __forceinline__ Unit<kTile> make_unit(const DenseAttnDev& a, const UnitRef& f) {
  Unit<kTile> u{f.b, 0, 0, f.s0, 0, 0, {0, 0, 0}};
  if (f.last < 0) return u;
  u.row0 = f.last & ~(R - 1);
  u.rows = f.last - u.row0 + 1;
  u.m_lo = f.p0 + u.row0 / a.G;
  u.m_hi = f.p0 + f.last / a.G;
  u.tr = tile_range<kTile>(a, u.m_lo, u.m_hi);
  return u;
}

// Row r of a unit in the [T][H] order of q and out.
template <int kTile>
__device__ __forceinline__ int64_t row_of(const DenseAttnDev& a, const Unit<kTile>& u, int hk, int r) {
  return int64_t(u.s0 + (u.row0 + r) / a.G) * a.H + hk * a.G + (u.row0 + r) % a.G;
}

// How a launch divides the units, which are numbered over the sequences' row
// groups (sequences without tokens in this launch have none): split = 1: the
// tiles of all units and KV heads form one line (unit by unit, KV head by KV head) that the CTAs divide
// evenly, each unit counted with `cost` tiles more than it has (its set-up and
// its end take about that long); split = 0: one CTA per unit and KV head.
struct SplitDev {
  int RG, U, split;               // row groups of the longest sequence; units at most (split = 2: dense_stream.cuh)
  int rows, grid, cost;           // R; CTAs of the launch and a unit's extra tiles (split)
  struct JoinDesc* join;          // [CTA]
  float *part_o, *part_ml;        // [CTA][2][R][dim], [CTA][2][R][2] (maximum in log2 units, sum)
  int rows_from, rows_to;         // the launch takes sequences of this many rows (tokens x group)
  // A call's two launches need nothing of each other: the one for few rows lets
  // the other start as its CTAs leave (early), which waits for it at its end (late)
  // and reads memory past the L1 throughout, since it does not wait for the writers
  // before (which had ended when the first of the two began its work).
  int early, late;
};

// A unit that starts in a CTA's range and goes on in the next CTAs' up to `last`:
// its pieces are this CTA's slot 1 and slot 0 of the others.  rows = 0: none.
struct alignas(16) JoinDesc { int rows, row0, s0, hk, last, pad[3]; };
static_assert(alignof(JoinDesc) <= 16 && sizeof(JoinDesc) == 32, "lies at the front of a workspace, which the caller aligns to 16 bytes");

// The most units (and sequences) of an even split: their table lies in shared
// memory.  More run one CTA each, which is as fast where they are about equally
// long (600 sequences at 1k, 32 + 8 heads of 128: 350 us, 7.2 TB/s) and not where
// one is far longer: 256k among 600 at 1k 2.8 ms (among 500, split: 475 us), 512
// tokens over 32k beside 600 decoding at 1k 870 us (beside 500: 560).
constexpr int kMaxSplitUnits = 512;
constexpr int kSms = 152;

// Units of R rows that a consistent batch has at most: a sequence of n rows has
// n / R and one more, and only sequences of rows_from rows or more count.
inline int64_t units_bound(const DenseAttnDev& a, int rows_from, int64_t RG, int R) {
  const int64_t rows = int64_t(a.T) * a.G, seqs = std::min<int64_t>(a.B, rows_from > 0 ? rows / rows_from : a.T);
  return RG == 1 ? a.B : std::min(a.B * RG, rows / R + seqs);
}
__host__ __device__ constexpr size_t split_smem(int split, int U) {
  return split ? U * sizeof(UnitRef) + (U + 1) * sizeof(int64_t) : sizeof(UnitRef);
}
__host__ __device__ constexpr size_t split_workspace(int R, int dim, int ctas) {
  return ctas * (sizeof(JoinDesc) + size_t(2) * R * (dim + 2) * sizeof(float));      // (a multiple of 16)
}
// f() where it has not been true on the current device yet (`done`: the devices where it was).
template <typename F>
inline bool once_per_device(std::atomic<uint64_t>* done, F f) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (dev < 64 && (done->load() >> dev & 1)) return true;
  if (!f()) return false;
  if (dev < 64) done->fetch_or(uint64_t(1) << dev);
  return true;
}
// Raises a kernel's dynamic shared memory limit on the current device.
template <typename K>
inline bool raise_smem(K kern, int bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
}

inline void split_carve(SplitDev* p, void* ws, int R, int dim, int ctas, int cost) {
  p->rows = R;
  p->grid = ctas;
  p->cost = cost;
  p->join = static_cast<JoinDesc*>(ws);
  p->part_o = reinterpret_cast<float*>(p->join + ctas);
  p->part_ml = p->part_o + size_t(ctas) * 2 * R * dim;
}

// The CTA's part of the line (or its unit), kept in shared memory behind `mem`.
// Dev: the arguments, with a seq_run and a make_unit of their own.
template <int R, int kTile, int kThreads, typename Dev = DenseAttnDev>
struct Line {
  const Dev& a;
  const SplitDev& p;
  UnitRef* refs;                  // [U], or the one
  int64_t* pre;                   // [U + 1] tiles before unit u, over its KV heads
  int64_t x0, x1, total, weight;
  int ctas, u_direct, hk_direct;

  struct Piece { int u, hk, tile; };
  struct Seq { SeqRun r; int first; };      // a sequence and the units before it

  __device__ __forceinline__ Line(const Dev& a_, const SplitDev& p_, void* mem) : a(a_), p(p_) {
    refs = static_cast<UnitRef*>(mem);
    pre = reinterpret_cast<int64_t*>(refs + p.U);
  }
  // `scan`: kThreads / 32 words of shared memory; `scratch`: kMaxSplitUnits Seq
  // of it, free again on return.  At least min_tiles tiles (or units' costs)
  // per CTA.  Called by the whole CTA; false when it has no tiles.
  __device__ __forceinline__ bool init(int64_t* scan, void* scratch, int min_tiles) {
    const int tid = threadIdx.x;
    int32_t* st = blockIdx.x == 0 ? a.status : nullptr;     // one CTA reports the batch's faults
    u_direct = hk_direct = ctas = 0;
    total = 0;
    if (!p.split) {
      u_direct = int(blockIdx.x / unsigned(a.K));
      hk_direct = int(blockIdx.x % unsigned(a.K));
      if (p.RG == 1) {
        if (tid == 0) refs[0] = ref(u_direct, 0, run(u_direct, hk_direct == 0 ? a.status : nullptr));
      } else {
        // units counted by the starts alone, each thread a run of sequences; the one found is checked then
        const int per = (a.B + kThreads - 1) / kThreads, b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
        if (tid == 0) refs[0] = UnitRef{0, 0, 0, -1};
        int64_t n = 0, all;
        for (int b = b0; b < b1; ++b) {
          n += groups(load(a.starts + b, p.late), load(a.starts + b + 1, p.late));
          if (st) run(b, st);
        }
        int64_t at = before(n, scan, &all);
        if (u_direct >= at && u_direct < at + n) {
          int b = b0;
          for (int64_t g; at + (g = groups(load(a.starts + b, p.late), load(a.starts + b + 1, p.late))) <= u_direct; ++b) at += g;
          refs[0] = ref(b, int(u_direct - at), run(b, nullptr));
        }
        if (st && tid == 0 && all > p.U) report(st, V4A_DEV_BAD_BATCH);       // sequences that share tokens
      }
      __syncthreads();
      x0 = 0;
      x1 = unit(u_direct).tr.tiles;
      return x1 > 0;
    }
    Seq* const seqs = static_cast<Seq*>(scratch);
    for (int b = tid; b < a.B; b += kThreads) seqs[b] = Seq{run(b, st), b};
    __syncthreads();
    int units = p.U;
    if (p.RG > 1) {
      const int per = (a.B + kThreads - 1) / kThreads, b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
      int64_t n = 0, all;
      for (int b = b0; b < b1; ++b) n += groups(seqs[b].r.s0, seqs[b].r.s0 + seqs[b].r.n);
      int64_t at = before(n, scan, &all);
      units = int(min(all, int64_t(p.U)));
      for (int b = b0; b < b1; ++b) {
        seqs[b].first = int(min(at, int64_t(units)));
        at += groups(seqs[b].r.s0, seqs[b].r.s0 + seqs[b].r.n);
      }
      if (st && tid == 0 && all > p.U) report(st, V4A_DEV_BAD_BATCH);         // sequences that share tokens
      __syncthreads();
    }
    // exclusive sums over the units: each thread a run of units, then the threads' totals
    const int per = (p.U + kThreads - 1) / kThreads, u0 = min(p.U, tid * per), u1 = min(p.U, u0 + per);
    int64_t sum = 0;
    for (int u = u0; u < u1; ++u) {
      int lo = u;                                 // the unit's sequence: the last whose first <= u
      if (p.RG > 1) {
        lo = 0;
        for (int hi = a.B; hi - lo > 1;) {
          const int mid = (lo + hi) >> 1;
          if (seqs[mid].first <= u) lo = mid; else hi = mid;
        }
      }
      refs[u] = u < units ? ref(lo, u - seqs[lo].first, seqs[lo].r) : UnitRef{0, 0, 0, -1};
      pre[u] = sum;
      sum += int64_t(unit(u).tr.tiles) * a.K;
    }
    const int64_t ahead = before(sum, scan, &total);
    for (int u = u0; u < u1; ++u) pre[u] += ahead;
    if (tid == 0) pre[p.U] = total;
    __syncthreads();
    weight = total + int64_t(p.cost) * a.K * units;
    ctas = int(min(int64_t(gridDim.x), (weight + min_tiles - 1) / min_tiles));
    x0 = x1 = 0;
    if (int(blockIdx.x) < ctas) {
      x0 = place(int64_t(blockIdx.x) * weight / ctas);
      x1 = place((int64_t(blockIdx.x) + 1) * weight / ctas);
    }
    if (x0 == x1 && tid == 0) p.join[blockIdx.x].rows = 0;
    return x0 < x1;
  }
  __device__ __forceinline__ UnitRef ref(int b, int rg, const SeqRun& r) const {
    return UnitRef{b, r.s0, r.p0, int(min(int64_t(r.n) * a.G, (int64_t(rg) + 1) * R)) - 1};
  }
  __device__ __forceinline__ SeqRun run(int b, int32_t* st) const { return seq_run(a, p.rows_from, p.rows_to, p.late, b, st); }
  // Row groups of a sequence of tokens [s0, s1) in this launch.
  __device__ __forceinline__ int64_t groups(int s0, int s1) const {
    const int64_t n = int64_t(s1) - s0, rows = n * a.G;
    return n > 0 && n <= a.max_new && rows >= p.rows_from && rows <= p.rows_to ? (rows + R - 1) / R : 0;
  }
  // The sum of the earlier threads' v, and of all (whole CTA; `scan` is free again behind a barrier).
  __device__ __forceinline__ int64_t before(int64_t v, int64_t* scan, int64_t* all) const {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t w = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += w;
    }
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    int64_t ahead = x - v;
    *all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) ahead += scan[w];
      *all += scan[w];
    }
    return ahead;
  }
  // The first tile at or behind position w of the line with the units' costs,
  // which are in front of their tiles.
  __device__ __forceinline__ int64_t place(int64_t w) const {
    const int64_t each = int64_t(p.cost) * a.K;
    if (w >= weight) return total;
    int lo = 0, hi = p.U;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] + each * mid <= w) lo = mid; else hi = mid;
    }
    const int tiles = unit(lo).tr.tiles;
    const int64_t rem = w - pre[lo] - each * lo, hk = rem / (tiles + p.cost);
    return pre[lo] + hk * tiles + max(int64_t(0), rem - hk * (tiles + p.cost) - p.cost);
  }
  __device__ __forceinline__ Unit<kTile> unit(int u) const { return make_unit<R, kTile>(a, refs[p.split ? u : 0]); }
  // Where tile x of the line lies.
  __device__ __forceinline__ Piece locate(int64_t x, Unit<kTile>* un) const {
    if (!p.split) {
      *un = unit(u_direct);
      return Piece{u_direct, hk_direct, int(x)};
    }
    int lo = 0, hi = p.U;                       // largest u with pre[u] <= x (empty units precede)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= x) lo = mid; else hi = mid;
    }
    *un = unit(lo);
    const int64_t rem = x - pre[lo];
    const int hk = rem <= INT32_MAX ? int(rem) / un->tr.tiles : int(rem / un->tr.tiles);
    return Piece{lo, hk, int(rem - int64_t(hk) * un->tr.tiles)};
  }
  // The description of a unit that leaves the CTA's range.
  __device__ __forceinline__ JoinDesc describe(const Piece& pc, const Unit<kTile>& un) const {
    const int64_t end = pre[pc.u] + int64_t(p.cost) * a.K * pc.u + int64_t(pc.hk + 1) * (un.tr.tiles + p.cost);
    return JoinDesc{un.rows, un.row0, un.s0, pc.hk, int((end * ctas - 1) / weight), {0, 0, 0}};
  }
};

// Joins the pieces of every split unit (dense_attn.cu).
int dense_join(const DenseAttnDev& a, const SplitDev& p, int dim, cudaStream_t stream);

// The tensor-core form for many rows (dense_prefill.cu): whether it takes the
// shape, its division (U = 0: no sequence of the call can have so many rows),
// its kernel's readiness on the current device (ahead of the call's first
// launch) and its launch, whose pieces are then to be joined (p.split).
bool dense_prefill_takes(const v4a_dense_attn_args* a);
size_t dense_prefill_workspace(const v4a_dense_attn_args* a);
int dense_prefill_plan(const v4a_dense_attn_args* a, const DenseAttnDev& d, int rows_from, void* ws, SplitDev* p);
bool dense_prefill_ready(const v4a_dense_attn_args* a, const DenseAttnDev& d);
int dense_prefill(const v4a_dense_attn_args* a, const DenseAttnDev& d, const SplitDev& p, cudaStream_t stream);

// The same for caches with a scale per group (dense_group.cu).  The division is shared with whole prompts
// (prompt_attn.cu); keys: what a sequence has at most or on the average, causal: its later queries see more.
size_t stream_workspace(int dim);
int stream_plan(const DenseAttnDev& d, int dim, int rows_from, int64_t keys, bool causal, void* ws, SplitDev* p);
bool dense_group_ready(int dim, const DenseAttnDev& d);
int dense_group(int dim, const DenseAttnDev& d, const SplitDev& p, cudaStream_t stream);

}  // namespace v4a
