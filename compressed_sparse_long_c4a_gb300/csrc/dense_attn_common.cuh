// What the dense attention kernels share: the arguments on the device, which
// keys a group of rows sees, and the tiles that cover them.
#pragma once
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

// One sequence's tokens of the call: first row, count and first position;
// n = 0 when there are none or the entries are inconsistent (reported).
struct SeqRun { int s0, n, p0; };

__device__ __forceinline__ SeqRun seq_run(const DenseAttnDev& a, int b, int32_t* status) {
  const int s0 = a.starts[b], s1 = a.starts[b + 1];
  SeqRun r{s0, 0, 0};
  if (s0 == s1 && s0 >= 0 && s1 <= a.T) return r;
  bool ok = s0 >= 0 && s1 > s0 && s1 <= a.T && s1 - s0 <= a.max_new;
  if (ok) {
    const int p0 = a.positions[s0], p1 = a.positions[s1 - 1];
    ok = p0 >= 0 && int64_t(p1) == int64_t(p0) + (s1 - s0) - 1 && p1 < int64_t(a.max_blocks) * kBlockPositions;
    r.p0 = p0;
  }
  if (ok) r.n = s1 - s0;
  else report(status, V4A_DEV_BAD_BATCH);
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

template <int R, int kTile>
__device__ __forceinline__ Unit<kTile> make_unit(const DenseAttnDev& a, int b, int rg, const SeqRun& s) {
  Unit<kTile> u;
  u.b = b;
  u.row0 = rg * R;
  u.rows = int(min(int64_t(R), int64_t(s.n) * a.G - u.row0));
  u.s0 = s.s0;
  u.m_lo = u.m_hi = 0;
  u.tr = TileRange<kTile>{0, 0, 0};
  if (u.rows <= 0) return u;
  u.m_lo = s.p0 + u.row0 / a.G;
  u.m_hi = s.p0 + (u.row0 + u.rows - 1) / a.G;
  u.tr = tile_range<kTile>(a, u.m_lo, u.m_hi);
  return u;
}

// Row r of a unit in the [T][H] order of q and out.
template <int kTile>
__device__ __forceinline__ int64_t row_of(const DenseAttnDev& a, const Unit<kTile>& u, int hk, int r) {
  return int64_t(u.s0 + (u.row0 + r) / a.G) * a.H + hk * a.G + (u.row0 + r) % a.G;
}

// How a launch divides the units: split = 1: the tiles of all units and KV
// heads form one line (unit by unit, KV head by KV head) that the CTAs divide
// evenly, each unit counted with `cost` tiles more than it has (its set-up and
// its end take about that long); split = 0: one CTA per unit and KV head.
struct SplitDev {
  int RG, U, split;               // row groups per sequence, units (sequences x row groups)
  int rows, grid, cost;           // R; CTAs of the launch and a unit's extra tiles (split)
  struct JoinDesc* join;          // [CTA]
  float *part_o, *part_ml;        // [CTA][2][R][dim], [CTA][2][R][2] (maximum in log2 units, sum)
};

// A unit that starts in a CTA's range and goes on in the next CTAs' up to `last`:
// its pieces are this CTA's slot 1 and slot 0 of the others.  rows = 0: none.
struct alignas(32) JoinDesc { int rows, row0, s0, hk, last, pad[3]; };

constexpr int kMaxSplitUnits = 512;   // more units than these fill the machine one by one
constexpr int kSms = 152;

__host__ __device__ constexpr size_t split_smem(int split, int U, int B) {
  return split ? (U + 1) * sizeof(int64_t) + B * sizeof(SeqRun) : sizeof(SeqRun);
}
__host__ __device__ constexpr size_t split_workspace(int R, int dim, int ctas) {
  return 16 + ctas * (sizeof(JoinDesc) + size_t(2) * R * (dim + 2) * sizeof(float));
}
// Raises a kernel's dynamic shared memory limit, once per device (`done`: the devices it is done on).
template <typename K>
inline bool raise_smem(K kern, int bytes, std::atomic<uint64_t>* done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (dev < 64 && (done->load() >> dev & 1)) return true;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  if (dev < 64) done->fetch_or(uint64_t(1) << dev);
  return true;
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
template <int R, int kTile, int kThreads>
struct Line {
  const DenseAttnDev& a;
  const SplitDev& p;
  int64_t* pre;                   // [U + 1] tiles before unit u, over its KV heads
  SeqRun* runs;                   // [B], or the one
  int64_t x0, x1, total, weight;
  int ctas, u_direct, hk_direct;

  struct Piece { int u, hk, tile; };

  // `scan`: kThreads / 32 words of shared memory.  At least min_tiles tiles per
  // CTA.  Called by the whole CTA; false when it has no tiles.
  __device__ __forceinline__ Line(const DenseAttnDev& a_, const SplitDev& p_, void* mem) : a(a_), p(p_) {
    pre = static_cast<int64_t*>(mem);
    runs = reinterpret_cast<SeqRun*>(pre + (p.split ? p.U + 1 : 0));
  }
  __device__ __forceinline__ bool init(int64_t* scan, int min_tiles) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    u_direct = hk_direct = ctas = 0;
    total = 0;
    if (!p.split) {
      u_direct = int(blockIdx.x / unsigned(a.K));
      hk_direct = int(blockIdx.x % unsigned(a.K));
      if (tid == 0) runs[0] = seq_run(a, u_direct / p.RG, hk_direct == 0 && u_direct % p.RG == 0 ? a.status : nullptr);
      __syncthreads();
      x0 = 0;
      x1 = unit(u_direct).tr.tiles;
      return x1 > 0;
    }
    int32_t* st = blockIdx.x == 0 ? a.status : nullptr;     // one CTA reports the batch's faults
    for (int b = tid; b < a.B; b += kThreads) runs[b] = seq_run(a, b, st);
    __syncthreads();
    // exclusive sums over the units: each thread a run of units, then the threads' totals
    const int per = (p.U + kThreads - 1) / kThreads, u0 = min(p.U, tid * per), u1 = min(p.U, u0 + per);
    int64_t sum = 0;
    for (int u = u0; u < u1; ++u) {
      pre[u] = sum;
      sum += int64_t(unit(u).tr.tiles) * a.K;
    }
    int64_t v = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t w = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += w;
    }
    if (lane == 31) scan[warp] = v;
    __syncthreads();
    int64_t before = v - sum;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += scan[w];
      total += scan[w];
    }
    for (int u = u0; u < u1; ++u) pre[u] += before;
    if (tid == 0) pre[p.U] = total;
    __syncthreads();
    weight = total + int64_t(p.cost) * a.K * p.U;
    ctas = int(min(int64_t(gridDim.x), (total + min_tiles - 1) / min_tiles));
    x0 = x1 = 0;
    if (int(blockIdx.x) < ctas) {
      x0 = place(int64_t(blockIdx.x) * weight / ctas);
      x1 = place((int64_t(blockIdx.x) + 1) * weight / ctas);
    }
    if (x0 == x1 && tid == 0) p.join[blockIdx.x].rows = 0;
    return x0 < x1;
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
  __device__ __forceinline__ Unit<kTile> unit(int u) const {
    return make_unit<R, kTile>(a, u / p.RG, u % p.RG, runs[p.split ? u / p.RG : 0]);
  }
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

// The tensor-core form for many rows (dense_prefill.cu): whether it takes the shape, and its launch.
bool dense_prefill_takes(const v4a_dense_attn_args* a);
size_t dense_prefill_workspace(const v4a_dense_attn_args* a);
int dense_prefill(const v4a_dense_attn_args* a, const DenseAttnDev& d, void* ws, cudaStream_t stream);

}  // namespace v4a
