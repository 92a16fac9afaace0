// What the dense attention kernels share: the arguments on the device, which
// keys a group of rows sees, and the tiles that cover them.
#pragma once
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

// The tensor-core form for many rows (dense_prefill.cu): whether it takes the shape, and its launch.
bool dense_prefill_takes(const v4a_dense_attn_args* a);
int dense_prefill(const DenseAttnDev& d, int dim, cudaStream_t stream);

}  // namespace v4a
