// The step plan: positions, slot maps and block tables from request lengths,
// on the GPU (v4a_dense.h, v4a_step_plan).
//
// Mathematics: three exclusive prefix sums over the sequences (fresh tokens,
// new blocks, given-back blocks) place every token, every new page and every
// given-back page, so each output entry is computed by itself: token t finds
// its sequence by a binary search in the token sums; new block n of the step
// takes pages n * L .. n * L + L - 1 of the free ring.  Pages are taken from
// the ring's front and given back behind its end, so no entry is read and
// written in one call and the fill needs no order.
//
// One CTA forms the sums (they are the only serial part).  Small steps are
// filled by the same CTA; larger ones by a second, wide kernel that starts
// while the first drains (programmatic dependent launch).
//
// Bound: latency.  The loads, the scan and the two launches one after the other
// take 5 to 6 us on the device (64 decoding sequences with 60 tables 5.6, 4 x
// 1024 tokens with 60 tables, whose slots are 2 MB, 5.7, 1000 sequences 6 to 7,
// 8000 19: the scan's eight rounds); 64 decoding sequences with one table 3.4.
// A step that ends long sequences moves their pages too: table rows lie far
// apart, so each page is a sector of its own (one sequence of 1M positions, 61
// tables, 250k pages: 8.9 us over 152 SMs, 156 in a step that one CTA fills).
#include <algorithm>

#include "tc_common.cuh"
#include "v4a_dense.h"
#include "v4a_dense_internal.h"

namespace v4a {
namespace {

constexpr int kScanThreads = 1024;
constexpr int kFillThreads = 256;
constexpr int kTablesPerItem = 4;     // tables one thread writes for its token
constexpr int kMaxSeqs = 8192;
constexpr uint32_t kBackBatch = 8;    // given-back pages a thread has under way
// Steps of at most this many (token, table group) items are filled by the
// scanning CTA: a second launch costs more than they take (64 items: 3.4 us
// inline, 4.6 wide; 960: 5.9 and 5.3; 2048: 6.5 and 5.5; 4096: 10.1 and 5.5).
// Given-back pages are not counted, since only the device knows them: a small
// step that ends a sequence of 4096 pages takes 5.7 us, of 31k 22, of 250k 156
// (wide 8.9), once in a sequence's life; the second launch would cost every
// small step 1.2 us.
constexpr int64_t kInlineItems = 512;

struct PlanHeader {                   // in the workspace, before the sums
  int32_t ok, tokens, fresh_blocks, back_blocks, first, count, pad[2];
};

struct PlanDev {
  v4a_plan_args a;
  PlanHeader* hdr;
  int32_t* sums;                      // [2][B + 1] new blocks, given-back blocks (wide fill only)
  int64_t items;                      // T * ceil(L / kTablesPerItem)
  int inline_fill;
};

__host__ __device__ __forceinline__ int groups_of(int tables) { return (tables + kTablesPerItem - 1) / kTablesPerItem; }

__device__ __forceinline__ int blocks_for(int64_t positions) { return int((positions + kBlockPositions - 1) / kBlockPositions); }

// Largest b in [0, B) with sum[b] <= x (sum is non-decreasing, sum[0] = 0 <= x < sum[B]).
__device__ __forceinline__ int find_row(const int32_t* sum, int B, int x) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sum[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int32_t ring_at(const v4a_plan_args& a, int first, int64_t n) {
  int64_t i = first + n;
  while (i >= a.ring_cap) i -= a.ring_cap;       // first < cap and n < 2 cap
  return int32_t(i);
}

// Fills the outputs with threads tid, tid + n, ...; st, nb, bb: the sums.
__device__ void fill(const PlanDev& p, const PlanHeader& h, const int32_t* st, const int32_t* nb, const int32_t* bb,
                     int64_t tid, int64_t n) {
  const v4a_plan_args& a = p.a;
  const int B = a.num_seqs, L = a.num_tables, T = a.max_tokens;
  for (int64_t it = tid; it < p.items; it += n) {
    int g, t;
    if (p.items <= INT32_MAX) {                  // 32-bit division where it suffices
      g = int(uint32_t(it) / uint32_t(T));
      t = int(uint32_t(it) - uint32_t(g) * uint32_t(T));
    } else {
      g = int(it / T);
      t = int(it - int64_t(g) * T);
    }
    int b = -1, pos = -1;
    bool held = false;
    int64_t nth = 0;                             // pages taken before this token's new block
    if (t < h.tokens) {
      b = find_row(st, B, t);
      const int c = a.cached[b], has = blocks_for(c);
      pos = c + (t - st[b]);
      held = pos / kBlockPositions < has;
      nth = int64_t(nb[b] + (pos / kBlockPositions - has)) * L;
    }
    if (g == 0) {
      a.seq_ids[t] = b;
      a.positions[t] = pos;
    }
    if (!a.slots) continue;
    int32_t page[kTablesPerItem];
#pragma unroll
    for (int i = 0; i < kTablesPerItem; ++i) {
      const int l = g * kTablesPerItem + i;
      page[i] = -1;
      if (b >= 0 && l < L)
        page[i] = held ? a.block_table[int64_t(l) * a.table_stride + int64_t(b) * a.max_blocks + pos / kBlockPositions]
                       : a.free_ring[ring_at(a, h.first, nth + l)];
    }
#pragma unroll
    for (int i = 0; i < kTablesPerItem; ++i) {
      const int l = g * kTablesPerItem + i;
      if (l >= L) break;
      int64_t slot = -1;
      if (b >= 0) {
        if (page[i] < 0 || page[i] >= a.num_blocks) report(a.status, V4A_DEV_BAD_BLOCK);
        else slot = int64_t(page[i]) * kBlockPositions + pos % kBlockPositions;
      }
      a.slots[int64_t(l) * T + t] = slot;
    }
  }
  // new table entries: (block, table) pairs, tables fastest (the ring's order); at most 2^30, as the ring has
  const uint32_t fresh = uint32_t(h.fresh_blocks) * uint32_t(L), step = uint32_t(n);
  for (uint32_t it = uint32_t(tid); it < fresh; it += step) {
    const int j = int(it / uint32_t(L)), l = int(it - uint32_t(j) * uint32_t(L));
    const int b = find_row(nb, B, j);
    const int k = blocks_for(a.cached[b]) + (j - nb[b]);
    const int32_t page = a.free_ring[ring_at(a, h.first, it)];
    if (page < 0 || page >= a.num_blocks) report(a.status, V4A_DEV_BAD_BLOCK);
    a.block_table[int64_t(l) * a.table_stride + int64_t(b) * a.max_blocks + k] = page;
  }
  // given-back pages, behind the last free one; a thread's loads of several are under way together
  const uint32_t back = uint32_t(h.back_blocks) * uint32_t(L);
  for (uint32_t i0 = uint32_t(tid); i0 < back; i0 += kBackBatch * step) {
    int32_t page[kBackBatch];
#pragma unroll
    for (uint32_t u = 0; u < kBackBatch; ++u) {
      const uint32_t it = i0 + u * step;
      page[u] = 0;
      if (it < back) {
        const int j = int(it / uint32_t(L)), l = int(it - uint32_t(j) * uint32_t(L));
        const int b = find_row(bb, B, j);
        page[u] = a.block_table[int64_t(l) * a.table_stride + int64_t(b) * a.max_blocks + (j - bb[b])];
      }
    }
#pragma unroll
    for (uint32_t u = 0; u < kBackBatch; ++u) {
      const uint32_t it = i0 + u * step;
      if (it >= back) break;
      if (page[u] < 0 || page[u] >= a.num_blocks) report(a.status, V4A_DEV_BAD_BLOCK);
      a.free_ring[ring_at(a, h.first, int64_t(h.count) + it)] = page[u];
    }
  }
}

struct Sum3 { int64_t x, y, z; };

__device__ __forceinline__ Sum3 warp_scan(Sum3 v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, v.x, o), y = __shfl_up_sync(0xffffffffu, v.y, o),
                  z = __shfl_up_sync(0xffffffffu, v.z, o);
    if (lane >= o) { v.x += x; v.y += y; v.z += z; }
  }
  return v;
}

__global__ void __launch_bounds__(kScanThreads, 1) plan_scan(const PlanDev p) {
  extern __shared__ int32_t sums[];                  // [3][B + 1]
  __shared__ Sum3 warp_tot[32];
  __shared__ PlanHeader h;
  const v4a_plan_args& a = p.a;
  const int B = a.num_seqs, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t *st = sums, *nb = sums + B + 1, *bb = nb + B + 1;
  pdl_trigger();
  pdl_wait();
  Sum3 carry{0, 0, 0};
  bool good = true;
  for (int b0 = 0; b0 < B; b0 += kScanThreads) {
    const int b = b0 + tid;
    Sum3 v{0, 0, 0};
    if (b < B) {
      const int c = a.cached[b], f = a.fresh[b];
      const int64_t end = int64_t(c) + (f > 0 ? f : 0);
      if (c < 0 || f < -1 || end > int64_t(a.max_blocks) * kBlockPositions) {
        good = false;
      } else {
        v.x = f > 0 ? f : 0;
        v.y = f > 0 ? blocks_for(end) - blocks_for(c) : 0;
        v.z = f < 0 ? blocks_for(c) : 0;
      }
    }
    const Sum3 own = v;
    v = warp_scan(v);
    if (lane == 31) warp_tot[warp] = v;
    __syncthreads();
    if (warp == 0) warp_tot[lane] = warp_scan(warp_tot[lane]);
    __syncthreads();
    const Sum3 before = warp ? warp_tot[warp - 1] : Sum3{0, 0, 0}, total = warp_tot[31];
    if (b < B) {                                     // exclusive sums (too large ones fail below)
      st[b] = int32_t(carry.x + before.x + v.x - own.x);
      nb[b] = int32_t(carry.y + before.y + v.y - own.y);
      bb[b] = int32_t(carry.z + before.z + v.z - own.z);
    }
    carry.x += total.x; carry.y += total.y; carry.z += total.z;
    __syncthreads();
  }
  good = __syncthreads_and(good);
  if (tid == 0) {
    st[B] = int32_t(carry.x); nb[B] = int32_t(carry.y); bb[B] = int32_t(carry.z);
    const int first = a.free_in[0], count = a.free_in[1];
    const int64_t take = carry.y * a.num_tables, give = carry.z * a.num_tables;
    int bad = 0;
    if (!good || carry.x > a.max_tokens || first < 0 || first >= a.ring_cap || count < 0 || count > a.ring_cap ||
        count + give > a.ring_cap)
      bad = V4A_DEV_BAD_BATCH;
    else if (take > count)
      bad = V4A_DEV_OUT_OF_PAGES;
    if (bad) report(a.status, bad);
    h = PlanHeader{};
    h.ok = !bad;
    h.first = first;
    h.count = count;
    if (!bad) {
      h.tokens = int32_t(carry.x);
      h.fresh_blocks = int32_t(carry.y);
      h.back_blocks = int32_t(carry.z);
      a.free_out[0] = ring_at(a, first, take);
      a.free_out[1] = int32_t(count - take + give);
    } else {
      a.free_out[0] = first;
      a.free_out[1] = count;
    }
    if (!p.inline_fill) *p.hdr = h;
  }
  __syncthreads();
  for (int b = tid; b <= B; b += kScanThreads) a.token_starts[b] = h.ok ? st[b] : 0;
  if (p.inline_fill) {
    fill(p, h, st, nb, bb, tid, kScanThreads);
  } else {
    for (int b = tid; b <= B; b += kScanThreads) {
      p.sums[b] = nb[b];
      p.sums[B + 1 + b] = bb[b];
    }
  }
}

__global__ void __launch_bounds__(kFillThreads) plan_fill(const PlanDev p) {
  extern __shared__ int32_t sums[];
  const int B = p.a.num_seqs, tid = threadIdx.x;
  int32_t *st = sums, *nb = sums + B + 1, *bb = nb + B + 1;
  pdl_trigger();
  pdl_wait();
  const PlanHeader h = *p.hdr;
  // (the CTAs that have tokens do not wait for the header before they load the sums)
  const int64_t first = int64_t(blockIdx.x) * kFillThreads;
  if (first >= p.items && first >= int64_t(max(h.fresh_blocks, h.back_blocks)) * p.a.num_tables) return;
  for (int b = tid; b <= B; b += kFillThreads) {
    st[b] = p.a.token_starts[b];
    nb[b] = p.sums[b];
    bb[b] = p.sums[B + 1 + b];
  }
  __syncthreads();
  fill(p, h, st, nb, bb, int64_t(blockIdx.x) * kFillThreads + tid, int64_t(gridDim.x) * kFillThreads);
}

// Host checks; V4A_OK or the error (the workspace size needs no pointer).
int check_shape(const v4a_plan_args* a) {
  if (!a || a->num_seqs < 0 || a->num_tables < 1 || a->max_tokens < 0 || a->max_blocks < 1 || a->ring_cap < 1 ||
      a->num_blocks < 1)
    return V4A_ERR_INVALID_ARG;
  if (a->num_seqs > kMaxSeqs || a->num_tables > 4096 || a->max_blocks > (1 << 22) || a->ring_cap > (1 << 30))
    return V4A_ERR_UNSUPPORTED;
  if (a->table_stride < int64_t(a->num_seqs) * a->max_blocks) return V4A_ERR_INVALID_ARG;
  return V4A_OK;
}

size_t plan_bytes(const v4a_plan_args* a) { return sizeof(PlanHeader) + 2 * (size_t(a->num_seqs) + 1) * sizeof(int32_t); }

}  // namespace

size_t plan_workspace_size(const v4a_plan_args* a) { return check_shape(a) ? 0 : plan_bytes(a); }

int step_plan(const v4a_plan_args* a, void* ws, size_t ws_bytes, cudaStream_t stream) {
  const int rc = check_shape(a);
  if (rc) return rc;
  if (!a->token_starts || !a->free_ring || !a->free_in || !a->free_out) return V4A_ERR_INVALID_ARG;
  if (a->num_seqs > 0 && (!a->cached || !a->fresh || !a->block_table)) return V4A_ERR_INVALID_ARG;
  if (a->max_tokens > 0 && (!a->seq_ids || !a->positions)) return V4A_ERR_INVALID_ARG;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 15) || ws_bytes < plan_bytes(a)) return V4A_ERR_WORKSPACE;
  PlanDev p{};
  p.a = *a;
  p.hdr = static_cast<PlanHeader*>(ws);
  p.sums = reinterpret_cast<int32_t*>(p.hdr + 1);
  p.items = int64_t(a->max_tokens) * (a->slots ? groups_of(a->num_tables) : 1);
  p.inline_fill = p.items <= kInlineItems;
  const size_t smem = 3 * (size_t(a->num_seqs) + 1) * sizeof(int32_t);
  if (smem > 48 * 1024) {     // past the default limit: raised on the current device, for both kernels
    const int most = 3 * (kMaxSeqs + 1) * int(sizeof(int32_t));
    if (cudaFuncSetAttribute(plan_scan, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess ||
        cudaFuncSetAttribute(plan_fill, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
      return V4A_ERR_CUDA;
  }
  cudaError_t e = launch_pdl(plan_scan, dim3(1), dim3(kScanThreads), smem, stream, p);
  if (e == cudaSuccess && !p.inline_fill) {
    // enough CTAs for the tokens, and one an SM for the pages that a step may give back (how many only the device
    // knows; CTAs that find nothing leave)
    const int64_t pages = std::min(int64_t(a->ring_cap), int64_t(a->num_seqs) * a->max_blocks * a->num_tables);
    const int64_t want = std::max((p.items + kFillThreads - 1) / kFillThreads, std::min((pages + kFillThreads - 1) / kFillThreads, int64_t(152)));
    const int grid = int(want < 152 * 8 ? want : 152 * 8);
    e = launch_pdl(plan_fill, dim3(grid), dim3(kFillThreads), smem, stream, p);
  }
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? V4A_OK : V4A_ERR_CUDA;
}

}  // namespace v4a
