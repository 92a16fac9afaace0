// Attention of a step's tokens over the dense paged cache (v4a_dense.h,
// v4a_dense_attn): the form for few query rows per KV head (decode, short
// chunks), which any shape may take.
//
// Mathematics: one pass over the keys with a running maximum m and sum l per
// row; o = sum_j 2^{z_j - m} v_j is rescaled when m grows.  Scores are formed
// transposed, S^T = K Q^T, so that the 16 rows of an mma.m16n8k16 are keys and
// its 8 columns are query rows (the heads of a KV head's group, times tokens):
// a group of up to 8 heads wastes nothing.  O^T = V^T P^T uses the same
// columns, so the softmax factors of a column sit in the threads that hold the
// column's accumulators.
//
// Bound: memory.  A KV head reads 2 dim elements per position for
// 4 dim flops per query row, so with up to 16 rows the warp-level MMA (which
// takes 8-column operands; tcgen05 needs 128 rows) is far from its rate and
// the cache's bytes set the time.
//
// Layout: the positions of all sequences and KV heads, in tiles, form one line
// that the CTAs divide evenly, so ragged lengths balance and one long sequence
// fills the machine.  A tile is 16 positions of bf16 or 32 of fp8 (twice that
// at dim 64): contiguous runs of one page, since both divide the
// 256-position block.  Warp w of a CTA takes tiles w, w + kWarps, ... of the
// CTA's range and streams them by itself through a private ring of stages in
// shared memory (16-byte cp.async, rows swizzled for ldmatrix), with its own
// m, l and o, so the main loop has no barrier.  The warps meet when the range
// leaves a (sequence, KV head, row group): each leaves o in the stage that it
// has just read.  Pieces of a unit that several CTAs hold go to the workspace
// and are joined by a second kernel in CTA order.
//
// A cache with a scale per group has one pair of scales a tile, which lies within a
// group: 4 sequences at 1M, 16 + 2 heads of 128, 320 to 327 us (a scale per row 332), 32
// at 32k to 64k, 64 + 8 heads, 439 to 448 us: 6.6 to 6.8 TB/s, a copy's rate.
//
// bf16 caches: P is taken as the sum of two bf16 operands (16 bits), since the
// tensor cores have the time; fp8 caches: P in f16, with the values' scales in
// its exponent.  Measured with 32 + 8 heads of 128: 8 sequences at 8k 49 us
// (268 MB: 5.4 TB/s) and fp8 34 (4.1), a call of 6.6 GB 6.9 TB/s, one sequence at
// 1000 positions 10.7 us (the two launches and the loads one after the other).
// Dim 192 and 256: 8 sequences at 8k 73 and 87 us (5.5 and 6.2 TB/s), fp8 49 and 58
// (4.2 and 4.7); 16 at 32k at the copy rate, fp8 at 85% and 94% of it.
#include "dense_attn_common.cuh"

namespace v4a {
namespace {

constexpr int kRingBytes = 192 * 1024;
// Tiles that a unit's set-up and merge take the time of (200 sequences of 1 to
// 600: 0 tiles 76 us, 16 54, 48 57; one of 30000 among 60 of 100: 46, 34, 38).
constexpr int kUnitCost = 16;

// kFmt: the cache's format, V4A_KV_BF16, V4A_KV_FP8_TOKEN or V4A_KV_FP8_GROUP.
template <int D, int NT, int kFmt>
struct Shape {
  static constexpr bool kFp8 = kFmt != V4A_KV_BF16;
  static constexpr int R = 8 * NT;                               // query rows of a unit
  static constexpr int kKeys = (kFp8 ? 32 : 16) * (D == 64 ? 2 : 1);   // positions per tile
  static constexpr int kRow = kFp8 ? D : 2 * D;                  // bytes of a row
  static constexpr int kHalf = kKeys * kRow;                     // keys (or values) of a tile: 32 D bytes (64 D at dim 64)
  // A group's two scales (a tile lies in one) have 256 bytes: stages that start between two rows of banks, as 16
  // bytes would have it, took 504 us instead of 469 for 32 sequences at 32k to 64k.
  static constexpr int kScales = kFmt == V4A_KV_FP8_GROUP ? 256 : kFp8 ? 2 * kKeys * 4 : 0;
  static constexpr int kStage = 2 * kHalf + kScales;             // holds R x D fp32 for the merge as well
  static constexpr int kWarps = 4;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kPerSm = D <= 128 ? 2 : 1;                // CTAs per SM: while one's warps meet, the other's stream
  static constexpr int kStages = kRingBytes / kPerSm / (kWarps * 2 * kHalf);
  static_assert(R * D * 4 <= 2 * kHalf && kStages >= 3, "a stage holds the merge rows");
  struct Tail {                                                  // behind the rings
    int64_t scan[kWarps];
    int buf[kWarps];                                             // the stage a warp left its o in
    float ml[kWarps][R][2];
  };
};

// 16-byte chunk `ch` of row r: rows of a multiple of 128 bytes rotate over the
// eight bank groups, rows of 64 and 192 bytes over four (two rows apart).
template <int kRow>
__device__ __forceinline__ uint32_t chunk_at(int r, int ch) {
  return uint32_t(r * kRow + ((ch ^ (kRow % 128 == 0 ? r & 7 : (r >> 1) & 3)) << 4));
}

__device__ __forceinline__ void ldsm(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, const uint32_t* b) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// The same product with f16 operands.
__device__ __forceinline__ void mma16816_f16(float* c, const uint32_t* a, const uint32_t* b) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// Two e4m3 codes (low byte first) as f16, exactly.
__device__ __forceinline__ uint32_t e4m3_f16(uint32_t codes) {
  uint32_t r;
  asm("{\n.reg .b16 c;\ncvt.u16.u32 c, %1;\ncvt.rn.f16x2.e4m3x2 %0, c;\n}\n" : "=r"(r) : "r"(codes));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// log2 of a value row's scale, at least -100 (a NaN stays one).
__device__ __forceinline__ float scale_log2(float s) { return s > 0x1p-100f ? log2f(s) : s <= 0x1p-100f ? -100.f : s; }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
template <int D, int NT, int kFmt>
__global__ void __launch_bounds__(Shape<D, NT, kFmt>::kThreads, Shape<D, NT, kFmt>::kPerSm) dense_attn_mma(const DenseAttnDev a, const SplitDev p) {
  using S = Shape<D, NT, kFmt>;
  constexpr bool kFp8 = S::kFp8, kGroup = kFmt == V4A_KV_FP8_GROUP;
  constexpr int R = S::R, kWarps = S::kWarps, kThreads = S::kThreads, kKeys = S::kKeys, MT = kKeys / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  typename S::Tail& s = *reinterpret_cast<typename S::Tail*>(smem + kWarps * S::kStages * S::kStage);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  if (p.early) pdl_trigger();
  Line<R, kKeys, kThreads> line(a, p, &s + 1);
  if (!line.init(s.scan, smem, kWarps)) return;          // a tile per warp at least
  const int64_t x0 = line.x0, x1 = line.x1;

  // ---- this warp's stream: tiles x0 + warp + j kWarps, j = 0, 1, ... ----
  // Lane l looks up tile j0 + l of a batch of 32, one batch ahead of its use:
  // its page (-1: missing) and its first row in the page (KV head x 256 + position).
  struct Where { int page, row; };
  const int mine = int((x1 - x0 - warp + kWarps - 1) / kWarps);
  const int64_t to_values = int64_t(a.K) * kBlockPositions * S::kRow;
  auto lookup = [&](int j) -> Where {
    if (j >= mine) return {-1, 0};
    Unit<kKeys> un;
    const auto pc = line.locate(x0 + warp + int64_t(j) * kWarps, &un);
    const int kt = un.tr.at(pc.tile);
    const int32_t page = a.bt[int64_t(un.b) * a.max_blocks + kt / (kBlockPositions / kKeys)];
    const int row = pc.hk * kBlockPositions + kt % (kBlockPositions / kKeys) * kKeys;
    if (page >= 0 && page < a.num_blocks) return {page, row};
    report(a.status, V4A_DEV_BAD_BLOCK);
    return {-1, row};
  };
  uint8_t* ring = smem + warp * (S::kStages * S::kStage);
  const uint32_t ring0 = tc::smem_u32(ring);
  Where now = lookup(lane), next = lookup(32 + lane);
  uint32_t missing = 0;                          // bit per stage
  int issued = 0, istage = 0;
  auto issue = [&]() {                           // copies tile `issued` into stage istage; one group per call
    if (issued < mine) {
      const int page = __shfl_sync(0xffffffffu, now.page, issued & 31);
      const int row = __shfl_sync(0xffffffffu, now.row, issued & 31);
      missing = page < 0 ? missing | (1u << istage) : missing & ~(1u << istage);
      if (page >= 0) {
        const uint8_t* block = a.pool + page * a.block_bytes;
        const uint8_t* src = block + int64_t(row) * S::kRow;
        uint8_t* dst = ring + istage * S::kStage;
#pragma unroll
        for (int i = 0; i < S::kHalf / 512; ++i) {
          const int c = lane + 32 * i, r = c / (S::kRow / 16), ch = c % (S::kRow / 16);
          const uint32_t to = chunk_at<S::kRow>(r, ch);
          tc::cp_async16(dst + to, src + c * 16);
          tc::cp_async16(dst + S::kHalf + to, src + to_values + c * 16);
        }
        if (kGroup && lane < 2)                  // the group's scales
          tc::cp_async4(dst + 2 * S::kHalf + lane * 4, block + 2 * to_values + (lane * a.K * kGroupsPerBlock + row / kGroupPositions) * 4);
        if (kFp8 && !kGroup && lane < kKeys / 2) {          // the rows' scales: keys' from the first half of these lanes, values' from the rest
          const int which = lane / (kKeys / 4), q = lane % (kKeys / 4);
          const uint8_t* sc = block + 2 * to_values + (row + int64_t(which) * a.K * kBlockPositions) * 4;
          tc::cp_async16(dst + 2 * S::kHalf + which * kKeys * 4 + q * 16, sc + q * 16);
        }
      }
      if ((++issued & 31) == 0) {
        now = next;
        next = lookup(issued + 32 + lane);
      }
      if (++istage == S::kStages) istage = 0;
    }
    tc::cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < S::kStages - 1; ++i) issue();

  JoinDesc desc{};
  const float f = a.scale_log2;
  const int g4 = lane >> 2, c2 = (lane & 3) * 2;
  int stage = 0;                                 // of this warp's next tile
  uint32_t qf[D / 16][NT][2];
  float fq[NT][2];                               // f for the columns c2, c2 + 1 (fp8: with their rows' powers of two)
  auto load_q = [&](const Unit<kKeys>& un, int hk) {
    // the query rows as B operands: column g4 of n-tile nt, dims of step ks
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = nt * 8 + g4;
      const bool live = r < un.rows;
      const uint16_t* q = a.q + row_of(a, un, hk, live ? r : 0) * D;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        if (kFp8) {           // fp8: a thread's four codes are dims 4 (lane % 4) .. + 3 of the step
          const uint2 w = live ? *reinterpret_cast<const uint2*>(q + ks * 16 + 2 * c2) : make_uint2(0, 0);
          qf[ks][nt][0] = w.x;
          qf[ks][nt][1] = w.y;
        } else {
          qf[ks][nt][0] = live ? *reinterpret_cast<const uint32_t*>(q + ks * 16 + c2) : 0;
          qf[ks][nt][1] = live ? *reinterpret_cast<const uint32_t*>(q + ks * 16 + 8 + c2) : 0;
        }
      }
    }
  };
  // fp8: e4m3 codes are exact in f16, so the query joins them there: its row times the power of two
  // that brings its largest element to [2^14, 2^15) is exact down to 2^-31 of that element (and
  // within 2^-40 of it below).
  auto fit_q = [&]() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      fq[nt][0] = fq[nt][1] = f;
      if constexpr (kFp8) {
        uint32_t top = 0;                        // |q| as bf16 bits, two at a time
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) top = __vmaxu2(top, __vmaxu2(qf[ks][nt][0] & 0x7fff7fffu, qf[ks][nt][1] & 0x7fff7fffu));
        top = max(top >> 16, top & 0xffffu);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = top == 0 ? 127 : min(253, max(1, 268 - int(top >> 7)));      // the power's exponent field
        const float up = __int_as_float(e << 23), down = __int_as_float((254 - e) << 23);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t w = qf[ks][nt][i];
            qf[ks][nt][i] = pack_f16(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up);
          }
        // at least the smallest normal number: flushed to zero, it would make NaNs of hidden keys' -inf
        fq[nt][0] = fmaxf(f * __shfl_sync(0xffffffffu, down, 4 * c2), 0x1p-126f);
        fq[nt][1] = fmaxf(f * __shfl_sync(0xffffffffu, down, 4 * c2 + 4), 0x1p-126f);
      }
    }
  };
  int64_t x = x0;
  Unit<kKeys> next_un;
  auto next_pc = line.locate(x, &next_un);
  load_q(next_un, next_pc.hk);
  while (x < x1) {
    const Unit<kKeys> un = next_un;
    const auto pc = next_pc;
    const int count = int(min(int64_t(un.tr.tiles - pc.tile), x1 - x));     // tiles of this segment
    fit_q();
    float o[D / 16][NT][4], m[NT][2], l[NT][2];
    int mrow[NT][2];                               // the columns' query positions
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nt][e] = -INFINITY;
        l[nt][e] = 0.f;
        mrow[nt][e] = un.m_lo + ((un.row0 % a.G) + min(nt * 8 + c2 + e, un.rows - 1)) / a.G;
      }
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[d][nt][e] = 0.f;
    }

    int last = stage;                              // the stage read last: free until the next issue()
    const int phase = int((x - x0) % kWarps);
    for (int i = (warp - phase + kWarps) % kWarps; i < count; i += kWarps) {
      tc::cp_async_wait_group<S::kStages - 2>();
      __syncwarp();                                // every lane's copies of the tile; every lane has left the stage read last
      const bool gone = missing >> stage & 1;
      const int cur = stage;
      if (++stage == S::kStages) stage = 0;
      last = cur;
      issue();                                     // into the stage read last
      if (gone) continue;
      const uint32_t kb = ring0 + cur * S::kStage, vb = kb + S::kHalf;
      const float* scale = reinterpret_cast<const float*>(ring + cur * S::kStage + 2 * S::kHalf);
      const int j0 = un.tr.at(pc.tile + i) * kKeys;
      float z[MT][NT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) z[mt][nt][e] = 0.f;
      // S^T = K Q^T
      const int lr = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        if constexpr (!kFp8) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t k[4];
            ldsm(kb + chunk_at<S::kRow>(mt * 16 + lr, 2 * ks + (lane >> 4)), k);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816(z[mt][nt], k, qf[ks][nt]);
          }
        } else {
          // matrices: keys 0-7 and 8-15 of 16-code chunk 2c, then of chunk 2c + 1
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t w[4];
            ldsm(kb + chunk_at<S::kRow>(mt * 16 + lr, 2 * c + (lane >> 4)), w);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t lo = w[2 * h], hi = w[2 * h + 1];
              const uint32_t k[4] = {e4m3_f16(lo), e4m3_f16(hi), e4m3_f16(lo >> 16), e4m3_f16(hi >> 16)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816_f16(z[mt][nt], k, qf[2 * c + h][nt]);
            }
          }
          if constexpr (!kGroup) {
            const float k0 = scale[mt * 16 + g4], k1 = scale[mt * 16 + g4 + 8];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              z[mt][nt][0] *= k0; z[mt][nt][1] *= k0;
              z[mt][nt][2] *= k1; z[mt][nt][3] *= k1;
            }
          }
        }
      }
      // mask, running maximum
      const bool full = all_visible(a, un.m_lo, un.m_hi, j0, kKeys);
      if (!full) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!visible(a, mrow[nt][e & 1], j0 + mt * 16 + g4 + (e >> 1) * 8)) z[mt][nt][e] = -INFINITY;
      }
      // In log2 units from here.  fp8: the values' scales are a part of the exponent (w_j = z_j + log2
      // sv_j, whose running maximum is taken), so that P = 2^{w - m} is 1 at its largest whatever the
      // scales are and fits f16, whose 11 bits keep the single dominating key exact to 2^-12 (a bf16
      // product p sv lost up to 2^-9 there); 2^15 P uses f16's upper range, so that keys down to
      // 2^-39 of the largest count.  l sums 2^{z - m} itself: at most 2^100 a key.
      float ls[MT][2], fz[NT][2];                // fz: the scores' factors (a group's key scale among them)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) fz[nt][e] = kGroup ? logit_factor(fq[nt][e] * scale[0]) : fq[nt][e];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        if constexpr (kGroup) {
          ls[mt][0] = ls[mt][1] = scale_log2(scale[1]);
          continue;
        }
        ls[mt][0] = kFp8 ? scale_log2(scale[kKeys + mt * 16 + g4]) : 0.f;
        ls[mt][1] = kFp8 ? scale_log2(scale[kKeys + mt * 16 + g4 + 8]) : 0.f;
      }
      bool grew = false;
      float alpha[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = -INFINITY;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            t = kFp8 ? fmaxf(t, fmaxf(fmaf(z[mt][nt][e], fz[nt][e], ls[mt][0]), fmaf(z[mt][nt][e + 2], fz[nt][e], ls[mt][1])))
                     : fmaxf(t, fmaxf(z[mt][nt][e], z[mt][nt][e + 2]));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
          if (!kFp8) t *= f;
          const float top = fmaxf(m[nt][e], t);
          grew |= top > m[nt][e];
          alpha[nt][e] = top == -INFINITY ? 1.f : exp2f(m[nt][e] - top);
          m[nt][e] = top;
        }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          l[nt][0] *= alpha[nt][0];
          l[nt][1] *= alpha[nt][1];
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            o[d][nt][0] *= alpha[nt][0]; o[d][nt][1] *= alpha[nt][1];
            o[d][nt][2] *= alpha[nt][0]; o[d][nt][3] *= alpha[nt][1];
          }
        }
      }
      // P^T as B operands: keys are rows of the k step
      uint32_t pf[MT][NT][2], pl[kFp8 ? 1 : MT][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float b0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0], b1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const float y0 = fmaf(z[mt][nt][0], fz[nt][0], -b0), y1 = fmaf(z[mt][nt][1], fz[nt][1], -b1);
          const float y2 = fmaf(z[mt][nt][2], fz[nt][0], -b0), y3 = fmaf(z[mt][nt][3], fz[nt][1], -b1);
          const float p0 = exp2f(y0), p1 = exp2f(y1), p2 = exp2f(y2), p3 = exp2f(y3);
          l[nt][0] += p0 + p2;
          l[nt][1] += p1 + p3;
          if constexpr (kFp8) {        // a hidden row has y = -inf; its scale may be anything
            auto weight = [](float y, float s) { return y == -INFINITY ? 0.f : exp2f(y + s); };
            const float s0 = ls[mt][0] + 15.f, s1 = ls[mt][1] + 15.f;
            pf[mt][nt][0] = transpose8(pack_f16(weight(y0, s0), weight(y1, s0)));
            pf[mt][nt][1] = transpose8(pack_f16(weight(y2, s1), weight(y3, s1)));
          } else {
            // two bf16 operands, p and what its rounding left: 16 bits (the products wait on memory anyway)
            auto split = [](float u, float w, uint32_t* hi, uint32_t* lo) {
              const uint32_t h = pack_bf16(u, w);
              *hi = transpose8(h);
              *lo = transpose8(pack_bf16(u - __uint_as_float(h << 16), w - __uint_as_float(h & 0xffff0000u)));
            };
            split(p0, p1, &pf[mt][nt][0], &pl[mt][nt][0]);
            split(p2, p3, &pf[mt][nt][1], &pl[mt][nt][1]);
          }
        }
      }
      // O^T += V^T P^T; value rows that no row of the unit sees become zeros
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
        if (!full) {
          uint32_t k[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = j0 + mt * 16 + c2 + (e & 1) + (e >> 1) * 8;
            k[e] = j <= un.m_hi && (a.window == 0 || j > un.m_lo - a.window || j < a.sinks) ? 0xffffu : 0u;
          }
          keep0 = k[0] | k[1] << 16;
          keep1 = k[2] | k[3] << 16;
        }
        if constexpr (!kFp8) {
          const int key = mt * 16 + (lane & 7) + (lane >> 4) * 8;
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            uint32_t v[4];
            ldsm_t(vb + chunk_at<S::kRow>(key, 2 * d + ((lane >> 3) & 1)), v);
            if (!full) { v[0] &= keep0; v[1] &= keep0; v[2] &= keep1; v[3] &= keep1; }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma16816(o[d][nt], v, pf[mt][nt]);
              mma16816(o[d][nt], v, pl[mt][nt]);
            }
          }
        } else {
          // matrices: keys 0-7 and 8-15 of 16-code chunk 2c, then of chunk 2c + 1; a transposed
          // word holds codes (key, dim 2 g4), (key, dim 2 g4 + 1) of two keys: the MMA's rows g4
          // and g4 + 8 are dims 2 g4 and 2 g4 + 1 of the chunk
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t w[4];
            ldsm_t(vb + chunk_at<S::kRow>(mt * 16 + lr, 2 * c + (lane >> 4)), w);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t lo = w[2 * h], hi = w[2 * h + 1];
              const uint32_t wl = __byte_perm(lo, 0, 0x3120), wh = __byte_perm(hi, 0, 0x3120);
              uint32_t v[4] = {e4m3_f16(wl), e4m3_f16(wl >> 16), e4m3_f16(wh), e4m3_f16(wh >> 16)};
              if (!full) { v[0] &= keep0; v[1] &= keep0; v[2] &= keep1; v[3] &= keep1; }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816_f16(o[2 * c + h][nt], v, pf[mt][nt]);
            }
          }
        }
      }
    }

    // ---- the warps' results meet: o [R][D] fp32 in the stage read last ----
    // (float index r D + (d with bits 3..4 turned by r / 2): the rows that one
    // store touches lie in different banks)
    if (x + count >= x1) pdl_trigger();      // the join may be set up (it waits for this kernel's end)
    if (x + count < x1) {          // the next segment's queries are on their way meanwhile
      next_pc = line.locate(x + count, &next_un);
      load_q(next_un, next_pc.hk);
    }
    __syncwarp();
    float* mine_o = reinterpret_cast<float*>(ring + last * S::kStage);
    if (lane == 0) s.buf[warp] = int(ring - smem) + last * S::kStage;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float t = l[nt][e];
        t += __shfl_xor_sync(0xffffffffu, t, 4);
        t += __shfl_xor_sync(0xffffffffu, t, 8);
        t += __shfl_xor_sync(0xffffffffu, t, 16);
        const int r = nt * 8 + c2 + e, turn = ((r >> 1) & 3) << 3;
        // a column without a key leaves nothing (a warp without a tile of this segment has no free
        // stage either); one whose logits are all NaN has m = -inf and a NaN sum, and is passed on
        const bool none = m[nt][e] == -INFINITY && t == 0.f;
        if (g4 == 0) {
          s.ml[warp][r][0] = none ? -INFINITY : m[nt][e] == -INFINITY ? 0.f : m[nt][e];
          s.ml[warp][r][1] = t;
        }
        if (!none) {
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            // rows of the accumulator: dims g4, g4 + 8 (fp8: dims 2 g4, 2 g4 + 1)
            constexpr float unit = kFp8 ? 0x1p-15f : 1.f;
            mine_o[r * D + ((d * 16 + (kFp8 ? 2 * g4 : g4)) ^ turn)] = o[d][nt][e] * unit;
            mine_o[r * D + ((d * 16 + (kFp8 ? 2 * g4 + 1 : g4 + 8)) ^ turn)] = o[d][nt][e + 2] * unit;
          }
        }
      }
    }
    __syncthreads();
    const bool begins = pc.tile == 0, ends = pc.tile + count == un.tr.tiles;
    const int64_t part = int64_t(blockIdx.x) * 2 + (begins ? 1 : 0);
    for (int i = tid; i < R * D / 4; i += kThreads) {
      const int r = i / (D / 4), d = i % (D / 4) * 4, turn = ((r >> 1) & 3) << 3;
      if (r >= un.rows) continue;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s.ml[w][r][0]);
      float sum = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (s.ml[w][r][0] == -INFINITY) continue;
        const float wt = exp2f(s.ml[w][r][0] - top);
        sum = fmaf(wt, s.ml[w][r][1], sum);
        const float4 t = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + s.buf[w]) + r * D + (d ^ turn));
        v[0] = fmaf(wt, t.x, v[0]); v[1] = fmaf(wt, t.y, v[1]);
        v[2] = fmaf(wt, t.z, v[2]); v[3] = fmaf(wt, t.w, v[3]);
      }
      if (begins && ends) {
        const int64_t row = row_of(a, un, pc.hk, r);
        const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;     // NaN stays NaN
        *reinterpret_cast<uint2*>(a.out + row * D + d) =
            make_uint2(pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv));
        if (d == 0 && a.lse) a.lse[row] = (top + log2f(sum)) * 0.6931471805599453f;
      } else {
        *reinterpret_cast<float4*>(p.part_o + (part * R + r) * D + d) = make_float4(v[0], v[1], v[2], v[3]);
        if (d == 0) {
          p.part_ml[(part * R + r) * 2] = top;
          p.part_ml[(part * R + r) * 2 + 1] = sum;
        }
      }
    }
    if (begins && !ends) desc = line.describe(pc, un);     // the unit goes on in the next CTAs
    __syncthreads();              // the stages are read
    x += count;
  }
  if (p.split && tid == 0) p.join[blockIdx.x] = desc;
}

// Joins the pieces of a unit that several CTAs hold: piece c's slot 1, then
// slot 0 of the CTAs behind it; weights 2^{m - max} of the pieces' maxima.  A
// CTA takes one row (grid.y = rows) of the unit that CTA blockIdx.x of the
// launch before describes; 8 groups of lanes share the pieces and meet in
// group order, so the result does not depend on timing.
template <int D>
__global__ void __launch_bounds__(256) dense_join_kernel(const DenseAttnDev a, const SplitDev p) {
  constexpr int kLanes = D / 4, kGroups = 256 / kLanes > 8 ? 8 : 256 / kLanes;
  __shared__ float4 acc[kGroups][kLanes];
  __shared__ float2 red[kGroups];
  const int c = blockIdx.x, r = blockIdx.y, tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  const JoinDesc j = p.join[c];
  if (r >= j.rows) return;
  // each group goes once through its pieces with a running maximum
  const int pieces = j.last - c + 1, g = tid / kLanes, l = tid % kLanes;
  float top = -INFINITY, sum = 0.f;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (g < kGroups) {
#pragma unroll 4
    for (int k = g; k < pieces; k += kGroups) {
      const int64_t part = (int64_t(c + k) * 2 + (k == 0 ? 1 : 0)) * p.rows + r;
      const float2 t = *reinterpret_cast<const float2*>(p.part_ml + part * 2);
      const float4 o = *reinterpret_cast<const float4*>(p.part_o + part * D + 4 * l);
      if (t.x == -INFINITY) continue;        // a piece without a key
      const float m = fmaxf(top, t.x), w0 = exp2f(top - m), w1 = exp2f(t.x - m);
      top = m;
      sum = fmaf(sum, w0, w1 * t.y);
      v.x = fmaf(v.x, w0, w1 * o.x); v.y = fmaf(v.y, w0, w1 * o.y);
      v.z = fmaf(v.z, w0, w1 * o.z); v.w = fmaf(v.w, w0, w1 * o.w);
    }
    acc[g][l] = v;
    if (l == 0) red[g] = make_float2(top, sum);
  }
  __syncthreads();
  if (tid >= kLanes) return;
  top = -INFINITY;
#pragma unroll
  for (int k = 0; k < kGroups; ++k) top = fmaxf(top, red[k].x);
  sum = 0.f;
  v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < kGroups; ++k) {
    const float2 t = red[k];
    if (t.x == -INFINITY) continue;
    const float w = exp2f(t.x - top);
    const float4 o = acc[k][l];
    sum = fmaf(w, t.y, sum);
    v.x = fmaf(w, o.x, v.x); v.y = fmaf(w, o.y, v.y); v.z = fmaf(w, o.z, v.z); v.w = fmaf(w, o.w, v.w);
  }
  const int i = j.row0 + r;
  const int64_t at = int64_t(j.s0 + i / a.G) * a.H + j.hk * a.G + i % a.G;
  const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;
  *reinterpret_cast<uint2*>(a.out + at * D + 4 * l) = make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
  if (l == 0 && a.lse) a.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

// The same for units of 128 or 256 rows (dense_prefill*.cu), whose pieces are few and
// lie as [slot][dim / 4][row][4]: a thread takes a row's 16 dims (grid.y =
// dim / 16) through the pieces in order.
template <int D>
__global__ void __launch_bounds__(256) dense_join_rows(const DenseAttnDev a, const SplitDev p) {
  const int c = blockIdx.x, r = threadIdx.x, d0 = blockIdx.y * 4;
  pdl_wait();
  pdl_trigger();
  const JoinDesc j = p.join[c];
  if (r >= j.rows) return;
  auto slot = [&](int k) { return int64_t(c + k) * 2 + (k == 0 ? 1 : 0); };
  auto ml = [&](int k) { return *reinterpret_cast<const float2*>(p.part_ml + (slot(k) * p.rows + r) * 2); };
  const int pieces = j.last - c + 1;
  float top = -INFINITY, sum = 0.f;
#pragma unroll 4
  for (int k = 0; k < pieces; ++k) top = fmaxf(top, ml(k).x);
  float4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int k = 0; k < pieces; ++k) {
    const float2 t = ml(k);
    float4 o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = reinterpret_cast<const float4*>(p.part_o)[(slot(k) * (D / 4) + d0 + i) * p.rows + r];
    if (t.x == -INFINITY) continue;
    const float w = exp2f(t.x - top);
    sum = fmaf(w, t.y, sum);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i].x = fmaf(w, o[i].x, v[i].x); v[i].y = fmaf(w, o[i].y, v[i].y);
      v[i].z = fmaf(w, o[i].z, v[i].z); v[i].w = fmaf(w, o[i].w, v[i].w);
    }
  }
  const int i = j.row0 + r;
  const int64_t at = int64_t(j.s0 + i / a.G) * a.H + j.hk * a.G + i % a.G;
  const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;
#pragma unroll
  for (int k = 0; k < 4; k += 2)
    *reinterpret_cast<uint4*>(a.out + at * D + 4 * (d0 + k)) =
        make_uint4(pack_bf16(v[k].x * inv, v[k].y * inv), pack_bf16(v[k].z * inv, v[k].w * inv),
                   pack_bf16(v[k + 1].x * inv, v[k + 1].y * inv), pack_bf16(v[k + 1].z * inv, v[k + 1].w * inv));
  if (blockIdx.y == 0 && a.lse) a.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

// A call whose sequences all bring many rows runs the form of dense_prefill*.cu, one
// whose sequences all bring few rows this file's, and a mixed one both, each
// launch taking its sequences: it is mixed when the token count leaves room
// for short sequences beside the longest.  The short ones go first, so that
// the few CTAs of a small chunk do not hold back an even share of theirs: 64
// decoding sequences (32 + 8 heads of 128) beside a chunk of 9 tokens 63 us (75
// in the other order), of 4096 295 (306), 256 beside 4096 312 (304; 146 and 147
// alone).  The launches for short sequences that are not there cost two chunks
// of 1024 9 us of 54.  (Choosing the order by the batch's mean rows saved 8 us
// there and cost every small decode call 4%: the form for few rows would have to
// read past the L1 as well.)
bool mixed(const v4a_dense_attn_args* a) {
  return dense_prefill_takes(a) && a->num_tokens < int64_t(a->num_seqs) * a->max_new_per_seq;
}

// The most rows a sequence brings to the form for few rows.
int64_t most_rows(const v4a_dense_attn_args* a) {
  const int64_t rows = int64_t(a->max_new_per_seq) * (a->num_heads / a->kv.num_kv_heads);
  return dense_prefill_takes(a) ? few_rows(a->kv.dim, a->kv.format) : rows;
}

int rows_of(const v4a_dense_attn_args* a) {
  return most_rows(a) > 8 && a->kv.dim <= 192 ? 16 : 8;      // 16 rows of dim 256 would not fit the registers
}

int64_t row_groups(const v4a_dense_attn_args* a) { return (most_rows(a) + rows_of(a) - 1) / rows_of(a); }

int ctas_of(const v4a_dense_attn_args* a) { return a->kv.dim <= 128 ? 2 * kSms : kSms; }

size_t few_workspace(const v4a_dense_attn_args* a) { return split_workspace(rows_of(a), a->kv.dim, ctas_of(a)); }

// Of every call of the shape, mixed or not.
size_t workspace_of(const v4a_dense_attn_args* a) {
  return few_workspace(a) + (dense_prefill_takes(a) ? dense_prefill_workspace(a) : 0);
}

template <int D, int NT, int kFmt>
int launch(const DenseAttnDev& a, const SplitDev& p, cudaStream_t stream) {
  using S = Shape<D, NT, kFmt>;
  const size_t smem = S::kWarps * S::kStages * S::kStage + sizeof(typename S::Tail) + split_smem(p.split, p.U);
  static_assert(S::kWarps * S::kStages * S::kStage + sizeof(typename S::Tail) + split_smem(1, kMaxSplitUnits) <= 227 * 1024, "shared memory of a CTA");
  auto kern = dense_attn_mma<D, NT, kFmt>;
  static std::atomic<uint64_t> done{0};
  if (!once_per_device(&done, [=] { return raise_smem(kern, 227 * 1024); })) return V4A_ERR_CUDA;
  const int64_t grid = p.split ? p.grid : int64_t(p.U) * a.K;
  const cudaError_t e = launch_pdl(kern, dim3(unsigned(grid)), dim3(S::kThreads), smem, stream, a, p);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? V4A_OK : V4A_ERR_CUDA;
}

template <int kFmt>
int launch_dim(const DenseAttnDev& a, const SplitDev& p, int dim, cudaStream_t stream) {
  const bool two = p.rows == 16;
  switch (dim) {
    case 64: return two ? launch<64, 2, kFmt>(a, p, stream) : launch<64, 1, kFmt>(a, p, stream);
    case 128: return two ? launch<128, 2, kFmt>(a, p, stream) : launch<128, 1, kFmt>(a, p, stream);
    case 192: return two ? launch<192, 2, kFmt>(a, p, stream) : launch<192, 1, kFmt>(a, p, stream);
    default: return launch<256, 1, kFmt>(a, p, stream);
  }
}

// Everything but the pointers of the call's own tensors.
int check_shape(const v4a_dense_attn_args* a) {
  if (!a || a->num_tokens < 0 || a->num_seqs < 0 || a->max_new_per_seq < 1 || a->num_heads < 1 || a->window < 0 || a->sinks < 0)
    return V4A_ERR_INVALID_ARG;
  const v4a_dense_cache& c = a->kv;
  if (c.num_kv_heads < 1 || c.num_kv_heads > 1024 || a->num_heads % c.num_kv_heads) return V4A_ERR_INVALID_ARG;
  if (c.dim != 64 && c.dim != 128 && c.dim != 192 && c.dim != 256) return V4A_ERR_UNSUPPORTED;
  if (c.format != V4A_KV_BF16 && c.format != V4A_KV_FP8_TOKEN && c.format != V4A_KV_FP8_GROUP) return V4A_ERR_UNSUPPORTED;
  if (a->num_heads > 1024 || a->max_new_per_seq > (1 << 22) || c.max_blocks > (1 << 22)) return V4A_ERR_UNSUPPORTED;
  if (int64_t(a->max_new_per_seq) * (a->num_heads / c.num_kv_heads) > INT32_MAX / 2) return V4A_ERR_UNSUPPORTED;   // rows are counted in 32 bits
  return V4A_OK;
}

}  // namespace

int dense_join(const DenseAttnDev& a, const SplitDev& p, int dim, cudaStream_t stream) {
  const bool many = p.rows > 16;
  auto kern = many ? (dim == 64 ? dense_join_rows<64> : dim == 128 ? dense_join_rows<128> : dim == 192 ? dense_join_rows<192> : dense_join_rows<256>)
                   : (dim == 64 ? dense_join_kernel<64> : dim == 128 ? dense_join_kernel<128> : dim == 192 ? dense_join_kernel<192> : dense_join_kernel<256>);
  const int y = many ? dim / 16 : int(std::min<int64_t>(p.rows, std::min<int64_t>(int64_t(a.max_new) * a.G, p.rows_to)));   // rows that a unit can have
  const cudaError_t e = launch_pdl(kern, dim3(unsigned(p.grid), unsigned(y)), dim3(many ? p.rows : 256), 0, stream, a, p);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? V4A_OK : V4A_ERR_CUDA;
}

size_t dense_attn_workspace_size(const v4a_dense_attn_args* a) { return check_shape(a) ? 0 : workspace_of(a); }

int dense_attn(const v4a_dense_attn_args* a, void* ws, size_t ws_bytes, cudaStream_t stream) {
  int rc = check_shape(a);
  if (rc) return rc;
  DenseAttnDev d{};
  rc = dense_cache_check(a->kv, &d.block_bytes);
  if (rc) return rc;
  if (a->kv.format == V4A_KV_FP8_GROUP && d.block_bytes >= int64_t(1) << 40) return V4A_ERR_UNSUPPORTED;      // (a tensor map's strides)
  if (!(a->softmax_scale > 0.f) || !std::isfinite(a->softmax_scale * 1.4426950408889634f) || a->kv.max_blocks < 1) return V4A_ERR_INVALID_ARG;
  if (a->num_tokens == 0 || a->num_seqs == 0) return V4A_OK;
  if (!a->positions || !a->token_starts || !a->kv.block_table || !a->q || !a->out) return V4A_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(a->q) & 15) || (reinterpret_cast<uintptr_t>(a->out) & 15) ||
      static_cast<const void*>(a->q) == static_cast<const void*>(a->out))
    return V4A_ERR_INVALID_ARG;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 15) || ws_bytes < workspace_of(a)) return V4A_ERR_WORKSPACE;
  d.T = a->num_tokens; d.B = a->num_seqs; d.H = a->num_heads; d.K = a->kv.num_kv_heads; d.G = d.H / d.K;
  d.max_new = a->max_new_per_seq; d.max_blocks = a->kv.max_blocks; d.sinks = a->sinks;
  // a window as long as a sequence can be hides nothing (and the kernels' differences stay in 32 bits)
  d.window = a->window < int64_t(a->kv.max_blocks) * kBlockPositions ? a->window : 0;
  d.num_blocks = a->kv.num_blocks;
  d.positions = a->positions; d.starts = a->token_starts; d.bt = a->kv.block_table;
  d.pool = static_cast<const uint8_t*>(a->kv.pool);
  d.q = a->q; d.out = a->out; d.lse = a->lse; d.status = a->status;
  d.scale_log2 = std::max(a->softmax_scale * 1.4426950408889634f, 0x1p-126f);      // (a subnormal one would be flushed)
  const bool fp8 = a->kv.format != V4A_KV_BF16, takes = dense_prefill_takes(a), both = takes && mixed(a);
  const int few = few_rows(a->kv.dim, a->kv.format);
  SplitDev p{}, many{};
  p.RG = int(row_groups(a));
  p.rows_to = both ? few : INT32_MAX;
  const int64_t units = units_bound(d, p.rows_from, p.RG, rows_of(a));
  // all refusals come before the first launch
  if (!takes || both)
    if (units > INT32_MAX || units * d.K > INT32_MAX) return V4A_ERR_UNSUPPORTED;
  if (takes) {
    rc = dense_prefill_plan(a, d, both ? few + 1 : 0, static_cast<uint8_t*>(ws) + few_workspace(a), &many);
    if (rc) return rc;
    if (many.U > 0 && !dense_prefill_ready(a, d)) return V4A_ERR_CUDA;
    if (!both) {
      rc = dense_prefill(a, d, many, stream);
      return rc == V4A_OK && many.split == 1 ? dense_join(d, many, a->kv.dim, stream) : rc;
    }
    p.early = many.late = many.U > 0;               // (no room for a sequence of the other form: no launch for it)
  }
  p.U = int(units);
  // One CTA per unit and KV head under a window of up to 4096 when there are enough of them to keep the memory
  // busy (one streams 50 GB/s of bf16 rows, 25 of fp8 ones), or it is short; an even split otherwise.  Unsplit /
  // split, us: 64 sequences x 8 heads of 64, window 1024: 29 / 34; heads of 128, 4096: 153 / 172; 64 x 2 heads,
  // 1024: 15 / 19; 20 x 2, 1024: 15 / 13, 4096: 45 / 18, 256: 8 / 12; fp8, 20 x 8, 4096: 50 / 41.  Longer windows
  // gain less (16384: 579 / 619) and would leave one long sequence among short ones to run alone.
  p.split = std::max(p.U, d.B) <= kMaxSplitUnits &&
            (d.window == 0 || d.window > 4096 || (units * d.K < (fp8 ? 256 : 128) && d.window > 512));
  split_carve(&p, ws, rows_of(a), a->kv.dim, ctas_of(a), kUnitCost);
  rc = a->kv.format == V4A_KV_FP8_GROUP ? launch_dim<V4A_KV_FP8_GROUP>(d, p, a->kv.dim, stream)
       : fp8 ? launch_dim<V4A_KV_FP8_TOKEN>(d, p, a->kv.dim, stream) : launch_dim<V4A_KV_BF16>(d, p, a->kv.dim, stream);
  if (rc == V4A_OK && many.U > 0) rc = dense_prefill(a, d, many, stream);
  if (rc == V4A_OK && p.split) rc = dense_join(d, p, a->kv.dim, stream);
  return rc == V4A_OK && many.U > 0 && many.split == 1 ? dense_join(d, many, a->kv.dim, stream) : rc;
}

}  // namespace v4a
