// Attention of chunks over the dense paged cache on the tensor cores
// (v4a_dense_attn with many query rows per KV head; dim 64 and 128): tcgen05
// kind::f16 with the accumulators in TMEM.
//
// Mathematics: as dense_attn.cu, one pass over the keys with a running
// maximum and sum per row.  The rows of a CTA are 256 consecutive (token,
// head of the group) pairs of one sequence and KV head, as two tiles of 128:
// both read each key tile, and while one tile is in its softmax the tensor
// cores work for the other.  The maximum that P is formed against is raised
// only when a row's logits pass it by more than 2^8, so the output
// accumulator is rescaled a few times per row instead of once per key tile;
// P <= 2^8 then, which bf16 holds as well as values up to one, and l uses the
// same maximum.
//
//   S_t = Q_t K^T   M = 128, N = 128 keys, K = dim     TMEM columns [128 t, +128)
//   P_t = 2^{S f - m} in bf16 (fp8: f16), over S_t's columns  [128 t, +64)
//   O_t += P_t V    M = 128, N = dim, K = 128 keys      [256 + 128 t, +dim)
//                   (P from TMEM, V as an MN-major operand)
//
// Roles: warps 0-3 and 4-7 the two tiles' softmax (a thread owns a row), 8
// issues the MMAs, the others copy keys and values into the 128-byte swizzle
// (bf16: 16-byte cp.async; fp8: through registers, the codes becoming bf16 keys
// and f16 values exactly, their scales applied to the logits and to P).  Rows
// that no row of the CTA sees are filled with zeros, so what they hold cannot
// reach a product.  Keys and values have two buffers each.
//
// P is rounded to bf16: by at most 2^-8 of each weight, so by at most 2^-8
// sum_j p_j |v_j| in the output, as much as the output's own rounding may be
// where nothing cancels; the two-operand P of dense_attn.cu would double
// the second product here, where the tensor cores set the time.
//
// Bound: no one unit.  A step is a chain of product, softmax and product for
// each of two row tiles, and two softmax warps a scheduler do not cover its
// waits: dim 128 bf16 keeps the tensor pipe 50% busy, the issue slots 40% and the
// exponential unit 25%; dim 64, with half of the flops for the same softmax,
// 30%, 44% and 30%.  Measured, 32 + 8 heads of 128, 2048 tokens over 10240
// positions: bf16 258 us (1200 TFLOP/s), fp8 480 us (645: the conversions of the
// codes); dim 64 bf16 211 us (733), fp8 396 (390); a window of 1024 with 1500
// tokens 61 us.
#include "dense_prefill_common.cuh"

namespace v4a {
namespace {

constexpr int kRows = 128;           // rows of a tile (MMA M)
constexpr int kKeys = 128;           // keys per step
constexpr int kUnit = 2 * kRows;     // rows of a unit
// Threads and registers of the two forms (2k tokens over 10k, 32 + 8 heads of
// 128).  bf16 rows are copied as they are: three warps and 200 registers for
// the softmax, 258 us; four warps among 512 threads, whose softmax has 192, 314
// us.  fp8 rows go through the registers of their copying warps, which convert
// them: four warps and 184 + 72 registers, 495 us, and 480 since their
// loads go past the L1 (192 + 64: 545; seven warps:
// 546; three among 384 threads: 587).  The registers of a thread at launch come
// in steps that four warps share, so 512 threads carry three warps that only
// wait.  softmax x 256 + rest x (threads - 256) = launch x threads.
template <bool kFp8>
struct Roles {
  static constexpr int kThreads = kFp8 ? 512 : 384;
  static constexpr int kLoaders = kFp8 ? 128 : 96;
  static constexpr int kSoftmaxRegs = kFp8 ? 184 : 200, kRestRegs = kFp8 ? 72 : 104, kLaunchRegs = kFp8 ? 128 : 168;
  static_assert(kSoftmaxRegs * 256 + kRestRegs * (kThreads - 256) == kLaunchRegs * kThreads, "the split of the registers");
};
// Steps that a unit's set-up and output take the time of (one chunk of 4096
// tokens, 32 + 8 heads: 0 steps 320 us, 1 223, 3 147, 6 151, 12 163).
constexpr int kUnitCost = 3;
constexpr int kMinSteps = 4;         // steps a CTA of an even split has at least

struct PreSmem {
  uint64_t q_full[2], k_full[2], v_full[2], k_free[2], v_free[2], s_full[2], p_full[2][2], o_full[2], drain;
  int64_t scan[16];
  uint32_t tmem_base;
  int abort_flag;
  int missing[4];                    // step n's page is missing: [n % 4]
  // fp8, step n's keys: softmax scale x log2(e) x key scale; log2 of the value scale; its inverse
  alignas(16) float scales[4][3][kKeys];
};

// Byte offset of 16-byte chunk `ch` of row r in an operand of [dim / 64][128 rows][128 bytes], swizzled.
__device__ __forceinline__ uint32_t chunk_at(int r, int ch) {
  return uint32_t((ch >> 3) * (128 * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(Roles<kFp8>::kThreads, 1) dense_prefill_kernel(const DenseAttnDev a, const SplitDev p) {
  constexpr int kThreads = Roles<kFp8>::kThreads, kLoaders = Roles<kFp8>::kLoaders;
  constexpr int kTileBytes = 128 * D * 2;      // a Q tile, a step's keys or its values
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t q0 = tc::smem_u32(base), k0 = q0 + 2 * kTileBytes, v0 = k0 + 2 * kTileBytes;
  PreSmem& s = *reinterpret_cast<PreSmem*>(base + 6 * kTileBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &s.abort_flag;

  if (!p.late) pdl_wait();
  Line<kUnit, kKeys, kThreads> line(a, p, &s + 1);
  if (!line.init(s.scan, base, kMinSteps)) {
    if (p.late) pdl_wait();
    return;
  }
  const int64_t x0 = line.x0, x1 = line.x1;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&s.q_full[i], kRows);
      tc::mbar_init(&s.k_full[i], kLoaders + (kFp8 ? 0 : 1));
      tc::mbar_init(&s.v_full[i], kLoaders);
      tc::mbar_init(&s.k_free[i], 1);
      tc::mbar_init(&s.v_free[i], 1);
      tc::mbar_init(&s.s_full[i], 1);
      tc::mbar_init(&s.p_full[i][0], 4);
      tc::mbar_init(&s.p_full[i][1], 4);
      tc::mbar_init(&s.o_full[i], 1);
    }
    tc::mbar_init(&s.drain, 1);
    s.abort_flag = 0;
    tc::mbar_fence_init();
  }
  __syncwarp();
  if (warp == 0) tc::tmem_alloc(&s.tmem_base, 512);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = s.tmem_base;

  // Every role walks the CTA's segments (the parts of units in [x0, x1)) by
  // itself.  Counters: n = steps of the CTA (key and value buffers), e = steps
  // of a tile (its S and P), g = segments of a tile (its Q and O).
  if (warp < 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Roles<kFp8>::kSoftmaxRegs));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Roles<kFp8>::kRestRegs));
  if (warp < 8) {
    // ---- a tile's queries, softmax and output ----
    const int t = warp >> 2, r = tid & 127;
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + 128 * t + lanes, o_at = tmem + 256 + 128 * t + lanes;
    const float f = a.scale_log2;
    bool ok = true;
    int n0 = 0, e = 0, g = 0;
    for (int64_t x = x0; x < x1 && ok;) {
      Unit<kKeys> un;
      const auto pc = line.locate(x, &un);
      const int count = int(min(int64_t(un.tr.tiles - pc.tile), x1 - x));
      if (un.rows > t * kRows) {
        // Q rows behind the last are zeros
#pragma unroll 4
        for (int c = r; c < kRows * (D / 8); c += kRows) {
          const int qr = c / (D / 8), ch = c % (D / 8), i = t * kRows + qr;
          const uint16_t* q = a.q + row_of(a, un, pc.hk, min(i, un.rows - 1)) * D;
          copy16(q0 + t * kTileBytes + chunk_at(qr, ch), q + ch * 8, i < un.rows);
        }
        tc::cp_async_wait_all();
        tc::fence_proxy_async();
        tc::mbar_arrive(&s.q_full[t]);
        const int row = t * kRows + r, m = un.m_lo + (un.row0 % a.G + min(row, un.rows - 1)) / a.G;
        float top = -INFINITY, ref = 0.f, l = 0.f;       // largest logit, the maximum in use, the sum against it
        bool any = false;                                // `ref` is set (a key has been seen)
        for (int i = 0; i < count; ++i, ++e) {
          ok = __all_sync(0xffffffffu, wait_for(&s.s_full[t], e & 1, a.status, abort_flag));
          if (!ok) break;
          tc::tc_fence_after();
          float z[128];
          tc::tmem_ld64(s_at, z);
          tc::tmem_ld64(s_at + 64, z + 64);
          const auto& sc = s.scales[(n0 + i) & 3];
          if constexpr (kFp8) {          // logits in log2 units plus log2 of the value's scale
#pragma unroll
            for (int c = 0; c < 128; c += 4) {
              const float4 k = *reinterpret_cast<const float4*>(&sc[0][c]), v = *reinterpret_cast<const float4*>(&sc[1][c]);
              const float2 lo = fma2(make_float2(z[c], z[c + 1]), make_float2(k.x, k.y), make_float2(v.x, v.y));
              const float2 hi = fma2(make_float2(z[c + 2], z[c + 3]), make_float2(k.z, k.w), make_float2(v.z, v.w));
              z[c] = lo.x; z[c + 1] = lo.y; z[c + 2] = hi.x; z[c + 3] = hi.y;
            }
          }
          const int j0 = un.tr.at(pc.tile + i) * kKeys;
          const bool gone = s.missing[(n0 + i) & 3] != 0;
          if (gone || !all_visible(a, un.m_lo, un.m_hi, j0, kKeys)) {
            // columns up to hi, and of those the ones behind lo or before sk; a warp whose rows see all skips each side
            const int hi = gone ? -1 : m - j0, lo = a.window ? m - a.window - j0 : -1, sk = a.window ? a.sinks - j0 : 0;
            if (__any_sync(0xffffffffu, hi < kKeys - 1)) {
#pragma unroll
              for (int c = 0; c < 128; ++c) z[c] = c <= hi ? z[c] : -INFINITY;
            }
            if (__any_sync(0xffffffffu, lo >= 0)) {
#pragma unroll
              for (int c = 0; c < 128; ++c) z[c] = c > lo || c < sk ? z[c] : -INFINITY;
            }
          }
          float mx[4] = {z[0], z[1], z[2], z[3]};
#pragma unroll
          for (int c = 4; c < 124; c += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k] = max3(mx[k], z[c + k], z[c + k + 4]);
          top = fmaxf(top, max3(max3(mx[0], mx[1], mx[2]), mx[3], fmaxf(max3(z[124], z[125], z[126]), z[127])) * (kFp8 ? 1.f : f));
          const bool raise = top > -INFINITY && (!any || top > ref + (kFp8 ? kRaiseFp8 : kRaise));
          if (__any_sync(0xffffffffu, raise && any)) {   // the step before has left the accumulator: its MMAs precede S
            const float w = raise && any ? exp2f(ref - top) : 1.f;
            l *= w;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float o[32];
              tmem_ld32(o_at + c, o);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] *= w;
              tmem_st32(o_at + c, reinterpret_cast<const uint32_t*>(o));
            }
            tmem_wait_st();
          }
          if (raise) {
            ref = top;
            any = true;
          }
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          const float2 f2 = make_float2(f, f), r2 = kFp8 ? make_float2(kShiftFp8 - ref, kShiftFp8 - ref) : make_float2(-ref, -ref);
#pragma unroll
          for (int h = 0; h < 2; ++h) {          // the first 64 keys' product runs while the other 64 are exponentiated
            uint32_t pk[32];
#pragma unroll
            for (int c = 0; c < 64; c += 2) {
              const float2 x2 = make_float2(z[64 * h + c], z[64 * h + c + 1]);
              float2 y = kFp8 ? add2(x2, r2) : fma2(x2, f2, r2);
              y.x = exp2f(y.x);
              y.y = exp2f(y.y);
              if (kFp8) {
                sum[(c >> 1) & 1] = fma2(y, *reinterpret_cast<const float2*>(&sc[2][64 * h + c]), sum[(c >> 1) & 1]);
                pk[c >> 1] = pack_f16(y.x, y.y);
              } else {
                sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], y);
                pk[c >> 1] = pack_bf16(y.x, y.y);
              }
            }
            tmem_st32(s_at + 32 * h, pk);
            tmem_wait_st();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&s.p_full[t][h]);
          }
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        }
        // ---- the output, or the piece for the join ----
        if (ok) ok = __all_sync(0xffffffffu, wait_for(&s.o_full[t], g & 1, a.status, abort_flag));
        ++g;
        if (ok) {
          tc::tc_fence_after();
          const bool begins = pc.tile == 0, whole = begins && pc.tile + count == un.tr.tiles;
          const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
          const int64_t at = row_of(a, un, pc.hk, min(row, un.rows - 1));
          const int64_t slot = int64_t(blockIdx.x) * 2 + (begins ? 1 : 0), part = slot * kUnit + row;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            tmem_ld32(o_at + c, o);
            if (row < un.rows && whole) {
#pragma unroll
              for (int k = 0; k < 32; k += 8)
                *reinterpret_cast<uint4*>(a.out + at * D + c + k) =
                    make_uint4(pack_bf16(o[k] * inv, o[k + 1] * inv), pack_bf16(o[k + 2] * inv, o[k + 3] * inv),
                               pack_bf16(o[k + 4] * inv, o[k + 5] * inv), pack_bf16(o[k + 6] * inv, o[k + 7] * inv));
            } else if (row < un.rows) {
#pragma unroll
              for (int k = 0; k < 32; k += 4)      // [slot][dim / 4][row][4]: a warp's rows side by side
                *reinterpret_cast<float4*>(p.part_o + (slot * (D / 4) + (c + k) / 4) * (kUnit * 4) + row * 4) =
                    make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
            }
            __syncwarp();
          }
          if (row < un.rows) {
            if (whole) {
              if (a.lse) a.lse[at] = any ? (ref - (kFp8 ? kShiftFp8 : 0.f) + log2f(l)) * 0.6931471805599453f : l == 0.f ? -INFINITY : l;
            } else {       // a piece without a key leaves nothing; one whose logits are all NaN is passed on
              p.part_ml[part * 2] = any || l != 0.f ? ref - (kFp8 ? kShiftFp8 : 0.f) : -INFINITY;
              p.part_ml[part * 2 + 1] = l;
            }
          }
          tc::tc_fence_before();       // O and Q are free for the next segment (announced by its q_full)
        }
      }
      n0 += count;
      x += count;
    }
  } else if (warp == 8) {
    // ---- the MMA issuer: tile 0's products, then tile 1's, so that one tile's run while the other is
    // in its softmax (with an issuer per tile the two ran in step: 4100 clocks a step instead of 3760) ----
    if (lane == 0) {
      const uint32_t idesc_s = tc::make_idesc(1, 1, kRows, kKeys);
      const uint32_t idesc_o = tc::make_idesc(kFp8 ? 0 : 1, kFp8 ? 0 : 1, kRows, D) | (1u << 16);       // f16 or bf16; B is MN-major
      auto scores = [&](int t, int n) {
        const uint32_t st = tmem + 128 * t, qa = q0 + t * kTileBytes, kb = k0 + (n & 1) * kTileBytes;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc::mma_f16(st, tc::desc_sw128(qa + (k >> 2) * (128 * 128)) + 2 * (k & 3),
                      tc::desc_sw128(kb + (k >> 2) * (128 * 128)) + 2 * (k & 3), idesc_s, k > 0);
        tc::mma_commit(&s.s_full[t]);
      };
      auto wait_keys = [&](int n) { return wait_for(&s.k_full[n & 1], (n >> 1) & 1, a.status, abort_flag); };
      auto wait_values = [&](int n) { return wait_for(&s.v_full[n & 1], (n >> 1) & 1, a.status, abort_flag); };
      bool ok = true;
      int n = 0, e[2] = {0, 0}, g[2] = {0, 0};
      for (int64_t x = x0; x < x1 && ok;) {
        Unit<kKeys> un;
        const auto pc = line.locate(x, &un);
        const int count = int(min(int64_t(un.tr.tiles - pc.tile), x1 - x));
        x += count;
        const int tiles = un.rows > kRows ? 2 : 1;
        ok = wait_keys(n);
        for (int t = 0; t < tiles && ok; ++t) {
          ok = wait_for(&s.q_full[t], g[t] & 1, a.status, abort_flag);
          ++g[t];
          if (!ok) break;
          tc::fence_proxy_async();     // the copying threads' writes, seen through the barrier, -> the tensor cores' reads
          tc::tc_fence_after();
          scores(t, n);
        }
        tc::mma_commit(&s.k_free[n & 1]);
        for (int i = 0; i < count && ok; ++i, ++n) {
          // the copies are waited for ahead of P, so that nothing but P separates the products
          const bool more = i + 1 < count;
          ok = wait_values(n) && (!more || wait_keys(n + 1));
          tc::fence_proxy_async();
          const uint32_t vb = v0 + (n & 1) * kTileBytes;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t >= tiles) break;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              ok = ok && wait_for(&s.p_full[t][h], e[t] & 1, a.status, abort_flag);
              if (!ok) break;
              tc::tc_fence_after();
#pragma unroll
              for (int k = 4 * h; k < 4 * h + 4; ++k)
                mma_ts(tmem + 256 + 128 * t, tmem + 128 * t + 8 * k, desc_mn(vb + k * 16 * 128, 128 * 128), idesc_o, i > 0 || k > 0);
            }
            if (!ok) break;
            ++e[t];
            if (more) scores(t, n + 1);
            else tc::mma_commit(&s.o_full[t]);
          }
          if (!ok) break;
          if (more) tc::mma_commit(&s.k_free[(n + 1) & 1]);
          tc::mma_commit(&s.v_free[n & 1]);
        }
      }
      if (!ok) {                      // after a timeout: what was issued ends before TMEM is freed
        tc::mma_commit(&s.drain);
        for (int k = 0; k < (1 << 22) && !tc::mbar_test(&s.drain, 0); ++k) {
        }
      }
    }
    __syncwarp();
  } else if (tid < 9 * 32 + kLoaders) {
    // ---- the copying warps: each step's keys, then its values, as soon as a buffer is free; a
    // buffer's barrier completes when every thread's copies into it have landed ----
    const int lt = tid - 9 * 32;
    bool ok = true;
    int n = 0;
    for (int64_t x = x0; x < x1 && ok;) {
      Unit<kKeys> un;
      const auto pc = line.locate(x, &un);
      const int count = int(min(int64_t(un.tr.tiles - pc.tile), x1 - x));
      x += count;
      auto entry = [&](int i) {      // step i's table entry, read a step ahead of its use
        return i < count ? __ldcg(a.bt + int64_t(un.b) * a.max_blocks + un.tr.at(pc.tile + i) / (kBlockPositions / kKeys)) : -1;
      };
      int32_t next = entry(0);
      for (int i = 0; i < count && ok; ++i, ++n) {
        int32_t page = next;
        next = entry(i + 1);
        if (page < 0 || page >= a.num_blocks) {
          if (lt == 0) report(a.status, V4A_DEV_BAD_BLOCK);
          page = -1;
        }
        const int j0 = un.tr.at(pc.tile + i) * kKeys;
        if (lt == 0) s.missing[n & 3] = page < 0;
        // rows up to hi, and of those the ones behind lo or before sk, are copied; the others are zeros
        const int hi = page < 0 ? -1 : un.m_hi - j0, lo = a.window ? un.m_lo - a.window - j0 : -1, sk = a.window ? a.sinks - j0 : 0;
        constexpr int kRow = kFp8 ? D : 2 * D;
        const uint8_t* block = a.pool + (page < 0 ? 0 : page * a.block_bytes);
        const int at = page < 0 ? 0 : pc.hk * kBlockPositions + j0 % kBlockPositions;       // first row of the step
        if constexpr (kFp8) {
          // codes are loaded ahead of their buffer, converted and stored into it; the step's scales with its keys
          // (a thread has one chunk of every kStep-th row, at the same place of the swizzle)
          constexpr int kPerRow = D / 16, kStep = kLoaders / kPerRow, kPasses = kKeys / kStep;
          static_assert(kStep % 8 == 0 && kLoaders % kPerRow == 0 && kKeys % kStep == 0 && kLoaders >= kKeys, "rows per pass");
          const int r0 = lt / kPerRow, ch = lt % kPerRow;
          if (lt < kKeys) {
            const float* row_scale = reinterpret_cast<const float*>(block + int64_t(2 * a.K) * kBlockPositions * D) + at + lt;
            const bool live = lt <= hi && (lt > lo || lt < sk);
            const float ks = live ? __ldcg(row_scale) : 0.f, vs = live ? __ldcg(row_scale + a.K * kBlockPositions) : 1.f;
            const float l = vs > 0x1p-100f ? log2f(vs) : vs <= 0x1p-100f ? -100.f : vs;
            float* const sc = &s.scales[n & 3][0][lt];
            sc[0] = ks * a.scale_log2;
            sc[kKeys] = l;
            sc[2 * kKeys] = exp2f(-l);
          }
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            const uint8_t* src = block + (int64_t(half * a.K) * kBlockPositions + at) * D + lt * 16;
            uint4 raw[kPasses];
#pragma unroll
            for (int k = 0; k < kPasses; ++k) {
              const int r = r0 + k * kStep;
              raw[k] = make_uint4(0, 0, 0, 0);
              if (r <= hi && (r > lo || r < sk)) raw[k] = __ldcg(reinterpret_cast<const uint4*>(src + k * (kStep * D)));
            }
            ok = wait_for(half ? &s.v_free[n & 1] : &s.k_free[n & 1], ((n >> 1) & 1) ^ 1, a.status, abort_flag);
            if (!ok) break;
            const uint32_t dst = (half ? v0 : k0) + (n & 1) * kTileBytes;
            const uint32_t even = dst + chunk_at(r0, 2 * ch), odd = dst + chunk_at(r0, 2 * ch + 1);
#pragma unroll
            for (int k = 0; k < kPasses; ++k) {
              st_shared16(even + k * (kStep * 128), half ? f16_of(raw[k].x) : bf16_of(raw[k].x), half ? f16_of(raw[k].y) : bf16_of(raw[k].y));
              st_shared16(odd + k * (kStep * 128), half ? f16_of(raw[k].z) : bf16_of(raw[k].z), half ? f16_of(raw[k].w) : bf16_of(raw[k].w));
            }
            tc::fence_proxy_async();
            tc::mbar_arrive(half ? &s.v_full[n & 1] : &s.k_full[n & 1]);
          }
        } else {
          const bool whole = hi >= kKeys - 1 && lo < 0;
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            ok = wait_for(half ? &s.v_free[n & 1] : &s.k_free[n & 1], ((n >> 1) & 1) ^ 1, a.status, abort_flag);
            if (!ok) break;
            // the copies' own arrivals release no plain store: s.missing has one of its own
            if (half == 0 && lt == 0) tc::mbar_arrive(&s.k_full[n & 1]);
            const uint8_t* src = block + (int64_t(half * a.K) * kBlockPositions + at) * kRow;
            const uint32_t dst = (half ? v0 : k0) + (n & 1) * kTileBytes;
            // thread lt: chunk lt % (dim / 8) of rows lt / (dim / 8) + k * (96 / (dim / 8))
            constexpr int kChunks = kKeys * (D / 8), kPasses = (kChunks + kLoaders - 1) / kLoaders;
            if (whole) {
#pragma unroll
              for (int k = 0; k < kPasses; ++k) {
                const int c = lt + k * kLoaders;
                if (c < kChunks) copy16(dst + chunk_at(c / (D / 8), c % (D / 8)), src + c * 16, true);
              }
            } else {
#pragma unroll
              for (int k = 0; k < kPasses; ++k) {
                const int c = lt + k * kLoaders, r = c / (D / 8);
                const bool live = r <= hi && (r > lo || r < sk);
                if (c < kChunks) copy16(dst + chunk_at(r, c % (D / 8)), live ? src + c * 16 : a.pool, live);
              }
            }
            arrive_copies(half ? &s.v_full[n & 1] : &s.k_full[n & 1]);
          }
        }
      }
    }
    tc::cp_async_wait_all();
  }
  __syncthreads();
  tc::tc_fence_after();
  if (warp == 0) tc::tmem_dealloc(tmem, 512);
  if (p.split && tid == 0) {          // at most the last unit goes on in the next CTAs
    Unit<kKeys> un;
    const auto pc = line.locate(x1 - 1, &un);
    // (its first tile has to lie in the range, its last one behind it)
    const bool tail = pc.tile + 1 < un.tr.tiles && x1 - 1 - pc.tile >= x0;
    p.join[blockIdx.x] = tail ? line.describe(pc, un) : JoinDesc{};
  }
  if (p.late) pdl_wait();
  pdl_trigger();
}

// The split of the registers adds up only with those that the kernel was to be built with: setmaxnreg would wait
// for ever with fewer.  (The build's tests read them from the compiler; this is what a library built otherwise meets.)
template <int D, bool kFp8>
bool ready() {
  static std::atomic<uint64_t> done{0};
  return once_per_device(&done, [] {
    auto kern = dense_prefill_kernel<D, kFp8>;
    cudaFuncAttributes attr;
    return cudaFuncGetAttributes(&attr, kern) == cudaSuccess && attr.numRegs == Roles<kFp8>::kLaunchRegs && raise_smem(kern, 227 * 1024);
  });
}

template <int D, bool kFp8>
int launch(const DenseAttnDev& d, const SplitDev& p, cudaStream_t stream) {
  // at least 116 KB: no two CTAs that allocate TMEM share an SM
  size_t bytes = 1024 + 6 * 128 * D * 2 + sizeof(PreSmem) + split_smem(p.split, p.U);
  if (bytes < 116 * 1024) bytes = 116 * 1024;
  static_assert(1024 + 6 * 128 * D * 2 + sizeof(PreSmem) + split_smem(1, kMaxSplitUnits) <= 227 * 1024, "shared memory of a CTA");
  auto kern = dense_prefill_kernel<D, kFp8>;
  const int64_t grid = p.split ? p.grid : int64_t(p.U) * d.K;
  const cudaError_t e = launch_pdl(kern, dim3(unsigned(grid)), dim3(Roles<kFp8>::kThreads), bytes, stream, d, p);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? V4A_OK : V4A_ERR_CUDA;
}

}  // namespace

bool dense_prefill_takes(const v4a_dense_attn_args* a) {
  const int64_t rows = int64_t(a->max_new_per_seq) * (a->num_heads / a->kv.num_kv_heads);
  return rows > few_rows(a->kv.dim, a->kv.format);
}

size_t dense_prefill_workspace(const v4a_dense_attn_args* a) {
  if (a->kv.format == V4A_KV_FP8_GROUP) return stream_workspace(a->kv.dim);
  return split_workspace(a->kv.dim > 128 ? kWideUnit : kUnit, a->kv.dim, kSms);
}

int dense_prefill_plan(const v4a_dense_attn_args* a, const DenseAttnDev& d, int rows_from, void* ws, SplitDev* out) {
  if (a->kv.format == V4A_KV_FP8_GROUP) return stream_plan(d, a->kv.dim, rows_from, int64_t(d.max_blocks) * kBlockPositions, true, ws, out);
  const bool wide = a->kv.dim > 128;
  const int unit = wide ? kWideUnit : kUnit;
  SplitDev p{};
  p.RG = int((int64_t(a->max_new_per_seq) * d.G + unit - 1) / unit);
  p.rows_from = rows_from;
  p.rows_to = INT32_MAX;
  if (rows_from > 0) p.RG = std::max(p.RG, 2);      // sequences of the other launch are not units
  const int64_t units = units_bound(d, rows_from, p.RG, unit);
  if (units > INT32_MAX || units * d.K > INT32_MAX) return V4A_ERR_UNSUPPORTED;
  p.U = int(units);
  // Under a window the units are about equally long, and one CTA each saves the cut units' pieces and their
  // join, unless the last wave of CTAs is so empty that more than nine steps of 128 keys go to waste on the
  // average SM (window 1024, 32 + 8 heads of 128: 6000 tokens 146 us unsplit, 169 split; 2048 tokens 58 and 71;
  // 1500 tokens, 1.2 waves, 57 both; 2 KV heads, 5000 tokens, 1.03 waves: 57 and 51).
  const int64_t ctas = int64_t(p.U) * d.K, idle = (ctas + kSms - 1) / kSms * kSms - ctas;
  p.split = std::max(p.U, d.B) <= kMaxSplitUnits && (d.window == 0 || idle * (d.window / 128 + 5) > 9 * kSms);
  split_carve(&p, ws, unit, a->kv.dim, kSms, wide ? kWideUnitCost : kUnitCost);
  *out = p;
  return V4A_OK;
}

bool dense_prefill_ready(const v4a_dense_attn_args* a, const DenseAttnDev& d) {
  if (a->kv.format == V4A_KV_FP8_GROUP) return dense_group_ready(a->kv.dim, d);
  const bool fp8 = a->kv.format == V4A_KV_FP8_TOKEN;
  if (a->kv.dim > 128) return dense_prefill_wide_ready(a->kv.dim, fp8);
  if (fp8) return a->kv.dim == 64 ? ready<64, true>() : ready<128, true>();
  return a->kv.dim == 64 ? ready<64, false>() : ready<128, false>();
}

int dense_prefill(const v4a_dense_attn_args* a, const DenseAttnDev& d, const SplitDev& p, cudaStream_t stream) {
  if (a->kv.format == V4A_KV_FP8_GROUP) return dense_group(a->kv.dim, d, p, stream);
  const bool wide = a->kv.dim > 128, fp8 = a->kv.format == V4A_KV_FP8_TOKEN;
  if (wide) return dense_prefill_wide(a->kv.dim, fp8, d, p, stream);
  if (fp8) return a->kv.dim == 64 ? launch<64, true>(d, p, stream) : launch<128, true>(d, p, stream);
  return a->kv.dim == 64 ? launch<64, false>(d, p, stream) : launch<128, false>(d, p, stream);
}

}  // namespace v4a
