// Attention of chunks over the dense paged cache on the tensor cores for heads
// of 192 and 256 dims (v4a_dense_attn with many query rows per KV head).
//
// Mathematics: as dense_prefill.cu.  An output accumulator of 128 rows takes up
// to 256 of the 512 TMEM columns here, so a CTA has one tile of rows, and what
// keeps the tensor cores busy during a softmax is the step before it and the
// step behind it: the scores have two buffers, and the products are issued as
// S(0), S(1), O += P(0) V(0), S(2), O += P(1) V(1), S(3), ...
//
//   S(n) = Q K(n)^T     M = 128, N = 64 keys, K = dim   TMEM columns [256 + 64 (n % 2), +64)
//   P(n) = 2^{S f - m} in bf16 (fp8: f16), over S(n)'s columns
//   O += P(n) V(n)      M = 128, N = dim, K = 64 keys   [0, dim)
//
// S(n) is issued behind P(n - 2)'s product and the tensor cores take one
// thread's products in order, so a buffer is free when it is written; the
// accumulator may only be rescaled once O += P(n - 1) V(n - 1) is done, which
// is the event that frees V(n - 1)'s buffer.
//
// Roles: warps 0-3 the softmax (a thread owns a row), 4 issues the MMAs, the
// others copy keys and values.  Steps of 64 keys: two buffers each of keys and values of 256 dims
// are 128 KB beside the 64 KB of queries.
//
// Bound: the tensor cores (4 dim flops per visible pair); a step's keys and
// values (4 dim bytes a key from the L2) serve 128 rows only.  Measured, 2048
// tokens over 10240 positions, 16 + 4 heads: dim 256 bf16 320 us (966 TFLOP/s;
// the form for few rows, which had them before, re-reads the cache per 8 rows),
// fp8 505 us (613: the conversions); dim 192 bf16 274 us (847), fp8 467 (497).
#include "dense_prefill_common.cuh"

namespace v4a {
namespace {

constexpr int kRows = kWideUnit;     // rows of a unit (MMA M)
constexpr int kKeys = 64;            // keys per step
constexpr int kMinSteps = 8;         // steps a CTA of an even split has at least

template <int D, bool kFp8>
struct Wide {
  // Whole rows a pass: bf16 four rows, fp8 (whose codes the threads convert) sixteen: eight took 610 us
  // instead of 519 for 2k tokens over 10k, 16 + 4 heads of 256.
  static constexpr int kLoaders = kFp8 ? D : D / 2;
  static constexpr int kStep = kLoaders / (D / 16);    // fp8: rows a pass
  static constexpr int kThreads = 5 * 32 + kLoaders;
  static constexpr int kQBytes = kRows * D * 2, kStepBytes = kKeys * D * 2;
};

struct WideSmem {
  uint64_t q_full, k_full[2], v_full[2], k_free[2], v_free[2], s_full[2], p_full[2], o_full, drain;
  int64_t scan[16];
  uint32_t tmem_base;
  int abort_flag;
  int missing[4];                    // step n's page is missing: [n % 4]
  // fp8, step n's keys: softmax scale x log2(e) x key scale; log2 of the value scale; its inverse
  alignas(16) float scales[4][3][kKeys];
};

// Byte offset of 16-byte chunk `ch` of row r in an operand of [dim / 64][kN rows][128 bytes], swizzled.
template <int kN>
__device__ __forceinline__ uint32_t chunk_at(int r, int ch) {
  return uint32_t((ch >> 3) * (kN * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(Wide<D, kFp8>::kThreads, 1) dense_prefill_wide_kernel(const DenseAttnDev a, const SplitDev p) {
  using W = Wide<D, kFp8>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t q0 = tc::smem_u32(base), k0 = q0 + W::kQBytes, v0 = k0 + 2 * W::kStepBytes;
  WideSmem& s = *reinterpret_cast<WideSmem*>(base + W::kQBytes + 4 * W::kStepBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &s.abort_flag;

  if (!p.late) pdl_wait();
  Line<kRows, kKeys, W::kThreads> line(a, p, &s + 1);
  if (!line.init(s.scan, base, kMinSteps)) {
    if (p.late) pdl_wait();
    return;
  }
  const int64_t x0 = line.x0, x1 = line.x1;

  if (tid == 0) {
    tc::mbar_init(&s.q_full, kRows);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&s.k_full[i], W::kLoaders + (kFp8 ? 0 : 1));
      tc::mbar_init(&s.v_full[i], W::kLoaders);
      tc::mbar_init(&s.k_free[i], 1);
      tc::mbar_init(&s.v_free[i], 1);
      tc::mbar_init(&s.s_full[i], 1);
      tc::mbar_init(&s.p_full[i], 4);
    }
    tc::mbar_init(&s.o_full, 1);
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
  // itself.  Counters: n = steps of the CTA, g = segments.
  if (warp < 4) {
    // ---- queries, softmax and output ----
    const int row = tid;
    const uint32_t lanes = uint32_t(warp * 32) << 16;
    const uint32_t o_at = tmem + lanes;
    const float f = a.scale_log2;
    bool ok = true;
    int n = 0, g = 0;
    for (int64_t x = x0; x < x1 && ok;) {
      Unit<kKeys> un;
      const auto pc = line.locate(x, &un);
      const int count = int(min(int64_t(un.tr.tiles - pc.tile), x1 - x));
      x += count;
      // Q rows behind the last are zeros
#pragma unroll 4
      for (int c = row; c < kRows * (D / 8); c += kRows) {
        const int qr = c / (D / 8), ch = c % (D / 8);
        const uint16_t* q = a.q + row_of(a, un, pc.hk, min(qr, un.rows - 1)) * D;
        copy16(q0 + chunk_at<kRows>(qr, ch), q + ch * 8, qr < un.rows);
      }
      tc::cp_async_wait_all();
      tc::fence_proxy_async();
      tc::mbar_arrive(&s.q_full);
      const int m = un.m_lo + (un.row0 % a.G + min(row, un.rows - 1)) / a.G;
      float top = -INFINITY, ref = 0.f, l = 0.f;       // largest logit, the maximum in use, the sum against it
      bool any = false;                                // `ref` is set (a key has been seen)
      for (int i = 0; i < count; ++i, ++n) {
        const uint32_t s_at = tmem + 256 + 64 * (n & 1) + lanes;
        ok = __all_sync(0xffffffffu, wait_for(&s.s_full[n & 1], (n >> 1) & 1, a.status, abort_flag));
        if (!ok) break;
        tc::tc_fence_after();
        float z[kKeys];
        tc::tmem_ld64(s_at, z);
        const auto& sc = s.scales[n & 3];
        if constexpr (kFp8) {          // logits in log2 units plus log2 of the value's scale
#pragma unroll
          for (int c = 0; c < kKeys; c += 4) {
            const float4 k = *reinterpret_cast<const float4*>(&sc[0][c]), v = *reinterpret_cast<const float4*>(&sc[1][c]);
            const float2 lo = fma2(make_float2(z[c], z[c + 1]), make_float2(k.x, k.y), make_float2(v.x, v.y));
            const float2 hi = fma2(make_float2(z[c + 2], z[c + 3]), make_float2(k.z, k.w), make_float2(v.z, v.w));
            z[c] = lo.x; z[c + 1] = lo.y; z[c + 2] = hi.x; z[c + 3] = hi.y;
          }
        }
        const int j0 = un.tr.at(pc.tile + i) * kKeys;
        const bool gone = s.missing[n & 3] != 0;
        if (gone || !all_visible(a, un.m_lo, un.m_hi, j0, kKeys)) {
          // columns up to hi, and of those the ones behind lo or before sk
          const int hi = gone ? -1 : m - j0, lo = a.window ? m - a.window - j0 : -1, sk = a.window ? a.sinks - j0 : 0;
#pragma unroll
          for (int c = 0; c < kKeys; ++c) z[c] = c <= hi && (c > lo || c < sk) ? z[c] : -INFINITY;
        }
        float mx[4] = {z[0], z[1], z[2], z[3]};
#pragma unroll
        for (int c = 4; c < kKeys - 4; c += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k) mx[k] = max3(mx[k], z[c + k], z[c + k + 4]);
        top = fmaxf(top, max3(max3(mx[0], mx[1], mx[2]), mx[3],
                              fmaxf(max3(z[kKeys - 4], z[kKeys - 3], z[kKeys - 2]), z[kKeys - 1])) * (kFp8 ? 1.f : f));
        const bool raise = top > -INFINITY && (!any || top > ref + (kFp8 ? kRaiseFp8 : kRaise));
        if (__any_sync(0xffffffffu, raise && any)) {       // (so i > 0)
          ok = __all_sync(0xffffffffu, wait_for(&s.v_free[(n - 1) & 1], ((n - 1) >> 1) & 1, a.status, abort_flag));
          if (!ok) break;
          tc::tc_fence_after();
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
        }
        if (raise) {
          ref = top;
          any = true;
        }
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const float2 f2 = make_float2(f, f), r2 = kFp8 ? make_float2(kShiftFp8 - ref, kShiftFp8 - ref) : make_float2(-ref, -ref);
        uint32_t pk[kKeys / 2];
#pragma unroll
        for (int c = 0; c < kKeys; c += 2) {
          const float2 x2 = make_float2(z[c], z[c + 1]);
          float2 y = kFp8 ? add2(x2, r2) : fma2(x2, f2, r2);
          y.x = exp2f(y.x);
          y.y = exp2f(y.y);
          if (kFp8) {
            sum[(c >> 1) & 1] = fma2(y, *reinterpret_cast<const float2*>(&sc[2][c]), sum[(c >> 1) & 1]);
            pk[c >> 1] = pack_f16(y.x, y.y);
          } else {
            sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], y);
            pk[c >> 1] = pack_bf16(y.x, y.y);
          }
        }
        tmem_st32(s_at, pk);
        tmem_wait_st();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&s.p_full[n & 1]);
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      }
      // ---- the output, or the piece for the join ----
      if (ok) ok = __all_sync(0xffffffffu, wait_for(&s.o_full, g & 1, a.status, abort_flag));
      ++g;
      if (ok) {
        tc::tc_fence_after();
        const bool begins = pc.tile == 0, whole = begins && pc.tile + count == un.tr.tiles;
        const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
        const int64_t at = row_of(a, un, pc.hk, min(row, un.rows - 1));
        const int64_t slot = int64_t(blockIdx.x) * 2 + (begins ? 1 : 0), part = slot * kRows + row;
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
              *reinterpret_cast<float4*>(p.part_o + (slot * (D / 4) + (c + k) / 4) * (kRows * 4) + row * 4) =
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
  } else if (warp == 4) {
    // ---- the MMA issuer ----
    if (lane == 0) {
      const uint32_t idesc_s = tc::make_idesc(1, 1, kRows, kKeys);
      const uint32_t idesc_o = tc::make_idesc(kFp8 ? 0 : 1, kFp8 ? 0 : 1, kRows, D) | (1u << 16);       // f16 or bf16; B is MN-major
      auto scores = [&](int n) {
        if (!wait_for(&s.k_full[n & 1], (n >> 1) & 1, a.status, abort_flag)) return false;
        tc::fence_proxy_async();     // the copying threads' writes, seen through the barrier, -> the tensor cores' reads
        tc::tc_fence_after();
        const uint32_t st = tmem + 256 + 64 * (n & 1), kb = k0 + (n & 1) * W::kStepBytes;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc::mma_f16(st, tc::desc_sw128(q0 + (k >> 2) * (kRows * 128)) + 2 * (k & 3),
                      tc::desc_sw128(kb + (k >> 2) * (kKeys * 128)) + 2 * (k & 3), idesc_s, k > 0);
        tc::mma_commit(&s.s_full[n & 1]);
        tc::mma_commit(&s.k_free[n & 1]);
        return true;
      };
      bool ok = true;
      int n = 0, g = 0;
      for (int64_t x = x0; x < x1 && ok;) {
        Unit<kKeys> un;
        const auto pc = line.locate(x, &un);
        const int count = int(min(int64_t(un.tr.tiles - pc.tile), x1 - x));
        x += count;
        ok = wait_for(&s.q_full, g & 1, a.status, abort_flag);
        ++g;
        ok = ok && scores(n) && (count < 2 || scores(n + 1));
        for (int i = 0; i < count && ok; ++i, ++n) {
          ok = wait_for(&s.v_full[n & 1], (n >> 1) & 1, a.status, abort_flag) &&
               wait_for(&s.p_full[n & 1], (n >> 1) & 1, a.status, abort_flag);
          if (!ok) break;
          tc::fence_proxy_async();
          tc::tc_fence_after();
          const uint32_t vb = v0 + (n & 1) * W::kStepBytes;
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            mma_ts(tmem, tmem + 256 + 64 * (n & 1) + 8 * k, desc_mn(vb + k * 16 * 128, kKeys * 128), idesc_o, i > 0 || k > 0);
          tc::mma_commit(&s.v_free[n & 1]);
          if (i + 1 == count) tc::mma_commit(&s.o_full);
          if (i + 2 < count) ok = scores(n + 2);
        }
      }
      if (!ok) {                      // after a timeout: what was issued ends before TMEM is freed
        tc::mma_commit(&s.drain);
        for (int k = 0; k < (1 << 22) && !tc::mbar_test(&s.drain, 0); ++k) {
        }
      }
    }
    __syncwarp();
  } else {
    // ---- the copying warps: each step's keys, then its values, as soon as a buffer is free; a
    // buffer's barrier completes when every thread's copies into it have landed ----
    const int lt = tid - 5 * 32;
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
        // rows up to hi, and of those the ones behind lo or before sk, are copied; the others are zeros
        const int hi = page < 0 ? -1 : un.m_hi - j0, lo = a.window ? un.m_lo - a.window - j0 : -1, sk = a.window ? a.sinks - j0 : 0;
        constexpr int kRow = kFp8 ? D : 2 * D;
        const uint8_t* block = a.pool + (page < 0 ? 0 : page * a.block_bytes);
        const int at = page < 0 ? 0 : pc.hk * kBlockPositions + j0 % kBlockPositions;       // first row of the step
        if (lt == 0) s.missing[n & 3] = page < 0;
        if (kFp8 && lt < kKeys) {
          const float* row_scale = reinterpret_cast<const float*>(block + int64_t(2 * a.K) * kBlockPositions * D) + at + lt;
          const bool live = lt <= hi && (lt > lo || lt < sk);
          const float ks = live ? __ldcg(row_scale) : 0.f, vs = live ? __ldcg(row_scale + a.K * kBlockPositions) : 1.f;
          const float l = vs > 0x1p-100f ? log2f(vs) : vs <= 0x1p-100f ? -100.f : vs;
          s.scales[n & 3][0][lt] = ks * a.scale_log2;
          s.scales[n & 3][1][lt] = l;
          s.scales[n & 3][2][lt] = exp2f(-l);
        }
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          const uint8_t* src = block + (int64_t(half * a.K) * kBlockPositions + at) * kRow + lt * 16;
          const uint32_t dst = (half ? v0 : k0) + (n & 1) * W::kStepBytes;
          uint64_t* const free = half ? &s.v_free[n & 1] : &s.k_free[n & 1];
          uint64_t* const full = half ? &s.v_full[n & 1] : &s.k_full[n & 1];
          if constexpr (kFp8) {
            // codes are loaded ahead of their buffer, converted and stored into it
            const int r0 = lt / (D / 16), ch = lt % (D / 16);
            uint4 raw[kKeys / W::kStep];
#pragma unroll
            for (int k = 0; k < kKeys / W::kStep; ++k) {
              const int r = r0 + W::kStep * k;
              raw[k] = make_uint4(0, 0, 0, 0);
              if (r <= hi && (r > lo || r < sk)) raw[k] = __ldcg(reinterpret_cast<const uint4*>(src + k * (W::kStep * D)));
            }
            ok = wait_for(free, ((n >> 1) & 1) ^ 1, a.status, abort_flag);
            if (!ok) break;
            const uint32_t even = dst + chunk_at<kKeys>(r0, 2 * ch), odd = dst + chunk_at<kKeys>(r0, 2 * ch + 1);
#pragma unroll
            for (int k = 0; k < kKeys / W::kStep; ++k) {
              st_shared16(even + k * (W::kStep * 128), half ? f16_of(raw[k].x) : bf16_of(raw[k].x), half ? f16_of(raw[k].y) : bf16_of(raw[k].y));
              st_shared16(odd + k * (W::kStep * 128), half ? f16_of(raw[k].z) : bf16_of(raw[k].z), half ? f16_of(raw[k].w) : bf16_of(raw[k].w));
            }
            tc::fence_proxy_async();
            tc::mbar_arrive(full);
          } else {
            ok = wait_for(free, ((n >> 1) & 1) ^ 1, a.status, abort_flag);
            if (!ok) break;
            // the copies' own arrivals release no plain store: s.missing has one of its own
            if (half == 0 && lt == 0) tc::mbar_arrive(full);
            const int r0 = lt / (D / 8), ch = lt % (D / 8);      // four rows a pass
#pragma unroll
            for (int k = 0; k < kKeys / 4; ++k) {
              const int r = r0 + 4 * k;
              const bool live = r <= hi && (r > lo || r < sk);
              copy16(dst + chunk_at<kKeys>(r, ch), live ? src + k * (4 * kRow) : a.pool, live);
            }
            arrive_copies(full);
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

template <int D, bool kFp8>
bool ready() {
  static std::atomic<uint64_t> done{0};
  return once_per_device(&done, [] { return raise_smem(dense_prefill_wide_kernel<D, kFp8>, 227 * 1024); });
}

template <int D, bool kFp8>
int launch(const DenseAttnDev& d, const SplitDev& p, cudaStream_t stream) {
  // more than 116 KB: no two CTAs that allocate TMEM share an SM
  const size_t bytes = 1024 + Wide<D, kFp8>::kQBytes + 4 * Wide<D, kFp8>::kStepBytes + sizeof(WideSmem) + split_smem(p.split, p.U);
  static_assert(1024 + Wide<D, kFp8>::kQBytes + 4 * Wide<D, kFp8>::kStepBytes + sizeof(WideSmem) + split_smem(1, kMaxSplitUnits) <= 227 * 1024, "shared memory of a CTA");
  auto kern = dense_prefill_wide_kernel<D, kFp8>;
  const int64_t grid = p.split ? p.grid : int64_t(p.U) * d.K;
  const cudaError_t e = launch_pdl(kern, dim3(unsigned(grid)), dim3(Wide<D, kFp8>::kThreads), bytes, stream, d, p);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? V4A_OK : V4A_ERR_CUDA;
}

}  // namespace

bool dense_prefill_wide_ready(int dim, bool fp8) {
  if (dim == 192) return fp8 ? ready<192, true>() : ready<192, false>();
  return fp8 ? ready<256, true>() : ready<256, false>();
}

int dense_prefill_wide(int dim, bool fp8, const DenseAttnDev& d, const SplitDev& p, cudaStream_t stream) {
  if (dim == 192) return fp8 ? launch<192, true>(d, p, stream) : launch<192, false>(d, p, stream);
  return fp8 ? launch<256, true>(d, p, stream) : launch<256, false>(d, p, stream);
}

}  // namespace v4a
