// Attention of many query rows per KV head on the tensor cores (tcgen05
// kind::f16, accumulators in TMEM), in steps of 64 keys.  Two sources of keys
// and values share it: a paged fp8 cache with a scale per 64 positions
// (dense_group.cu) and packed bf16 rows (prompt_attn.cu).
//
// Mathematics: one pass over the keys with a running maximum and sum per row.
// A CTA has one tile of 128 rows (dim 192, 256) or two (dim 64, 128), rows
// being consecutive (token, head of the group) pairs of one sequence and KV
// head.  The scores of a tile have two buffers of 64 columns, so a tile's
// softmax goes from one step to the next without waiting for its own products:
// the tensor cores work for the other tile and for the step behind it.
//
//   S_t(n) = Q_t K(n)^T     M = 128, N = 64 keys, K = dim    TMEM columns [128 t + 64 (n % 2), +64)
//   P_t(n) = 2^{S f - m}    16 bits, over S_t(n)'s columns
//   O_t += P_t(n) V(n)      M = 128, N = dim, K = 64 keys    [128 tiles + dim t, +dim)
//
// issued as S(0), S(1), O += P(0) V(0), S(2), O += P(1) V(1), S(3), ... for the
// tiles in turn.  One thread's products run in order, so S(n + 2), behind
// P(n)'s product, may take its buffer.  The maximum that P is formed against is
// raised only when a row's logits pass it by 2^kRaise, so the accumulator is
// rescaled a few times per row; it then waits for the product before.
//
// Source: what differs (the arguments, the copying warps, scaled or not).
#pragma once
#include "dense_prefill_common.cuh"

namespace v4a {

constexpr int kStreamKeys = 64;      // keys per step
constexpr int kTileRows = 128;       // rows of a tile (MMA M)
constexpr int kStreamCost = 6;       // steps that a unit's set-up and output take the time of
constexpr int kStreamMinSteps = 8;   // steps a CTA of an even split has at least

template <int D>
struct Stream {
  static constexpr int kTiles = D <= 128 ? 2 : 1;
  static constexpr int kUnit = kTiles * kTileRows;
  static constexpr int kStages = D <= 128 ? 4 : D == 192 ? 3 : 2;      // of keys, and of values
  static constexpr int kQBytes = kTileRows * D * 2;                    // of a tile
  static constexpr int kStepBytes = kStreamKeys * D * 2;               // a step's keys, or its values
  static constexpr int kSoftmax = kTiles * 128;                        // threads
};
constexpr int stream_unit(int dim) { return dim <= 128 ? 256 : 128; }

struct StreamSmem {
  uint64_t q_full[2], s_full[2][2], p_full[2][2], o_done[2][2], k_full[4], k_free[4], v_full[4], v_free[4], drain;
  int64_t scan[16];
  uint32_t tmem_base;
  int abort_flag;
  // step n at [n % 8] (a buffer's step can be six steps ahead of the slowest softmax): its page is missing;
  // softmax scale x log2(e) x key scale, log2 of the value scale, its inverse
  int missing[8];
  alignas(16) float scales[8][4];
};

// Byte offset of 16-byte chunk `ch` of row r in an operand of [dim / 64][kN rows][128 bytes], swizzled.
template <int kN>
__device__ __forceinline__ uint32_t stream_chunk(int r, int ch) {
  return uint32_t((ch >> 3) * (kN * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}

template <int D, class Src>
__global__ void __launch_bounds__(Src::template threads<D>(), 1)
stream_attn_kernel(const __grid_constant__ typename Src::Dev a, const SplitDev p) {
  using W = Stream<D>;
  constexpr int kThreads = Src::template threads<D>(), kLoaders = Src::template loaders<D>(), S = W::kStages;
  constexpr bool kScaled = Src::kScaled;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t q0 = tc::smem_u32(base), k0 = q0 + W::kTiles * W::kQBytes, v0 = k0 + S * W::kStepBytes;
  StreamSmem& s = *reinterpret_cast<StreamSmem*>(base + W::kTiles * W::kQBytes + 2 * S * W::kStepBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &s.abort_flag;

  if (!p.late) pdl_wait();
  Line<W::kUnit, kStreamKeys, kThreads, typename Src::Dev> line(a, p, &s + 1);
  if (!line.init(s.scan, base, kStreamMinSteps)) {
    if (p.late) pdl_wait();
    return;
  }
  const int64_t x0 = line.x0, x1 = line.x1;

  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      tc::mbar_init(&s.q_full[t], kTileRows);
      for (int i = 0; i < 2; ++i) {
        tc::mbar_init(&s.s_full[t][i], 1);
        tc::mbar_init(&s.p_full[t][i], 4);
        tc::mbar_init(&s.o_done[t][i], 1);
      }
    }
    for (int i = 0; i < S; ++i) {
      tc::mbar_init(&s.k_full[i], Src::template arrivals<D>());
      tc::mbar_init(&s.v_full[i], Src::template arrivals<D>());
      tc::mbar_init(&s.k_free[i], 1);
      tc::mbar_init(&s.v_free[i], 1);
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
  const uint32_t tmem = s.tmem_base, tmem_o = tmem + 128 * W::kTiles;

  // Every role walks the CTA's segments (the parts of units in [x0, x1)) by
  // itself.  Counters: n = steps of the CTA, e = steps of a tile, g = its segments.
  if (tid < W::kSoftmax) {
    // ---- a tile's queries, softmax and output ----
    const int t = warp >> 2, r = tid & 127, row = t * kTileRows + r;
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + 128 * t + lanes, o_at = tmem_o + D * t + lanes;
    bool ok = true;
    int n = 0, e = 0;
    // step e's product is in the accumulator (asked behind S(e + 1) or P(e): step e - 2's is, so the phase is the one meant)
    auto done = [&](int e) { return wait_for(&s.o_done[t][e & 1], (e >> 1) & 1, a.status, abort_flag); };
    for (int64_t x = x0; x < x1 && ok;) {
      Unit<kStreamKeys> un;
      const auto pc = line.locate(x, &un);
      const int count = int(min(int64_t(un.tr.tiles - pc.tile), x1 - x));
      x += count;
      if (un.rows <= t * kTileRows) {
        n += count;
        continue;
      }
      // a row's logits in log2 units: its scores times f (fp8: and the key scale)
      const float f = Src::template load_q<D>(a, un, pc.hk, t, r, q0 + t * W::kQBytes);
      tc::fence_proxy_async();
      tc::mbar_arrive(&s.q_full[t]);
      const int m = Src::row_position(a, un, min(row, un.rows - 1));
      float top = -INFINITY, ref = 0.f, l = 0.f;       // largest logit, the maximum in use, the sum against it
      bool any = false;                                // `ref` is set (a key has been seen)
      for (int i = 0; i < count; ++i, ++e, ++n) {
        ok = __all_sync(0xffffffffu, wait_for(&s.s_full[t][e & 1], (e >> 1) & 1, a.status, abort_flag));
        if (!ok) break;
        tc::tc_fence_after();
        float z[kStreamKeys];
        tc::tmem_ld64(s_at + 64 * (e & 1), z);
        float fk = f, lv = 0.f, inv_v = 1.f;
        if constexpr (kScaled) {
          const float4 sc = *reinterpret_cast<const float4*>(s.scales[n & 7]);
          fk = fmaxf(f * sc.x, 0x1p-126f);             // (flushed to zero, it would make NaNs of hidden keys' -inf)
          lv = sc.y;
          inv_v = sc.z;
        }
        const int j0 = un.tr.at(pc.tile + i) * kStreamKeys;
        const bool gone = Src::kPaged && s.missing[n & 7] != 0;
        if (gone || !all_visible(a, un.m_lo, un.m_hi, j0, kStreamKeys)) {
          // columns up to hi, and of those the ones behind lo or before sk; a warp whose rows see all skips each side
          const int hi = gone ? -1 : m - j0, lo = a.window ? m - a.window - j0 : -1, sk = a.window ? a.sinks - j0 : 0;
          if (__any_sync(0xffffffffu, hi < kStreamKeys - 1)) {
#pragma unroll
            for (int c = 0; c < kStreamKeys; ++c) z[c] = c <= hi ? z[c] : -INFINITY;
          }
          if (__any_sync(0xffffffffu, lo >= 0)) {
#pragma unroll
            for (int c = 0; c < kStreamKeys; ++c) z[c] = c > lo || c < sk ? z[c] : -INFINITY;
          }
        }
        float mx[4] = {z[0], z[1], z[2], z[3]};
#pragma unroll
        for (int c = 4; c < kStreamKeys - 4; c += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k) mx[k] = max3(mx[k], z[c + k], z[c + k + 4]);
        top = fmaxf(top, fmaf(max3(max3(mx[0], mx[1], mx[2]), mx[3],
                                   fmaxf(max3(z[kStreamKeys - 4], z[kStreamKeys - 3], z[kStreamKeys - 2]), z[kStreamKeys - 1])), fk, lv));
        const bool raise = top > -INFINITY && (!any || top > ref + (kScaled ? kRaiseFp8 : kRaise));
        if (__any_sync(0xffffffffu, raise && any)) {       // (so i > 0)
          ok = __all_sync(0xffffffffu, done(e - 1));
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
        const float up = kScaled ? lv + kShiftFp8 - ref : -ref;
        const float2 f2 = make_float2(fk, fk), r2 = make_float2(up, up);
        uint32_t pk[kStreamKeys / 2];
#pragma unroll
        for (int c = 0; c < kStreamKeys; c += 2) {
          float2 y = fma2(make_float2(z[c], z[c + 1]), f2, r2);
          y.x = exp2f(y.x);
          y.y = exp2f(y.y);
          sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], y);
          pk[c >> 1] = kScaled ? pack_f16(y.x, y.y) : pack_bf16(y.x, y.y);
        }
        tmem_st32(s_at + 64 * (e & 1), pk);
        tmem_wait_st();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&s.p_full[t][e & 1]);
        l = fmaf((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y), inv_v, l);
      }
      // ---- the output, or the piece for the join ----
      if (ok) ok = __all_sync(0xffffffffu, done(e - 1));
      if (ok) {
        tc::tc_fence_after();
        const bool begins = pc.tile == 0, whole = begins && pc.tile + count == un.tr.tiles;
        const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
        const int64_t at = row_of(a, un, pc.hk, min(row, un.rows - 1));
        const int64_t slot = int64_t(blockIdx.x) * 2 + (begins ? 1 : 0), part = slot * W::kUnit + row;
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
              *reinterpret_cast<float4*>(p.part_o + (slot * (D / 4) + (c + k) / 4) * (W::kUnit * 4) + row * 4) =
                  make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
          }
          __syncwarp();
        }
        if (row < un.rows) {
          if (whole) {
            if (a.lse) a.lse[at] = any ? (ref - (kScaled ? kShiftFp8 : 0.f) + log2f(l)) * 0.6931471805599453f : l == 0.f ? -INFINITY : l;
          } else {       // a piece without a key leaves nothing; one whose logits are all NaN is passed on
            p.part_ml[part * 2] = any || l != 0.f ? ref - (kScaled ? kShiftFp8 : 0.f) : -INFINITY;
            p.part_ml[part * 2 + 1] = l;
          }
        }
        tc::tc_fence_before();       // O and Q are free for the next segment (announced by its q_full)
      }
    }
  } else if (tid < W::kSoftmax + 32) {
    // ---- the MMA issuer ----
    if (lane == 0) {
      constexpr uint32_t kFmt = kScaled ? 0 : 1;       // f16 or bf16
      const uint32_t idesc_s = tc::make_idesc(kFmt, kFmt, kTileRows, kStreamKeys);
      const uint32_t idesc_o = tc::make_idesc(kFmt, kFmt, kTileRows, D) | (1u << 16);       // B is MN-major
      auto scores = [&](int t, int e, int n) {
        const uint32_t st = tmem + 128 * t + 64 * (e & 1), qa = q0 + t * W::kQBytes, kb = k0 + (n % S) * W::kStepBytes;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc::mma_f16(st, tc::desc_sw128(qa + (k >> 2) * (kTileRows * 128)) + 2 * (k & 3),
                      tc::desc_sw128(kb + (k >> 2) * (kStreamKeys * 128)) + 2 * (k & 3), idesc_s, k > 0);
        tc::mma_commit(&s.s_full[t][e & 1]);
      };
      auto wait_keys = [&](int n) { return wait_for(&s.k_full[n % S], (n / S) & 1, a.status, abort_flag); };
      bool ok = true;
      int n = 0, e[2] = {0, 0}, g[2] = {0, 0};
      for (int64_t x = x0; x < x1 && ok;) {
        Unit<kStreamKeys> un;
        const auto pc = line.locate(x, &un);
        const int count = int(min(int64_t(un.tr.tiles - pc.tile), x1 - x));
        x += count;
        const int tiles = W::kTiles == 2 && un.rows > kTileRows ? 2 : 1;
        for (int t = 0; t < tiles && ok; ++t) {
          ok = wait_for(&s.q_full[t], g[t] & 1, a.status, abort_flag);
          ++g[t];
        }
        for (int j = 0; j < min(count, 2) && ok; ++j) {
          ok = wait_keys(n + j);
          if (!ok) break;
          tc::fence_proxy_async();
          tc::tc_fence_after();
          for (int t = 0; t < tiles; ++t) scores(t, e[t] + j, n + j);
          tc::mma_commit(&s.k_free[(n + j) % S]);
        }
        for (int i = 0; i < count && ok; ++i, ++n) {
          // the copies are waited for ahead of P, so that nothing but P separates the products
          const bool more = i + 2 < count;
          ok = wait_for(&s.v_full[n % S], (n / S) & 1, a.status, abort_flag) && (!more || wait_keys(n + 2));
          tc::fence_proxy_async();
          const uint32_t vb = v0 + (n % S) * W::kStepBytes;
#pragma unroll
          for (int t = 0; t < W::kTiles; ++t) {
            if (t >= tiles) break;
            ok = ok && wait_for(&s.p_full[t][e[t] & 1], (e[t] >> 1) & 1, a.status, abort_flag);
            if (!ok) break;
            tc::tc_fence_after();
#pragma unroll
            for (int k = 0; k < kStreamKeys / 16; ++k)
              mma_ts(tmem_o + D * t, tmem + 128 * t + 64 * (e[t] & 1) + 8 * k, desc_mn(vb + k * 16 * 128, kStreamKeys * 128), idesc_o,
                     i > 0 || k > 0);
            tc::mma_commit(&s.o_done[t][e[t] & 1]);
            if (more) scores(t, e[t] + 2, n + 2);
            ++e[t];
          }
          if (!ok) break;
          tc::mma_commit(&s.v_free[n % S]);
          if (more) tc::mma_commit(&s.k_free[(n + 2) % S]);
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
    // ---- the copying warps: one half the keys, the other the values, as soon as a buffer is free ----
    const int lt = tid - W::kSoftmax - 32, half = lt / kLoaders;
    bool ok = true;
    int n = 0;
    for (int64_t x = x0; x < x1 && ok;) {
      Unit<kStreamKeys> un;
      const auto pc = line.locate(x, &un);
      const int count = int(min(int64_t(un.tr.tiles - pc.tile), x1 - x));
      x += count;
      ok = Src::template copy<D>(a, un, pc.hk, pc.tile, count, n, half, lt % kLoaders, base + W::kTiles * W::kQBytes + half * S * W::kStepBytes, s);
      n += count;
    }
  }
  __syncthreads();
  tc::tc_fence_after();
  if (warp == 0) tc::tmem_dealloc(tmem, 512);
  if (p.split && tid == 0) {          // at most the last unit goes on in the next CTAs
    Unit<kStreamKeys> un;
    const auto pc = line.locate(x1 - 1, &un);
    // (its first tile has to lie in the range, its last one behind it)
    const bool tail = pc.tile + 1 < un.tr.tiles && x1 - 1 - pc.tile >= x0;
    p.join[blockIdx.x] = tail ? line.describe(pc, un) : JoinDesc{};
  }
  if (p.late) pdl_wait();
  pdl_trigger();
}

template <int D>
constexpr size_t stream_smem(int split, int U) {
  return 1024 + Stream<D>::kTiles * Stream<D>::kQBytes + 2 * Stream<D>::kStages * Stream<D>::kStepBytes + sizeof(StreamSmem) + split_smem(split, U);
}

template <int D, class Src>
bool stream_ready() {
  static std::atomic<uint64_t> done{0};
  return once_per_device(&done, [] { return raise_smem(stream_attn_kernel<D, Src>, 227 * 1024); });
}

template <int D, class Src>
int stream_launch(const typename Src::Dev& d, const SplitDev& p, cudaStream_t stream) {
  static_assert(stream_smem<D>(1, kMaxSplitUnits) <= 227 * 1024, "shared memory of a CTA");
  static_assert(Stream<D>::kTiles * Stream<D>::kQBytes + 2 * Stream<D>::kStages * Stream<D>::kStepBytes >= int(kMaxSplitUnits * 16), "scratch of the line");
  // at least 116 KB: no two CTAs that allocate TMEM share an SM
  const size_t bytes = std::max(stream_smem<D>(p.split, p.U), size_t(116 * 1024));
  const int64_t grid = p.split ? p.grid : int64_t(p.U) * d.K;
  const cudaError_t e = launch_pdl(stream_attn_kernel<D, Src>, dim3(unsigned(grid)), dim3(Src::template threads<D>()), bytes, stream, d, p);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? V4A_OK : V4A_ERR_CUDA;
}

}  // namespace v4a
