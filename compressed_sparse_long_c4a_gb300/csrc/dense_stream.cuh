// Attention of many query rows per KV head on the tensor cores (tcgen05
// kind::f16, accumulators in TMEM).  Two sources of keys and values share it: a
// paged fp8 cache with a scale per 64 positions (dense_group.cu) and packed bf16
// rows (prompt_attn.cu).
//
// Mathematics: one pass over the keys with a running maximum and sum per row.
// A CTA has tiles of 128 rows, a row being a (token, head of the group) pair of
// one sequence and KV head: two tiles at dim 64 and 128, in steps of 128 keys,
// each tile in its softmax while the tensor cores work for the other; one at dim
// 192 and 256, in steps of 64 keys whose scores have two buffers, so that the
// tensor cores work for the step before and the step behind.
//
//   S_t(n) = Q_t K(n)^T     M = 128, N = keys, K = dim       TMEM columns [128 t, +128), or [64 (n % 2), +64)
//   P_t(n) = 2^{S f - m}    16 bits, over S_t(n)'s columns
//   O_t += P_t(n) V(n)      M = 128, N = dim, K = keys       [128 tiles + dim t, +dim)
//
// issued as S(0), O += P(0) V(0), S(1), ... for the tiles in turn, or with two
// buffers S(0), S(1), O += P(0) V(0), S(2), ...  One thread's products run in
// order, so a score behind a product may take the columns of the product's P, and
// a score that is there says that the products before it are.  The maximum that P
// is formed against is raised only when a row's logits pass it by 2^kRaise, so the
// accumulator is rescaled a few times per row.
//
// Bound: a step is a chain of score, softmax and product for each tile, in which the
// two tiles alternate.  Of about 2,850 clocks a step of 128 keys at dim 128 takes
// (prompts, by time stamps), the products are 2,048 at the tensor cores' rate; a tile's chain is
// 520 for its scores' load and maximum of the first 64 keys and as much for the
// rest, 400 for the exponentials of each half, 300 until the issuer has seen P, 700
// to issue the products and 330 until the next scores are there.  Measured and not
// kept: against the form of its time, for a prompt of 16384 tokens, 32 + 8 heads: scores
// in two buffers of 64 columns at dim 128 (1722 us for 1373) and 64 (the same), an
// issuing warp per tile (1994 for 1688), polling without suspension (1745 for 1665), the
// exponentials beside the search for the maximum (1436 for 1341), the second half's load
// beside the first's maximum (1413 for 1341).
//
// What differs is in the source, a class: the arguments, the operands of the
// scores (scores), the queries' way into shared memory (load_q, or Feed's), what
// the waiting warp copies (Feed) and what the copying warps do (copy).
#pragma once
#include <new>
#include <type_traits>

#include "dense_prefill_common.cuh"

namespace v4a {

constexpr int kTileRows = 128;       // rows of a tile (MMA M)

template <int D>
struct Stream {
  static constexpr int kTiles = D <= 128 ? 2 : 1;
  static constexpr int kUnit = kTiles * kTileRows;
  static constexpr int kKeys = kTiles * 64;                            // keys per step
  static constexpr int kParts = kKeys / 64;                            // parts of a step's P, announced one by one
  static constexpr int kBuffers = 3 - kTiles;                          // of a tile's scores
  static constexpr int kQBytes = kTileRows * D * 2;                    // of a tile
  static constexpr int kStepBytes = kKeys * D * 2;                     // a step's values (and bf16 keys)
  static constexpr int kSoftmax = kTiles * 128;                        // threads
  static constexpr bool kSplitRegs = kTiles == 2;                      // (384 threads)
  static constexpr int kCost = 6 / kTiles;                             // steps that a unit's set-up and output take the time of
  static constexpr int kMinSteps = 8 / kTiles;                         // steps a CTA of an even split has at least
};
// A softmax thread of a 128-key step holds 128 scores: the 384 threads of a CTA of two tiles give it registers.
constexpr int kStreamLaunchRegs = 168, kStreamSoftmaxRegs = 200, kStreamRestRegs = 104;
static_assert(kStreamSoftmaxRegs * 256 + kStreamRestRegs * 128 == kStreamLaunchRegs * 384, "the split of the registers");
// P in bf16 has fp32's range, so its maximum may lag far behind: the first keys of a window, few for some rows, would have
// most rows raised at the next step (8 prompts of 1000 to 4096 tokens, window 1024: 2^8 608 us, 2^24 575).  The maximum in
// use is set that far above the largest logit, so that no weight passes one and the accumulator stays below the sum of the
// values' sizes, as with a maximum that does not lag; what it loses are elements of an output below 2^-102, which it may
// hold as less than 2^-126.
constexpr float kRaiseRows = 24.f;
// P in f16 is 2^kTopFp8 2^{w - m}, m again the lag above the largest logit: from 2^11 to 2^15 for the largest weight.  The
// sum is kept without that factor, so groups of zeros, whose value scale is read as 2^-100, add 2^100 a key at most (with
// the factor and a maximum below the logits 2^13 of them, with it alone 2^17, made an infinite lse).
constexpr float kTopFp8 = kShiftFp8 + kRaiseFp8, kTopFp8Inv = 0x1p-15f;
static_assert(kTopFp8 == 15.f, "its inverse");
constexpr int stream_unit(int dim) { return dim <= 128 ? 256 : 128; }

struct StreamSmem {
  uint64_t q_full[2], s_full[2][2], p_full[2][2], o_full[2], k_full[4], k_free[4], v_full[4], v_free[4], raw_full[2], raw_free[2], drain;
  int64_t scan[16];
  alignas(16) uint8_t line[128];     // the CTA's Segments: what they hold would take every role's registers
  uint32_t tmem_base;
  int abort_flag;
  // step n at [n % 8] (a buffer's step can be six steps ahead of the slowest softmax): its page is missing;
  // of its groups of 64 keys: softmax scale x log2(e) x key scale, log2 of the value scale, its inverse
  int missing[8], raw_missing[2];
  alignas(16) float scales[8][2][4];
};

// Byte offset of 16-byte chunk `ch` of row r in an operand of [dim / 64][kN rows][128 bytes], swizzled.
template <int kN>
__device__ __forceinline__ uint32_t stream_chunk(int r, int ch) {
  return uint32_t((ch >> 3) * (kN * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}

// Whether all queries of a sequence are at its run's first position.
__device__ __forceinline__ bool one_position(const DenseAttnDev&) { return false; }

// Units dealt out (split = 2): a CTA's list lies in shared memory or, longer, in its part of the workspace.
template <int kTile>
struct DealtUnit { Unit<kTile> un; int hk; };
constexpr int kDealtItems = 400, kDealtBytes = kDealtItems * int(sizeof(DealtUnit<128>));
constexpr int kMaxDealtSeqs = 4096, kLengthEntries = 8192;      // of the table they are found in
__host__ __device__ constexpr int dealt_bytes(int unit) { return int(split_workspace(unit, 64, 1)); }      // of the workspace, for a CTA

struct Segment { int hk, tile, count; bool whole; };      // tile: the first of `count`; whole: the unit's all

// The CTA's segments (parts of units), one after the other: of SplitDev::split = 0 and 1.
template <int R, int kTile, int kThreads, typename Dev>
struct Segments : Line<R, kTile, kThreads, Dev> {
  using Base = Line<R, kTile, kThreads, Dev>;
  using Base::x0, Base::x1;

  __device__ __forceinline__ Segments(const Dev& a_, const SplitDev& p_, void* mem) : Base(a_, p_, mem) {}
  // The segment at x, and x moved behind it.
  __device__ __forceinline__ Segment next(int64_t* x, Unit<kTile>* un) const {
    const auto pc = this->locate(*x, un);
    const int count = int(min(int64_t(un->tr.tiles - pc.tile), x1 - *x));
    *x += count;
    return Segment{pc.hk, pc.tile, count, pc.tile == 0 && count == un->tr.tiles};
  }
  __device__ __forceinline__ JoinDesc tail() const {      // (split = 1) what the CTA leaves to the next ones
    Unit<kTile> un;
    const auto pc = this->locate(x1 - 1, &un);      // at most the last unit goes on: its first tile has to lie in the range, its last one behind it
    return pc.tile + 1 < un.tr.tiles && x1 - 1 - pc.tile >= x0 ? this->describe(pc, un) : JoinDesc{};
  }
};

// Those of split = 2: whole units, the (unit, KV head) pairs dealt out to the CTAs in turn, forth and back, the longest
// units first.  A unit's length is the tile that its last row sees last (up to the window's length, behind which all are
// alike), or several tiles are one where the table, an entry for each length and sequence, would be too long.
template <int R, int kTile, int kThreads, typename Dev>
struct DealtUnits : Line<R, kTile, kThreads, Dev> {
  using Base = Line<R, kTile, kThreads, Dev>;
  using Base::a, Base::p, Base::x0, Base::x1;
  DealtUnit<kTile>* list;

  __device__ __forceinline__ DealtUnits(const Dev& a_, const SplitDev& p_, void* mem) : Base(a_, p_, mem), list(static_cast<DealtUnit<kTile>*>(mem)) {}
  __device__ __forceinline__ bool init(int64_t* scan, void* scratch, int) {
    SeqRun* const runs = static_cast<SeqRun*>(scratch);
    int* const table = reinterpret_cast<int*>(runs + a.B);      // [length, longest first][B] units before the sequence's
    const int tid = threadIdx.x;
    int32_t* st = blockIdx.x == 0 ? a.status : nullptr;     // one CTA reports the batch's faults
    int top = 0;
    for (int b = tid; b < a.B; b += kThreads) {
      const SeqRun r = runs[b] = this->run(b, st);
      if (r.n > 0) top = max(top, (r.p0 + (one_position(a) ? 0 : r.n - 1)) / kTile);
    }
    int lengths = 1, shift = 0;      // a length: 2^shift tiles
    if (int64_t(p.U) * a.K > gridDim.x) {
      top = __reduce_max_sync(0xffffffffu, top);
      if ((tid & 31) == 0) scan[tid >> 5] = top;
      __syncthreads();
      for (int w = 0; w < kThreads / 32; ++w) top = max(top, int(scan[w]));
      if (a.window) top = min(top, (a.window + kTile - 1) / kTile);
      while (int64_t((top >> shift) + 1) * a.B > kLengthEntries) ++shift;
      lengths = (top >> shift) + 1;
    }
    __syncthreads();
    auto shorter = [&](const SeqRun& r, int len) {      // units of a sequence that are shorter than length `len`
      const int64_t all = this->groups(r.s0, r.s0 + r.n), m = (int64_t(len) << shift) * kTile;      // the first position of this length
      if (len <= 0) return int64_t(0);
      if (len >= lengths || r.p0 + (one_position(a) ? 1 : r.n) <= m) return all;
      return one_position(a) ? 0 : max(int64_t(0), m - r.p0) * a.G / R;
    };
    const int entries = lengths * a.B, per = (entries + kThreads - 1) / kThreads, e0 = min(entries, tid * per), e1 = min(entries, e0 + per);
    int64_t n = 0, all;
    for (int pass = 0; pass < 2; ++pass) {              // counted, then written
      int64_t at = 0;
      if (pass == 1) at = this->before(n, scan, &all);
      for (int e = e0, b = e0 % a.B, len = lengths - 1 - e0 / a.B; e < e1; ++e) {
        const int64_t units = shorter(runs[b], len + 1) - shorter(runs[b], len);
        if (pass == 1) table[e] = int(min(at, int64_t(p.U)));
        at += units;
        if (++b == a.B) b = 0, --len;
      }
      n = at;
    }
    if (st && tid == 0 && all > p.U) report(st, V4A_DEV_BAD_BATCH);         // sequences that share tokens
    __syncthreads();
    const unsigned pairs = unsigned(min(all, int64_t(p.U))) * unsigned(a.K), turns = pairs / gridDim.x;        // (below 2^31: stream_plan)
    auto pair_of = [&](unsigned turn) { return turn * gridDim.x + (turn & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x); };
    x0 = 0;
    x1 = turns + (pair_of(turns) < pairs);
    if (turns >= kDealtItems) list = reinterpret_cast<DealtUnit<kTile>*>(reinterpret_cast<uint8_t*>(p.join) + blockIdx.x * dealt_bytes(R));
    for (int i = tid; i < x1; i += kThreads) {
      const unsigned pair = pair_of(i);
      const int u = int(pair / unsigned(a.K));
      int lo = 0;                                     // the last entry <= u (those without units precede)
      for (int hi = entries; hi - lo > 1;) {
        const int mid = (lo + hi) >> 1;
        if (table[mid] <= u) lo = mid; else hi = mid;
      }
      const int b = lo % a.B, rg = int(shorter(runs[b], lengths - 1 - lo / a.B)) + u - table[lo];
      list[i] = DealtUnit<kTile>{make_unit<R, kTile>(a, this->ref(b, rg, runs[b])), int(pair % unsigned(a.K))};
    }
    __syncthreads();
    return x1 > 0;
  }
  __device__ __forceinline__ Segment next(int64_t* x, Unit<kTile>* un) const {
    const DealtUnit<kTile>& it = list[*x];
    *un = it.un;
    ++*x;
    return Segment{it.hk, 0, un->tr.tiles, true};
  }
};

// A value that a warp's lanes share, said so to the compiler: what an MMA takes from uniform registers need not be
// moved there for each.
template <typename T>
__device__ __forceinline__ T uniform(T x) { return __shfl_sync(0xffffffffu, x, 0); }

// One step of the exchange of four lanes' four pieces (lane l's v[k] becomes lane k's v[l] with steps 1 and 2): pieces
// whose number differs from the lane's in bit kBit change places with the partner's.
template <int kBit>
__device__ __forceinline__ void exchange(uint4 (&v)[4], int lane) {
  const bool high = lane & kBit;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (k & kBit) continue;
    const uint4 give = high ? v[k] : v[k + kBit];
    const uint4 got = make_uint4(__shfl_xor_sync(0xffffffffu, give.x, kBit), __shfl_xor_sync(0xffffffffu, give.y, kBit),
                                 __shfl_xor_sync(0xffffffffu, give.z, kBit), __shfl_xor_sync(0xffffffffu, give.w, kBit));
    if (high) v[k] = got; else v[k + kBit] = got;
  }
}

// The n lowest bits (none for n <= 0, all from 32 on).
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? ~0u : (1u << max(n, 0)) - 1u; }

// Shared memory: queries, the keys' stages, the values', what the source adds, StreamSmem, the line's table.
template <int D, class Src>
struct StreamLayout {
  static constexpr int kThreads = Stream<D>::kSoftmax + 64 + Src::template copiers<D>();
  static constexpr int kKeyStages = Src::template key_stages<D>(), kValueStages = Src::template value_stages<D>();
  static constexpr int kKeyBytes = Src::template key_bytes<D>();       // of a step
  static constexpr int kKeys = Stream<D>::kTiles * Stream<D>::kQBytes;
  static constexpr int kValues = kKeys + kKeyStages * kKeyBytes;
  static constexpr int kExtra = kValues + kValueStages * Stream<D>::kStepBytes;
  static constexpr int kRest = kExtra + Src::template extra_bytes<D>();
  static_assert(kKeyStages <= 4 && kValueStages <= 4 && kKeyBytes % 1024 == 0, "stages");
};

template <int D, class Src, bool kDealt>
__device__ __forceinline__ void stream_attn(const typename Src::Dev& a, const SplitDev& p) {
  using W = Stream<D>;
  using L = StreamLayout<D, Src>;
  constexpr int kThreads = L::kThreads, SK = L::kKeyStages, SV = L::kValueStages;
  constexpr int kKeys = W::kKeys, kBuffers = W::kBuffers;
  constexpr bool kScaled = Src::kScaled;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t q0 = tc::smem_u32(base), k0 = q0 + L::kKeys, v0 = q0 + L::kValues;
  StreamSmem& s = *reinterpret_cast<StreamSmem*>(base + L::kRest);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &s.abort_flag;

  if (!p.late) pdl_wait();
  using Line = std::conditional_t<kDealt, DealtUnits<W::kUnit, kKeys, kThreads, typename Src::Dev>, Segments<W::kUnit, kKeys, kThreads, typename Src::Dev>>;
  static_assert(sizeof(Line) <= sizeof(StreamSmem::line), "room for the line");
  {
    Line mine(a, p, &s + 1);
    if (!mine.init(s.scan, base, W::kMinSteps)) {
      if (p.late) pdl_wait();
      return;
    }
    if (tid == 0) new (s.line) Line(mine);
  }
  const Line& line = *reinterpret_cast<const Line*>(s.line);
  const bool q_copied = Src::q_copied(a);      // the queries come with Feed, ahead of the unit before's output

  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      tc::mbar_init(&s.q_full[t], q_copied ? 1 : kTileRows);
      tc::mbar_init(&s.o_full[t], 1);
      for (int i = 0; i < 2; ++i) {
        tc::mbar_init(&s.s_full[t][i], 1);
        tc::mbar_init(&s.p_full[t][i], t == 0 && (i == 0 || kBuffers == 2) ? 5 : 4);
      }
    }
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(&s.k_full[i], 1);
      tc::mbar_init(&s.v_full[i], Src::template value_arrivals<D>());
      tc::mbar_init(&s.k_free[i], 1);
      tc::mbar_init(&s.v_free[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&s.raw_full[i], 1);
      tc::mbar_init(&s.raw_free[i], Src::template value_arrivals<D>());
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
  if constexpr (W::kSplitRegs) {
    if (warp < 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kStreamSoftmaxRegs));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kStreamRestRegs));
  }
  if (tid < W::kSoftmax) {
    // ---- a tile's queries, softmax and output ----
    const int t = warp >> 2, r = tid & 127, row = t * kTileRows + r;
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + 128 * t + lanes, o_at = tmem_o + D * t + lanes;
    bool ok = true;
    int n = 0, e = 0, g = 0;
    for (int64_t x = line.x0; x < line.x1 && ok;) {
      Unit<kKeys> un;
      const auto sg = line.next(&x, &un);
      const int count = sg.count;
      if (un.rows <= t * kTileRows) {
        n += count;
        continue;
      }
      // a row's logits in log2 units: its scores times f (fp8: and the key scale)
      float f = a.scale_log2;
      if (!q_copied) {
        f = Src::template load_q<D>(a, un, sg.hk, t, r, q0 + t * W::kQBytes);
        tc::fence_proxy_async();
        tc::mbar_arrive(&s.q_full[t]);
      }
      const int m = Src::template row_position<kKeys>(a, un, min(row, un.rows - 1));
      float top = -INFINITY, ref = 0.f, l = 0.f;       // largest logit, the maximum in use, the sum against it
      bool any = false;                                // `ref` is set (a key has been seen)
      for (int i = 0; i < count; ++i, ++e, ++n) {
        const uint32_t at = s_at + 64 * (kBuffers == 2 ? e & 1 : 0);
        ok = __all_sync(0xffffffffu, wait_for(&s.s_full[t][e % kBuffers], (e / kBuffers) & 1, a.status, abort_flag));
        if (!ok) break;
        tc::tc_fence_after();
        float fk[W::kParts], lv[W::kParts], inv_v[W::kParts];
#pragma unroll
        for (int h = 0; h < W::kParts; ++h) {
          fk[h] = f;
          lv[h] = 0.f;
          inv_v[h] = 1.f;
          if constexpr (kScaled) {
            const float4 sc = *reinterpret_cast<const float4*>(s.scales[n & 7][h]);
            fk[h] = logit_factor(f * sc.x);
            lv[h] = sc.y;
            inv_v[h] = sc.z;
          }
        }
        const int j0 = un.tr.at(sg.tile + i) * kKeys;
        const bool gone = Src::kPaged && s.missing[n & 7] != 0;
        const bool hides = gone || !all_visible(a, un.m_lo, un.m_hi, j0, kKeys);
        // columns up to hi, and of those the ones behind lo or before sk; a warp whose rows see all skips each side
        const int hi = gone ? -1 : m - j0, lo = a.window ? m - a.window - j0 : -1, sk = a.window ? a.sinks - j0 : 0;
        auto mask = [&](float* z, int h) {             // (part h)
          if ((W::kParts == 1 && !hides) || __all_sync(0xffffffffu, hi >= 64 * h + 63 && lo < 64 * h)) return;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const int c0 = 64 * h + 32 * w;
            const uint32_t keep = low_bits(hi + 1 - c0) & (~low_bits(lo + 1 - c0) | low_bits(sk - c0));
            if (__all_sync(0xffffffffu, keep == ~0u)) continue;
#pragma unroll
            for (int c = 0; c < 32; ++c) z[32 * w + c] = keep & (1u << c) ? z[32 * w + c] : -INFINITY;
          }
        };
        auto largest = [&](const float* z, int h) {
          float mx[4] = {z[0], z[1], z[2], z[3]};
#pragma unroll
          for (int c = 4; c < 60; c += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k] = max3(mx[k], z[c + k], z[c + k + 4]);
          return fmaf(max3(max3(mx[0], mx[1], mx[2]), mx[3], fmaxf(max3(z[60], z[61], z[62]), z[63])), fk[h], lv[h]);
        };
        uint32_t pk[32];
        auto weights = [&](const float* z, int h) {    // P of part h into pk; their sum
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          const float up = kScaled ? lv[h] + kTopFp8 - ref : -ref;
          const float2 f2 = make_float2(fk[h], fk[h]), r2 = make_float2(up, up);
#pragma unroll
          for (int c = 0; c < 64; c += 2) {
            float2 y = fma2(make_float2(z[c], z[c + 1]), f2, r2);
            y.x = exp2f(y.x);
            y.y = exp2f(y.y);
            sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], y);
            pk[c >> 1] = kScaled ? pack_f16(y.x, y.y) : pack_bf16(y.x, y.y);
          }
          const float all = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          return kScaled ? all * inv_v[h] * kTopFp8Inv : all;
        };
        auto announce = [&](int h) {
          tmem_st32(at + 32 * h, pk);
          tmem_wait_st();
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&s.p_full[t][kBuffers == 2 ? e & 1 : h]);
        };
        float z[kKeys];
        auto find = [&](auto masked) {
#pragma unroll
          for (int h = 0; h < W::kParts; ++h) {
            tc::tmem_ld64(at + 64 * h, z + 64 * h);
            if constexpr (decltype(masked)::value) mask(z + 64 * h, h);
            top = fmaxf(top, largest(z + 64 * h, h));
          }
        };
        if (W::kParts == 1 || hides) find(std::true_type{}); else find(std::false_type{});
        const bool raise = top > -INFINITY && (!any || top > ref);
        const float next = top + (kScaled ? kRaiseFp8 : kRaiseRows);      // what the maximum in use is raised to
        if (__any_sync(0xffffffffu, raise && any)) {       // (so i > 0)
          if constexpr (kBuffers == 2) {      // the step before has to leave the accumulator, which frees its values (one buffer: S says so)
            ok = __all_sync(0xffffffffu, wait_for(&s.v_free[(n - 1) % SV], ((n - 1) / SV) & 1, a.status, abort_flag));
            if (!ok) break;
            tc::tc_fence_after();
          }
          const float w = raise && any ? exp2f(ref - next) : 1.f;
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
          ref = next;
          any = true;
        }
        float sum = weights(z, 0);
        announce(0);
        l += sum;
        if constexpr (W::kParts == 2) {         // (the first part's product runs meanwhile)
          sum = weights(z + 64, 1);
          announce(1);
          l += sum;
        }
      }
      // ---- the output, or the piece for the join ----
      if (ok) ok = __all_sync(0xffffffffu, wait_for(&s.o_full[t], g & 1, a.status, abort_flag));
      ++g;
      if (ok) {
        tc::tc_fence_after();
        const bool begins = sg.tile == 0, whole = sg.whole;
        if (any && l == 0.f) l = NAN;                  // the largest logit is past fp32: it has no weight against itself
        const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
        const int64_t at = row_of(a, un, sg.hk, min(row, un.rows - 1));
        const int64_t slot = int64_t(blockIdx.x) * 2 + (begins ? 1 : 0), part = slot * W::kUnit + row;
        // A lane has a row; four lanes exchange their rows' 16-byte pieces, so that a store covers 64 bytes of each of
        // eight rows instead of 16 of each of 32 (32 prompts of 300 to 700 tokens 111 us instead of 135; chunks of 4096
        // tokens over 28672, heads of 64, 1157 instead of 1208, of 128 1558 and 1565).
        int64_t to[4];
        const int live = un.rows - (row & ~3);         // of the four rows
#pragma unroll
        for (int k = 0; k < 4; ++k) to[k] = __shfl_sync(0xffffffffu, at, (lane & ~3) + k) * D + (lane & 3) * 8;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tmem_ld32(o_at + c, o);
          if constexpr (kScaled) {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] *= kTopFp8Inv;
          }
          if (whole) {
            uint4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              v[k] = make_uint4(pack_bf16(o[8 * k] * inv, o[8 * k + 1] * inv), pack_bf16(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
                                pack_bf16(o[8 * k + 4] * inv, o[8 * k + 5] * inv), pack_bf16(o[8 * k + 6] * inv, o[8 * k + 7] * inv));
            exchange<1>(v, lane);
            exchange<2>(v, lane);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k < live) *reinterpret_cast<uint4*>(a.out + to[k] + c) = v[k];
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
            if (a.lse) a.lse[at] = any ? (ref + log2f(l)) * 0.6931471805599453f : l == 0.f ? -INFINITY : l;
          } else {       // a piece without a key leaves nothing; one whose logits are all NaN is passed on
            p.part_ml[part * 2] = any || l != 0.f ? ref : -INFINITY;
            p.part_ml[part * 2 + 1] = l;
          }
        }
        tc::tc_fence_before();       // O and Q are free for the next segment (announced by its q_full)
      }
    }
  } else if (tid < W::kSoftmax + 32) {
    // ---- the MMA issuer: the warp walks together and one elected lane issues (a branch on the lane's number, which
    // the compiler does not know to leave one lane, took 20 clocks more a product) ----
    constexpr uint32_t kFmt = kScaled ? 0 : 1;       // f16 or bf16
    const uint32_t idesc_o = tc::make_idesc(kFmt, kFmt, kTileRows, D) | (1u << 16);       // B is MN-major
    auto s_of = [&](int t, int e) { return tmem + 128 * t + 64 * (kBuffers == 2 ? e & 1 : 0); };
    auto scores = [&](int t, int e, int n) {         // (by the elected lane)
      Src::template scores<D>(s_of(t, e), q0 + t * W::kQBytes, k0 + (n % SK) * L::kKeyBytes);
      tc::mma_commit(&s.s_full[t][e % kBuffers]);
    };
    auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_for(bar, parity, a.status, abort_flag); };
    bool ok = true;
    int n = 0, e[2] = {0, 0}, g[2] = {0, 0};
    for (int64_t x = line.x0; x < line.x1 && ok;) {
      Unit<kKeys> un;
      const auto sg = line.next(&x, &un);
      const int count = uniform(sg.count);
      const int tiles = uniform(W::kTiles == 2 && un.rows > kTileRows ? 2 : 1);
      for (int j = 0; j < min(count, kBuffers) && ok; ++j) {
        ok = __all_sync(0xffffffffu, wait(&s.k_full[(n + j) % SK], ((n + j) / SK) & 1));
#pragma unroll
        for (int t = 0; t < W::kTiles; ++t) {
          if (t >= tiles) break;
          if (j == 0) ok = __all_sync(0xffffffffu, ok && wait(&s.q_full[t], g[t]++ & 1));
          tc::tc_fence_after();
          if (ok && tc::elect_one()) scores(t, e[t] + j, n + j);
          __syncwarp();
        }
        if (tc::elect_one()) tc::mma_commit(&s.k_free[(n + j) % SK]);
        __syncwarp();
      }
      for (int i = 0; i < count && ok; ++i, ++n) {
        const bool more = i + kBuffers < count;
        const uint32_t vb = v0 + (n % SV) * W::kStepBytes;
#pragma unroll
        for (int t = 0; t < W::kTiles; ++t) {
          if (t >= tiles) break;
#pragma unroll
          for (int h = 0; h < W::kParts; ++h) {
            ok = __all_sync(0xffffffffu, wait(&s.p_full[t][kBuffers == 2 ? e[t] & 1 : h], (e[t] / kBuffers) & 1));
            if (!ok) break;
            tc::tc_fence_after();
            if (tc::elect_one()) {
#pragma unroll
              for (int k = 4 * h; k < 4 * h + 4; ++k)
                mma_ts(tmem_o + D * t, s_of(t, e[t]) + 8 * k, desc_mn(vb + k * 16 * 128, kKeys * 128), idesc_o, i > 0 || k > 0);
              if (h == W::kParts - 1) {
                if (more) scores(t, e[t] + kBuffers, n + kBuffers);
                else if (i + 1 == count) tc::mma_commit(&s.o_full[t]);
              }
              if (h == W::kParts - 1 && t + 1 == tiles) {
                tc::mma_commit(&s.v_free[n % SV]);
                if (more) tc::mma_commit(&s.k_free[(n + kBuffers) % SK]);
              }
            }
            __syncwarp();
          }
          if (!ok) break;
          ++e[t];
        }
      }
    }
    if (!ok) {                      // after a timeout: what was issued ends before TMEM is freed
      if (tc::elect_one()) tc::mma_commit(&s.drain);
      for (int k = 0; k < (1 << 22) && !tc::mbar_test(&s.drain, 0); ++k) {
      }
    }
    __syncwarp();
  } else if (tid < W::kSoftmax + 64) {
    // ---- a warp that copies what TMA brings without a conversion (Feed), and waits for all copies in the issuer's
    // place (a test of a barrier takes it 180 clocks, which would lie between two products): step n's first P is
    // announced when the values of n and the keys of the scores behind its product are there too ----
    typename Src::template Feed<D> feed(a, base, s);
    auto wait = [&](uint64_t* bar, int phase) { return wait_for(bar, phase & 1, a.status, abort_flag); };
    bool ok = true;
    int n = 0, e = 0;
    for (int64_t x = line.x0; x < line.x1 && ok;) {
      Unit<kKeys> un;
      const auto sg = line.next(&x, &un);
      const int count = sg.count;
      ok = feed.begin(un, sg.hk, sg.tile, count, n);
      for (int j = 0; j < min(count, kBuffers) && ok; ++j)      // (a phase is asked for when the one before it has been)
        ok = __all_sync(0xffffffffu, wait(&s.k_full[(n + j) % SK], (n + j) / SK));
      for (int i = 0; i < count && ok; ++i, ++n, ++e) {
        uint64_t* const p_first = &s.p_full[0][kBuffers == 2 ? e & 1 : 0];
        ok = feed.step(i, n) && (i + kBuffers >= count || wait(&s.k_full[(n + kBuffers) % SK], (n + kBuffers) / SK)) &&
             wait(&s.v_full[n % SV], n / SV) && (e < kBuffers || wait(p_first, e / kBuffers - 1));        // (the arrival is for this phase)
        ok = __all_sync(0xffffffffu, ok);
        if (ok && lane == 0) tc::mbar_arrive(p_first);
      }
    }
    if (!ok) feed.drain();
  } else {
    // ---- the copying warps ----
    bool ok = true;
    int n = 0;
    for (int64_t x = line.x0; x < line.x1 && ok;) {
      Unit<kKeys> un;
      const auto sg = line.next(&x, &un);
      const int count = sg.count;
      ok = Src::template copy<D>(a, un, sg.hk, sg.tile, count, n, tid - W::kSoftmax - 64, base, s);
      n += count;
    }
  }
  __syncthreads();
  tc::tc_fence_after();
  if (warp == 0) tc::tmem_dealloc(tmem, 512);
  if constexpr (!kDealt) {
    if (p.split == 1 && tid == 0) p.join[blockIdx.x] = line.tail();
  }
  if (p.late) pdl_wait();
  pdl_trigger();
}

// Two kernels, since what finds the segments of an even split costs the other form time (its code and registers: chunks over
// a long cache 1632 us for 1812 in one kernel).
template <int D, class Src>
__global__ void __launch_bounds__(StreamLayout<D, Src>::kThreads, 1)
stream_attn_kernel(const __grid_constant__ typename Src::Dev a, const __grid_constant__ SplitDev p) {
  stream_attn<D, Src, false>(a, p);
}
template <int D, class Src>
__global__ void __launch_bounds__(StreamLayout<D, Src>::kThreads, 1)
dealt_attn_kernel(const __grid_constant__ typename Src::Dev a, const __grid_constant__ SplitDev p) {
  stream_attn<D, Src, true>(a, p);
}

template <int D, class Src>
constexpr size_t stream_smem(int split, int U) { return 1024 + StreamLayout<D, Src>::kRest + sizeof(StreamSmem) + split_smem(split, U); }

// After a timeout: the copies of steps before `n` into a ring of stages end before the CTA does (waited for with a limit).
__device__ __forceinline__ void drain_copies(uint64_t* full, int stages, int n) {
  for (int m = max(0, n - stages); m < n; ++m)
    for (int k = 0; k < (1 << 20) && !tc::mbar_test(&full[m % stages], (m / stages) & 1); ++k) {
    }
}

// The split of the registers adds up only with those that the kernel was to be built with: setmaxnreg would wait
// for ever with fewer.
template <int D, class Src>
bool stream_ready() {
  static std::atomic<uint64_t> done{0};
  return once_per_device(&done, [] {
    auto fits = [](auto kern) {
      cudaFuncAttributes attr;
      return (!Stream<D>::kSplitRegs || (cudaFuncGetAttributes(&attr, kern) == cudaSuccess && attr.numRegs == kStreamLaunchRegs)) &&
             raise_smem(kern, 227 * 1024);
    };
    return fits(stream_attn_kernel<D, Src>) && fits(dealt_attn_kernel<D, Src>);
  });
}

template <int D, class Src>
int stream_launch(const typename Src::Dev& d, const SplitDev& p, cudaStream_t stream) {
  using L = StreamLayout<D, Src>;
  static_assert(!Stream<D>::kSplitRegs || L::kThreads == 384, "the split of the registers");
  static_assert(stream_smem<D, Src>(1, kMaxSplitUnits) <= 227 * 1024, "shared memory of a CTA");
  static_assert(stream_smem<D, Src>(0, 0) + kDealtBytes <= 227 * 1024, "shared memory of a CTA");
  static_assert(L::kRest >= int(kMaxSplitUnits * 16), "scratch of the line");
  static_assert(L::kRest >= kMaxDealtSeqs * int(sizeof(SeqRun)) + kLengthEntries * 4, "scratch of the dealt units");
  // at least 116 KB: no two CTAs that allocate TMEM share an SM
  const size_t table = p.split == 2 ? kDealtBytes : 0;
  const size_t bytes = std::max(stream_smem<D, Src>(p.split == 1, p.U) + table, size_t(116 * 1024));
  const int64_t pairs = int64_t(p.U) * d.K, grid = p.split == 1 ? p.grid : p.split == 2 ? std::min<int64_t>(p.grid, pairs) : pairs;
  const cudaError_t e = launch_pdl(p.split == 2 ? dealt_attn_kernel<D, Src> : stream_attn_kernel<D, Src>, dim3(unsigned(grid)), dim3(L::kThreads), bytes, stream, d, p);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? V4A_OK : V4A_ERR_CUDA;
}

}  // namespace v4a
