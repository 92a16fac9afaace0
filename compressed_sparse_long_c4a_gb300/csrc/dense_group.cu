// Attention of chunks over the dense paged cache whose fp8 rows have one scale
// per 64 positions and KV head (v4a_dense_attn, V4A_KV_FP8_GROUP, many query
// rows per KV head): dense_stream.cuh over that cache.
//
// Mathematics: the keys of a group share a scale, so a step's key scales are one
// factor of the logits of each 64 keys and the value scales one shift of their
// exponents: the softmax costs what it does over bf16 rows.  The scores are an
// 8-bit product of the key codes as they lie in the cache: a query row times the
// power of two that brings its largest element to [2^7, 2^8) is taken as the sum
// of two e4m3 numbers, the nearest one and what that leaves, each multiplied with
// the keys at twice the 16-bit rate.  A bf16 has 8 bits, a nearest e4m3 4 of them
// and the rest at most 4, so the sum is exact down to 2^-9 of the row's largest
// element and within 2^-17 of that element below.  Value codes become f16, exactly:
// P in 8 bits would be too coarse.  P is f16 and holds 2^{w - m}, w the logit plus
// log2 of the value scale, times a power that makes 2^11 to 2^15 of the largest:
// weights down to 2^-25 of it are rounded to 11 bits.
//
// Copies: one lane has TMA bring the key codes into the swizzle that the MMA reads,
// and the value codes as they are; two to four warps convert the latter from shared
// memory.  Key rows that no row sees hold anything: their scores are replaced, not
// multiplied; hidden value rows become zeros.
//
// Bound: as prompts (dense_stream.cuh); the conversions share the softmax's
// schedulers (as integer operations instead of cvt: 2362 us for 1605; four warps of
// them among 512 threads: 1708), and the second e4m3 of the query takes 3% of the
// time.  Measured, 32 + 8 heads of 128: 4096 tokens over 28672 1568 us (1314 TFLOP/s;
// ncu, 2048 over 8192: tensor pipe 47% busy), 1000 over 4000 92 us, 4096 over none 168 (both
// with a table no wider than the sequence: stream_plan); 16 + 4 heads of 256,
// 2048 over 10240 367 us (1030; row scales 505), of 192 330 us (860); heads of 64 over
// 28672 1157 us (891).
#include "dense_stream.cuh"

namespace v4a {
namespace {

struct GroupDev : DenseAttnDev {
  CUtensorMap km;                   // [pages][2 K 256 rows][dim codes]
};

// K-major operand of 64-byte rows with the 64-byte swizzle: 8-row groups 512 bytes apart.
__device__ __forceinline__ uint64_t desc_sw64(uint32_t saddr) {
  return uint64_t((saddr & 0x3FFFFu) >> 4) | (uint64_t(1) << 16) | (uint64_t(512 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(4) << 61);
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint32_t r;
  asm("{\n.reg .b16 c;\ncvt.rn.satfinite.e4m3x2.f32 c, %2, %1;\ncvt.u32.u16 %0, c;\n}\n" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_values(uint32_t codes) {
  uint32_t r;
  asm("{\n.reg .b16 c;\ncvt.u16.u32 c, %1;\ncvt.rn.f16x2.e4m3x2 %0, c;\n}\n" : "=r"(r) : "r"(codes));
  return __half22float2(*reinterpret_cast<const __half2*>(&r));
}

struct GroupCache {
  using Dev = GroupDev;
  static constexpr bool kScaled = true, kPaged = true;
  static constexpr int kLead = 2;                  // steps that copies are issued ahead
  template <int D> static constexpr int copiers() { return D == 192 ? 96 : D == 256 ? 128 : 64; }
  template <int D> static constexpr int key_stages() { return 3; }
  template <int D> static constexpr int value_stages() { return 2; }
  template <int D> static constexpr int key_bytes() { return Stream<D>::kKeys * D; }
  template <int D> static constexpr int raw_stages() { return 2; }        // of value codes as they are
  template <int D> static constexpr int extra_bytes() { return raw_stages<D>() * key_bytes<D>(); }
  template <int D> static constexpr int value_arrivals() { return copiers<D>(); }
  // Codes of an operand lie in blocks of this many bytes a row, the span of its swizzle.
  template <int D> static constexpr int block() { return D % 128 ? 64 : 128; }

  // Byte offset of 16-byte chunk `ch` of row r in an operand of [dim / block][kN rows][block].
  template <int D, int kN>
  static __device__ __forceinline__ uint32_t code_chunk(int r, int ch) {
    constexpr int kPer = block<D>() / 16;
    return uint32_t(ch / kPer * (kN * block<D>()) + r * block<D>() + (((ch % kPer) ^ (kPer == 8 ? r & 7 : (r >> 1) & 3)) << 4));
  }

  template <int kKeys>
  static __device__ __forceinline__ int row_position(const Dev& a, const Unit<kKeys>& un, int row) {
    return un.m_lo + (un.row0 % a.G + row) / a.G;
  }

  template <int D>
  static __device__ __forceinline__ void scores(uint32_t st, uint32_t qa, uint32_t kb) {
    constexpr int kKeys = Stream<D>::kKeys, kPer = block<D>() / 32;
    constexpr uint32_t idesc = tc::make_idesc(0, 0, kTileRows, kKeys);
    auto desc = [](uint32_t at) { return block<D>() == 128 ? tc::desc_sw128(at) : desc_sw64(at); };
#pragma unroll
    for (int k = 0; k < 2 * (D / 32); ++k) {       // the nearest e4m3, then the rest, against the same codes
      const int j = k % (D / 32);
      tc::mma_f8f6f4(st, desc(qa + (k / (D / 32)) * (kTileRows * D) + j / kPer * (kTileRows * block<D>())) + 2 * (j % kPer),
                     desc(kb + j / kPer * (kKeys * block<D>())) + 2 * (j % kPer), idesc, k > 0);
    }
  }

  static __device__ __forceinline__ bool q_copied(const Dev&) { return false; }

  // Row r of tile t as two e4m3 operands at q0 and behind; zeros behind the unit's last row.
  template <int D>
  static __device__ __forceinline__ float load_q(const Dev& a, const Unit<Stream<D>::kKeys>& un, int hk, int t, int r, uint32_t q0) {
    const int row = t * kTileRows + r;
    const bool live = row < un.rows;
    const uint4* q = reinterpret_cast<const uint4*>(a.q + row_of(a, un, hk, live ? row : 0) * D);
    uint32_t top = 0;                          // |q| as bf16 bits, two at a time
#pragma unroll 8
    for (int ch = 0; ch < D / 8; ++ch) {
      const uint4 w = __ldcg(q + ch);
      top = __vmaxu2(top, __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
    }
    top = max(top >> 16, top & 0xffffu);
    const int e = top == 0 ? 127 : min(253, max(1, 261 - int(top >> 7)));      // the power's exponent field
    // (a row with an infinity becomes NaN: e4m3 has none, and would make it 448)
    const float up = !live ? 0.f : top >= 0x7f80 ? NAN : __int_as_float(e << 23), down = __int_as_float((254 - e) << 23);
#pragma unroll 4
    for (int ch = 0; ch < D / 16; ++ch) {
      const uint4 u = __ldcg(q + 2 * ch), w = __ldcg(q + 2 * ch + 1);
      const uint32_t in[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
      uint32_t near[4], rest[4];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float x = __uint_as_float(in[k] << 16) * up, y = __uint_as_float(in[k] & 0xffff0000u) * up;
        const uint32_t c = e4m3x2(x, y);
        const float2 v = e4m3x2_values(c);
        const uint32_t d = e4m3x2(x - v.x, y - v.y);
        near[k >> 1] = k & 1 ? near[k >> 1] | c << 16 : c;
        rest[k >> 1] = k & 1 ? rest[k >> 1] | d << 16 : d;
      }
      const uint32_t at = q0 + code_chunk<D, kTileRows>(r, ch);
      st_shared16(at, make_uint2(near[0], near[1]), make_uint2(near[2], near[3]));
      st_shared16(at + kTileRows * D, make_uint2(rest[0], rest[1]), make_uint2(rest[2], rest[3]));
    }
    return fmaxf(a.scale_log2 * down, 0x1p-126f);
  }

  // Who issues the copies of the value codes: with two tiles Feed, beside the keys' (4096 tokens over 28672, 32 + 8 heads
  // of 128: 1605 us; the converting warps, whose lanes then wait for the one that issues: 1957), with one tile the
  // converting warps, as soon as a buffer is read (2048 over 10240, 16 + 4 heads of 256: 371 us; Feed, which then holds
  // the keys' copies back: 412).
  template <int D>
  static constexpr bool copiers_issue() { return Stream<D>::kTiles == 1; }
  // Issues the copy of the value codes of step i of the segment, step n of the CTA (one lane).
  template <int D>
  static __device__ __forceinline__ bool issue_values(const Dev& a, const Unit<Stream<D>::kKeys>& un, int hk, int tile, int i, int n, int32_t page,
                                                      uint8_t* base, StreamSmem& s) {
    using L = StreamLayout<D, GroupCache>;
    constexpr int SR = raw_stages<D>();
    if (!wait_for(&s.raw_free[n % SR], ((n / SR) & 1) ^ 1, a.status, &s.abort_flag)) return false;
    const bool gone = page < 0 || page >= a.num_blocks;
    s.raw_missing[n % SR] = gone;
    if (gone) {
      tc::mbar_arrive(&s.raw_full[n % SR]);
    } else {
      const int at = hk * kBlockPositions + un.tr.at(tile + i) * Stream<D>::kKeys % kBlockPositions;       // first row of the step
      tc::mbar_arrive_expect_tx(&s.raw_full[n % SR], L::kKeyBytes);
      tc::bulk_load(base + L::kExtra + (n % SR) * L::kKeyBytes, a.pool + page * a.block_bytes + (int64_t(a.K) * kBlockPositions + at) * D,
                    L::kKeyBytes, &s.raw_full[n % SR]);
    }
    return true;
  }

  // The copies of a step's key codes, issued by one lane kLead steps ahead.  Table entries are read two steps before
  // they are used and the scales one step.
  template <int D>
  struct Feed {
    using W = Stream<D>;
    using L = StreamLayout<D, GroupCache>;
    static constexpr int kGroups = W::kKeys / kGroupPositions;
    const Dev& a;
    uint8_t* base;
    StreamSmem& s;
    const Unit<W::kKeys>* un = nullptr;
    int hk = 0, tile = 0, count = 0, issued = 0;       // issued: steps of the CTA whose copies are on their way
    int32_t entry = -1;                                // table entry of the step behind `page`'s
    int32_t page = -1;                                 // of the step to be issued; -1: missing
    float scale = 1.f;                                 // lanes 0..3: its groups' key scales, then value scales

    __device__ __forceinline__ Feed(const Dev& a_, uint8_t* base_, StreamSmem& s_) : a(a_), base(base_), s(s_) {}
    __device__ __forceinline__ int lane() const { return threadIdx.x & 31; }
    __device__ __forceinline__ int32_t lookup(int i) const {
      return i < count ? __ldcg(a.bt + int64_t(un->b) * a.max_blocks + un->tr.at(tile + i) / (kBlockPositions / W::kKeys)) : -1;
    }
    // Takes `entry`, of step i, for the next step to be issued, and reads its scales and the entry behind.
    __device__ __forceinline__ void advance(int i) {
      page = entry;
      entry = lookup(i + 1);
      if (i < count && (page < 0 || page >= a.num_blocks)) {
        if (lane() == 0) report(a.status, V4A_DEV_BAD_BLOCK);
        page = -1;
      }
      scale = 1.f;
      if (page >= 0 && lane() < 2 * kGroups) {
        const int which = lane() / kGroups, g = lane() % kGroups;
        const int j = un->tr.at(tile + i) * W::kKeys + g * kGroupPositions;       // the group's first position
        const float* at = reinterpret_cast<const float*>(a.pool + page * a.block_bytes + int64_t(2 * a.K) * kBlockPositions * D);
        // (of a group that no row sees the scale may be anything)
        if (j <= un->m_hi && (a.window == 0 || j + kGroupPositions - 1 > un->m_lo - a.window || j < a.sinks))
          scale = __ldcg(at + (which * a.K + hk) * kGroupsPerBlock + j % kBlockPositions / kGroupPositions);
      }
    }
    // Issues the copies of step i of the segment, step n of the CTA.
    __device__ __forceinline__ bool issue(int i, int n) {
      constexpr int SK = key_stages<D>();
      if (!__all_sync(0xffffffffu, wait_for(&s.k_free[n % SK], ((n / SK) & 1) ^ 1, a.status, &s.abort_flag))) return false;
      if (lane() < 2 * kGroups) {
        const int which = lane() / kGroups, g = lane() % kGroups;
        float* const to = s.scales[n & 7][g];
        if (which == 0) {
          to[0] = scale;
        } else {
          const float l = scale > 0x1p-100f ? log2f(scale) : scale <= 0x1p-100f ? -100.f : scale;
          to[1] = l;
          to[2] = exp2f(-l);
        }
      }
      if (lane() == 0) s.missing[n & 7] = page < 0;
      __syncwarp();
      if (lane() == 0) {
        if (page < 0) {
          tc::mbar_arrive(&s.k_full[n % SK]);
        } else {
          const int at = hk * kBlockPositions + un->tr.at(tile + i) * W::kKeys % kBlockPositions;       // first row of the step
          uint8_t* const keys = base + L::kKeys + (n % SK) * L::kKeyBytes;
          tc::mbar_arrive_expect_tx(&s.k_full[n % SK], L::kKeyBytes);
#pragma unroll
          for (int c = 0; c < D / block<D>(); ++c)
            tc::tma_load_3d(keys + c * (W::kKeys * block<D>()), &a.km, c * block<D>(), at, page, &s.k_full[n % SK]);
        }
      }
      bool ok = true;
      if (!copiers_issue<D>() && lane() == 0) ok = issue_values<D>(a, *un, hk, tile, i, n, page, base, s);
      issued = n + 1;
      if (!__all_sync(0xffffffffu, ok)) return false;
      advance(i + 1);
      return true;
    }
    __device__ __forceinline__ bool begin(const Unit<W::kKeys>& un_, int hk_, int tile_, int count_, int n) {
      un = &un_;
      hk = hk_; tile = tile_; count = count_;
      entry = lookup(0);
      advance(0);
      for (int i = 0; i < min(count, kLead); ++i)
        if (!issue(i, n + i)) return false;
      return true;
    }
    // (4096 tokens over 28672 with three stages of value codes and two of keys, issued behind step i's announcement: 1716 us)
    __device__ __forceinline__ bool step(int i, int n) { return i + kLead >= count || issue(i + kLead, n + kLead); }
    __device__ __forceinline__ void drain() {
      drain_copies(s.k_full, key_stages<D>(), issued);
      if (!copiers_issue<D>()) drain_copies(s.raw_full, raw_stages<D>(), issued);
    }
  };

  // Value codes of `count` steps from tile `tile` of the unit on, step n of the CTA first, as f16.
  template <int D>
  static __device__ __forceinline__ bool copy(const Dev& a, const Unit<Stream<D>::kKeys>& un, int hk, int tile, int count, int n, int lt,
                                              uint8_t* base, StreamSmem& s) {
    using L = StreamLayout<D, GroupCache>;
    constexpr int SV = value_stages<D>(), SR = raw_stages<D>(), kKeys = Stream<D>::kKeys, kPerRow = D / 16, kStep = copiers<D>() / kPerRow, kPasses = kKeys / kStep;
    static_assert(kStep % 8 == 0 && copiers<D>() % kPerRow == 0 && kKeys % kStep == 0, "a thread's chunks lie at the same place of the swizzle");
    const int r0 = lt / kPerRow, ch = lt % kPerRow;
    const uint32_t values = tc::smem_u32(base + L::kValues);
    const uint32_t even = values + stream_chunk<kKeys>(r0, 2 * ch), odd = values + stream_chunk<kKeys>(r0, 2 * ch + 1);
    volatile int* abort_flag = &s.abort_flag;
    auto entry = [&](int i) {        // step i's table entry, read a step ahead of its use
      return i < count && lt == 0 ? __ldcg(a.bt + int64_t(un.b) * a.max_blocks + un.tr.at(tile + i) / (kBlockPositions / kKeys)) : -1;
    };
    constexpr bool kIssue = copiers_issue<D>();
    auto fail = [&](int issued) {
      if (kIssue && lt == 0) drain_copies(s.raw_full, SR, issued);
      return false;
    };
    int32_t next = -1;
    if (kIssue && lt == 0) {         // two steps ahead
      const int32_t first = entry(0), second = entry(1);
      if (!issue_values<D>(a, un, hk, tile, 0, n, first, base, s) || (count > 1 && !issue_values<D>(a, un, hk, tile, 1, n + 1, second, base, s)))
        return fail(n + 1);
      next = entry(2);
    }
    for (int i = 0; i < count; ++i, ++n) {
      const int issued = n + min(count - i, 2);
      if (!wait_for(&s.raw_full[n % SR], (n / SR) & 1, a.status, abort_flag)) return fail(issued);
      const int j0 = un.tr.at(tile + i) * kKeys;
      // rows up to hi, and of those the ones behind lo or before sk, are values, the others zeros
      const int hi = s.raw_missing[n % SR] ? -1 : un.m_hi - j0, lo = a.window ? un.m_lo - a.window - j0 : -1, sk = a.window ? a.sinks - j0 : 0;
      const uint4* raw = reinterpret_cast<const uint4*>(base + L::kExtra + (n % SR) * L::kKeyBytes) + lt;
      if (!wait_for(&s.v_free[n % SV], ((n / SV) & 1) ^ 1, a.status, abort_flag)) return fail(issued);
      const uint32_t to = (n % SV) * Stream<D>::kStepBytes;
#pragma unroll
      for (int k = 0; k < kPasses; ++k) {
        const int r = r0 + k * kStep;
        uint4 w = raw[k * copiers<D>()];
        if (!(r <= hi && (r > lo || r < sk))) w = make_uint4(0, 0, 0, 0);
        st_shared16(even + to + k * (kStep * 128), f16_of(w.x), f16_of(w.y));
        st_shared16(odd + to + k * (kStep * 128), f16_of(w.z), f16_of(w.w));
      }
      tc::mbar_arrive(&s.raw_free[n % SR]);
      tc::fence_proxy_async();
      tc::mbar_arrive(&s.v_full[n % SV]);
      if (kIssue && lt == 0 && i + 2 < count) {
        if (!issue_values<D>(a, un, hk, tile, i + 2, n + 2, next, base, s)) return fail(issued);
        next = entry(i + 3);
      }
    }
    return true;
  }
};

bool make_map(CUtensorMap* map, const DenseAttnDev& d, int dim) {
  auto fn = tc::encode_fn();
  if (!fn) return false;
  const int block = dim % 128 ? 64 : 128;
  const cuuint64_t dims[3] = {cuuint64_t(dim), cuuint64_t(2 * d.K) * kBlockPositions, cuuint64_t(d.num_blocks)};
  const cuuint64_t strides[2] = {cuuint64_t(dim), cuuint64_t(d.block_bytes)};
  const cuuint32_t box[3] = {cuuint32_t(block), cuuint32_t(dim <= 128 ? 128 : 64), 1}, step[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(d.pool), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            block == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool dense_group_ready(int dim, const DenseAttnDev& d) {
  CUtensorMap map;
  if (!make_map(&map, d, dim)) return false;
  return dim == 64 ? stream_ready<64, GroupCache>() : dim == 128 ? stream_ready<128, GroupCache>()
       : dim == 192 ? stream_ready<192, GroupCache>() : stream_ready<256, GroupCache>();
}

int dense_group(int dim, const DenseAttnDev& d, const SplitDev& p, cudaStream_t stream) {
  GroupDev g{};
  static_cast<DenseAttnDev&>(g) = d;
  if (!make_map(&g.km, d, dim)) return V4A_ERR_CUDA;
  switch (dim) {
    case 64: return stream_launch<64, GroupCache>(g, p, stream);
    case 128: return stream_launch<128, GroupCache>(g, p, stream);
    case 192: return stream_launch<192, GroupCache>(g, p, stream);
    default: return stream_launch<256, GroupCache>(g, p, stream);
  }
}

size_t stream_workspace(int dim) { return split_workspace(stream_unit(dim), dim, kSms); }

// Whole units are dealt out unless an even split of the steps should take less time: that has no idle CTAs, but cut units
// leave pieces to be joined, which costs the time of about 11 steps of 128 keys, and its CTAs walk several sequences'
// keys at different places.  Even split / dealt out, us, 32 + 8 heads of 128: prompts of 16384 tokens 1348 / 1276, 2048
// 57 / 37, 4 + 1 heads 8192 74 / 104, 4096 41 / 57, 16384 195 / 195; 4 of 1500 to 2500 139 / 96; a window of 1024 over
// 16384 276 / 217; group caches, 4096 tokens over 28672 1565 / 1806, over none 277 / 168, 2048 over 2000 156 / 125, 1000
// over 4000 111 / 94, 4 sequences of 1000 over 8000 533 / 557, of 500 to 2000 over up to 8000 378 / 314, 16 of 256 over
// 1000 to 30000 963 / 846.
// `keys` of a paged cache is the width of its block table, the only bound on the lengths that the host has.  Where the
// table is far wider than its sequences they look long, and chunks that would gain from being dealt out are split evenly:
// with a table of 8192 positions or more the chunks over none, 2000 and 4000 above take the first of the two times.
int stream_plan(const DenseAttnDev& d, int dim, int rows_from, int64_t keys, bool causal, void* ws, SplitDev* out) {
  const int unit = stream_unit(dim);
  SplitDev p{};
  p.RG = int((int64_t(d.max_new) * d.G + unit - 1) / unit);
  p.rows_from = rows_from;
  p.rows_to = INT32_MAX;
  if (rows_from > 0) p.RG = std::max(p.RG, 2);      // sequences of the other launch are not units
  const int64_t units = units_bound(d, rows_from, p.RG, unit);
  if (units > INT32_MAX || units * d.K > INT32_MAX) return V4A_ERR_UNSUPPORTED;
  p.U = int(units);
  // Times in steps of 128 keys.  Units' lengths are taken to be spread evenly: of one sequence between its first and its
  // last query's, of several between none and the longest.  Dealt out, the full turns have the longest of them, and the
  // last turn's first is the next.
  const double longest = double(d.window ? std::min<int64_t>(keys, int64_t(d.window) + 256) : keys) / 128;
  const double spread = d.window ? 0 : d.B > 1 ? longest : causal ? std::min(longest, double(d.max_new) / 128) : 0;
  const double rounds = double(p.U) * d.K / kSms, full = std::floor(rounds);
  const double even = (rounds * (longest - spread / 2) + 11) * (d.B > 1 ? 1.15 : 1);
  const double dealt = full * (longest - spread * full / (2 * rounds)) + (rounds > full ? longest - spread * full / rounds : 0);
  const bool can_split = std::max(p.U, d.B) <= kMaxSplitUnits, can_deal = d.B <= kMaxDealtSeqs && (units * d.K / kSms + 1) * int(sizeof(DealtUnit<128>)) <= dealt_bytes(unit);
  p.split = can_split && (even < dealt || !can_deal) ? 1 : can_deal ? 2 : 0;
  split_carve(&p, ws, unit, dim, kSms, dim <= 128 ? Stream<128>::kCost : Stream<256>::kCost);
  *out = p;
  return V4A_OK;
}

}  // namespace v4a
