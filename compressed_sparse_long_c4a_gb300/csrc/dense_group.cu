// Attention of chunks over the dense paged cache whose fp8 rows have one scale
// per 64 positions and KV head (v4a_dense_attn, V4A_KV_FP8_GROUP, many query
// rows per KV head): dense_stream.cuh over that cache.
//
// Mathematics: a step of 64 keys is one group, so its key scale is one factor of
// the step's logits and its value scale one shift of their exponents: the softmax
// costs what it does over bf16 rows.  Codes become f16 on their way into shared
// memory, exactly; the query joins them there as f16 times the power of two that
// brings its row's largest element to [2^14, 2^15), exact down to 2^-31 of that
// element.  P is f16 and holds 2^11 2^{w - m}, w the logit plus log2 of the value
// scale: weights down to 2^-25 of the largest are rounded to 11 bits.
#include "dense_stream.cuh"

namespace v4a {
namespace {

struct GroupCache {
  using Dev = DenseAttnDev;
  static constexpr bool kScaled = true, kPaged = true;
  // Threads that copy the keys (and as many the values): each has one 16-code chunk of every kStep-th row.
  template <int D>
  static constexpr int loaders() { return D == 64 ? 64 : D / 2; }
  template <int D>
  static constexpr int threads() { return Stream<D>::kSoftmax + 32 + 2 * loaders<D>(); }
  template <int D>
  static constexpr int arrivals() { return loaders<D>(); }

  static __device__ __forceinline__ int row_position(const Dev& a, const Unit<kStreamKeys>& un, int row) {
    return un.m_lo + (un.row0 % a.G + row) / a.G;
  }

  // Row r of tile t as f16 into the operand at q0; zeros behind the unit's last row.
  template <int D>
  static __device__ __forceinline__ float load_q(const Dev& a, const Unit<kStreamKeys>& un, int hk, int t, int r, uint32_t q0) {
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
    const int e = top == 0 ? 127 : min(253, max(1, 268 - int(top >> 7)));      // the power's exponent field
    const float up = __int_as_float(e << 23), down = __int_as_float((254 - e) << 23);
    auto f16 = [&](uint32_t w) { return live ? pack_f16(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up) : 0u; };
#pragma unroll 8
    for (int ch = 0; ch < D / 8; ++ch) {
      const uint4 w = __ldcg(q + ch);
      st_shared16(q0 + stream_chunk<kTileRows>(r, ch), make_uint2(f16(w.x), f16(w.y)), make_uint2(f16(w.z), f16(w.w)));
    }
    return fmaxf(a.scale_log2 * down, 0x1p-126f);
  }

  // Keys (half 0) or values of `count` steps from tile `tile` of the unit on, step n of the CTA first.
  template <int D>
  static __device__ __forceinline__ bool copy(const Dev& a, const Unit<kStreamKeys>& un, int hk, int tile, int count, int n, int half, int lt,
                                              uint8_t* buffers, StreamSmem& s) {
    constexpr int S = Stream<D>::kStages, kPerRow = D / 16, kStep = loaders<D>() / kPerRow, kPasses = kStreamKeys / kStep;
    static_assert(kStep % 8 == 0 && loaders<D>() % kPerRow == 0, "a thread's chunks lie at the same place of the swizzle");
    const int r0 = lt / kPerRow, ch = lt % kPerRow;
    const uint32_t even = tc::smem_u32(buffers) + stream_chunk<kStreamKeys>(r0, 2 * ch), odd = tc::smem_u32(buffers) + stream_chunk<kStreamKeys>(r0, 2 * ch + 1);
    uint64_t* const full = half ? s.v_full : s.k_full;
    uint64_t* const free = half ? s.v_free : s.k_free;
    volatile int* abort_flag = &s.abort_flag;
    auto entry = [&](int i) {        // step i's table entry, read ahead of its use
      return i < count ? __ldcg(a.bt + int64_t(un.b) * a.max_blocks + un.tr.at(tile + i) / (kBlockPositions / kStreamKeys)) : -1;
    };
    // step i's rows and scales; rows up to hi, and of those the ones behind lo or before sk, are read, the others are zeros
    struct Step { uint4 raw[kPasses]; float ks, vs; bool missing; };
    auto read = [&](int i, int32_t page, Step& st) {
      st.missing = page < 0 || page >= a.num_blocks;
      if (st.missing && lt == 0 && half == 0) report(a.status, V4A_DEV_BAD_BLOCK);
      const int j0 = un.tr.at(tile + i) * kStreamKeys;
      const int hi = st.missing ? -1 : un.m_hi - j0, lo = a.window ? un.m_lo - a.window - j0 : -1, sk = a.window ? a.sinks - j0 : 0;
      const uint8_t* block = a.pool + (st.missing ? 0 : page * a.block_bytes);
      const int at = st.missing ? 0 : hk * kBlockPositions + j0 % kBlockPositions;       // first row of the step
      const uint8_t* src = block + (int64_t(half * a.K) * kBlockPositions + at) * D + lt * 16;
#pragma unroll
      for (int k = 0; k < kPasses; ++k) {
        const int r = r0 + k * kStep;
        st.raw[k] = make_uint4(0, 0, 0, 0);
        if (r <= hi && (r > lo || r < sk)) st.raw[k] = __ldcg(reinterpret_cast<const uint4*>(src + k * (kStep * D)));
      }
      st.ks = st.vs = 1.f;
      if (lt == 0 && half == 0 && !st.missing) {
        const float* scale = reinterpret_cast<const float*>(block + int64_t(2 * a.K) * kBlockPositions * D) + at / kStreamKeys;
        st.ks = __ldcg(scale);
        st.vs = __ldcg(scale + a.K * (kBlockPositions / kStreamKeys));
      }
    };
    Step cur, next;
    read(0, entry(0), cur);
    int32_t page = entry(1);
    for (int i = 0; i < count; ++i, ++n) {
      if (i + 1 < count) read(i + 1, page, next);
      page = entry(i + 2);
      if (!wait_for(&free[n % S], ((n / S) & 1) ^ 1, a.status, abort_flag)) return false;
      if (lt == 0 && half == 0) {
        const float l = cur.vs > 0x1p-100f ? log2f(cur.vs) : cur.vs <= 0x1p-100f ? -100.f : cur.vs;
        s.missing[n & 7] = cur.missing;
        *reinterpret_cast<float4*>(s.scales[n & 7]) = make_float4(cur.ks, l, exp2f(-l), 0.f);
      }
      const uint32_t to = (n % S) * Stream<D>::kStepBytes;
#pragma unroll
      for (int k = 0; k < kPasses; ++k) {
        st_shared16(even + to + k * (kStep * 128), f16_of(cur.raw[k].x), f16_of(cur.raw[k].y));
        st_shared16(odd + to + k * (kStep * 128), f16_of(cur.raw[k].z), f16_of(cur.raw[k].w));
      }
      tc::fence_proxy_async();
      tc::mbar_arrive(&full[n % S]);
      cur = next;
    }
    return true;
  }
};

}  // namespace

bool dense_group_ready(int dim) {
  return dim == 64 ? stream_ready<64, GroupCache>() : dim == 128 ? stream_ready<128, GroupCache>()
       : dim == 192 ? stream_ready<192, GroupCache>() : stream_ready<256, GroupCache>();
}

int dense_group(int dim, const DenseAttnDev& d, const SplitDev& p, cudaStream_t stream) {
  switch (dim) {
    case 64: return stream_launch<64, GroupCache>(d, p, stream);
    case 128: return stream_launch<128, GroupCache>(d, p, stream);
    case 192: return stream_launch<192, GroupCache>(d, p, stream);
    default: return stream_launch<256, GroupCache>(d, p, stream);
  }
}

size_t stream_workspace(int dim) { return split_workspace(stream_unit(dim), dim, kSms); }

int stream_plan(const DenseAttnDev& d, int dim, int rows_from, void* ws, SplitDev* out) {
  const int unit = stream_unit(dim);
  SplitDev p{};
  p.RG = int((int64_t(d.max_new) * d.G + unit - 1) / unit);
  p.rows_from = rows_from;
  p.rows_to = INT32_MAX;
  if (rows_from > 0) p.RG = std::max(p.RG, 2);      // sequences of the other launch are not units
  const int64_t units = units_bound(d, rows_from, p.RG, unit);
  if (units > INT32_MAX || units * d.K > INT32_MAX) return V4A_ERR_UNSUPPORTED;
  p.U = int(units);
  // under a window one CTA per unit and KV head, unless the last wave of CTAs is nearly empty (as dense_prefill_plan)
  const int64_t ctas = int64_t(p.U) * d.K, idle = (ctas + kSms - 1) / kSms * kSms - ctas;
  p.split = std::max(p.U, d.B) <= kMaxSplitUnits && (d.window == 0 || idle * (d.window / 128 + 5) > 9 * kSms);
  split_carve(&p, ws, unit, dim, kSms, kStreamCost);
  *out = p;
  return V4A_OK;
}

}  // namespace v4a
