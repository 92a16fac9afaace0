// Attention of whole packed prompts over packed keys and values
// (v4a_dense.h, v4a_prompt_attn): dense_stream.cuh over bf16 rows.
//
// Keys and values come by TMA (a box of a step's rows x 64 dims of one head lands in
// the 128-byte swizzle that the MMA reads), but for a step that reaches past
// its sequence: its rows behind the last are zeros, so that the next
// sequence's cannot reach a product, and are copied by the warp.
//
// Bound: 4 dim flops per visible pair on the tensor cores, which are 63% busy (ncu,
// 4096 tokens; XU pipe 32%, DRAM 7%): dense_stream.cuh says what the rest is.
// Measured alone (calls one behind the other heat the GPU: the longest takes 1413 us
// then, 1556 TFLOP/s), 32 + 8 heads of 128: 16384 tokens 1292 us (1702 TFLOP/s), 4096 104
// us (1316), 16 prompts of 1000 to 3000 447 (1340), 64 of 1 to 256 (16 + 4 heads) 37 us; 16 +
// 4 heads of 256, 8192 tokens 412 us (1336), of 192 326 (1266); heads of 64, 16384 tokens
// 1141 us (964: half of the flops for the same softmax); 8 prompts of 1000 to 4096, 64 + 8
// heads of 64, window 1024 575 us (660, of which masks take about 40 us).
#include "dense_stream.cuh"

namespace v4a {
namespace {

struct PromptDev : DenseAttnDev {
  const int32_t* kv_starts;
  int Tk, causal;
  int64_t qs, ks, vs;               // elements between tokens
  const uint16_t *k, *v;
  CUtensorMap km, vm;               // [Tk][K][dim]
  CUtensorMap qm;                   // [T][K][G][dim]
  int q_copied;
};

// One sequence's rows: p0 is its first row's position among its keys (not causal: every row's, the last key's).
__device__ __forceinline__ SeqRun seq_run(const PromptDev& a, int64_t rows_from, int64_t rows_to, bool, int b, int32_t* status) {
  const int s0 = a.starts[b], s1 = a.starts[b + 1], k0 = a.kv_starts[b], k1 = a.kv_starts[b + 1];
  SeqRun r{s0, 0, 0};
  if (s0 == s1 && s0 >= 0 && s1 <= a.T) return r;
  if (s0 >= 0 && s1 > s0 && s1 <= a.T && s1 - s0 <= a.max_new && k0 >= 0 && k1 >= k0 && k1 <= a.Tk) {
    r.n = s1 - s0;
    r.p0 = (k1 - k0) - (a.causal ? s1 - s0 : 1);
  } else {
    report(status, V4A_DEV_BAD_BATCH);
  }
  return r;
}

__device__ __forceinline__ bool one_position(const PromptDev& a) { return !a.causal; }

template <int R, int kTile>
__device__ __forceinline__ Unit<kTile> make_unit(const PromptDev& a, const UnitRef& f) {
  Unit<kTile> u{f.b, 0, 0, f.s0, 0, 0, {0, 0, 0}};
  if (f.last < 0) return u;
  u.row0 = f.last & ~(R - 1);
  u.rows = f.last - u.row0 + 1;
  u.m_lo = f.p0 + (a.causal ? u.row0 / a.G : 0);
  u.m_hi = f.p0 + (a.causal ? f.last / a.G : 0);
  u.tr = tile_range<kTile>(a, max(u.m_lo, 0), max(u.m_hi, 0));      // (rows without a key have one step, of zeros)
  return u;
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(tc::smem_u32(bar))
      : "memory");
}

struct PackedRows {
  using Dev = PromptDev;
  static constexpr bool kScaled = false, kPaged = false;
  template <int D> static constexpr int copiers() { return 64; }       // a warp for the keys, one for the values
  template <int D> static constexpr int key_stages() { return D == 64 ? 4 : D == 192 ? 3 : 2; }
  template <int D> static constexpr int value_stages() { return key_stages<D>(); }
  template <int D> static constexpr int key_bytes() { return Stream<D>::kStepBytes; }
  template <int D> static constexpr int extra_bytes() { return 0; }
  template <int D> static constexpr int value_arrivals() { return 1; }

  template <int kKeys>
  static __device__ __forceinline__ int row_position(const Dev& a, const Unit<kKeys>& un, int row) {
    return un.m_lo + (a.causal ? (un.row0 % a.G + row) / a.G : 0);
  }

  template <int D>
  static __device__ __forceinline__ void scores(uint32_t st, uint32_t qa, uint32_t kb) {
    constexpr int kKeys = Stream<D>::kKeys;
    constexpr uint32_t idesc = tc::make_idesc(1, 1, kTileRows, kKeys);
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
      tc::mma_f16(st, tc::desc_sw128(qa + (k >> 2) * (kTileRows * 128)) + 2 * (k & 3),
                  tc::desc_sw128(kb + (k >> 2) * (kKeys * 128)) + 2 * (k & 3), idesc, k > 0);
  }

  // Rows are (token, head of the group) pairs: where a group divides a tile, a tile's are a box.
  static __device__ __forceinline__ bool q_copied(const Dev& a) { return a.q_copied != 0; }

  template <int D>
  struct Feed {
    using W = Stream<D>;
    const Dev& a;
    uint8_t* base;
    StreamSmem& s;
    int tiles[2] = {0, 0};
    __device__ __forceinline__ Feed(const Dev& a_, uint8_t* base_, StreamSmem& s_) : a(a_), base(base_), s(s_) {}
    __device__ __forceinline__ bool begin(const Unit<W::kKeys>& un, int hk, int, int, int n) {
      if (!a.q_copied) return true;
      // Q is free when the unit before's last scores, the last to read its keys, are there
      constexpr int SK = key_stages<D>();
      const bool ok = n == 0 || wait_for(&s.k_free[(n - 1) % SK], ((n - 1) / SK) & 1, a.status, &s.abort_flag);
      if (!__all_sync(0xffffffffu, ok)) return false;
#pragma unroll
      for (int t = 0; t < W::kTiles; ++t) {
        if (un.rows <= t * kTileRows) continue;
        if ((threadIdx.x & 31) == 0) {
          tc::mbar_arrive_expect_tx(&s.q_full[t], W::kQBytes);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(base + t * W::kQBytes + c * (kTileRows * 128), &a.qm, 64 * c, 0, hk, un.s0 + (un.row0 + t * kTileRows) / a.G, &s.q_full[t]);
        }
        ++tiles[t];
      }
      return true;
    }
    __device__ __forceinline__ bool step(int, int) { return true; }
    __device__ __forceinline__ void drain() {
      if (!a.q_copied) return;
#pragma unroll
      for (int t = 0; t < W::kTiles; ++t)
        if (tiles[t]) drain_copies(&s.q_full[t], 1, tiles[t]);
    }
  };

  template <int D>
  static __device__ __forceinline__ float load_q(const Dev& a, const Unit<Stream<D>::kKeys>& un, int hk, int t, int r, uint32_t q0) {
#pragma unroll 4
    for (int c = r; c < kTileRows * (D / 8); c += kTileRows) {
      const int qr = c / (D / 8), ch = c % (D / 8), row = t * kTileRows + qr, i = un.row0 + min(row, un.rows - 1);
      const uint16_t* q = a.q + (un.s0 + i / a.G) * a.qs + (hk * a.G + i % a.G) * D;
      copy16(q0 + stream_chunk<kTileRows>(qr, ch), q + ch * 8, row < un.rows);
    }
    tc::cp_async_wait_all();
    return a.scale_log2;
  }

  // Keys (the first warp) or values of `count` steps from tile `tile` of the unit on, step n of the CTA first.
  template <int D>
  static __device__ __forceinline__ bool copy(const Dev& a, const Unit<Stream<D>::kKeys>& un, int hk, int tile, int count, int n, int lt,
                                              uint8_t* base, StreamSmem& s) {
    using L = StreamLayout<D, PackedRows>;
    constexpr int S = key_stages<D>(), kKeys = Stream<D>::kKeys;
    const int half = lt / 32, lane = lt % 32;
    uint8_t* const buffers = base + (half ? L::kValues : L::kKeys);
    const int k0 = a.kv_starts[un.b], nk = a.kv_starts[un.b + 1] - k0;
    const CUtensorMap* map = half ? &a.vm : &a.km;
    const uint16_t* rows = half ? a.v : a.k;
    const int64_t stride = half ? a.vs : a.ks;
    uint64_t* const full = half ? s.v_full : s.k_full;
    uint64_t* const free = half ? s.v_free : s.k_free;
    volatile int* abort_flag = &s.abort_flag;
    for (int i = 0; i < count; ++i, ++n) {
      if (!__all_sync(0xffffffffu, wait_for(&free[n % S], ((n / S) & 1) ^ 1, a.status, abort_flag))) {
        drain_copies(full, S, n);
        return false;
      }
      uint8_t* const to = buffers + (n % S) * Stream<D>::kStepBytes;
      const int j0 = un.tr.at(tile + i) * kKeys;
      if (j0 + kKeys <= nk) {
        if (lane == 0) {
          tc::mbar_arrive_expect_tx(&full[n % S], Stream<D>::kStepBytes);
#pragma unroll
          for (int c = 0; c < D / 64; ++c) tc::tma_load_3d(to + c * (kKeys * 128), map, 64 * c, hk, k0 + j0, &full[n % S]);
        }
      } else {
        const uint32_t dst = tc::smem_u32(to);
#pragma unroll 4
        for (int c = lane; c < kKeys * (D / 8); c += 32) {
          const int r = c / (D / 8), ch = c % (D / 8);
          const bool live = j0 + r < nk;
          copy16(dst + stream_chunk<kKeys>(r, ch), rows + (live ? (int64_t(k0) + j0 + r) * stride + hk * D + ch * 8 : 0), live);
        }
        tc::cp_async_wait_all();
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&full[n % S]);
      }
    }
    return true;
  }
};

// A map of [rows][heads][dim] whose boxes are a step's rows x 64 dims of one head.
bool make_map(CUtensorMap* map, const uint16_t* rows, int64_t n, int heads, int dim, int64_t stride) {
  auto fn = tc::encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {cuuint64_t(dim), cuuint64_t(heads), cuuint64_t(n)};
  const cuuint64_t strides[2] = {cuuint64_t(dim) * 2, cuuint64_t(stride) * 2};
  const cuuint32_t box[3] = {64, 1, cuuint32_t(dim <= 128 ? 128 : 64)}, step[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(rows), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A map of queries [tokens][KV heads][group][dim] whose boxes are a tile's rows x 64 dims of one KV head.
bool make_q_map(CUtensorMap* map, const PromptDev& d, int dim) {
  auto fn = tc::encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {cuuint64_t(dim), cuuint64_t(d.G), cuuint64_t(d.K), cuuint64_t(d.T)};
  const cuuint64_t strides[3] = {cuuint64_t(dim) * 2, cuuint64_t(d.G) * dim * 2, cuuint64_t(d.qs) * 2};
  const cuuint32_t box[4] = {64, cuuint32_t(d.G), 1, cuuint32_t(kTileRows / d.G)}, step[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t*>(d.q), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool ready(int dim) {
  return dim == 64 ? stream_ready<64, PackedRows>() : dim == 128 ? stream_ready<128, PackedRows>()
       : dim == 192 ? stream_ready<192, PackedRows>() : stream_ready<256, PackedRows>();
}

// Everything but the pointers of the call's own tensors.
int check_shape(const v4a_prompt_attn_args* a) {
  if (!a || a->num_tokens < 0 || a->num_kv_tokens < 0 || a->num_seqs < 0 || a->max_new_per_seq < 1 || a->num_heads < 1 || a->num_kv_heads < 1 ||
      a->window < 0 || a->sinks < 0 || a->causal < 0 || a->causal > 1 || (a->window > 0 && !a->causal))
    return V4A_ERR_INVALID_ARG;
  if (a->num_heads % a->num_kv_heads) return V4A_ERR_INVALID_ARG;
  if (a->dim != 64 && a->dim != 128 && a->dim != 192 && a->dim != 256) return V4A_ERR_UNSUPPORTED;
  if (a->num_heads > 1024 || a->max_new_per_seq > (1 << 22) || a->num_kv_tokens > (1 << 30)) return V4A_ERR_UNSUPPORTED;
  if (int64_t(a->max_new_per_seq) * (a->num_heads / a->num_kv_heads) > INT32_MAX / 2) return V4A_ERR_UNSUPPORTED;   // rows are counted in 32 bits
  return V4A_OK;
}

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool row_stride(int64_t stride, int heads, int dim) {
  return stride >= int64_t(heads) * dim && stride % 8 == 0 && stride < (int64_t(1) << 38);      // (a tensor map's strides are below 2^40 bytes)
}

}  // namespace

size_t prompt_attn_workspace_size(const v4a_prompt_attn_args* a) { return check_shape(a) ? 0 : stream_workspace(a->dim); }

int prompt_attn(const v4a_prompt_attn_args* a, void* ws, size_t ws_bytes, cudaStream_t stream) {
  int rc = check_shape(a);
  if (rc) return rc;
  if (!(a->softmax_scale > 0.f) || !std::isfinite(a->softmax_scale * 1.4426950408889634f)) return V4A_ERR_INVALID_ARG;
  if (a->num_tokens == 0 || a->num_seqs == 0) return V4A_OK;
  if (!a->token_starts || !a->q || !a->out || !aligned(a->q) || !aligned(a->out) || static_cast<const void*>(a->q) == a->out)
    return V4A_ERR_INVALID_ARG;
  if (!row_stride(a->q_stride, a->num_heads, a->dim)) return V4A_ERR_INVALID_ARG;
  if (a->num_kv_tokens > 0 && (!a->k || !a->v || !aligned(a->k) || !aligned(a->v) || !row_stride(a->k_stride, a->num_kv_heads, a->dim) ||
                               !row_stride(a->v_stride, a->num_kv_heads, a->dim)))
    return V4A_ERR_INVALID_ARG;
  if (!ws || !aligned(ws) || ws_bytes < stream_workspace(a->dim)) return V4A_ERR_WORKSPACE;
  PromptDev d{};
  d.T = a->num_tokens; d.B = a->num_seqs; d.H = a->num_heads; d.K = a->num_kv_heads; d.G = d.H / d.K;
  d.max_new = a->max_new_per_seq; d.sinks = a->sinks; d.causal = a->causal; d.Tk = a->num_kv_tokens;
  d.window = a->window < a->num_kv_tokens ? a->window : 0;       // one as long as the keys hides nothing
  d.starts = a->token_starts; d.kv_starts = a->kv_starts ? a->kv_starts : a->token_starts;
  d.q = a->q; d.k = d.Tk ? a->k : a->q; d.v = d.Tk ? a->v : a->q;      // (no keys: nothing is read there)
  d.qs = a->q_stride; d.ks = a->k_stride; d.vs = a->v_stride;
  d.out = a->out; d.lse = a->lse; d.status = a->status;
  d.scale_log2 = std::max(a->softmax_scale * 1.4426950408889634f, 0x1p-126f);      // (a subnormal one would be flushed)
  SplitDev p{};
  rc = stream_plan(d, a->dim, 0, (int64_t(d.Tk) + d.B - 1) / d.B, d.causal != 0, ws, &p);
  if (rc) return rc;
  if (a->num_kv_tokens > 0 && (!make_map(&d.km, a->k, d.Tk, d.K, a->dim, d.ks) || !make_map(&d.vm, a->v, d.Tk, d.K, a->dim, d.vs))) return V4A_ERR_CUDA;
  d.q_copied = kTileRows % d.G == 0;
  if (d.q_copied && !make_q_map(&d.qm, d, a->dim)) return V4A_ERR_CUDA;
  if (!ready(a->dim)) return V4A_ERR_CUDA;
  switch (a->dim) {
    case 64: rc = stream_launch<64, PackedRows>(d, p, stream); break;
    case 128: rc = stream_launch<128, PackedRows>(d, p, stream); break;
    case 192: rc = stream_launch<192, PackedRows>(d, p, stream); break;
    default: rc = stream_launch<256, PackedRows>(d, p, stream);
  }
  return rc == V4A_OK && p.split == 1 ? dense_join(d, p, a->dim, stream) : rc;
}

}  // namespace v4a
