// Attention of whole packed prompts over packed keys and values
// (v4a_dense.h, v4a_prompt_attn): dense_stream.cuh over bf16 rows.
//
// Keys and values come by TMA (a box of 64 rows x 64 dims of one head lands in
// the 128-byte swizzle that the MMA reads), but for a step that reaches past
// its sequence: its rows behind the last are zeros, so that the next
// sequence's cannot reach a product, and are copied by the warp.
#include "dense_stream.cuh"

namespace v4a {
namespace {

struct PromptDev : DenseAttnDev {
  const int32_t* kv_starts;
  int Tk, causal;
  int64_t qs, ks, vs;               // elements between tokens
  const uint16_t *k, *v;
  CUtensorMap km, vm;               // [Tk][K][dim]
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

struct PackedRows {
  using Dev = PromptDev;
  static constexpr bool kScaled = false, kPaged = false;
  template <int D>
  static constexpr int loaders() { return 32; }
  template <int D>
  static constexpr int threads() { return Stream<D>::kSoftmax + 32 + 64; }
  template <int D>
  static constexpr int arrivals() { return 1; }

  static __device__ __forceinline__ int row_position(const Dev& a, const Unit<kStreamKeys>& un, int row) {
    return un.m_lo + (a.causal ? (un.row0 % a.G + row) / a.G : 0);
  }

  template <int D>
  static __device__ __forceinline__ float load_q(const Dev& a, const Unit<kStreamKeys>& un, int hk, int t, int r, uint32_t q0) {
#pragma unroll 4
    for (int c = r; c < kTileRows * (D / 8); c += kTileRows) {
      const int qr = c / (D / 8), ch = c % (D / 8), row = t * kTileRows + qr, i = un.row0 + min(row, un.rows - 1);
      const uint16_t* q = a.q + (un.s0 + i / a.G) * a.qs + (hk * a.G + i % a.G) * D;
      copy16(q0 + stream_chunk<kTileRows>(qr, ch), q + ch * 8, row < un.rows);
    }
    tc::cp_async_wait_all();
    return a.scale_log2;
  }

  template <int D>
  static __device__ __forceinline__ bool copy(const Dev& a, const Unit<kStreamKeys>& un, int hk, int tile, int count, int n, int half, int lane,
                                              uint8_t* buffers, StreamSmem& s) {
    constexpr int S = Stream<D>::kStages;
    const int k0 = a.kv_starts[un.b], nk = a.kv_starts[un.b + 1] - k0;
    const CUtensorMap* map = half ? &a.vm : &a.km;
    const uint16_t* rows = half ? a.v : a.k;
    const int64_t stride = half ? a.vs : a.ks;
    uint64_t* const full = half ? s.v_full : s.k_full;
    uint64_t* const free = half ? s.v_free : s.k_free;
    volatile int* abort_flag = &s.abort_flag;
    for (int i = 0; i < count; ++i, ++n) {
      if (!__all_sync(0xffffffffu, wait_for(&free[n % S], ((n / S) & 1) ^ 1, a.status, abort_flag))) return false;
      uint8_t* const to = buffers + (n % S) * Stream<D>::kStepBytes;
      const int j0 = un.tr.at(tile + i) * kStreamKeys;
      if (j0 + kStreamKeys <= nk) {
        if (lane == 0) {
          tc::mbar_arrive_expect_tx(&full[n % S], Stream<D>::kStepBytes);
#pragma unroll
          for (int c = 0; c < D / 64; ++c) tc::tma_load_3d(to + c * (kStreamKeys * 128), map, 64 * c, hk, k0 + j0, &full[n % S]);
        }
      } else {
        const uint32_t dst = tc::smem_u32(to);
#pragma unroll 4
        for (int c = lane; c < kStreamKeys * (D / 8); c += 32) {
          const int r = c / (D / 8), ch = c % (D / 8);
          const bool live = j0 + r < nk;
          copy16(dst + stream_chunk<kStreamKeys>(r, ch), rows + (live ? (int64_t(k0) + j0 + r) * stride + hk * D + ch * 8 : 0), live);
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

// A map of [rows][heads][dim] whose boxes are 64 rows x 64 dims of one head.
bool make_map(CUtensorMap* map, const uint16_t* rows, int64_t n, int heads, int dim, int64_t stride) {
  auto fn = tc::encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {cuuint64_t(dim), cuuint64_t(heads), cuuint64_t(n)};
  const cuuint64_t strides[2] = {cuuint64_t(dim) * 2, cuuint64_t(stride) * 2};
  const cuuint32_t box[3] = {64, 1, kStreamKeys}, step[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(rows), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
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
  rc = stream_plan(d, a->dim, 0, ws, &p);
  if (rc) return rc;
  if (a->num_kv_tokens > 0 && (!make_map(&d.km, a->k, d.Tk, d.K, a->dim, d.ks) || !make_map(&d.vm, a->v, d.Tk, d.K, a->dim, d.vs))) return V4A_ERR_CUDA;
  if (!ready(a->dim)) return V4A_ERR_CUDA;
  switch (a->dim) {
    case 64: rc = stream_launch<64, PackedRows>(d, p, stream); break;
    case 128: rc = stream_launch<128, PackedRows>(d, p, stream); break;
    case 192: rc = stream_launch<192, PackedRows>(d, p, stream); break;
    default: rc = stream_launch<256, PackedRows>(d, p, stream);
  }
  return rc == V4A_OK && p.split ? dense_join(d, p, a->dim, stream) : rc;
}

}  // namespace v4a
