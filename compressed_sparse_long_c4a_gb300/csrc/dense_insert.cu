// Per-head RMSNorm of queries and keys, the position rotation, and the keys'
// and values' insert into the dense paged cache, in one pass
// (v4a_dense.h, v4a_dense_insert).
//
// Mathematics: y = x / sqrt(mean(x^2) + eps) * gamma over a head's dims, then
// pairs (a, b) turn by the angle p f_j.  The angle is formed in turns as a
// 64-bit fraction: F_j = f_j / (2 pi) 2^64 on the host, p F_j mod 2^64 is one
// integer product, and its top 32 bits are the signed fraction of a turn, so
// no fp64 and no range reduction runs on the device and far positions lose
// nothing.
//
// Bound: memory, if the arithmetic keeps out of its way.  Every row is read
// once and written once.  A row is held by dim / 8 lanes, each with two runs of
// four dims: in the half layout a lane takes the two halves of its pairs, so
// the rotation needs no exchange, and its cosines and sines are the same for
// every row that it handles and stay in registers.  The norm
// and the fp8 row maximum are shuffles inside the row's lanes.  A CTA takes one
// token (or part of its rows when tokens are few): its angles are computed once
// and shared by all its heads, and all its loads are issued before the first use.
// Measured, 64 + 8 + 8 heads of 128, one call behind the other: 16384 tokens, bf16
// 123 us (671 MB: 5.5 TB/s of the 6.7 that a copy reaches), fp8 147 us (the row
// maxima and the codes); one token 2.9 us.  With packed keys 129 and 152 us.
//
// A cache with a scale per group takes two launches (v4a_dense_insert_rows): this
// kernel for queries and keys as rows, then dense_quant.cu for the codes, which
// needs all rows of a group at once.
#include <type_traits>

#include "tc_common.cuh"
#include "v4a_dense.h"
#include "v4a_dense_internal.h"

namespace v4a {
namespace {

constexpr int kThreads = 128;     // eight CTAs an SM: 121 us for 16384 tokens of 64 + 8 + 8 heads; four of 256 threads took 124
static_assert(kThreads == 1 << 7, "threads of a token");
constexpr int kPasses = 5;        // rows per lane group held in registers (16 bytes a lane each; 3: 142 us, 10: 147 us)

struct InsertDev {
  uint64_t turn[128];             // F_j: turns per position as a 64-bit fraction
  float magnitude;
  int R, first, half;
  int D, H, K, NR, passes;        // NR = H + 2K rows a token
  int tokens, share;              // T; tokens per CTA, log2
  float eps;
  const int32_t* positions;
  const int64_t* slots;
  const uint16_t *q, *k, *v;
  uint16_t *q_out, *k_out;         // k_out: the keys as packed rows (kPacked)
  int64_t qs, qos, ks, vs, kos;
  const float *qg, *kg;
  uint8_t* pool;
  int64_t num_slots, block_bytes;
  int32_t* status;
};

__device__ __forceinline__ void unpack4(uint2 w, float* x) {
  x[0] = __uint_as_float(w.x << 16);
  x[1] = __uint_as_float(w.x & 0xffff0000u);
  x[2] = __uint_as_float(w.y << 16);
  x[3] = __uint_as_float(w.y & 0xffff0000u);
}
__device__ __forceinline__ uint2 pack4(const float* x) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// kLanes: lanes of one row (dim / 8, or 32 with the last eight idle at dim 192).
// kMode: what the cache gets, bf16 rows, fp8 rows with a scale each, or nothing (values are not read).
// kPacked: the keys go to k_out too (a test of the pointer cost calls without it 4 to 6%: 16384 tokens of 64 + 8 + 8 heads,
// bf16 128 us against 123, fp8 156 against 147).
// kShare: several tokens of few rows in a CTA (the division costs the others 5%: 121 us against 127).
enum { kBf16, kFp8Rows, kRowsOnly };
template <int kLanes, int kMode, bool kPacked, bool kShare>
__global__ void __launch_bounds__(kThreads, 8) dense_insert_kernel(const __grid_constant__ InsertDev p) {
  constexpr bool kFp8 = kMode == kFp8Rows;
  constexpr int kRows = kThreads / kLanes;      // rows per pass
  __shared__ alignas(16) float angles[kShare ? 4 : 1][256];      // of a token: cos [0, R/2), sin [R/2, R)
  // a CTA's threads are divided among its tokens
  const int share = kShare ? p.share : 0, threads = kThreads >> share, rows = kRows >> share;
  const int part = kShare ? threadIdx.x >> (7 - share) : 0, tid = kShare ? threadIdx.x & (threads - 1) : threadIdx.x;
  const int t = (blockIdx.x << share) + part;
  float* const cs = angles[part];
  const int l = tid % kLanes, r0 = blockIdx.y * (rows * p.passes) + tid / kLanes;
  const int D = p.D;
  const bool live = 8 * l < D;
  // this lane's dims: d0 .. d0 + 3 and d1 .. d1 + 3; with `rot` their pairs' cosines start at cs[j]
  int d0 = 8 * l, d1 = 8 * l + 4, j = 0;
  bool rot;
  if (p.half) {
    rot = l < p.R / 8;
    if (rot) {
      j = 4 * l;
      d0 = p.first + j;
      d1 = d0 + p.R / 2;
    } else {                                    // the dims beside the rotated ones, eight at a time
      d0 = 8 * l - p.R;
      if (d0 >= p.first) d0 += p.R;
      d1 = d0 + 4;
    }
  } else {
    rot = d0 >= p.first && d0 < p.first + p.R;
    if (rot) j = (d0 - p.first) / 2;
  }
  rot = rot && live;
  pdl_trigger();
  pdl_wait();
  const bool some = !kShare || t < p.tokens;
  const int64_t slot = some ? p.slots[t] : -1;
  const int P = some ? p.positions[t] : 0;
  uint2 lo[kPasses], hi[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = r0 + i * rows;
    lo[i] = hi[i] = make_uint2(0, 0);
    if (i < p.passes && r < p.NR && live && some) {
      const uint16_t* src = r < p.H ? p.q + int64_t(t) * p.qs + r * D
                            : r < p.H + p.K ? p.k + int64_t(t) * p.ks + (r - p.H) * D
                                            : p.v + int64_t(t) * p.vs + (r - p.H - p.K) * D;
      lo[i] = *reinterpret_cast<const uint2*>(src + d0);
      hi[i] = *reinterpret_cast<const uint2*>(src + d1);
    }
  }
  const bool skip = slot < 0 || slot >= p.num_slots || P < 0;      // all threads of the token
  if (skip && tid == 0 && slot != -1) report(p.status, slot < 0 || slot >= p.num_slots ? V4A_DEV_BAD_BLOCK : V4A_DEV_BAD_BATCH);
  if (!kShare && skip) return;
  for (int i = kShare && skip ? p.R : tid; i < p.R / 2; i += threads) {
    const int32_t frac = int32_t((uint64_t(uint32_t(P)) * p.turn[i]) >> 32);
    float sn, co;
    sincospif(float(frac) * 0x1p-31f, &sn, &co);
    cs[i] = co * p.magnitude;
    cs[p.R / 2 + i] = sn * p.magnitude;
  }
  __syncthreads();
  if (kShare && skip) return;
  float co[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
  if (rot) {
    const float4 c = *reinterpret_cast<const float4*>(cs + j), s = *reinterpret_cast<const float4*>(cs + p.R / 2 + j);
    co[0] = c.x; co[1] = c.y; co[2] = c.z; co[3] = c.w;
    sn[0] = s.x; sn[1] = s.y; sn[2] = s.z; sn[3] = s.w;
  }
  uint8_t* block = p.pool + (slot / kBlockPositions) * p.block_bytes;
  const int at = int(slot % kBlockPositions);
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = r0 + i * rows;
    if (i >= p.passes) break;                    // the same for the whole CTA
    const bool is_q = r < p.H, is_v = r >= p.H + p.K;
    float x[8];
    unpack4(lo[i], x);
    unpack4(hi[i], x + 4);
    const float* gamma = is_q ? p.qg : is_v ? nullptr : p.kg;
    if (gamma) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
      // a group of lanes that shares a row is here together
      const uint32_t group = kLanes == 32 ? 0xffffffffu : ((1u << (kLanes & 31)) - 1u) << ((threadIdx.x & 31) / kLanes * kLanes);
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(group, ss, o);
      const float mean = ss / float(D) + p.eps;
      const float inv = rsqrtf(mean < 0x1p-126f ? 0x1p-126f : mean);     // (squares that small are flushed; a NaN stays one)
      const int at0 = live ? d0 : 0, at1 = live ? d1 : 0;
      const float4 g0 = __ldg(reinterpret_cast<const float4*>(gamma + at0)), g1 = __ldg(reinterpret_cast<const float4*>(gamma + at1));
      x[0] *= inv * g0.x; x[1] *= inv * g0.y; x[2] *= inv * g0.z; x[3] *= inv * g0.w;
      x[4] *= inv * g1.x; x[5] *= inv * g1.y; x[6] *= inv * g1.z; x[7] *= inv * g1.w;
    }
    if (rot && !is_v) {
      auto turn = [](float& u, float& w, float c, float s) {
        const float a = fmaf(-w, s, u * c), b = fmaf(w, c, u * s);
        u = a;
        w = b;
      };
      if (p.half) {
#pragma unroll
        for (int e = 0; e < 4; ++e) turn(x[e], x[4 + e], co[e], sn[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) turn(x[2 * e], x[2 * e + 1], co[e], sn[e]);
      }
    }
    if (kPacked && !is_q && !is_v && live) {
      uint16_t* dst = p.k_out + int64_t(t) * p.kos + (r - p.H) * D;
      *reinterpret_cast<uint2*>(dst + d0) = pack4(x);
      *reinterpret_cast<uint2*>(dst + d1) = pack4(x + 4);
    }
    if (kMode == kRowsOnly && !is_q) continue;
    const int64_t row = int64_t(r - p.H) * kBlockPositions + at;     // keys' heads, then values'
    if (is_q || !kFp8) {
      if (r < p.NR && live) {
        uint16_t* dst = is_q ? p.q_out + int64_t(t) * p.qos + r * D : reinterpret_cast<uint16_t*>(block) + row * D;
        *reinterpret_cast<uint2*>(dst + d0) = pack4(x);
        *reinterpret_cast<uint2*>(dst + d1) = pack4(x + 4);
      }
    } else {
      // row maximum of |x| as bits: a NaN is the largest of them, and makes the
      // row's scale NaN (readers may decode the code itself as a number)
      const uint32_t group = kLanes == 32 ? 0xffffffffu : ((1u << (kLanes & 31)) - 1u) << ((threadIdx.x & 31) / kLanes * kLanes);
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(group, top, o));
      if (r < p.NR && live) {
        // exact divisions: the codes are those of the definition in fp32, but for subnormals, which the
        // library's fast math flushes: a quotient below the smallest normal number would be a scale of zero and
        // the row's zeros 0 / 0, so it is raised to that number (as bits: a NaN and an infinity stay what they are)
        const float s = top ? __uint_as_float(max(__float_as_uint(__fdiv_rn(__uint_as_float(top), 448.f)), 0x00800000u)) : 1.f;
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e >> 2] |= uint32_t(f32_to_e4m3(__fdiv_rn(x[e], s))) << (8 * (e & 3));
        *reinterpret_cast<uint32_t*>(block + row * D + d0) = w[0];
        *reinterpret_cast<uint32_t*>(block + row * D + d1) = w[1];
        if (l == 0) reinterpret_cast<float*>(block + int64_t(2 * p.K) * kBlockPositions * D)[row] = s;
      }
    }
  }
}

bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// The turns per position of each pair; V4A_OK or V4A_ERR_INVALID_ARG.
int fill_rope(const v4a_rope& r, int dim, InsertDev* d) {
  if (r.dims < 0 || r.dims > 256 || r.dims % 16 || r.first < 0 || r.first % 8 || r.first + r.dims > dim) return V4A_ERR_INVALID_ARG;
  d->R = r.dims;
  d->first = r.first;
  d->half = r.layout == V4A_ROPE_HALF;
  d->magnitude = float(r.magnitude);
  if (r.dims == 0) {
    d->half = 0;
    return V4A_OK;
  }
  if (r.layout != V4A_ROPE_INTERLEAVED && r.layout != V4A_ROPE_HALF) return V4A_ERR_INVALID_ARG;
  if (r.scaling < V4A_ROPE_PLAIN || r.scaling > V4A_ROPE_TABLE) return V4A_ERR_INVALID_ARG;
  if (!std::isfinite(d->magnitude)) return V4A_ERR_INVALID_ARG;     // (as the kernel takes it, in fp32)
  if (r.scaling == V4A_ROPE_TABLE ? !r.inv_freq : !(r.theta > 0)) return V4A_ERR_INVALID_ARG;
  if ((r.scaling == V4A_ROPE_LINEAR || r.scaling == V4A_ROPE_YARN) && !(r.factor > 0)) return V4A_ERR_INVALID_ARG;
  if (r.scaling == V4A_ROPE_YARN && (!(r.original > 0) || !(r.beta_fast > r.beta_slow))) return V4A_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925286766559;
  for (int j = 0; j < r.dims / 2; ++j) {
    double f = r.scaling == V4A_ROPE_TABLE ? r.inv_freq[j] : std::pow(r.theta, -2.0 * j / r.dims);
    if (r.scaling == V4A_ROPE_LINEAR) f /= r.factor;
    if (r.scaling == V4A_ROPE_YARN) {
      double g = (r.original * f / two_pi - r.beta_slow) / (r.beta_fast - r.beta_slow);
      g = g < 0 ? 0 : g > 1 ? 1 : g;
      f = f * g + f / r.factor * (1 - g);
    }
    if (!(f >= 0 && f <= two_pi / 2)) return V4A_ERR_INVALID_ARG;     // at most half a turn a position
    d->turn[j] = uint64_t(std::ldexp(f / two_pi, 64));
  }
  return V4A_OK;
}

}  // namespace

int dense_cache_check(const v4a_dense_cache& c, int64_t* block_bytes) {
  if (c.num_kv_heads < 1 || c.num_kv_heads > 1024 || c.num_blocks < 1 || !c.pool) return V4A_ERR_INVALID_ARG;
  if (c.format != V4A_KV_BF16 && c.format != V4A_KV_FP8_TOKEN && c.format != V4A_KV_FP8_GROUP) return V4A_ERR_UNSUPPORTED;
  if (c.dim != 64 && c.dim != 128 && c.dim != 192 && c.dim != 256) return V4A_ERR_UNSUPPORTED;
  const int64_t need = v4a_dense_block_bytes(c.num_kv_heads, c.dim, c.format);
  *block_bytes = c.block_bytes ? c.block_bytes : need;
  if (*block_bytes < need || *block_bytes % 16 || !aligned(c.pool, 16)) return V4A_ERR_INVALID_ARG;
  if (c.num_blocks > INT32_MAX) return V4A_ERR_UNSUPPORTED;
  return V4A_OK;
}

int dense_insert(const v4a_dense_insert_args* a, bool with_rows, uint16_t* k_out, int64_t k_out_stride, cudaStream_t stream) {
  if (!a || a->num_tokens < 0 || a->num_heads < 0 || !(a->eps >= 0.f)) return V4A_ERR_INVALID_ARG;
  if (a->num_heads > 1024) return V4A_ERR_UNSUPPORTED;
  InsertDev d{};
  int rc = dense_cache_check(a->kv, &d.block_bytes);
  if (rc) return rc;
  const bool group = a->kv.format == V4A_KV_FP8_GROUP;
  if (group && !with_rows) return V4A_ERR_UNSUPPORTED;
  const int D = a->kv.dim, K = a->kv.num_kv_heads, H = a->num_heads;
  if (H % K) return V4A_ERR_INVALID_ARG;
  rc = fill_rope(a->rope, D, &d);
  if (rc) return rc;
  if (a->num_tokens == 0) return V4A_OK;
  if (!a->positions || !a->slots || !a->k || !a->v || (H > 0 && (!a->q || !a->q_out))) return V4A_ERR_INVALID_ARG;
  if (!aligned(a->q, 16) || !aligned(a->q_out, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) ||
      !aligned(a->q_gamma, 16) || !aligned(a->k_gamma, 16))
    return V4A_ERR_INVALID_ARG;
  if ((H > 0 && (a->q_stride < int64_t(H) * D || a->q_out_stride < int64_t(H) * D || a->q_stride % 8 || a->q_out_stride % 8)) ||
      a->k_stride < int64_t(K) * D || a->v_stride < int64_t(K) * D || a->k_stride % 8 || a->v_stride % 8)
    return V4A_ERR_INVALID_ARG;
  if (with_rows) {
    if (!k_out || !aligned(k_out, 16) || k_out_stride < int64_t(K) * D || k_out_stride % 8 || (k_out == a->k && k_out_stride != a->k_stride))
      return V4A_ERR_INVALID_ARG;
    d.k_out = k_out;
    d.kos = k_out_stride;
  }
  if (H > 0 && a->q == a->q_out && a->q_stride != a->q_out_stride) return V4A_ERR_INVALID_ARG;
  d.D = D; d.H = H; d.K = K; d.NR = H + (group ? 1 : 2) * K; d.eps = a->eps;
  d.positions = a->positions; d.slots = a->slots;
  d.q = a->q; d.k = a->k; d.v = a->v; d.q_out = a->q_out;
  d.qs = a->q_stride; d.qos = a->q_out_stride; d.ks = a->k_stride; d.vs = a->v_stride;
  d.qg = a->q_gamma; d.kg = a->k_gamma;
  d.pool = static_cast<uint8_t*>(a->kv.pool);
  d.num_slots = a->kv.num_blocks * kBlockPositions;
  d.status = a->status;
  const int lanes = D == 64 ? 8 : D == 128 ? 16 : 32;
  const int rows = kThreads / lanes, need = (d.NR + rows - 1) / rows;
  // few tokens: one pass per CTA, so that a token's rows spread over more SMs (64 + 8 + 8 heads of 128: 4 tokens
  // 2.2 us, five passes a CTA 3.4; 128 tokens 3.7 and 4.1; 256 tokens 5.2 and 5.4; 512 tokens 8.5 and 5.7)
  int y = (need + kPasses - 1) / kPasses;
  if (int64_t(a->num_tokens) * y < 2 * 152) y = need;
  d.passes = (need + y - 1) / y;
  y = (need + d.passes - 1) / d.passes;
  // many tokens of few rows: two or four a CTA while the machine stays full (16384
  // tokens of 4 + 1 + 1 heads of 64: one 20 us, two 13, four 12; 2500 tokens 4.7, 3.9, 4.2)
  d.tokens = a->num_tokens;
  auto passes = [&](int share) { return (d.NR + (rows >> share) - 1) / (rows >> share); };
  while (y == 1 && d.share < 2 && passes(d.share + 1) <= kPasses && a->num_tokens >> (d.share + 1) >= 152 * 8) d.passes = passes(++d.share);
  auto pick = [&](auto mode, auto packed, auto share) {
    constexpr int kMode = decltype(mode)::value;
    constexpr bool kPacked = decltype(packed)::value, kShare = decltype(share)::value;
    return lanes == 8    ? dense_insert_kernel<8, kMode, kPacked, kShare>
           : lanes == 16 ? dense_insert_kernel<16, kMode, kPacked, kShare>
                         : dense_insert_kernel<32, kMode, kPacked, kShare>;
  };
  auto pick_mode = [&](auto share) {
    const std::integral_constant<int, kBf16> bf16;
    const std::integral_constant<int, kFp8Rows> fp8;
    if (group) return pick(std::integral_constant<int, kRowsOnly>{}, std::true_type{}, share);
    if (a->kv.format == V4A_KV_FP8_TOKEN) return with_rows ? pick(fp8, std::true_type{}, share) : pick(fp8, std::false_type{}, share);
    return with_rows ? pick(bf16, std::true_type{}, share) : pick(bf16, std::false_type{}, share);
  };
  auto kern = d.share ? pick_mode(std::true_type{}) : pick_mode(std::false_type{});
  const cudaError_t e = launch_pdl(kern, dim3(unsigned(a->num_tokens + (int64_t(1) << d.share) - 1) >> d.share, y), dim3(kThreads), 0, stream, d);
  rc = e == cudaSuccess && cudaGetLastError() == cudaSuccess ? V4A_OK : V4A_ERR_CUDA;
  return rc == V4A_OK && group ? dense_quant(*a, k_out, k_out_stride, d.block_bytes, stream) : rc;
}

}  // namespace v4a
