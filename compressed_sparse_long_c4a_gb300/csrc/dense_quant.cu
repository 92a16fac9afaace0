// Quantising a dense paged cache as it is written, one scale per group of 64
// positions and KV head (v4a_dense_insert_rows, V4A_KV_FP8_GROUP), and reading
// cached rows back (v4a_dense_read).
//
// Mathematics: the scale is the smallest power of two s with amax / s <= 448,
// so x / s is exact in fp32 and a code is one rounding of x.  A power of two
// costs e4m3 nothing above its subnormals: it moves the exponents.  A group
// fills over many steps; its scale only grows, and rows that are there already
// are then brought to the new scale, code by code (exact but for codes that
// become subnormal: half a step of 2^-9 s each time).
//
// Bound: memory.  The rows of a group (64 x dim bf16, 16 KB at dim 128) lie in a
// CTA's registers between the maximum and the codes, so they are read once.
// Measured: the insert's two launches, 16384 tokens of 64 + 8 + 8 heads of 128 150 us
// (ncu, half of the tokens, each alone: 61 and 25; a CTA waits for its rows and then
// for the maximum, and loading the next plane ahead was slower), 4097 tokens of 64
// dims 27 us, 64 tokens of 16 + 4 + 4 heads 6 (one call behind the other; alone and from cold
// caches 154, 35 and 10.9); the read back of 133 thousand positions of 8 heads of 128
// 133 us (6.1 TB/s of the 6.7 that a copy reaches), of row-scaled ones 136.
#include <algorithm>

#include "tc_common.cuh"
#include "v4a_dense.h"
#include "v4a_dense_internal.h"

namespace v4a {
namespace {

constexpr int kThreads = 128;

struct QuantDev {
  int T, K, tokens, planes;       // of a CTA: tokens among which it looks for groups' first ones; KV heads' keys or values
  const int32_t* positions;
  const int64_t* slots;
  const uint16_t *k, *v;
  int64_t ks, vs, num_slots, block_bytes;
  uint8_t* pool;
};

// Largest finite |x| of two bf16 each, as bf16 bits.
__device__ __forceinline__ uint32_t finite_max(uint32_t top, uint32_t w) {
  const uint32_t m = w & 0x7fff7fffu;
  return __vmaxu2(top, m & ~__vcmpgeu2(m, 0x7f807f80u));
}
// e4m3 codes of four values, low byte first.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n.reg .b16 l, h;\ncvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\ncvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\nmov.b32 %0, {l, h};\n}\n"
      : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
// Two e4m3 codes as f16, exactly.
__device__ __forceinline__ float2 values2(uint32_t codes) {
  uint32_t r;
  asm("{\n.reg .b16 c;\ncvt.u16.u32 c, %1;\ncvt.rn.f16x2.e4m3x2 %0, c;\n}\n" : "=r"(r) : "r"(codes));
  return __half22float2(*reinterpret_cast<const __half2*>(&r));
}
__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// x s with x or the product below 2^-126 kept (the library's fast math would take them as zeros).
__device__ __forceinline__ float times(float x, float s) {
  float r;
  asm("mul.rn.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(s));
  return r;
}
// 2^(field - 127), 0 below the normal numbers.
__device__ __forceinline__ float power(int field) { return __uint_as_float(uint32_t(max(field, 0)) << 23); }

// A CTA takes the groups whose first token of the call is among `tokens` tokens from
// blockIdx.x * tokens on, for `planes` KV heads' keys or values (planes: keys' heads, then values') from blockIdx.y *
// planes on.
template <int D>
__global__ void __launch_bounds__(kThreads) dense_quant_kernel(const __grid_constant__ QuantDev p) {
  constexpr int kChunks = D / 16, kPasses = kGroupPositions * kChunks / kThreads;      // a chunk: 16 elements of a row
  constexpr int kBefore = kGroupPositions - 1;
  __shared__ int64_t slot[kBefore + 8 + kGroupPositions];      // of tokens x0 - kBefore ..; -1: skipped
  __shared__ uint32_t red[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, x0 = blockIdx.x * p.tokens;
  pdl_trigger();
  pdl_wait();
  for (int i = tid; i < kBefore + p.tokens + kGroupPositions; i += kThreads) {
    const int t = x0 - kBefore + i;
    int64_t s = -1;
    if (t >= 0 && t < p.T) {
      s = p.slots[t];
      if (s < 0 || s >= p.num_slots || p.positions[t] < 0) s = -1;      // (reported by the launch before)
    }
    slot[i] = s;
  }
  __syncthreads();
  for (int i = kBefore; i < kBefore + p.tokens; ++i) {
    const int64_t first = slot[i], group = first / kGroupPositions;
    if (first < 0) continue;
    // the group's tokens are among this one and the 63 behind it, if none of the 63 before it is; the rows that they
    // write (every warp by itself)
    auto in_group = [&](int64_t s) { return s >= 0 && s / kGroupPositions == group; };
    const int64_t sa = slot[i + lane], sb = slot[i + 32 + lane];
    if (__any_sync(0xffffffffu, in_group(slot[i - 1 - lane]) || (lane < 31 && in_group(slot[i - 33 - lane])))) continue;
    const bool ma = in_group(sa), mb = in_group(sb);
    const uint32_t member[2] = {__ballot_sync(0xffffffffu, ma), __ballot_sync(0xffffffffu, mb)};      // bit: the token
    uint32_t rows[2];                              // bit r: row r of the group is written
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int ra = int(sa % kGroupPositions), rb = int(sb % kGroupPositions);
      rows[w] = __reduce_or_sync(0xffffffffu, (ma && ra >> 5 == w ? 1u << (ra & 31) : 0u) | (mb && rb >> 5 == w ? 1u << (rb & 31) : 0u));
    }
    const int t0 = x0 - kBefore + i, in_block = int(first % kBlockPositions) / kGroupPositions;
    uint8_t* block = p.pool + first / kBlockPositions * p.block_bytes;
    const bool anew = rows[0] & 1;
    for (int plane = blockIdx.y * p.planes; plane < min(2 * p.K, int(blockIdx.y + 1) * p.planes); ++plane) {
      const int which = plane >= p.K, h = which ? plane - p.K : plane;
      uint8_t* dst = block + (int64_t(plane) * kBlockPositions + in_block * kGroupPositions) * D;
      float* const scale = reinterpret_cast<float*>(block + int64_t(2 * p.K) * kBlockPositions * D) + plane * kGroupsPerBlock + in_block;
      const uint16_t* src = which ? p.v + t0 * p.vs + h * D : p.k + t0 * p.ks + h * D;
      const int64_t stride = which ? p.vs : p.ks;
      const uint32_t old_bits = anew ? 0 : __float_as_uint(*scale);
      uint4 a[kPasses], b[kPasses];
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < kPasses; ++k) {
        const int c = tid + k * kThreads, r = c / kChunks, ch = c % kChunks;
        a[k] = b[k] = make_uint4(0, 0, 0, 0);
        if (member[r >> 5] >> (r & 31) & 1) {
          const uint4* x = reinterpret_cast<const uint4*>(src + r * stride + ch * 16);
          a[k] = x[0];
          b[k] = x[1];
        }
      }
#pragma unroll
      for (int k = 0; k < kPasses; ++k) {
        top = finite_max(finite_max(finite_max(finite_max(top, a[k].x), a[k].y), a[k].z), a[k].w);
        top = finite_max(finite_max(finite_max(finite_max(top, b[k].x), b[k].y), b[k].z), b[k].w);
      }
      top = __reduce_max_sync(0xffffffffu, max(top >> 16, top & 0xffffu));
      if (lane == 0) red[tid >> 5] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) top = max(top, red[w]);
      // exponent fields of the scales: 448 = 1.75 x 2^8, and a bf16's mantissa of 0.75 is 0x60
      const int old = anew ? 1 : min(253, max(1, int(old_bits >> 23 & 0xff)));
      const int now = max(old, max(1, int(top >> 7) - 8 + ((top & 0x7f) > 0x60)));
      if (tid == 0) *scale = power(now);
      if (now > old && !anew) {
        const float shrink = power(127 + old - now);
        for (int c = tid; c < kGroupPositions * kChunks; c += kThreads) {
          const int r = c / kChunks;
          if (rows[r >> 5] >> (r & 31) & 1) continue;
          uint4 w = *reinterpret_cast<const uint4*>(dst + c * 16);
          uint32_t* const u = &w.x;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 x = values2(u[k] & 0xffffu), y = values2(u[k] >> 16);
            u[k] = codes4(x.x * shrink, x.y * shrink, y.x * shrink, y.y * shrink);
          }
          *reinterpret_cast<uint4*>(dst + c * 16) = w;
        }
      }
      const float inv = power(254 - now);
#pragma unroll
      for (int k = 0; k < kPasses; ++k) {
        const int c = tid + k * kThreads, r = c / kChunks, ch = c % kChunks;
        if (!(member[r >> 5] >> (r & 31) & 1)) continue;
        auto four = [&](uint32_t x, uint32_t y) { return codes4(times(lo_of(x), inv), times(hi_of(x), inv), times(lo_of(y), inv), times(hi_of(y), inv)); };
        *reinterpret_cast<uint4*>(dst + int64_t(slot[i + r] % kGroupPositions) * D + ch * 16) =
            make_uint4(four(a[k].x, a[k].y), four(a[k].z, a[k].w), four(b[k].x, b[k].y), four(b[k].z, b[k].w));
      }
      __syncthreads();                             // `red` is read
    }
  }
}

// ---- reading back --------------------------------------------------------------------

constexpr int kReadThreads = 256, kReadRows = 64;

struct ReadDev {
  int N, B, K, D, rows, max_blocks;      // rows: of a CTA
  const int32_t *starts, *first, *bt;
  const uint8_t* pool;
  int64_t num_blocks, block_bytes, ks, vs;
  uint16_t *k, *v;
  int32_t* status;
};

__device__ __forceinline__ uint32_t two(float a, float b) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}

// x s for a code x and a row's scale s, so that rounding the result to bf16 rounds the product once.  The product has 28
// bits, of which fp32 keeps 24; cut off, the last bit set says that it is larger.  That bit may be set for an exact
// product too unless this is a tie of bf16, which takes a scale of at most nine bits: those have exact products (and an
// infinite scale is one of them).  Both neighbours of the product, to see whether it is exact, took 165 us for 132.
__device__ __forceinline__ uint32_t lost_bit(float s) { return (__float_as_uint(s) & 0x7fffu) != 0; }
__device__ __forceinline__ float times_to_odd(float x, float s, uint32_t lost) {
  float r;
  asm("mul.rz.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(s));
  return __uint_as_float(__float_as_uint(r) | lost);
}

// A CTA takes `rows` packed rows, a thread 16 elements of one at a time.
template <int kFmt>
__global__ void __launch_bounds__(kReadThreads) dense_read_kernel(const __grid_constant__ ReadDev p) {
  __shared__ const uint8_t* from[kReadRows];      // the row's block, nullptr: skipped
  __shared__ int at[kReadRows];                   // its row in the block
  const int tid = threadIdx.x, r0 = blockIdx.x * p.rows;
  pdl_trigger();
  pdl_wait();
  if (tid < p.rows) {
    const int r = r0 + tid;
    const uint8_t* block = nullptr;
    if (r < p.N) {
      int lo = -1, hi = p.B;                      // the last sequence that starts at or before row r
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.starts[mid] <= r) lo = mid; else hi = mid;
      }
      if (lo >= 0 && r < p.starts[lo + 1]) {
        const int64_t pos = int64_t(p.first ? p.first[lo] : 0) + (r - p.starts[lo]);
        if (p.starts[lo] < 0 || pos < 0 || pos >= int64_t(p.max_blocks) * kBlockPositions) {
          report(p.status, V4A_DEV_BAD_BATCH);
        } else {
          const int32_t page = p.bt[int64_t(lo) * p.max_blocks + pos / kBlockPositions];
          if (page < 0 || page >= p.num_blocks) report(p.status, V4A_DEV_BAD_BLOCK);
          else block = p.pool + page * p.block_bytes;
          at[tid] = int(pos % kBlockPositions);
        }
      }
    }
    from[tid] = block;
  }
  __syncthreads();
  const int chunks = p.D / 16, per = 2 * p.K * chunks, all = min(p.rows, p.N - r0) * per;
#pragma unroll 2
  for (int i = tid; i < all; i += kReadThreads) {
    const int r = i / per, u = i % per, plane = u / chunks, ch = u % chunks;      // plane: keys' heads, then values'
    const uint8_t* block = from[r];
    if (!block) continue;
    const int64_t row = int64_t(plane) * kBlockPositions + at[r];
    uint4 a, b;
    if constexpr (kFmt == V4A_KV_BF16) {
      const uint4* x = reinterpret_cast<const uint4*>(block + (row * p.D + ch * 16) * 2);
      a = x[0];
      b = x[1];
    } else {
      const uint4 w = *reinterpret_cast<const uint4*>(block + row * p.D + ch * 16);
      const float* scales = reinterpret_cast<const float*>(block + int64_t(2 * p.K) * kBlockPositions * p.D);
      const float s = scales[kFmt == V4A_KV_FP8_GROUP ? row / kGroupPositions : row];
      const uint32_t lost = lost_bit(s);
      auto pair = [&](uint32_t codes) {
        const float2 x = values2(codes);
        // (a code times a power of two is exact)
        return kFmt == V4A_KV_FP8_GROUP ? two(times(x.x, s), times(x.y, s)) : two(times_to_odd(x.x, s, lost), times_to_odd(x.y, s, lost));
      };
      a = make_uint4(pair(w.x & 0xffffu), pair(w.x >> 16), pair(w.y & 0xffffu), pair(w.y >> 16));
      b = make_uint4(pair(w.z & 0xffffu), pair(w.z >> 16), pair(w.w & 0xffffu), pair(w.w >> 16));
    }
    const bool is_v = plane >= p.K;
    uint4* to = reinterpret_cast<uint4*>((is_v ? p.v + (r0 + r) * p.vs + (plane - p.K) * p.D : p.k + (r0 + r) * p.ks + plane * p.D) + ch * 16);
    to[0] = a;
    to[1] = b;
  }
}

}  // namespace

int dense_quant(const v4a_dense_insert_args& a, const uint16_t* k_out, int64_t k_out_stride, int64_t block_bytes, cudaStream_t stream) {
  QuantDev d{};
  d.T = a.num_tokens; d.K = a.kv.num_kv_heads;
  // A CTA takes its tokens' groups one after the other, which suits prompts, where most tokens begin none, and not steps
  // of single tokens, where all do; the host cannot tell them apart.  The insert's two launches with 1, 2 and 8 tokens a
  // CTA, us, 64 + 8 + 8 heads of 128: single tokens, 512 25, 29, 33; 1025 44, 46, 54; 2048 86, 87, 108; 4096 171, 171, 185;
  // one prompt, 600 tokens 11.7, 11.3, 9.9; 1025 16, 15, 14; 2000 27, 24, 24; 4097 51, 45, 43.  Single tokens of 8 + 1 + 1
  // heads of 64, 1024 8, 9, 26; 4096 19, 19, 28.
  d.tokens = a.num_tokens <= 1024 ? 1 : a.num_tokens <= 4096 ? 2 : 8;
  // CTAs without a first token cost their start: with many, each looks once for four planes (the insert's two
  // launches from cold caches, 1, 2, 4, 8 and 16 planes: 16384 tokens, 8 heads of 128, 197, 167, 154, 152 and 165 us; 4097
  // tokens of 64 dims 42, 36, 36, 38 and 44)
  const int64_t blocks = (int64_t(d.T) + d.tokens - 1) / d.tokens;
  d.planes = blocks * 2 * d.K >= 16 * 152 ? 4 : 1;
  d.positions = a.positions; d.slots = a.slots;
  d.k = k_out; d.ks = k_out_stride; d.v = a.v; d.vs = a.v_stride;
  d.num_slots = a.kv.num_blocks * kBlockPositions; d.block_bytes = block_bytes;
  d.pool = static_cast<uint8_t*>(a.kv.pool);
  auto kern = a.kv.dim == 64 ? dense_quant_kernel<64> : a.kv.dim == 128 ? dense_quant_kernel<128>
            : a.kv.dim == 192 ? dense_quant_kernel<192> : dense_quant_kernel<256>;
  const cudaError_t e = launch_pdl(kern, dim3(unsigned(blocks), unsigned((2 * d.K + d.planes - 1) / d.planes)), dim3(kThreads), 0, stream, d);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? V4A_OK : V4A_ERR_CUDA;
}

int dense_read(const v4a_dense_read_args* a, cudaStream_t stream) {
  if (!a || a->num_rows < 0 || a->num_seqs < 0) return V4A_ERR_INVALID_ARG;
  ReadDev d{};
  const int rc = dense_cache_check(a->kv, &d.block_bytes);
  if (rc) return rc;
  const int D = a->kv.dim, K = a->kv.num_kv_heads;
  if (a->kv.max_blocks < 1) return V4A_ERR_INVALID_ARG;
  if (a->kv.max_blocks > (1 << 22)) return V4A_ERR_UNSUPPORTED;
  if (a->num_rows == 0 || a->num_seqs == 0) return V4A_OK;
  if (!a->row_starts || !a->kv.block_table || !a->k || !a->v) return V4A_ERR_INVALID_ARG;
  for (const uint16_t* x : {a->k, a->v})
    if (reinterpret_cast<uintptr_t>(x) & 15) return V4A_ERR_INVALID_ARG;
  for (const int64_t s : {a->k_stride, a->v_stride})
    if (s < int64_t(K) * D || s % 8) return V4A_ERR_INVALID_ARG;
  d.N = a->num_rows; d.B = a->num_seqs; d.K = K; d.D = D; d.max_blocks = a->kv.max_blocks;
  d.starts = a->row_starts; d.first = a->first; d.bt = a->kv.block_table;
  d.pool = static_cast<const uint8_t*>(a->kv.pool); d.num_blocks = a->kv.num_blocks;
  d.k = a->k; d.v = a->v; d.ks = a->k_stride; d.vs = a->v_stride; d.status = a->status;
  // about eight chunks a thread, and few enough rows that all SMs have work
  const int per = 2 * K * (D / 16);
  d.rows = std::max(1, std::min({kReadRows, 8 * kReadThreads / per, d.N / (2 * 152)}));
  auto kern = a->kv.format == V4A_KV_BF16 ? dense_read_kernel<V4A_KV_BF16>
            : a->kv.format == V4A_KV_FP8_TOKEN ? dense_read_kernel<V4A_KV_FP8_TOKEN> : dense_read_kernel<V4A_KV_FP8_GROUP>;
  const cudaError_t e = launch_pdl(kern, dim3(unsigned((int64_t(d.N) + d.rows - 1) / d.rows)), dim3(kReadThreads), 0, stream, d);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? V4A_OK : V4A_ERR_CUDA;
}

}  // namespace v4a
