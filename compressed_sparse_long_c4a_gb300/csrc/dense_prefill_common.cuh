// What the tensor-core forms of the dense attention share (dense_prefill.cu,
// dense_prefill_wide.cu): TMEM access, waits, copies and conversions.
#pragma once
#include "dense_attn_common.cuh"

namespace v4a {

// Log2 units by which logits may pass the maximum in use before it is raised:
// with 0 the accumulator is rescaled whenever a maximum grows (269 us instead
// of 258; mean relative error 0.0020 instead of 0.0024, since the largest
// weight is then exactly one).  The bound is the same half step of each weight:
// a float's relative step does not depend on its size.
constexpr float kRaise = 8.f;
// f16 P has 2^-14 as its smallest normal value, so it is held at 2^11 2^{w - m}
// <= 2^15: weights down to 2^-25 of the largest are rounded to 11 bits.
constexpr float kRaiseFp8 = 4.f, kShiftFp8 = 11.f;

// MN-major operand (as in attn_tc.cu): 64-element rows along N, 8-row groups
// 1024 bytes apart, the next 64 columns `lbo` bytes further.
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t lbo) {
  return uint64_t((saddr & 0x3FFFFu) >> 4) | (uint64_t((lbo >> 4) & 0x3FFFu) << 16) | (uint64_t(1024 >> 4) << 32) |
         (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// D += A B with A in TMEM (bf16 pairs, one row per lane).
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 32 lanes x 32 columns of 32 bits into TMEM (not waited for).
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};\n" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
      "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
      "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
        "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// tc::mbar_wait with a suspending test: the waiting warps here would otherwise
// poll shared memory against the copies and the tensor cores' operand reads
// (2k tokens over 10k: 269 us polling, 256 us suspended).
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, int32_t* status, volatile int* abort_flag) {
  if (tc::mbar_test(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (tc::mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > 4000000000LL) {
      report(status, V4A_DEV_TIMEOUT);
      *abort_flag = 1;
      return false;
    }
  }
}

// 16 bytes global -> shared, or zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

// Arrives on `bar` when this thread's copies so far have landed.
__device__ __forceinline__ void arrive_copies(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}

// (x, y) * (f, f) + (b, b), (x, y) + (u, v): one instruction for two values.
__device__ __forceinline__ float2 fma2(float2 x, float2 f, float2 b) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r) : "l"(*reinterpret_cast<uint64_t*>(&x)), "l"(*reinterpret_cast<uint64_t*>(&f)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(*reinterpret_cast<uint64_t*>(&x)), "l"(*reinterpret_cast<uint64_t*>(&y)));
  return *reinterpret_cast<float2*>(&r);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Four e4m3 codes as bf16, exactly: the code's bits in place of a bf16's, with
// the exponent biased by 127 instead of 7, times 2^120 (subnormal codes too).
__device__ __forceinline__ uint2 bf16_of(uint32_t w) {
  const uint32_t a = __byte_perm(w, 0u, 0x1404), b = __byte_perm(w, 0u, 0x3424);
  const uint32_t ma = ((a >> 4) & 0x07F007F0u) | (a & 0x80008000u), mb = ((b >> 4) & 0x07F007F0u) | (b & 0x80008000u);
  uint2 r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r.x) : "r"(ma), "r"(0x7B807B80u));
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r.y) : "r"(mb), "r"(0x7B807B80u));
  return r;
}
// ... and as f16.
__device__ __forceinline__ uint2 f16_of(uint32_t w) {
  uint2 r;
  asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\ncvt.rn.f16x2.e4m3x2 %0, l;\ncvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
      : "=r"(r.x), "=r"(r.y) : "r"(w));
  return r;
}
__device__ __forceinline__ void st_shared16(uint32_t dst, uint2 lo, uint2 hi) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(lo.x), "r"(lo.y), "r"(hi.x), "r"(hi.y) : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// The form for dim 192 and 256 (dense_prefill_wide.cu).
constexpr int kWideUnit = 128;       // rows of a unit
// Steps that a unit's set-up and output take the time of (a chunk of 4096 tokens, 16 + 4 heads of 256: 3 steps 233
// us, 6 175, 12 183).
constexpr int kWideUnitCost = 6;
bool dense_prefill_wide_ready(int dim, bool fp8);
int dense_prefill_wide(int dim, bool fp8, const DenseAttnDev& d, const SplitDev& p, cudaStream_t stream);

}  // namespace v4a
