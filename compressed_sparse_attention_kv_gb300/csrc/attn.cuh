// What the attention kernels over lists and chunks share: long waits, products issued by one
// lane, and the decoding of 16 dims of a cache row to bf16.
#pragma once

#include "codec.cuh"

namespace cskv {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The hardware suspends a waiting thread for up to about 4 us at a time: a waiting warp takes no
// issue slots from the working ones.
__device__ __forceinline__ bool try_wait_long(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 4000;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
  return ok != 0;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// The issuing lane's MMAs are unrolled with constant descriptor offsets and constant
// accumulate flags: about 40 cycles each, near what a 128 x 64 x 16 product takes; computed
// in a rolled loop, descriptors cost 100 to 190 cycles per MMA whatever its size.
__device__ __forceinline__ bool elect_lane() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void mma_add(uint32_t d, uint64_t da, uint64_t db, uint32_t id) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.eq.u32 p, 0, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(da), "l"(db), "r"(id)
      : "memory");
}
__device__ __forceinline__ void mma_set(uint32_t d, uint64_t da, uint64_t db, uint32_t id) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, 0, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(da), "l"(db), "r"(id)
      : "memory");
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

// ---------------------------------------------------------------------------
// rows: 16 dims of a row from its bytes to bf16, exactly
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t byte_of(uint32_t w, int i) { return (w >> (8 * i)) & 0xFFu; }

// x * y on two bf16 (rounded to nearest, subnormals kept)
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
// two fp16 to two bf16 (through fp32)
__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t h) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf16(f.x, f.y);
}
// e4m3 pairs to fp16 and to bf16 (4 significant bits: exact), times the block's scale 2^e
// (one rounding, where bf16 does not hold the value)
__device__ __forceinline__ void convert(const uint4& r, uint32_t scale, uint32_t (&w)[8]) {
  const uint32_t f = scale == 0u ? 0x0040u : scale << 7, ff = f | (f << 16);   // 255: infinite
  const uint32_t c[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(c[i]));
    w[2 * i] = mul_bf16x2(f16x2_to_bf16x2(lo), ff);
    w[2 * i + 1] = mul_bf16x2(f16x2_to_bf16x2(hi), ff);
  }
}
// e2m1 pairs to fp16, times the e4m3 scale (6 significant bits, 2^-10 .. 2688: exact in fp16
// and in bf16)
__device__ __forceinline__ void convert(const uint2& r, uint32_t scale, uint32_t (&w)[8]) {
  uint32_t s2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s2) : "h"(static_cast<uint16_t>(scale * 0x0101u)));
  const uint32_t c[2] = {r.x, r.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\tcvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(c[i]));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(h[j]) : "r"(h[j]), "r"(s2));
      w[4 * i + j] = f16x2_to_bf16x2(h[j]);
    }
  }
}

}  // namespace cskv
