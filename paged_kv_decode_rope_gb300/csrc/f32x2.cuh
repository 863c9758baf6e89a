// f32x2.cuh -- paired fp32 arithmetic and the other fp32 helpers of sm_100 and
// later that the streaming kernels share.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace pkv {

// Two fp32 values in one 64-bit register, and the paired fp32 arithmetic of
// sm_100 and later (each half rounded exactly as the scalar operation).
__device__ __forceinline__ uint64_t f32x2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack_f32x2(uint64_t v) {
  float a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
  return make_float2(a, b);
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t sub_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// p0 - h.lo and p1 - h.hi for the two bf16 halves of h, each in one
// mixed-precision fma (bf16 times bf16 -1, plus fp32; sm_100 and later):
// exact when h is p rounded to bf16, so the remainder of the split
__device__ __forceinline__ float2 bf16x2_remainder(uint32_t h, float p0, float p1) {
  float r0, r1;
  asm("{\n\t.reg .b16 h0, h1, m1;\n\t"
      "mov.b32 {h0, h1}, %2;\n\t"
      "mov.b16 m1, 0xBF80;\n\t"
      "fma.rn.f32.bf16 %0, h0, m1, %3;\n\t"
      "fma.rn.f32.bf16 %1, h1, m1, %4;\n\t}"
      : "=f"(r0), "=f"(r1)
      : "r"(h), "f"(p0), "f"(p1));
  return make_float2(r0, r1);
}

// max of three floats in one instruction (sm_100 and later)
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

}  // namespace pkv
