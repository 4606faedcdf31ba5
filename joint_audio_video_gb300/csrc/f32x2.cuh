// What the attention kernels do with scores in registers: pairs of fp32 in one 64-bit
// register, exponentials, masks.
#pragma once

#include <cstdint>

namespace h3 {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Packed pairs of fp32 in one 64-bit register (low word = first value).
__device__ __forceinline__ uint64_t f2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unf2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t ffma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

constexpr uint32_t kNegInf = 0xFF800000u;

// 32 consecutive columns from `base` on: those outside [lo_rel, hi_rel) become -infinity.
__device__ __forceinline__ void mask32(uint32_t (&r)[32], int base, int lo_rel, int hi_rel) {
#pragma unroll
  for (int c = 0; c < 32; ++c)
    if (c + base < lo_rel || c + base >= hi_rel) r[c] = kNegInf;
}

// Bits lo .. hi - 1 of 32 (none if hi <= lo; lo and hi may lie outside).
__device__ __forceinline__ uint32_t bits32(int lo, int hi) {
  const uint32_t from = lo <= 0 ? 0xffffffffu : lo >= 32 ? 0u : 0xffffffffu << lo;
  const uint32_t to = hi >= 32 ? 0xffffffffu : hi <= 0 ? 0u : ~(0xffffffffu << hi);
  return from & to;
}
// 32 consecutive columns: those whose bit is not set become the value with the bits `fill`.
// The empty statement keeps a branch around the call a branch.
__device__ __forceinline__ void keep32(uint32_t (&r)[32], uint32_t bits, uint32_t fill) {
  asm volatile("" ::: "memory");
#pragma unroll
  for (int c = 0; c < 32; ++c)
    if (!(bits & (1u << c))) r[c] = fill;
}

}  // namespace h3
