// An accumulated sum times the factors of its two rows.
#pragma once

#include <cstdint>

namespace h3 {
namespace {

// Neither vanishing nor large: 2^-62 <= |f| < 2^63.  The product of two such is normal.
__device__ __forceinline__ bool mid_range(float f) {
  return (__float_as_uint(f) & 0x7FFFFFFFu) - (uint32_t(127 - 62) << 23) < uint32_t(62 + 63) << 23;
}

// v a b where a b may leave fp32 although v a b does not: the mantissas' product with v, a small
// v raised first (exactly, also from below the normal numbers), then the exponents' sum at
// once.  For an a b that is a normal number it is v (a b), bit for bit.
__device__ __forceinline__ float times_apart(float v, float a, float b) {
  int ea = 0, eb = 0;
  const float m = frexpf(a, &ea) * frexpf(b, &eb);   // [1/4, 1)
  if (fabsf(v) < 1.f) {
    v *= 0x1p64f;
    ea -= 64;
  }
  return ldexpf(v * m, ea + eb);
}
// The same for v[i], b[i]: seldom needed, so one call for all of them (a call for each cost
// the product for few rows 4 %).
static __device__ __noinline__ void times_apart_n(float* v, int n, float a, const float* b) {
#pragma unroll 1
  for (int i = 0; i < n; ++i) v[i] = times_apart(v[i], a, b[i]);
}

}  // namespace
}  // namespace h3
