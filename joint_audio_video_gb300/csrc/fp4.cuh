// Microscaled 4-bit values: E2M1 codes with one scale for a block of columns.
//   H3_FP4_MX  blocks of 32, scale 2^k (E8M0),  k = min{k : amax <= 6 2^k}
//   H3_FP4_NV  blocks of 16, scale E4M3(amax / (6 2^e)), with one 2^e for the row,
//              e = min{e : row amax <= 2688 2^e}   (2688 = 6 x 448)
// A thread owns 16 consecutive columns: half an MX block or one NV block.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/h3attn_lowp.h"
#include "ptx.cuh"

namespace h3 {
namespace {

constexpr uint32_t kInfBits = 0x7F800000u;

template <int FMT>
__host__ __device__ constexpr int fp4_block() { return FMT == H3_FP4_MX ? 32 : 16; }

__device__ __forceinline__ float pow2f(int e) {   // -126 <= e <= 127
  return __uint_as_float(uint32_t(e + 127) << 23);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// E2M1 codes of v[0..7] (to nearest even, 6 at most), v[0] in the lowest nibble.
__device__ __forceinline__ uint32_t e2m1x8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
// The two values of code byte i of w, as halves.
template <int I>
__device__ __forceinline__ __half2 e2m1_pair(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b%2;\n\t}"
      : "=r"(r)
      : "r"(w), "n"(I));
  return *reinterpret_cast<__half2*>(&r);
}
// An E4M3 byte of a value >= 0 (to nearest even, 448 at most), and back.
__device__ __forceinline__ uint32_t e4m3_byte(float v) {
  uint16_t q;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(q) : "f"(0.f), "f"(v));
  return q & 0xFFu;
}
__device__ __forceinline__ float e4m3_value(uint32_t b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(b)));
  return __low2float(*reinterpret_cast<__half2*>(&h));
}

// Exponent of the row factor of an NV row whose largest finite |x| has these bits.
// 2688 = 1.3125 x 2^11, so e = E - 11 for a mantissa up to 1.3125, else E - 10.
__device__ __forceinline__ int nv_row_exponent(uint32_t amax_bits) {
  if (amax_bits == 0) return 0;
  const int E = int(amax_bits >> 23) - 127;
  const int e = (amax_bits & 0x7FFFFFu) <= 0x280000u ? E - 11 : E - 10;
  return e < -117 ? -117 : e;   // 1 / (scale 2^e) stays below 2^127
}

struct BlockScale {
  uint32_t byte;   // as stored
  float inv;       // 1 / (scale x row factor); 0 for a scale of 0 or NaN
};
// Scale of a block whose largest |x| has these bits (infinity or NaN included);
// `e` is the row's exponent (NV).  amax / 6 and 1 / scale are products with, and an
// approximation of, an inverse, within 2^-22.  For a bf16 amax (8 significant bits) that
// changes no scale: 6 x a value half way between two E4M3 values has at most 7 bits, so a
// quotient that is no tie is 2^-8 of it away from one, and rounded to 12 bits first a true
// tie is met exactly.  quantize16 says the same of the codes.
template <int FMT, bool SNAP>
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits, int e) {
  BlockScale s;
  const bool bad = amax_bits >= kInfBits;
  if constexpr (FMT == H3_FP4_MX) {
    // 6 = 1.5 x 2^2
    int k = int(amax_bits >> 23) - 127 - ((amax_bits & 0x7FFFFFu) <= 0x400000u ? 2 : 1);
    k = k < -127 ? -127 : k;
    s.byte = bad ? 0xFFu : uint32_t(k + 127);
    s.inv = bad ? 0.f : pow2f(-k);
  } else {
    float t = __uint_as_float(amax_bits) * pow2f(-e) * (1.f / 6.f);
    if constexpr (SNAP) t = __uint_as_float((__float_as_uint(t) + 0x800u) & ~0xFFFu);
    s.byte = bad ? 0x7Fu : e4m3_byte(t);
    const float v = e4m3_value(s.byte);
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    s.inv = bad || v == 0.f ? 0.f : r * pow2f(-e);
  }
  return s;
}

// Codes of 16 values under one scale.  SNAP (bf16 inputs): v x inv is within 2^-23 of
// x / scale, and since x has 8 significant bits and scale x tie at most 7, a quotient that
// is no tie is at least 2^-8 of it, 2^-10, away from one; adding and taking off 1.5 x 2^13
// rounds the product to a multiple of 2^-10 first, which lands exactly on a tie that the
// true quotient is and never crosses one that it is not: the codes are those of real
// arithmetic.  Two values an instruction.
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
template <bool SNAP>
__device__ __forceinline__ uint2 quantize16(const float (&v)[16], float inv) {
  float t[16];
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    if constexpr (SNAP) {
      constexpr float kSnap = 12288.f;
      uint64_t d;
      asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d)
          : "l"(f32x2(v[i], v[i + 1])), "l"(f32x2(inv, inv)), "l"(f32x2(kSnap, kSnap)));
      asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(d), "l"(f32x2(-kSnap, -kSnap)));
      asm("mov.b64 {%0, %1}, %2;" : "=f"(t[i]), "=f"(t[i + 1]) : "l"(d));
    } else {
      t[i] = v[i] * inv;
      t[i + 1] = v[i + 1] * inv;
    }
  }
  return make_uint2(e2m1x8(t), e2m1x8(t + 8));
}

// Bytes of the scale array: tiles of 128 rows x 4 blocks, 512 bytes each.
__device__ __forceinline__ size_t scale_bytes(int R, int tiles_k) {
  return (size_t(R) + 127) / 128 * size_t(tiles_k) * 512;
}
// The 4-byte word of row r in tile column tc.
__device__ __forceinline__ size_t scale_word(size_t r, int tc, int tiles_k) {
  return ((r >> 7) * size_t(tiles_k) + size_t(tc)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

// Stores the scale bytes of the 16-column groups held by consecutive lanes (group g
// on this lane; whole runs of 8 lanes are live together) for a matrix of R rows.
template <int FMT>
__device__ __forceinline__ void store_scales(uint8_t* bs, size_t r, int g, int tiles_k,
                                             uint32_t byte, bool live, int R, int* status) {
  const uint32_t lane = lane_id();
  uint32_t w;
  if constexpr (FMT == H3_FP4_MX) {   // lanes 2i, 2i + 1 hold the same byte
    w = byte << (8 * ((lane >> 1) & 3));
    w |= __shfl_xor_sync(0xffffffffu, w, 2);
    w |= __shfl_xor_sync(0xffffffffu, w, 4);
    if (live && (lane & 7) == 0 && H3_IN(scale_word(r, g >> 3, tiles_k) + 4 <= scale_bytes(R, tiles_k), status))
      *reinterpret_cast<uint32_t*>(bs + scale_word(r, g >> 3, tiles_k)) = w;
  } else {
    w = byte << (8 * (lane & 3));
    w |= __shfl_xor_sync(0xffffffffu, w, 1);
    w |= __shfl_xor_sync(0xffffffffu, w, 2);
    if (live && (lane & 3) == 0 && H3_IN(scale_word(r, g >> 2, tiles_k) + 4 <= scale_bytes(R, tiles_k), status))
      *reinterpret_cast<uint32_t*>(bs + scale_word(r, g >> 2, tiles_k)) = w;
  }
}

// Reduction over the W warps, from `first` on, that share a row; `red` holds one word a
// warp and is the caller's again after the next CTA barrier.
struct MaxU32 {
  static __device__ __forceinline__ uint32_t op(uint32_t a, uint32_t b) { return max(a, b); }
};
template <class Op, class T>
__device__ __forceinline__ T row_reduce(T v, int W, int first, T* red, Op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = Op::op(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (W > 1) {
    if (lane_id() == 0) red[warp_id()] = v;
    __syncthreads();
    v = red[first];
    for (int i = 1; i < W; ++i) v = Op::op(v, red[first + i]);
  }
  return v;
}

}  // namespace
}  // namespace h3
