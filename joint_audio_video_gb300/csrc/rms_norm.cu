// Root-mean-square norm with the residual's addition and a quantised output (HBM-bound):
//   sum = bf16(x + res),  y = sum * weight * rsqrt(mean sum^2 + eps),
//   out = E4M3 with one scale for the row, or microscaled 4 bits (fp4.cuh).
// W warps share a row; a thread owns the same columns (16 at a time, ITERS times) of
// every row it meets, so its weights stay in registers; the row's sum stays there as
// bf16 pairs between the passes that need it (squares, maximum, codes).  Algorithmic
// traffic: 4 bytes read, 2 + 1 (8 bits) or 2 + 0.53 .. 0.56 (4 bits) written an element.
#include "fp4.cuh"
#include "kernels.hpp"

namespace h3 {
namespace {

constexpr int kWarps = 8;
constexpr int kOutE4M3 = 0;   // other OUT values: the H3_FP4 formats

struct SumF32 {
  static __device__ __forceinline__ float op(float a, float b) { return a + b; }
};
struct MaxF32 {
  static __device__ __forceinline__ float op(float a, float b) { return fmaxf(a, b); }
};

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return uint32_t(lo) | (uint32_t(hi) << 16);
}

template <int OUT, int ITERS>
__global__ void __launch_bounds__(512)
    rms_norm_kernel(const uint4* x, const uint4* res, const float4* __restrict__ weight, int L,
                    int d, int W, float eps, uint4* sum, uint8_t* __restrict__ q,
                    uint8_t* __restrict__ bs, float* __restrict__ scale, int* status) {
  __shared__ float red_sum[2][16];
  __shared__ float red_max[2][16];
  __shared__ uint32_t red_top[2][16];
  const int rows_per_cta = int(blockDim.x >> 5) / W;
  const int t = int(threadIdx.x) & (32 * W - 1);
  const int groups = d >> 4;
  const float inv_d = 1.f / float(d);
  float wt[ITERS][16];
#pragma unroll
  for (int i = 0; i < ITERS; ++i) {
    const int g = t + i * 32 * W;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 f = g < groups ? __ldg(weight + 4 * g + j) : make_float4(0.f, 0.f, 0.f, 0.f);
      wt[i][4 * j] = f.x;
      wt[i][4 * j + 1] = f.y;
      wt[i][4 * j + 2] = f.z;
      wt[i][4 * j + 3] = f.w;
    }
  }
  int parity = 0;
  for (int64_t row0 = int64_t(blockIdx.x) * rows_per_cta; row0 < L;
       row0 += int64_t(gridDim.x) * rows_per_cta, parity ^= 1) {
    const int64_t row = row0 + int(warp_id()) / W;
    const bool row_ok = row < L;
    const size_t at = size_t(row) * (groups * 2);
    uint32_t v[ITERS][8];
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
      const int g = t + i * 32 * W;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0u;
      if (row_ok && g < groups && H3_IN(row >= 0 && g >= 0, status)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 a = x[at + 2 * g + h];
          v[i][4 * h] = a.x;
          v[i][4 * h + 1] = a.y;
          v[i][4 * h + 2] = a.z;
          v[i][4 * h + 3] = a.w;
          if (res != nullptr) {
            const uint4 b = res[at + 2 * g + h];
            const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              v[i][4 * h + j] = pack_bf16x2(bf16_lo(v[i][4 * h + j]) + bf16_lo(bw[j]),
                                            bf16_hi(v[i][4 * h + j]) + bf16_hi(bw[j]));
          }
        }
      }
    }
    // squares: a sum for each of eight positions, joined in pairs
    float part[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < ITERS; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float lo = bf16_lo(v[i][j]), hi = bf16_hi(v[i][j]);
        part[j] = fmaf(lo, lo, fmaf(hi, hi, part[j]));
      }
    const float ss = row_reduce(((part[0] + part[1]) + (part[2] + part[3])) +
                                    ((part[4] + part[5]) + (part[6] + part[7])),
                                W, red_sum[parity], SumF32());
    const float rstd = rsqrtf(ss * inv_d + eps);
    if (sum != nullptr && row_ok) {
#pragma unroll
      for (int i = 0; i < ITERS; ++i) {
        const int g = t + i * 32 * W;
        if (g < groups) {
          sum[at + 2 * g] = make_uint4(v[i][0], v[i][1], v[i][2], v[i][3]);
          sum[at + 2 * g + 1] = make_uint4(v[i][4], v[i][5], v[i][6], v[i][7]);
        }
      }
    }
    auto y_of = [&](int i, float (&y)[16]) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y[2 * j] = bf16_lo(v[i][j]) * rstd * wt[i][2 * j];
        y[2 * j + 1] = bf16_hi(v[i][j]) * rstd * wt[i][2 * j + 1];
      }
    };
    if constexpr (OUT == kOutE4M3) {
      float am = 0.f;
#pragma unroll
      for (int i = 0; i < ITERS; ++i) {
        float y[16];
        y_of(i, y);
#pragma unroll
        for (int j = 0; j < 16; ++j) am = fmaxf(am, fabsf(y[j]));
      }
      am = row_reduce(am, W, red_max[parity], MaxF32());
      const float inv = am > 0.f ? 448.f / am : 1.f;
      if (row_ok && t == 0) scale[row] = am > 0.f ? am / 448.f : 1.f;
      if (row_ok) {
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
          const int g = t + i * 32 * W;
          if (g < groups) {
            float y[16];
            y_of(i, y);
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              o[j] = e4m3x4(y[4 * j] * inv, y[4 * j + 1] * inv, y[4 * j + 2] * inv, y[4 * j + 3] * inv);
            reinterpret_cast<uint4*>(q)[size_t(row) * groups + g] = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
      }
    } else {
      const int tiles_k = d / (4 * fp4_block<OUT>());
      uint32_t am[ITERS];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < ITERS; ++i) {
        float y[16];
        y_of(i, y);
        am[i] = 0;
#pragma unroll
        for (int j = 0; j < 16; ++j) am[i] = max(am[i], __float_as_uint(y[j]) & 0x7FFFFFFFu);
        if constexpr (OUT == H3_FP4_MX) am[i] = max(am[i], __shfl_xor_sync(0xffffffffu, am[i], 1));
        else top = max(top, am[i] < kInfBits ? am[i] : 0u);
      }
      int e = 0;
      if constexpr (OUT == H3_FP4_NV) {
        e = nv_row_exponent(row_reduce(top, W, red_top[parity], MaxU32()));
        if (row_ok && t == 0) scale[row] = pow2f(e);
      }
#pragma unroll
      for (int i = 0; i < ITERS; ++i) {
        const int g = t + i * 32 * W;
        const bool live = row_ok && g < groups;
        const BlockScale sc = block_scale<OUT>(am[i], e);
        store_scales<OUT>(bs, size_t(row), g, tiles_k, sc.byte, live);
        if (live) {
          float y[16];
          y_of(i, y);
          reinterpret_cast<uint2*>(q)[size_t(row) * groups + g] =
              sc.inv == 0.f ? make_uint2(0u, 0u) : quantize16<false>(y, sc.inv);
        }
      }
    }
  }
}

template <int OUT, int ITERS>
cudaError_t launch_iters(const RmsNormArgs& a, int W, const DevCtx& ctx, cudaStream_t st) {
  const int warps = W > kWarps ? W : kWarps;
  int per_sm = 0;
  cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
      &per_sm, rms_norm_kernel<OUT, ITERS>, warps * 32, 0);
  if (e != cudaSuccess) return e;
  const int64_t want = (int64_t(a.L) + warps / W - 1) / (warps / W);
  const int64_t room = int64_t(ctx.num_sms) * (per_sm < 1 ? 1 : per_sm);
  rms_norm_kernel<OUT, ITERS><<<unsigned(want < room ? want : room), warps * 32, 0, st>>>(
      static_cast<const uint4*>(a.x), static_cast<const uint4*>(a.res),
      reinterpret_cast<const float4*>(a.weight), a.L, a.d, W, a.eps, static_cast<uint4*>(a.sum),
      static_cast<uint8_t*>(a.q), static_cast<uint8_t*>(a.bs), a.scale, ctx.status);
  return cudaGetLastError();
}

template <int OUT>
cudaError_t launch_out(const RmsNormArgs& a, const DevCtx& ctx, cudaStream_t st) {
  const int groups = a.d >> 4;
  int W = 1;
  while (groups > 32 * W * 3) W *= 2;   // d <= 16384: at most 16
  switch ((groups + 32 * W - 1) / (32 * W)) {
    case 1: return launch_iters<OUT, 1>(a, W, ctx, st);
    case 2: return launch_iters<OUT, 2>(a, W, ctx, st);
    default: return launch_iters<OUT, 3>(a, W, ctx, st);
  }
}

}  // namespace

cudaError_t launch_rms_norm(const RmsNormArgs& a, const DevCtx& ctx, cudaStream_t st) {
  switch (a.fmt) {
    case H3_FP4_MX: return launch_out<H3_FP4_MX>(a, ctx, st);
    case H3_FP4_NV: return launch_out<H3_FP4_NV>(a, ctx, st);
    default: return launch_out<kOutE4M3>(a, ctx, st);
  }
}

}  // namespace h3
