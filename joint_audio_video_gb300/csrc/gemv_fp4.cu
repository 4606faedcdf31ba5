// The 4-bit product for one or two rows of A: weights read once, no tensor cores.
//
// A warp takes four weight rows r, r + 32, r + 64, r + 96 of a 128-row group, whose scale
// words lie side by side (one 16-byte load serves 64 or 128 columns of all four), and a lane
// 16 columns of each at a time.  Codes become halves; the 16 products of a block half are
// whole multiples of 1/4 up to 36, so eight of them sum exactly in half precision (at most
// 288 = 1152 quarters); from there on everything is fp32: the two halves' sum, its product
// with the two block scales, the sum over blocks, and the tree over the lanes, in a fixed
// order.  `split` warps share a row's columns when there are few rows.
//
// Bound by the decoding, ~3 instructions a weight (the conversion instruction is the cheapest
// way: a table in PRMT took 1.5 times as long, integer products, dp4a, 1.4 times): 5.3 us
// (NV) or 5.2 (MX) for one row through 5,120 x 5,120 (14.8 MB; 2.2 us at the copy rate), 2.8
// through 2,048 x 2,048, 3.1 and 2.9 for two rows of that.  The scales of two rows of weights are
// converted by one instruction; one at a time by integer steps MX took 105 registers, one CTA
// an SM less, and 7.4 us for the former.
#include "factors.cuh"
#include "fp4.cuh"
#include "kernels.hpp"
#include "launch.hpp"

namespace h3 {
namespace {

constexpr int kThreads = 128;
constexpr int kCols = 512;      // columns of a warp's step
constexpr int kPerSm = 5;       // CTAs an SM that the registers allow (at most 102 a thread)

// Two scale bytes as floats.
template <int FMT>
__device__ __forceinline__ float2 scale_pair(uint32_t bytes) {
  uint32_t h;
  if constexpr (FMT == H3_FP4_MX) {
    asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(h) : "h"(uint16_t(bytes)));
    return make_float2(__uint_as_float(h << 16), __uint_as_float(h & 0xFFFF0000u));
  } else {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(bytes)));
    return __half22float2(reinterpret_cast<const __half2&>(h));
  }
}
__device__ __forceinline__ void halves16(const uint2& w, __half2 (&h)[8]) {
  h[0] = e2m1_pair<0>(w.x);
  h[1] = e2m1_pair<1>(w.x);
  h[2] = e2m1_pair<2>(w.x);
  h[3] = e2m1_pair<3>(w.x);
  h[4] = e2m1_pair<0>(w.y);
  h[5] = e2m1_pair<1>(w.y);
  h[6] = e2m1_pair<2>(w.y);
  h[7] = e2m1_pair<3>(w.y);
}

template <int EPI, int FMT, int MT>
__global__ void __launch_bounds__(kThreads, kPerSm)
    gemv_fp4_kernel(const __grid_constant__ GemmFp4Args a, int split, int* status) {
  constexpr int kAhead = MT == 1 ? 4 : 2;
  __shared__ float part[kThreads / 32][4 * MT];
  const int lane = int(lane_id()), warp = int(warp_id());
  const int quad = int(blockIdx.x) * (kThreads / 32 / split) + warp / split, slice = warp % split;
  const int group = quad >> 5, r0 = quad & 31;       // rows 128 group + r0 + 32 i
  constexpr int kPer = FMT == H3_FP4_MX ? 8 : 4;     // lanes of a scale word
  const int tiles_k = a.K / (16 * kPer), steps = (a.K + kCols - 1) / kCols;
  const size_t kbytes = size_t(a.K) >> 1;
  const uint8_t* wq = static_cast<const uint8_t*>(a.B) + (size_t(group) * 128 + r0) * kbytes;
  const uint8_t* wb = static_cast<const uint8_t*>(a.b_bs) + size_t(group) * tiles_k * 512 + r0 * 16;
  const uint8_t* xq = static_cast<const uint8_t*>(a.A);
  const uint8_t* xb = static_cast<const uint8_t*>(a.a_bs);
  const int byte_at = FMT == H3_FP4_MX ? (lane >> 1) & 3 : lane & 3;
  const uint32_t pick = uint32_t(byte_at) * 0x11u + 0x40u;   // that byte of two words
  // MX scales reach 2^127 and a block half's sum 576: the weights' scales are taken 2^-10 times,
  // exactly, so that only a sum that is itself out of range overflows
  constexpr float kDown = FMT == H3_FP4_MX ? 1.f / 1024.f : 1.f;
  pdl_trigger();
  // the weights' codes into L2 while the work ahead of this kernel ends (6.2 -> 5.5 us for 5,120
  // x 5,120 among others; the tensor-core kernel for few rows, whose ring asks for its bytes at
  // once, lost 5 to 15 % by the same)
  if (lane < 4 && slice == 0 && H3_IN(group * 128 + r0 + 32 * lane < a.N, status))
    bulk_prefetch_1d(wq + size_t(lane) * 32 * kbytes, uint32_t(kbytes));
  pdl_wait();
  float acc[4][MT];
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[r][m] = 0.f;

  for (int i0 = slice; i0 < steps; i0 += split * kAhead) {
    uint2 w[kAhead][4], x[kAhead][MT];
    uint4 ws[kAhead];
    uint32_t xs[kAhead][MT];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int col = (i0 + u * split) * kCols + lane * 16;
      const size_t tile = size_t(col / (16 * kPer)) * 512;
      // 16 columns of four rows, their scale words, and the words of the first rows of A
      const bool in = col < a.K && H3_IN(group * 128 + r0 + 96 < a.N && col >= 0 && col + 16 <= a.K &&
                                             tile + r0 * 16 + 16 <= size_t(tiles_k) * 512,
                                         status);
      ws[u] = in ? ld_dep(reinterpret_cast<const uint4*>(wb + tile)) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int r = 0; r < 4; ++r)
        w[u][r] = in ? ld_dep_cs(reinterpret_cast<const uint2*>(wq + size_t(r) * 32 * kbytes + (col >> 1)))
                     : make_uint2(0u, 0u);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const bool on = in && m < a.M;
        x[u][m] = on ? ld_dep(reinterpret_cast<const uint2*>(xq + m * kbytes + (col >> 1)))
                     : make_uint2(0u, 0u);
        xs[u][m] = on ? ld_dep(xb + tile + m * 16 + byte_at) : 0u;
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (i0 + u * split >= steps) break;   // the same for the whole warp
      __half2 xh[MT][8];
      float xsf[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        halves16(x[u][m], xh[m]);
        xsf[m] = scale_pair<FMT>(xs[u][m]).x;
      }
      const float2 s01 = scale_pair<FMT>(__byte_perm(ws[u].x, ws[u].y, pick));
      const float2 s23 = scale_pair<FMT>(__byte_perm(ws[u].z, ws[u].w, pick));
      const float wsf[4] = {s01.x * kDown, s01.y * kDown, s23.x * kDown, s23.y * kDown};
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        __half2 wh[8];
        halves16(w[u][r], wh);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          __half2 d = __hmul2(wh[0], xh[m][0]);
#pragma unroll
          for (int j = 1; j < 8; ++j) d = __hfma2(wh[j], xh[m][j], d);
          const float2 f = __half22float2(d);
          acc[r][m] = fmaf((f.x + f.y) * wsf[r], xsf[m], acc[r][m]);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[r][m] += __shfl_xor_sync(0xffffffffu, acc[r][m], o);
  // value i = (row i % 4, token i / 4) goes to lane i
  float v = 0.f;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (lane == m * 4 + r) v = acc[r][m];
  if (split > 1) {
    if (lane < 4 * MT) part[warp][lane] = v;
    __syncthreads();
    if (slice != 0) return;
    if (lane < 4 * MT)
      for (int s = 1; s < split; ++s) v += part[warp + s][lane];
  }
  const int m = lane >> 2, n = group * 128 + r0 + 32 * (lane & 3);
  if (lane >= 4 * MT || m >= a.M || !H3_IN(n < a.N, status)) return;
  v *= 1.f / kDown;
  const float fa = a.a_s != nullptr ? ld_dep(a.a_s + m) : 1.f;
  const float fb = a.b_s != nullptr ? ld_dep(a.b_s + n) : 1.f;
  v = mid_range(fa) && mid_range(fb) ? v * (fa * fb) : times_apart(v, fa, fb);
  if constexpr (EPI == EPI_GELU) {
    float t;   // tanh form, as in gemm_epilogue.cuh
    asm("tanh.approx.f32 %0, %1;" : "=f"(t) : "f"(0.7978845608028654f * fmaf(0.044715f * v, v * v, v)));
    v = 0.5f * v * (1.f + t);
  }
  if constexpr (EPI == EPI_GATED_RESIDUAL) {
    const int md = a.mod[m];
    if (md >= a.n_mod) {
      atomicCAS(status, H3_DEV_OK, H3_DEV_BAD_INDEX);
      v = __uint_as_float(0x7FC00000u);
    } else {
      const float xr = __bfloat162float(static_cast<const __nv_bfloat16*>(a.x_res)[size_t(m) * a.N + n]);
      v = fmaf(ld_dep(a.gate + size_t(md) * a.N + n), v, xr);
    }
  }
  static_cast<__nv_bfloat16*>(a.C)[size_t(m) * a.N + n] = __float2bfloat16_rn(v);
}

template <int EPI, int FMT, int MT>
cudaError_t launch_mt(const GemmFp4Args& a, const DevCtx& ctx, cudaStream_t st) {
  // rows alone, or two or four warps for the columns of each, as long as all run at once (4,096 x
  // 4,096 by four warps a row, 1.3 waves: 4.8 MX and 5.1 NV; by two, in one: 4.0 and 4.1)
  const int quads = a.N / 4, steps = (a.K + kCols - 1) / kCols;
  int split = 1;
  while (split < 4 && quads * split * 2 <= kThreads / 32 * kPerSm * ctx.num_sms && split * 2 <= steps)
    split *= 2;
  const Launch l(unsigned(quads / (kThreads / 32 / split)), kThreads, 0, st);
  if (cudaError_t e = cudaLaunchKernelEx(&l.cfg, gemv_fp4_kernel<EPI, FMT, MT>, a, split, ctx.status))
    return e;
  return cudaGetLastError();
}

template <int EPI, int FMT>
cudaError_t launch_fmt(const GemmFp4Args& a, const DevCtx& ctx, cudaStream_t st) {
  if (a.M == 1) return launch_mt<EPI, FMT, 1>(a, ctx, st);
  return launch_mt<EPI, FMT, 2>(a, ctx, st);
}

template <int EPI>
cudaError_t launch_epi(const GemmFp4Args& a, const DevCtx& ctx, cudaStream_t st) {
  return a.fmt == H3_FP4_MX ? launch_fmt<EPI, H3_FP4_MX>(a, ctx, st)
                            : launch_fmt<EPI, H3_FP4_NV>(a, ctx, st);
}

}  // namespace

cudaError_t launch_gemv_fp4(const GemmFp4Args& a, const DevCtx& ctx, cudaStream_t st) {
  switch (a.epilogue) {
    case EPI_PLAIN: return launch_epi<EPI_PLAIN>(a, ctx, st);
    case EPI_GATED_RESIDUAL: return launch_epi<EPI_GATED_RESIDUAL>(a, ctx, st);
    case EPI_GELU: return launch_epi<EPI_GELU>(a, ctx, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace h3
