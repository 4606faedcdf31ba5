// Row-wise microscaled 4-bit quantisation and its inverse (HBM-bound); formats and
// arithmetic in fp4.cuh.
//
// Quantisation: W warps share a row, a thread owns 16 consecutive columns at a time
// and keeps all its columns in registers (ITERS groups of 8 words), so a row is read
// once although an NV row's factor needs its maximum before the first code.
#include "fp4.cuh"
#include "kernels.hpp"
#include "launch.hpp"

namespace h3 {
namespace {

constexpr int kWarps = 8;         // warps of a CTA (16 for the widest rows)
constexpr int kMaxIters = 8;

// Largest |x| of 16 bf16 values as fp32 bits; a NaN among them gives a NaN.
__device__ __forceinline__ uint32_t amax_bits16(const uint4& a, const uint4& b) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  __nv_bfloat162 m = __habs2(reinterpret_cast<const __nv_bfloat162&>(w[0]));
#pragma unroll
  for (int i = 1; i < 8; ++i)
    m = __hmax2_nan(m, __habs2(reinterpret_cast<const __nv_bfloat162&>(w[i])));
  const uint32_t r = reinterpret_cast<const uint32_t&>(m);
  return max(r << 16, r & 0xFFFF0000u);
}

template <int FMT, int ITERS>
__global__ void __launch_bounds__(512, ITERS <= 5 ? 2 : 1)   // 64 registers, else 128
    quantize_fp4_kernel(const uint4* x, int R, int K, int W, uint2* q, uint8_t* bs, float* s,
                        int* status) {
  __shared__ uint32_t red[2][16];
  const int rows_per_cta = int(blockDim.x >> 5) / W;
  const int t = int(threadIdx.x) & (32 * W - 1);      // thread of the row
  const int groups = K >> 4, tiles_k = K / (4 * fp4_block<FMT>());
  int parity = 0;
  pdl_trigger();
  pdl_wait();
  for (int64_t row0 = int64_t(blockIdx.x) * rows_per_cta; row0 < R;
       row0 += int64_t(gridDim.x) * rows_per_cta, parity ^= 1) {
    const int64_t row = row0 + int(warp_id()) / W;
    const bool row_ok = row < R;
    const uint4* xr = x + size_t(row) * (groups * 2);
    uint4 v[ITERS][2];
    uint32_t am[ITERS];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
      const int g = t + i * 32 * W;
      v[i][0] = v[i][1] = make_uint4(0u, 0u, 0u, 0u);
      if (row_ok && g < groups && H3_IN(size_t(row) * groups + size_t(g) < size_t(R) * groups, status)) {
        v[i][0] = ld_dep_cs(xr + 2 * g);
        v[i][1] = ld_dep_cs(xr + 2 * g + 1);
      }
    }
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
      am[i] = amax_bits16(v[i][0], v[i][1]);
      if constexpr (FMT == H3_FP4_MX) am[i] = max(am[i], __shfl_xor_sync(0xffffffffu, am[i], 1));
      else top = max(top, am[i] < kInfBits ? am[i] : 0u);
    }
    int e = 0;
    if constexpr (FMT == H3_FP4_NV) {
      e = nv_row_exponent(row_reduce(top, W, int(warp_id()) & ~(W - 1), red[parity], MaxU32()));
      if (row_ok && t == 0 && H3_IN(row >= 0 && row < R, status)) s[row] = pow2f(e);
    }
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
      const int g = t + i * 32 * W;
      const bool live = row_ok && g < groups;
      const BlockScale sc = block_scale<FMT, true>(am[i], e);
      store_scales<FMT>(bs, size_t(row), g, tiles_k, sc.byte, live, R, status);
      if (live && H3_IN(size_t(row) * groups + size_t(g) < size_t(R) * groups, status)) {
        const uint32_t w[8] = {v[i][0].x, v[i][0].y, v[i][0].z, v[i][0].w,
                               v[i][1].x, v[i][1].y, v[i][1].z, v[i][1].w};
        float f[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          f[2 * j] = bf16_lo(w[j]);
          f[2 * j + 1] = bf16_hi(w[j]);
        }
        q[size_t(row) * groups + g] =
            sc.inv == 0.f ? make_uint2(0u, 0u) : quantize16<true>(f, sc.inv);
      }
    }
  }
}

// One warp for a row, one thread for 8 columns at a time: 4 bytes of codes in, 16 bytes of
// bf16 out, both contiguous over the warp; kAhead of each are in flight.  The eight warps of
// a CTA take the eight rows whose scale words share 32-byte sectors (2g, 2g + 1 and those 32,
// 64 and 96 further on), so a sector comes to the SM once.  code x scale is exact (at most 6
// significant bits), so with a power of two for the row the only rounding is the store, and
// that is exact too unless the value is subnormal (factors of any kind: one rounding more).
//
// Five ahead: with four, six and eight 58,758 x 5,120 MX took 129.9, 134.5 and 129.2 us against
// 130.4, x 1,152 37.8, 32.6 and 36.6 against 30.5, x 384 20.1, 26.6 and 33.0 against 23.2; only
// eight is faster for wide rows (4,096 x 20,480 41.2 us against 51.1).
constexpr int kAhead = 5;
template <int FMT>
__global__ void __launch_bounds__(256)
    dequantize_fp4_kernel(const uint32_t* q, const uint8_t* bs, const float* s, int R, int K,
                          uint4* y, int* status) {
  const int vecs = K >> 3, tiles_k = K / (4 * fp4_block<FMT>());
  const int lane = int(lane_id()), warp = int(warp_id());
  const int64_t groups = (int64_t(R) + 127) / 128 * 16;   // of 8 rows
  pdl_trigger();
  pdl_wait();
  for (int64_t g = blockIdx.x; g < groups; g += gridDim.x) {
    const int64_t row = (g >> 4) * 128 + (g & 15) * 2 + (warp & 1) + 32 * (warp >> 1);
    if (row >= R || !H3_IN(row >= 0, status)) continue;
    const float f = s != nullptr ? ld_dep(s + row) : 1.f;
    const uint32_t* qr = q + size_t(row) * vecs;
    uint4* yr = y + size_t(row) * vecs;
    const uint8_t* br = bs + scale_word(size_t(row), 0, tiles_k);
    for (int v0 = lane; v0 < vecs; v0 += 32 * kAhead) {
      uint32_t w[kAhead], byte[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int v = v0 + 32 * i, b = FMT == H3_FP4_MX ? v >> 2 : v >> 1;
        const size_t at = size_t(b >> 2) * 512 + (b & 3);
        const bool in = v < vecs && H3_IN(size_t(row) * vecs + v < size_t(R) * vecs &&
                                              scale_word(size_t(row), 0, tiles_k) + at < scale_bytes(R, tiles_k),
                                          status);
        w[i] = in ? ld_dep_cs(qr + v) : 0u;
        byte[i] = in ? ld_dep(br + at) : 0u;
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int v = v0 + 32 * i;
        float sc;
        if constexpr (FMT == H3_FP4_MX)   // byte 0 is 2^-127, below the normal numbers
          sc = byte[i] == 255u ? __uint_as_float(0x7FC00000u)
                               : __uint_as_float(byte[i] == 0u ? 0x400000u : byte[i] << 23);
        else
          sc = e4m3_value(byte[i]);
        const float2 c[4] = {__half22float2(e2m1_pair<0>(w[i])), __half22float2(e2m1_pair<1>(w[i])),
                             __half22float2(e2m1_pair<2>(w[i])), __half22float2(e2m1_pair<3>(w[i]))};
        // code x scale first, which is exact, then the factor: one rounding, out of range only if
        // the value is.  Codes times 2^126 and 2^127 would overflow, so those lend 2^2 to the end.
        const bool top = FMT == H3_FP4_MX && sc > 0x1p125f;
        const float ahead = top ? 0.25f * sc : sc, after = top ? 4.f : 1.f;
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[j] = pack_bf16x2(c[j].x * ahead * f * after, c[j].y * ahead * f * after);
        if (v < vecs && H3_IN(size_t(row) * vecs + v < size_t(R) * vecs, status))
          yr[v] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

template <int FMT, int ITERS>
cudaError_t launch_iters(const void* x, int R, int K, int W, void* q, void* bs, float* s,
                         const DevCtx& ctx, cudaStream_t st) {
  const int warps = W > kWarps ? W : kWarps;
  static KernelState state;
  const auto kern = quantize_fp4_kernel<FMT, ITERS>;
  int per_sm = 0;
  if (cudaError_t e = ctas_per_sm(&state, kern, warps * 32, 0, ctx, &per_sm)) return e;
  const int64_t want = (int64_t(R) + warps / W - 1) / (warps / W);
  const int64_t room = int64_t(ctx.num_sms) * per_sm;
  const Launch l(unsigned(want < room ? want : room), warps * 32, 0, st);
  if (cudaError_t e = cudaLaunchKernelEx(&l.cfg, kern, static_cast<const uint4*>(x), R, K, W,
                                         static_cast<uint2*>(q), static_cast<uint8_t*>(bs), s,
                                         ctx.status))
    return e;
  return cudaGetLastError();
}

template <int FMT>
cudaError_t launch_quant(const void* x, int R, int K, void* q, void* bs, float* s,
                         const DevCtx& ctx, cudaStream_t st) {
  const int groups = K >> 4;
  int W = 1;
  while (groups > 32 * W * kMaxIters) W *= 2;   // K <= 65536: at most 16
  switch ((groups + 32 * W - 1) / (32 * W)) {
    case 1: return launch_iters<FMT, 1>(x, R, K, W, q, bs, s, ctx, st);
    case 2: return launch_iters<FMT, 2>(x, R, K, W, q, bs, s, ctx, st);
    case 3: return launch_iters<FMT, 3>(x, R, K, W, q, bs, s, ctx, st);
    case 4: return launch_iters<FMT, 4>(x, R, K, W, q, bs, s, ctx, st);
    case 5: return launch_iters<FMT, 5>(x, R, K, W, q, bs, s, ctx, st);
    case 6: return launch_iters<FMT, 6>(x, R, K, W, q, bs, s, ctx, st);
    default: return launch_iters<FMT, 8>(x, R, K, W, q, bs, s, ctx, st);
  }
}

}  // namespace

cudaError_t launch_quantize_fp4(const void* x, int fmt, int R, int K, void* q, void* bs, float* s,
                                const DevCtx& ctx, cudaStream_t st) {
  return fmt == H3_FP4_MX ? launch_quant<H3_FP4_MX>(x, R, K, q, bs, s, ctx, st)
                          : launch_quant<H3_FP4_NV>(x, R, K, q, bs, s, ctx, st);
}

cudaError_t launch_dequantize_fp4(const void* q, const void* bs, const float* s, int fmt, int R,
                                  int K, void* y, const DevCtx& ctx, cudaStream_t st) {
  const int64_t want = (int64_t(R) + 127) / 128 * 16, room = int64_t(ctx.num_sms) * 8;
  const auto kern = fmt == H3_FP4_MX ? dequantize_fp4_kernel<H3_FP4_MX>
                                     : dequantize_fp4_kernel<H3_FP4_NV>;
  const Launch l(unsigned(want < room ? want : room), 256, 0, st);
  if (cudaError_t e = cudaLaunchKernelEx(&l.cfg, kern, static_cast<const uint32_t*>(q),
                                         static_cast<const uint8_t*>(bs), s, R, K,
                                         static_cast<uint4*>(y), ctx.status))
    return e;
  return cudaGetLastError();
}

}  // namespace h3
