// Root-mean-square norm with the residual's addition and a quantised output (HBM-bound):
//   sum = bf16(x + res),  y = sum * weight * rsqrt(mean sum^2 + eps),
//   out = E4M3 with one scale for the row, or microscaled 4 bits (fp4.cuh).
// W warps share a row, 4 / W rows share a CTA.  One thread keeps the CTA's next two to four
// groups of rows in flight as 1-D bulk copies into a ring of shared-memory slots, so HBM
// reads go on while the warps reduce and write.  A thread owns the same columns of every row
// it meets (8 at a time, ITERS times), so its weights stay in registers; the row's sum stays
// there too, as bf16 pairs, between the passes that need it (squares, maximum, codes).
// Algorithmic traffic: 4 bytes read, 2 + 1 (8 bits) or 2 + 0.53 .. 0.56 (4 bits) written an
// element.
#include "fp4.cuh"
#include "kernels.hpp"
#include "launch.hpp"

namespace h3 {
namespace {

constexpr int kWarps = 4;      // of a CTA, rows permitting
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

__device__ __forceinline__ uint4 add_bf16x8(uint4 a, const uint4& b) {
  a.x = pack_bf16x2(bf16_lo(a.x) + bf16_lo(b.x), bf16_hi(a.x) + bf16_hi(b.x));
  a.y = pack_bf16x2(bf16_lo(a.y) + bf16_lo(b.y), bf16_hi(a.y) + bf16_hi(b.y));
  a.z = pack_bf16x2(bf16_lo(a.z) + bf16_lo(b.z), bf16_hi(a.z) + bf16_hi(b.z));
  a.w = pack_bf16x2(bf16_lo(a.w) + bf16_lo(b.w), bf16_hi(a.w) + bf16_hi(b.w));
  return a;
}

// Scale word of 8-column vectors held by consecutive lanes (vector v on this lane): NV two
// lanes a block, MX four; whole runs of 16 lanes are live together; a matrix of R rows.
template <int FMT>
__device__ __forceinline__ void store_scales8(uint8_t* bs, size_t r, int v, int tiles_k,
                                              uint32_t byte, bool live, int R, int* status) {
  constexpr int kPer = FMT == H3_FP4_MX ? 4 : 2;   // lanes of a block
  uint32_t w = byte << (8 * ((lane_id() / kPer) & 3));
  w |= __shfl_xor_sync(0xffffffffu, w, kPer);
  w |= __shfl_xor_sync(0xffffffffu, w, 2 * kPer);
  if (live && (lane_id() & (4 * kPer - 1)) == 0 &&
      H3_IN(scale_word(r, v / (4 * kPer), tiles_k) + 4 <= scale_bytes(R, tiles_k), status))
    *reinterpret_cast<uint32_t*>(bs + scale_word(r, v / (4 * kPer), tiles_k)) = w;
}

constexpr int kMaxStages = 4;

// Squares of values above ~1e17 leave fp32, and with an eps below 2^-126 those of small values
// lose bits that count (TINY: kernels for such an eps).  Where the mean square is out of range
// it is taken again, of the row times 2^-72 or 2^96 with eps times the factor's square: rolled
// loops behind a vote, the values from global memory and the threads' sums through shared
// memory, which cost other rows nothing (58,758 x 5,120 in NV 339 us with and without; the same
// over the registers, with shuffles, or in a call: 350 to 375).  The factor goes to the inverse
// square root (2^-72: it is 2^-128 at least, two bits below the normal numbers) or, if TINY,
// where that could overflow, to the values.
template <int OUT, int ITERS, bool TINY>
__global__ void __launch_bounds__(512)
    rms_norm_kernel(const uint4* x, const uint4* res, const float4* weight, int L,
                    int d, int W_of, int rows, int stages, float eps, uint4* sum,
                    uint8_t* q, uint8_t* bs, float* scale,
                    int* status, uint64_t wait_ns) {
  extern __shared__ __align__(128) uint8_t ring[];   // stages x (x rows, then res rows)
  __shared__ uint64_t full[kMaxStages];
  __shared__ float red_sum[16];
  __shared__ float red_max[16];
  __shared__ uint32_t red_top[16];
  __shared__ float part_far[512];
  __shared__ int abort_flag;
  const int W = ITERS <= 2 ? 1 : W_of;           // narrow rows: one warp, known here
  const int vecs = d >> 3;                       // 16-byte vectors of a row
  const int r_cta = int(warp_id()) / W;          // row of the CTA's group
  const int t = int(threadIdx.x) - r_cta * 32 * W;
  const float inv_d = 1.f / float(d);
  const size_t row_bytes = size_t(d) * 2, half = row_bytes * rows;
  const size_t stage_bytes = res != nullptr ? 2 * half : half;
  // groups of rows of this CTA: blockIdx.x + k G, k < nk
  const int groups = (L - 1) / rows + 1, G = int(gridDim.x);
  const int nk = (groups - 1 - int(blockIdx.x)) / G + 1;
  const WaitCtx wc{&abort_flag, status, wait_ns};
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < stages; ++s) mbar_init(smem_u32(&full[s]), 1);
    fence_barrier_init();
  }
  __syncthreads();
  pdl_trigger();
  pdl_wait();
  const auto issue = [&](int k) {   // group k of this CTA into ring slot k % stages
    const int s = k % stages;
    const uint32_t bar = smem_u32(&full[s]);
    const int64_t row0 = (int64_t(blockIdx.x) + int64_t(k) * G) * rows;
    const int n = int(L - row0 < rows ? L - row0 : rows);
    uint8_t* slot = ring + s * stage_bytes;
    if (H3_IN(row0 >= 0 && n >= 1 && row0 + n <= L, status)) {
      const uint32_t bytes = uint32_t(n * row_bytes);
      mbar_arrive_expect_tx(bar, res != nullptr ? 2 * bytes : bytes);
      bulk_load_1d(smem_u32(slot), x + size_t(row0) * vecs, bytes, bar);
      if (res != nullptr) bulk_load_1d(smem_u32(slot + half), res + size_t(row0) * vecs, bytes, bar);
    } else {
      mbar_arrive(bar);
    }
  };
  int issued = 0;
  if (threadIdx.x == 0)
    for (; issued < stages && issued < nk; ++issued) issue(issued);

  float wt[ITERS][8];
#pragma unroll
  for (int i = 0; i < ITERS; ++i) {
    const int c = t + i * 32 * W;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    if (c < vecs && H3_IN(c >= 0 && 8 * c + 8 <= d, status)) {
      a = ld_dep(weight + 2 * c);
      b = ld_dep(weight + 2 * c + 1);
    }
    wt[i][0] = a.x, wt[i][1] = a.y, wt[i][2] = a.z, wt[i][3] = a.w;
    wt[i][4] = b.x, wt[i][5] = b.y, wt[i][6] = b.z, wt[i][7] = b.w;
  }
  int k = 0;
  for (; k < nk; ++k) {
    const int s = k % stages;
    const bool ok = mbar_wait(smem_u32(&full[s]), uint32_t(k / stages) & 1u, wc);
    if (__syncthreads_or(!ok)) break;
    const int64_t row = (int64_t(blockIdx.x) + int64_t(k) * G) * rows + r_cta;
    const bool row_ok = row < L;
    const uint4* xr = reinterpret_cast<const uint4*>(ring + s * stage_bytes) + r_cta * vecs;
    const uint4* rr = reinterpret_cast<const uint4*>(ring + s * stage_bytes + half) + r_cta * vecs;
    uint32_t v[ITERS][4];
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
      const int c = t + i * 32 * W;
      uint4 a = make_uint4(0u, 0u, 0u, 0u);
      if (row_ok && c < vecs) {
        a = xr[c];
        if (res != nullptr) a = add_bf16x8(a, rr[c]);
        if (sum != nullptr && H3_IN(size_t(row) * vecs + c < size_t(L) * vecs, status))
          sum[size_t(row) * vecs + c] = a;
      }
      v[i][0] = a.x, v[i][1] = a.y, v[i][2] = a.z, v[i][3] = a.w;
    }
    // squares: a sum for each of four positions, joined in pairs
    float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < ITERS; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float lo = bf16_lo(v[i][j]), hi = bf16_hi(v[i][j]);
        part[j] = fmaf(lo, lo, fmaf(hi, hi, part[j]));
      }
    // every thread has read its part of the slot before the barrier inside (W == 1: the one
    // below), after which it is filled again
    const float ss = row_reduce((part[0] + part[1]) + (part[2] + part[3]), W, r_cta * W, red_sum,
                                SumF32());
    if (W == 1) __syncthreads();
    if (threadIdx.x == 0 && issued < nk) issue(issued++);
    float ms = ss * inv_d + eps, f = 1.f;
    // the same for all of the row's warps
    if (__any_sync(0xffffffffu, !((!TINY || ms >= pow2f(-126)) && ms < __uint_as_float(kInfBits)))) {
      f = TINY && ms < 1.f ? pow2f(96) : pow2f(-72);
      float far = 0.f;   // this thread's part
#pragma unroll 1
      for (int c = t; row_ok && c < vecs; c += 32 * W) {
        const size_t at = size_t(row) * vecs + c;   // this thread has stored its part of the sum
        if (!H3_IN(at < size_t(L) * vecs, status)) continue;
        uint4 a = ld_dep((sum != nullptr ? sum : x) + at);
        if (sum == nullptr && res != nullptr) a = add_bf16x8(a, ld_dep(res + at));
        float each = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t w = (&a.x)[j];
          const float lo = bf16_lo(w) * f, hi = bf16_hi(w) * f;
          each = fmaf(lo, lo, fmaf(hi, hi, each));
        }
        far += each;
      }
      part_far[threadIdx.x] = far;
      if (W > 1) asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + r_cta), "r"(32 * W) : "memory");
      else __syncwarp();
      far = 0.f;
#pragma unroll 1
      for (int w = 0; w < W; ++w) {
        float each = 0.f;
#pragma unroll 1
        for (int i = 0; i < 32; ++i) each += part_far[(r_cta * W + w) * 32 + i];
        far += each;
      }
      ms = far * inv_d + eps * f * f;
      if (TINY && ms == 0.f) ms = __uint_as_float(kInfBits);   // a row of zeros is zeros
    }
    const float rstd = TINY ? rsqrtf(ms) : rsqrtf(ms) * f;
    const auto y_of = [&](int i, float (&y)[8]) {
      const float g = TINY ? f : 1.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[2 * j] = bf16_lo(v[i][j]) * g * rstd * wt[i][2 * j];
        y[2 * j + 1] = bf16_hi(v[i][j]) * g * rstd * wt[i][2 * j + 1];
      }
    };
    if constexpr (OUT == kOutE4M3) {
      float am = 0.f;
#pragma unroll
      for (int i = 0; i < ITERS; ++i) {
        float y[8];
        y_of(i, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) am = fmaxf(am, fabsf(y[j]));
      }
      am = row_reduce(am, W, r_cta * W, red_max, MaxF32());
      // the scale is at least 2^-126, so that its inverse stays in range
      const float sc = am > 0.f ? fmaxf(am / 448.f, pow2f(-126)) : 1.f;
      const float inv = sc > pow2f(-126) && am > 0.f ? 448.f / am : 1.f / sc;
      if (row_ok && t == 0 && H3_IN(row >= 0 && row < L, status)) scale[row] = sc;
#pragma unroll
      for (int i = 0; i < ITERS; ++i) {
        const int c = t + i * 32 * W;
        if (row_ok && c < vecs && H3_IN(size_t(row) * vecs + c < size_t(L) * vecs, status)) {
          float y[8];
          y_of(i, y);
          reinterpret_cast<uint2*>(q)[size_t(row) * vecs + c] =
              make_uint2(e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                         e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
        }
      }
    } else {
      const int tiles_k = d / (4 * fp4_block<OUT>());
      uint32_t am[ITERS];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < ITERS; ++i) {
        float y[8];
        y_of(i, y);
        am[i] = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) am[i] = max(am[i], __float_as_uint(y[j]) & 0x7FFFFFFFu);
        am[i] = max(am[i], __shfl_xor_sync(0xffffffffu, am[i], 1));
        if constexpr (OUT == H3_FP4_MX) am[i] = max(am[i], __shfl_xor_sync(0xffffffffu, am[i], 2));
        else top = max(top, am[i] < kInfBits ? am[i] : 0u);
      }
      int e = 0;
      if constexpr (OUT == H3_FP4_NV) {
        e = nv_row_exponent(row_reduce(top, W, r_cta * W, red_top, MaxU32()));
        if (row_ok && t == 0 && H3_IN(row >= 0 && row < L, status)) scale[row] = pow2f(e);
      }
#pragma unroll
      for (int i = 0; i < ITERS; ++i) {
        const int c = t + i * 32 * W;
        const bool live = row_ok && c < vecs;
        const BlockScale sc = block_scale<OUT, false>(am[i], e);
        store_scales8<OUT>(bs, size_t(row), c, tiles_k, sc.byte, live, L, status);
        if (live && H3_IN(size_t(row) * vecs + c < size_t(L) * vecs, status)) {
          float y[8];
          y_of(i, y);
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] *= sc.inv;
          reinterpret_cast<uint32_t*>(q)[size_t(row) * vecs + c] = sc.inv == 0.f ? 0u : e2m1x8(y);
        }
      }
    }
  }
  // a wait that gave up: let the copies still in flight land before the CTA
  // (and its shared memory) goes away
  if (k < nk && threadIdx.x == 0) {
    volatile int no_abort = 0;
    WaitCtx drain{&no_abort, status, kDrainWaitNs};
    for (int j = k; j < issued; ++j)
      mbar_wait(smem_u32(&full[j % stages]), uint32_t(j / stages) & 1u, drain);
  }
}

template <int OUT, int ITERS, bool TINY>
cudaError_t launch_iters(const RmsNormArgs& a, int W, const DevCtx& ctx, cudaStream_t st) {
  const int rows = W >= kWarps ? 1 : kWarps / W, threads = 32 * W * rows;
  // a ring of two to four slots of at most 36 KB in all (more for the widest rows): many small
  // CTAs rather than few large ones (8 warps and 72 KB: 367 instead of 357 us for 58,758 x
  // 5,120, 13.1 instead of 12.5 for 4,099 x 2,048)
  const size_t stage = size_t(rows) * a.d * 2 * (a.res != nullptr ? 2 : 1);
  int stages = int(36 * 1024 / stage);
  stages = stages < 2 ? 2 : (stages > kMaxStages ? kMaxStages : stages);
  const size_t smem = stage * stages;
  static KernelState state;
  const auto kern = rms_norm_kernel<OUT, ITERS, TINY>;
  // two slots of the widest rows with a residual
  if (cudaError_t e = allow_smem(&state, kern, 128 * 1024, ctx)) return e;
  int per_sm = 0;
  if (cudaError_t e = ctas_per_sm(&state, kern, threads, smem, ctx, &per_sm)) return e;
  const int64_t want = (int64_t(a.L) + rows - 1) / rows;
  const int64_t room = int64_t(ctx.num_sms) * per_sm;
  const Launch l(unsigned(want < room ? want : room), threads, smem, st);
  if (cudaError_t e = cudaLaunchKernelEx(
          &l.cfg, kern, static_cast<const uint4*>(a.x), static_cast<const uint4*>(a.res),
          reinterpret_cast<const float4*>(a.weight), a.L, a.d, W, rows, stages, a.eps,
          static_cast<uint4*>(a.sum), static_cast<uint8_t*>(a.q), static_cast<uint8_t*>(a.bs),
          a.scale, ctx.status, ctx.wait_ns))
    return e;
  return cudaGetLastError();
}

template <int OUT, bool TINY>
cudaError_t launch_width(const RmsNormArgs& a, const DevCtx& ctx, cudaStream_t st) {
  const int vecs = a.d >> 3;   // d <= 16384: at most 2048, 16 warps of 4 vectors a thread
  if (vecs <= 32) return launch_iters<OUT, 1, TINY>(a, 1, ctx, st);
  if (vecs <= 64) return launch_iters<OUT, 2, TINY>(a, 1, ctx, st);
  return launch_iters<OUT, 4, TINY>(a, (vecs + 127) / 128, ctx, st);
}

template <int OUT>
cudaError_t launch_out(const RmsNormArgs& a, const DevCtx& ctx, cudaStream_t st) {
  return a.eps < 0x1p-126f ? launch_width<OUT, true>(a, ctx, st) : launch_width<OUT, false>(a, ctx, st);
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
