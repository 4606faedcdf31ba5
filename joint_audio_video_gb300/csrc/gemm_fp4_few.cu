// The 4-bit product for few rows of A (tokens): the weights' bytes and the launch are the
// cost, so the weights take the wide side of the tensor cores and the work is split along K.
//
//   D[128 weight rows][T tokens] = W[128][K] X[T][K]^T   (T = 16, 32, 64 or 128)
//
// A cluster of S CTAs shares one such tile, each a slice of the k-blocks: every CTA
// streams its slice of W and X through a TMA ring (two CTAs fit an SM, so a slice's loads
// are nearly all in flight at once), accumulates in tensor memory, and leaves its partial
// tile in shared memory; the CTAs then add the S partials of their share of the tokens,
// read through distributed shared memory in a fixed order, and write rows of C.
#include <cuda_bf16.h>

#include "../../include/h3attn_lowp.h"
#include "kernels.hpp"
#include "ptx.cuh"
#include "tmap.hpp"

namespace h3 {
namespace {

constexpr int kThreads = 128;
constexpr int kBlockK = 256;
constexpr uint32_t kWBytes = 128 * 128;

template <int FMT, int T>
struct FewCfg {
  static constexpr int kVec = FMT == H3_FP4_MX ? 2 : 4;
  static constexpr int kTiles = kVec;                       // scale tiles of a k-block
  static constexpr uint32_t kScaleBytes = kTiles * 512;
  static constexpr uint32_t kXBytes = T * 128;
  static constexpr uint32_t kStageBytes = kWBytes + kXBytes + 2 * kScaleBytes;
  static constexpr uint32_t kStageStride = (kStageBytes + 1023) / 1024 * 1024;
  // two CTAs an SM: at most 113 KB each
  static constexpr int kStages = 111 * 1024 / kStageStride;
  static constexpr size_t kSmem = size_t(kStages) * kStageStride + 1024;
  static constexpr uint32_t kColSfw = T, kColSfx = T + 16;
  static constexpr uint32_t kCols = T + 32 <= 64 ? 64 : (T + 32 <= 128 ? 128 : 256);
  static_assert(size_t(T) * 512 <= size_t(kStages) * kStageStride, "");   // the partial tile
};

struct FewDev {
  __nv_bfloat16* C;
  int M, N, K;
  const float* x_scale;   // a_s: [M] or nullptr
  const float* w_scale;   // b_s: [N] or nullptr
  const __nv_bfloat16* x_res;
  const uint8_t* mod;
  const float* gate;
  int n_mod;
  int* status;
  uint64_t wait_ns;
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

template <int EPI, int FMT, int T>
__global__ void __launch_bounds__(kThreads, 2)
    gemm_fp4_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                        const __grid_constant__ CUtensorMap tmSW, const __grid_constant__ CUtensorMap tmSX,
                        const __grid_constant__ FewDev p, int S) {
  using Cfg = FewCfg<FMT, T>;
  constexpr int kStages = Cfg::kStages;
  constexpr bool mx = FMT == H3_FP4_MX;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bar_full[kStages], bar_empty[kStages], bar_acc;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;

  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  float* partial = reinterpret_cast<float*>(smem_raw + (base - smem_u32(smem_raw)));
  const int warp = warp_id();
  const int rank = S > 1 ? int(cluster_ctarank()) : 0;
  const int unit = int(blockIdx.x) / S;
  const int num_n = p.N >> 7;
  const int nt = unit % num_n, mt = unit / num_n;   // weight tile, token tile
  const int kblocks = (p.K + kBlockK - 1) / kBlockK;
  const int kb0 = int(int64_t(kblocks) * rank / S), kb1 = int(int64_t(kblocks) * (rank + 1) / S);
  const WaitCtx wc{&abort_flag, p.status, p.wait_ns};

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&bar_full[s]), 1);
      mbar_init(smem_u32(&bar_empty[s]), 1);
    }
    mbar_init(smem_u32(&bar_acc), 1);
    fence_barrier_init();
  }
  const auto load = [&](int kb, int stage) {
    const uint32_t fb = smem_u32(&bar_full[stage]);
    const uint32_t sa = base + stage * Cfg::kStageStride;
    mbar_arrive_expect_tx(fb, Cfg::kStageBytes);
    tma_load_2d(sa, &tmW, fb, kb * 128, nt * 128);
    tma_load_2d(sa + kWBytes, &tmX, fb, kb * 128, mt * T);
    tma_load_2d(sa + kWBytes + Cfg::kXBytes, &tmSW, fb, kb * Cfg::kTiles * 64, nt);
    // T < 128 serves M <= T: the tokens' scales start a 128-row group either way
    tma_load_2d(sa + kWBytes + Cfg::kXBytes + Cfg::kScaleBytes, &tmSX, fb, kb * Cfg::kTiles * 64, mt);
  };
  // the first loads go out before the CTA has met: only this thread has used the barriers
  int issued = kb0;
  if (threadIdx.x == 0)
    for (; issued < kb1 && issued - kb0 < kStages; ++issued) load(issued, issued - kb0);
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_base_sh), Cfg::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;

  bool ok = true;
  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (lane_id() == 0) {
      int stage = 0;
      uint32_t phase = 1;   // the refills start with the second use of stage 0
      if (issued - kb0 < kStages) issued = kb1;
      for (; issued < kb1; ++issued) {
        if (!mbar_wait(smem_u32(&bar_empty[stage]), phase ^ 1u, wc)) { ok = false; break; }
        load(issued, stage);
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    const bool leader = elect_one();
    const SDesc dW0 = sdesc_split(sdesc_sw128(base, 16, 1024));
    const SDesc dX0 = sdesc_split(sdesc_sw128(base + kWBytes, 16, 1024));
    const SDesc dS0 = sdesc_split(sdesc_plain(base + kWBytes + Cfg::kXBytes));
    int stage = 0;
    uint32_t phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar_full[stage]), phase, wc));
      if (!ok) break;
      tc_fence_after();
      const uint32_t soff = stage * (Cfg::kStageStride >> 4);
      const SDesc dW{dW0.lo + soff, dW0.hi}, dX{dX0.lo + soff, dX0.hi}, dS{dS0.lo + soff, dS0.hi};
      const int steps = min(4, (p.K - kb * kBlockK) >> 6);
      if (leader) {
#pragma unroll
        for (int c = 0; c < Cfg::kTiles; ++c) {
          if (c * 4 >= steps * Cfg::kTiles) break;   // tiles past K
          tmem_cp_scales<1>(tmem + Cfg::kColSfw + 4 * c, sdesc_at(dS, c * 512));
          tmem_cp_scales<1>(tmem + Cfg::kColSfx + 4 * c, sdesc_at(dS, Cfg::kScaleBytes + c * 512));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k >= steps) break;
          const uint32_t col = 4u * uint32_t(mx ? k >> 1 : k);
          mma_f4_ss<Cfg::kVec, 1>(tmem, sdesc_at(dW, k * 32), sdesc_at(dX, k * 32),
                                  idesc_e2m1_f32(128, T, mx, mx ? (k & 1) * 2 : 0),
                                  tmem + Cfg::kColSfw + col, tmem + Cfg::kColSfx + col,
                                  ((kb - kb0) | k) != 0);
        }
        tc_commit(smem_u32(&bar_empty[stage]));
      }
      __syncwarp();
      if (++stage == kStages) { stage = 0; phase ^= 1u; }
    }
    if (leader) tc_commit(smem_u32(&bar_acc));   // also after a failure: what was issued is done
    __syncwarp();
  }
  // ------------------------------------------------------------------ partial tile
  {
    // the issuer waits for its own products whatever happens: it frees their tensor memory
    volatile int no_abort = 0;
    const WaitCtx own{&no_abort, p.status, kDrainWaitNs};
    ok = mbar_wait(smem_u32(&bar_acc), 0, warp == 1 ? own : wc) && ok;
    if (!ok && threadIdx.x == 0) {
      // let the copies still in flight land: each armed stage completes its last phase
      WaitCtx land{&no_abort, p.status, kDrainWaitNs};
      for (int kb = issued - kStages < kb0 ? kb0 : issued - kStages; kb < issued; ++kb)
        mbar_wait(smem_u32(&bar_full[(kb - kb0) % kStages]), uint32_t((kb - kb0) / kStages) & 1u, land);
    }
  }
  ok = !__syncthreads_or(!ok);
  tc_fence_after();
  const int m0 = mt * T;
  const int live = min(T, p.M - m0);   // tokens of this tile
  if (ok) {
    // the ring is done with: weight row `lane` of token t at partial[t][lane]
    const uint32_t tacc = tmem + (uint32_t(warp * 32) << 16);
#pragma unroll 1
    for (int c = 0; c < live; c += 32) {
      uint32_t r[32];
      tmem_ld32(tacc + c, r);   // T = 16: the upper half are scale columns, not stored
      tmem_ld_wait(r);
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (c + i < live) partial[(c + i) * 128 + threadIdx.x] = __uint_as_float(r[i]);
    }
  }
  tc_fence_before();
  if (S > 1) cluster_sync();
  else __syncthreads();

  // ------------------------------------------------------------------ rows of C
  bool bad = false;
  const int n0 = nt * 128 + int(lane_id()) * 4;
  float4 ws = make_float4(1.f, 1.f, 1.f, 1.f);
  if (p.w_scale != nullptr) ws = __ldg(reinterpret_cast<const float4*>(p.w_scale + n0));
  for (int t = rank * 4 + warp; ok && t < live; t += 4 * S) {
    const int m = m0 + t;
    if (!H3_IN(m >= 0 && m < p.M && n0 + 4 <= p.N, p.status)) continue;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    const uint32_t at = base + uint32_t(t * 128 + int(lane_id()) * 4) * 4;
    if (S > 1) {
      float4 f[8];   // all loads before the first sum
#pragma unroll
      for (int r = 0; r < 8; ++r)
        f[r] = r < S ? ld_cluster_f4(cluster_addr(at, uint32_t(r))) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int r = 0; r < 8; ++r) v[0] += f[r].x, v[1] += f[r].y, v[2] += f[r].z, v[3] += f[r].w;
    } else {
      const float4 f = *reinterpret_cast<const float4*>(partial + t * 128 + lane_id() * 4);
      v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    }
    const float xs = p.x_scale != nullptr ? __ldg(p.x_scale + m) : 1.f;
    v[0] *= xs * ws.x, v[1] *= xs * ws.y, v[2] *= xs * ws.z, v[3] *= xs * ws.w;
    if constexpr (EPI == EPI_GELU) {
      // tanh form, as in gemm_epilogue.cuh
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float u = v[i];
        float th;
        asm("tanh.approx.f32 %0, %1;" : "=f"(th) : "f"(0.7978845608028654f * fmaf(0.044715f * u, u * u, u)));
        v[i] = 0.5f * u * (1.f + th);
      }
    }
    if constexpr (EPI == EPI_GATED_RESIDUAL) {
      const int md = p.mod[m];
      if (md >= p.n_mod) {
        bad = true;
        v[0] = v[1] = v[2] = v[3] = __uint_as_float(0x7FC00000u);
      } else {
        const uint2 xr = *reinterpret_cast<const uint2*>(p.x_res + size_t(m) * p.N + n0);
        const float4 g = __ldg(reinterpret_cast<const float4*>(p.gate + size_t(md) * p.N + n0));
        v[0] = fmaf(g.x, v[0], __uint_as_float(xr.x << 16));
        v[1] = fmaf(g.y, v[1], __uint_as_float(xr.x & 0xFFFF0000u));
        v[2] = fmaf(g.z, v[2], __uint_as_float(xr.y << 16));
        v[3] = fmaf(g.w, v[3], __uint_as_float(xr.y & 0xFFFF0000u));
      }
    }
    *reinterpret_cast<uint2*>(p.C + size_t(m) * p.N + n0) =
        make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  }
  if (bad) atomicCAS(p.status, H3_DEV_OK, H3_DEV_BAD_INDEX);
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, Cfg::kCols);
  if (S > 1) cluster_sync();   // no CTA leaves while another may still read its partial tile
}

template <int EPI, int FMT, int T>
cudaError_t launch_t(const GemmFp4Args& a, const DevCtx& ctx, cudaStream_t st) {
  using Cfg = FewCfg<FMT, T>;
  CUtensorMap tmW, tmX, tmSW, tmSX;
  const uint64_t kbytes = uint64_t(a.K) / 2, tiles = uint64_t(a.K) / (FMT == H3_FP4_MX ? 128 : 64);
  if (!make_tmap_u8_2d(&tmW, a.B, a.N, kbytes, kbytes, 128) ||
      !make_tmap_u8_2d(&tmX, a.A, a.M, kbytes, kbytes, T) ||
      !make_tmap_scales(&tmSW, a.b_bs, a.N / 128, tiles, 1, Cfg::kTiles) ||
      !make_tmap_scales(&tmSX, a.a_bs, (a.M + 127ull) / 128, tiles, 1, Cfg::kTiles))
    return cudaErrorInvalidValue;
  const FewDev p{static_cast<__nv_bfloat16*>(a.C), a.M, a.N, a.K, a.a_s, a.b_s,
                 static_cast<const __nv_bfloat16*>(a.x_res), a.mod, a.gate, a.n_mod, ctx.status,
                 ctx.wait_ns};
  const int units = a.N / 128 * ((a.M + T - 1) / T);
  const int kblocks = (a.K + kBlockK - 1) / kBlockK;
  int S = 1;
  while (S < 8 && units * S * 2 <= 2 * ctx.num_sms + ctx.num_sms / 8 && S * 2 <= kblocks) S *= 2;
  auto kern = gemm_fp4_few_kernel<EPI, FMT, T>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       int(Cfg::kSmem));
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(S);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(units) * unsigned(S));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg::kSmem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = S > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kern, tmW, tmX, tmSW, tmSX, p, S);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

template <int EPI, int FMT>
cudaError_t launch_fmt(const GemmFp4Args& a, const DevCtx& ctx, cudaStream_t st) {
  if (a.M <= 16) return launch_t<EPI, FMT, 16>(a, ctx, st);
  if (a.M <= 32) return launch_t<EPI, FMT, 32>(a, ctx, st);
  if (a.M <= 64) return launch_t<EPI, FMT, 64>(a, ctx, st);
  return launch_t<EPI, FMT, 128>(a, ctx, st);
}

template <int EPI>
cudaError_t launch_epi(const GemmFp4Args& a, const DevCtx& ctx, cudaStream_t st) {
  return a.fmt == H3_FP4_MX ? launch_fmt<EPI, H3_FP4_MX>(a, ctx, st)
                            : launch_fmt<EPI, H3_FP4_NV>(a, ctx, st);
}

}  // namespace

cudaError_t launch_gemm_fp4_few(const GemmFp4Args& a, const DevCtx& ctx, cudaStream_t st) {
  switch (a.epilogue) {
    case EPI_PLAIN: return launch_epi<EPI_PLAIN>(a, ctx, st);
    case EPI_GATED_RESIDUAL: return launch_epi<EPI_GATED_RESIDUAL>(a, ctx, st);
    case EPI_GELU: return launch_epi<EPI_GELU>(a, ctx, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace h3
