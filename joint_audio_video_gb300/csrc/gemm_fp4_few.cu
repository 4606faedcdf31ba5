// The 4-bit product for few rows of A (tokens): the weights' bytes and the launch are the
// cost, so the weights take the wide side of the tensor cores and the work is split along K.
//
//   D[128 weight rows][T tokens] = W[128][K] X[T][K]^T   (T = 16, 32 or 64 tokens, M <= T)
//
// A cluster of S CTAs shares one such tile, each a slice of the k-blocks: every CTA streams
// its slice of W and X through a TMA ring and accumulates in tensor memory, then sends each
// token's partial sums to the CTA that owns the token (stores into its shared memory), and
// after one cluster barrier every CTA adds the S partials of its tokens in a fixed order
// and writes rows of C.
//
// Latency bounds it: 6.6 us for 16 tokens through 5,120 x 5,120 (14.8 MB) among others, of
// which a small product (1 x 1,024 x 1,024) takes 3.4 us.  A first version, whose CTAs read the others'
// partials between two cluster barriers, took 9.6; partial sums sent four bytes a store
// instead of sixteen, and factors loaded row by row, 17 instead of 9.4 at 64 tokens.
#include <cuda_bf16.h>

#include "../../include/h3attn_lowp.h"
#include "factors.cuh"
#include "kernels.hpp"
#include "launch.hpp"
#include "ptx.cuh"
#include "tmap.hpp"

namespace h3 {
namespace {

constexpr int kThreads = 128;
constexpr int kBlockK = 256;
constexpr uint32_t kWBytes = 128 * 128;

constexpr int kMaxSplit = 8;

// PER: CTAs an SM (two halve the ring: for more tiles than SMs)
template <int FMT, int T, int PER>
struct FewCfg {
  static constexpr int kVec = FMT == H3_FP4_MX ? 2 : 4;
  static constexpr int kTiles = kVec;                       // scale tiles of a k-block
  static constexpr uint32_t kScaleBytes = kTiles * 512;
  static constexpr uint32_t kXBytes = T * 128;
  static constexpr uint32_t kStageStride = (kWBytes + kXBytes + 2 * kScaleBytes + 1023) / 1024 * 1024;
  // partial sums received: [source CTA][128 weight rows][own tokens, a multiple of 4] fp32;
  // S shares of ceil(T / S / 4) * 4 tokens are max(T, 4 S) tokens
  static constexpr uint32_t kPartialBytes = (T > 4 * kMaxSplit ? T : 4 * kMaxSplit) * 512;
  static constexpr int kFit = ((PER == 2 ? 111 : 225) * 1024 - kPartialBytes) / kStageStride;
  static constexpr int kStages = kFit < 9 ? kFit : 9;
  static constexpr size_t kSmem = size_t(kStages) * kStageStride + kPartialBytes + 1024;
  static constexpr uint32_t kColSfw = T, kColSfx = T + 16;
  static constexpr uint32_t kCols = T + 32 <= 64 ? 64 : (T + 32 <= 128 ? 128 : 256);
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
  const uint8_t* x_bs;    // tiled block scales of X and of W
  const uint8_t* w_bs;
  int* status;
  uint64_t wait_ns;
};

__device__ __forceinline__ void st_cluster_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                              uint32_t d) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                             uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

template <int EPI, int FMT, int T, int PER>
__global__ void __launch_bounds__(kThreads)
    gemm_fp4_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                        const __grid_constant__ FewDev p, int S) {
  using Cfg = FewCfg<FMT, T, PER>;
  constexpr int kStages = Cfg::kStages;
  constexpr bool mx = FMT == H3_FP4_MX;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bar_full[kStages], bar_empty[kStages], bar_acc;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  __shared__ int apart_sh;        // a token's factor is far from 1
  __shared__ float xs_sh[T];      // the tokens' factors
  __shared__ uint8_t md_sh[T];    // and modalities

  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t partial_at = base + kStages * Cfg::kStageStride;
  const float* partial = reinterpret_cast<const float*>(smem_raw + (partial_at - smem_u32(smem_raw)));
  const int warp = warp_id();
  const int rank = S > 1 ? int(cluster_ctarank()) : 0;
  const int nt = int(blockIdx.x) / S;   // weight tile
  const int kblocks = (p.K + kBlockK - 1) / kBlockK;
  const int kb0 = int(int64_t(kblocks) * rank / S), kb1 = int(int64_t(kblocks) * (rank + 1) / S);
  const int tiles_k = p.K / (mx ? 128 : 64);        // scale tiles along K
  const WaitCtx wc{&abort_flag, p.status, p.wait_ns};
  // K = 64 steps of k-block kb: 4, or 2 in the last one of an odd multiple of 128
  const auto steps_of = [&](int kb) { return min(4, (p.K - kb * kBlockK) >> 6); };
  const int live = p.M;                                 // tokens, at most T
  const int share = ((live + S - 1) / S + 3) & ~3;      // of them a CTA's: rank * share ...
  const int n = nt * 128 + int(threadIdx.x);            // this thread's weight row
  if (threadIdx.x == 0) {
    abort_flag = 0;
    apart_sh = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&bar_full[s]), 1);
      mbar_init(smem_u32(&bar_empty[s]), 1);
    }
    mbar_init(smem_u32(&bar_acc), 1);
    fence_barrier_init();
  }
  __syncthreads();
  if (S > 1) cluster_arrive_relaxed();   // waited for below: no store goes to a CTA that has not started
  pdl_trigger();
  pdl_wait();
  // read ahead of their use at the end
  if (int(threadIdx.x) < live && H3_IN(threadIdx.x < T, p.status)) {
    const float xs = p.x_scale != nullptr ? ld_dep(p.x_scale + threadIdx.x) : 1.f;
    xs_sh[threadIdx.x] = xs;
    if (!mid_range(xs)) apart_sh = 1;
    if constexpr (EPI == EPI_GATED_RESIDUAL) md_sh[threadIdx.x] = p.mod[threadIdx.x];
  }
  const float ws = p.w_scale != nullptr && H3_IN(n < p.N, p.status) ? ld_dep(p.w_scale + n) : 1.f;

  bool ok = true;
  int issued = kb0;
  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (lane_id() == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (; issued < kb1; ++issued) {
        if (!mbar_wait(smem_u32(&bar_empty[stage]), phase ^ 1u, wc)) { ok = false; break; }
        const int kb = issued;
        const uint32_t fb = smem_u32(&bar_full[stage]);
        const uint32_t sa = base + stage * Cfg::kStageStride, ss = sa + kWBytes + Cfg::kXBytes;
        // scale tiles of this k-block that exist; columns of codes past K read as zero
        const uint32_t sb = uint32_t(steps_of(kb) * Cfg::kTiles / 4) * 512;
        const size_t w_at = (size_t(nt) * tiles_k + size_t(kb) * Cfg::kTiles) * 512;
        const size_t x_at = size_t(kb) * Cfg::kTiles * 512;
        const bool in = H3_IN(w_at + sb <= size_t(p.N / 128) * tiles_k * 512 &&
                                  x_at + sb <= size_t(tiles_k) * 512,
                              p.status);
        mbar_arrive_expect_tx(fb, kWBytes + Cfg::kXBytes + (in ? 2 * sb : 0));
        tma_load_2d(sa, &tmW, fb, kb * 128, nt * 128);
        tma_load_2d(sa + kWBytes, &tmX, fb, kb * 128, 0);
        if (in) {
          bulk_load_1d(ss, p.w_bs + w_at, sb, fb);
          bulk_load_1d(ss + Cfg::kScaleBytes, p.x_bs + x_at, sb, fb);
        }
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    tmem_alloc(smem_u32(&tmem_base_sh), Cfg::kCols);
    tmem_relinquish();
    __syncwarp();
    tc_fence_after();
    const uint32_t tmem = *static_cast<volatile uint32_t*>(&tmem_base_sh);
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
      const int steps = steps_of(kb);
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
  // ------------------------------------------------------------------ partial sums
  {
    // the issuer waits for its own products whatever happens: it frees their tensor memory
    volatile int no_abort = 0;
    const WaitCtx own{&no_abort, p.status, kDrainWaitNs};
    ok = mbar_wait(smem_u32(&bar_acc), 0, warp == 1 ? own : wc) && ok;
    if (!ok && threadIdx.x == 0) {
      // let the copies still in flight land: each armed stage completes its last phase
      for (int kb = issued - kStages < kb0 ? kb0 : issued - kStages; kb < issued; ++kb)
        mbar_wait(smem_u32(&bar_full[(kb - kb0) % kStages]), uint32_t((kb - kb0) / kStages) & 1u, own);
    }
  }
  ok = !__syncthreads_or(!ok);
  if (S > 1) cluster_wait();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  // Four tokens of a row are one 16-byte piece; the pieces of a row start at its own place
  // and wrap around, so that neighbouring rows' pieces lie in different banks.
  const int pieces = share >> 2;
  const int turn = int(threadIdx.x) % pieces;
  const uint32_t row_at = partial_at + uint32_t(threadIdx.x) * uint32_t(share) * 4;
  if (ok) {
    const uint32_t tacc = tmem + (uint32_t(warp * 32) << 16);
    const uint32_t from = row_at + uint32_t(rank) * 512u * uint32_t(share);
    int owner = 0, piece = 0;   // of the next four tokens
#pragma unroll 1
    for (int c = 0; c < live; c += 32) {
      uint32_t r[32];
      tmem_ld32(tacc + c, r);   // T = 16: the upper half are scale columns, not stored
      tmem_ld_wait(r);
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        if (c + i < live) {
          const int at = piece + turn >= pieces ? piece + turn - pieces : piece + turn;
          const uint32_t to = from + uint32_t(at) * 16;
          if (S > 1) st_cluster_v4(cluster_addr(to, uint32_t(owner)), r[i], r[i + 1], r[i + 2], r[i + 3]);
          else st_shared_v4(to, r[i], r[i + 1], r[i + 2], r[i + 3]);
          if (++piece == pieces) {
            piece = 0;
            ++owner;
          }
        }
      }
    }
  }
  tc_fence_before();
  if (S > 1) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, Cfg::kCols);

  // ------------------------------------------------------------------ rows of C
  bool bad = false;
  const int t0 = rank * share;
  const bool odd = lane_id() & 1;
  // some product of two factors may leave fp32
  const bool apart = __any_sync(0xffffffffu, apart_sh != 0 || !mid_range(ws));
#pragma unroll 1
  for (int g = 0; ok && g < pieces && t0 + 4 * g < live; ++g) {
    const int at = g + turn >= pieces ? g + turn - pieces : g + turn;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    for (int r = 0; r < S; ++r) {
      const float4 f = *reinterpret_cast<const float4*>(
          partial + (size_t(r) * 128 + threadIdx.x) * share + 4 * at);
      v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
    }
    const int t = t0 + 4 * g, left = live - t;   // tokens t .. t + 3, `left` of them live
    float xr[4], gt[4];
    bool mine_bad[4] = {false, false, false, false};
    if constexpr (EPI == EPI_GATED_RESIDUAL) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int md = q < left ? int(md_sh[t + q]) : 0;
        mine_bad[q] = md >= p.n_mod;
        const bool in = H3_IN(q >= left || t + q < p.M, p.status) && H3_IN(n < p.N, p.status);
        xr[q] = q < left && in ? __bfloat162float(p.x_res[size_t(t + q) * p.N + n]) : 0.f;
        gt[q] = mine_bad[q] || !in ? 0.f : ld_dep(p.gate + size_t(md) * p.N + n);
      }
    }
    if (apart) {
      float far[4] = {v[0], v[1], v[2], v[3]};
      times_apart_n(far, left < 4 ? left : 4, ws, xs_sh + t);
      v[0] = far[0], v[1] = far[1], v[2] = far[2], v[3] = far[3];
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] *= (q < left ? xs_sh[t + q] : 0.f) * ws;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if constexpr (EPI == EPI_GELU) {
        float th;   // tanh form, as in gemm_epilogue.cuh
        asm("tanh.approx.f32 %0, %1;" : "=f"(th)
            : "f"(0.7978845608028654f * fmaf(0.044715f * v[q], v[q] * v[q], v[q])));
        v[q] = 0.5f * v[q] * (1.f + th);
      }
      if constexpr (EPI == EPI_GATED_RESIDUAL) {
        v[q] = mine_bad[q] ? __uint_as_float(0x7FC00000u) : fmaf(gt[q], v[q], xr[q]);
        bad |= mine_bad[q];
      }
    }
    // neighbouring lanes swap tokens, so that a lane writes two columns of two tokens
    const float s0 = __shfl_xor_sync(0xffffffffu, odd ? v[0] : v[2], 1);
    const float s1 = __shfl_xor_sync(0xffffffffu, odd ? v[1] : v[3], 1);
    const uint32_t o0 = odd ? pack_bf16x2(s0, v[2]) : pack_bf16x2(v[0], s0);
    const uint32_t o1 = odd ? pack_bf16x2(s1, v[3]) : pack_bf16x2(v[1], s1);
    const int q0 = odd ? 2 : 0;
    __nv_bfloat16* c = p.C + size_t(t + q0) * p.N + (n & ~1);
    if (q0 < left && H3_IN(t + q0 < p.M && n < p.N, p.status))
      *reinterpret_cast<uint32_t*>(c) = o0;
    if (q0 + 1 < left && H3_IN(t + q0 + 1 < p.M && n < p.N, p.status))
      *reinterpret_cast<uint32_t*>(c + p.N) = o1;
  }
  if (bad) atomicCAS(p.status, H3_DEV_OK, H3_DEV_BAD_INDEX);
}

template <int EPI, int FMT, int T, int PER>
cudaError_t launch_per(const GemmFp4Args& a, int S, const DevCtx& ctx, cudaStream_t st) {
  using Cfg = FewCfg<FMT, T, PER>;
  CUtensorMap tmW, tmX;
  const uint64_t kbytes = uint64_t(a.K) / 2;
  if (!make_tmap_u8_2d(&tmW, a.B, a.N, kbytes, kbytes, 128) ||
      !make_tmap_u8_2d(&tmX, a.A, a.M, kbytes, kbytes, T))
    return cudaErrorInvalidValue;
  const FewDev p{static_cast<__nv_bfloat16*>(a.C), a.M, a.N, a.K, a.a_s, a.b_s,
                 static_cast<const __nv_bfloat16*>(a.x_res), a.mod, a.gate, a.n_mod,
                 static_cast<const uint8_t*>(a.a_bs), static_cast<const uint8_t*>(a.b_bs),
                 ctx.status, ctx.wait_ns};
  const int units = a.N / 128;
  static KernelState state;
  const auto kern = gemm_fp4_few_kernel<EPI, FMT, T, PER>;
  if (cudaError_t e = allow_smem(&state, kern, Cfg::kSmem, ctx)) return e;
  const Launch l(unsigned(units) * unsigned(S), kThreads, Cfg::kSmem, st, S);
  if (cudaError_t e = cudaLaunchKernelEx(&l.cfg, kern, tmW, tmX, p, S)) return e;
  return cudaGetLastError();
}

template <int EPI, int FMT, int T>
cudaError_t launch_t(const GemmFp4Args& a, const DevCtx& ctx, cudaStream_t st) {
  // The split with the least estimated time, in units of a k-block (0.2 us at T = 16): waves
  // of clusters times the fixed part of a wave (21, launch included) and its k-blocks, but
  // no less than the weights' bytes take.  Clusters of four and eight leave some SMs out: 36 and
  // 15 of them, of 38 and 19, are taken to run at once on 152 SMs.
  const int64_t units = a.N / 128;
  const int64_t kblocks = (a.K + kBlockK - 1) / kBlockK;
  const int64_t floor = 21 + int64_t(a.N) * a.K / 2200000;
  int S = 1, per = 1;
  int64_t best = INT64_MAX;
  for (int c = 1; c <= (T <= 32 ? 2 : 1); ++c)
    for (int s = 1; s <= kMaxSplit && s <= kblocks; s *= 2) {
      const int64_t room =
          c * (s <= 2 ? ctx.num_sms / s : (s == 4 ? ctx.num_sms * 9 / 38 : ctx.num_sms / 10));
      const int64_t t = (units + room - 1) / room * (21 + (kblocks + s - 1) / s);
      const int64_t cost = t > floor ? t : floor;
      if (cost < best) {
        best = cost;
        S = s;
        per = c;
      }
    }
  if constexpr (T <= 32) {
    if (per == 2) return launch_per<EPI, FMT, T, 2>(a, S, ctx, st);
  }
  return launch_per<EPI, FMT, T, 1>(a, S, ctx, st);
}

template <int EPI, int FMT>
cudaError_t launch_fmt(const GemmFp4Args& a, const DevCtx& ctx, cudaStream_t st) {
  if (a.M <= 16) return launch_t<EPI, FMT, 16>(a, ctx, st);
  if (a.M <= 32) return launch_t<EPI, FMT, 32>(a, ctx, st);
  return launch_t<EPI, FMT, 64>(a, ctx, st);
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
