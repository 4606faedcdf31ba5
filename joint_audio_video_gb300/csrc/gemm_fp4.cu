// Persistent tcgen05 GEMM over microscaled 4-bit operands (h3attn_lowp.h):
//   C[M][N] = a_s[m] b_s[n] sum_k A[m][k] B[n][k],  fp32 accumulation, with the
// epilogues of gemm_epilogue.cuh.
//
// The tensor cores multiply E2M1 codes and apply one scale of A and one of B to every
// block of columns (kind::mxf4nvf4, E4M3 scales of 16; kind::mxf4, E8M0 of 32), so the
// codes go from global memory to the product as they are, 128 bytes (256 columns) of a
// row per k-block, and the scales follow them: a k-block's scale tiles arrive by TMA
// next to the codes and are copied from shared to tensor memory (tcgen05.cp) just
// before the products that read them.  The copies and the products of a k-block are
// issued by one thread and run in order, so one set of scale columns serves every
// k-block.
//
// Two forms here, both persistent: one CTA for a 128 x 128 tile (192 threads: TMA producer,
// MMA issuer, four epilogue warps, two accumulators, as in gemm.cu), and a CTA pair for a
// 256 x 256 tile, below.  Few rows of A take other kernels; launch_fmt at the end chooses.
#include <cuda_bf16.h>

#include "../../include/h3attn_lowp.h"
#include "gemm_epilogue.cuh"
#include "kernels.hpp"
#include "launch.hpp"
#include "ptx.cuh"
#include "tmap.hpp"

namespace h3 {
namespace {

constexpr int kThreads = 192;
constexpr int kGroupM = 16;
constexpr int BN = 128;
constexpr int kBlockK = 256;                          // columns of a k-block: 128 bytes of codes
constexpr int kStages = 5;
constexpr uint32_t kTileBytes = 128 * 128;            // 128 rows of a k-block

template <int FMT>
struct Fp4Cfg {
  static constexpr int kVec = FMT == H3_FP4_MX ? 2 : 4;            // scales of a K = 64 step
  static constexpr int kTiles = kVec;                              // scale tiles of a k-block
  static constexpr uint32_t kScaleBytes = kTiles * 512;            // of 128 rows
  static constexpr uint32_t kStageBytes = 2 * kTileBytes + 2 * kScaleBytes;
  static constexpr size_t kSmem = size_t(kStages) * kStageBytes + 2 * kStageC + 1024;
};
// tensor memory columns: two accumulators, then the scales of A and of B
constexpr uint32_t kColSfa = 2 * BN, kColSfb = kColSfa + 16, kTmemCols = 512;

template <int EPI, int FMT>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_fp4_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                    const __grid_constant__ CUtensorMap tmC, const __grid_constant__ GemmDev p) {
  using Cfg = Fp4Cfg<FMT>;
  constexpr int S = kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bar_full[S], bar_empty[S], bar_acc_full[2], bar_acc_empty[2], bar_drain;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;

  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int warp = warp_id();
  const WaitCtx wc{&abort_flag, p.status, p.wait_ns};

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&bar_full[s]), 1);
      mbar_init(smem_u32(&bar_empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&bar_acc_full[a]), 1);
      mbar_init(smem_u32(&bar_acc_empty[a]), 128);
    }
    mbar_init(smem_u32(&bar_drain), 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_base_sh), kTmemCols);
    tmem_relinquish();
  }
  if (warp == 0 && lane_id() == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmSA);
    tma_prefetch_desc(&tmSB);
    tma_prefetch_desc(&tmC);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  pdl_wait();
  const uint32_t tmem = tmem_base_sh;

  const int num_tiles = p.num_m * p.num_n;
  const int kblocks = (p.K + kBlockK - 1) / kBlockK;

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (lane_id() == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < num_tiles && ok; t += gridDim.x) {
        int mb, nb;
        tile_coords(t, p.num_m, p.num_n, mb, nb, kGroupM);
        for (int kb = 0; kb < kblocks; ++kb) {
          if (!mbar_wait(smem_u32(&bar_empty[stage]), phase ^ 1u, wc)) { ok = false; break; }
          const uint32_t fb = smem_u32(&bar_full[stage]);
          const uint32_t sa = base + stage * Cfg::kStageBytes;
          // columns and tiles past K read as zero; their bytes count all the same
          mbar_arrive_expect_tx(fb, Cfg::kStageBytes);
          tma_load_2d(sa, &tmA, fb, kb * 128, mb * BM);
          tma_load_2d(sa + kTileBytes, &tmB, fb, kb * 128, nb * BN);
          tma_load_2d(sa + 2 * kTileBytes, &tmSA, fb, kb * Cfg::kTiles * 64, mb);
          tma_load_2d(sa + 2 * kTileBytes + Cfg::kScaleBytes, &tmSB, fb, kb * Cfg::kTiles * 64, nb);
          if (++stage == S) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok) {
        // unwind: let copies already in flight land before the CTA exits
        WaitCtx drain{&abort_flag, p.status, kDrainWaitNs};
        volatile int no_abort = 0;
        drain.abort = &no_abort;
        for (int s = 0; s < S; ++s) {
          // a stage is in flight iff its full barrier is one phase behind the ring
          const uint32_t par = (s < stage) ? phase : (phase ^ 1u);
          mbar_wait(smem_u32(&bar_full[s]), par, drain);
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    const bool leader = elect_one();
    const SDesc dA0 = sdesc_split(sdesc_sw128(base, 16, 1024));
    const SDesc dB0 = sdesc_split(sdesc_sw128(base + kTileBytes, 16, 1024));
    const SDesc dS0 = sdesc_split(sdesc_plain(base + 2 * kTileBytes));
    int stage = 0;
    uint32_t phase = 0;
    int it = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < num_tiles && ok; t += gridDim.x, ++it) {
      const int acc = it & 1;
      const uint32_t acc_phase = (it >> 1) & 1;
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar_acc_empty[acc]), acc_phase ^ 1u, wc));
      if (!ok) break;
      tc_fence_after();
      const uint32_t dtm = tmem + acc * BN;
      for (int kb = 0; kb < kblocks; ++kb) {
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar_full[stage]), phase, wc));
        if (!ok) break;
        tc_fence_after();
        const uint32_t soff = stage * (Cfg::kStageBytes >> 4);
        const SDesc dA{dA0.lo + soff, dA0.hi}, dB{dB0.lo + soff, dB0.hi}, dS{dS0.lo + soff, dS0.hi};
        // K = 64 steps of this k-block: 4, or 2 in the last one of an odd multiple of 128
        const int steps = min(4, (p.K - kb * kBlockK) >> 6);
        if (leader) {
#pragma unroll
          for (int c = 0; c < Cfg::kTiles; ++c) {
            if (c * 4 >= steps * Cfg::kTiles) break;   // tiles past K
            tmem_cp_scales<1>(tmem + kColSfa + 4 * c, sdesc_at(dS, c * 512));
            tmem_cp_scales<1>(tmem + kColSfb + 4 * c, sdesc_at(dS, Cfg::kScaleBytes + c * 512));
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k >= steps) break;
            constexpr bool mx = FMT == H3_FP4_MX;
            const uint32_t col = 4u * uint32_t(mx ? k >> 1 : k);
            mma_f4_ss<Cfg::kVec, 1>(dtm, sdesc_at(dA, k * 32), sdesc_at(dB, k * 32),
                                    idesc_e2m1_f32(BM, BN, mx, mx ? (k & 1) * 2 : 0),
                                    tmem + kColSfa + col, tmem + kColSfb + col, (kb | k) != 0);
          }
          tc_commit(smem_u32(&bar_empty[stage]));
        }
        __syncwarp();
        if (++stage == S) { stage = 0; phase ^= 1u; }
      }
      if (!ok) break;
      if (leader) tc_commit(smem_u32(&bar_acc_full[acc]));
      __syncwarp();
    }
    // drain: every MMA issued so far has finished before TMEM is released
    if (leader) tc_commit(smem_u32(&bar_drain));
    __syncwarp();
    WaitCtx drain{&abort_flag, p.status, kDrainWaitNs};
    volatile int no_abort = 0;
    drain.abort = &no_abort;
    mbar_wait(smem_u32(&bar_drain), 0, drain);
  } else {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3;                 // TMEM lane quarter of this warp
    const int row_in_tile = q * 32 + lane_id();
    const bool leader = threadIdx.x == 64;   // issues the C stores
    const uint32_t sC = base + S * Cfg::kStageBytes;
    const RopeTable rt{};
    int chunk = 0;                           // C chunks staged so far (buffer parity)
    int it = 0;
    for (int t = blockIdx.x; t < num_tiles; t += gridDim.x, ++it) {
      int mb, nb;
      tile_coords(t, p.num_m, p.num_n, mb, nb, kGroupM);
      const int acc = it & 1;
      const uint32_t acc_phase = (it >> 1) & 1;
      // all four epilogue warps leave together (they share the staging barrier)
      const bool ok = epi_bar_and(mbar_wait(smem_u32(&bar_acc_full[acc]), acc_phase, wc));
      if (!ok) break;
      tc_fence_after();
      const uint32_t tacc = tmem + acc * BN + (uint32_t(q * 32) << 16);
      const bool bad = epilogue_tile<BN, EPI, 2>(p, rt, &tmC, tacc, mb * BM, nb * BN, row_in_tile,
                                                 leader, sC, chunk);
      if (bad) atomicCAS(p.status, H3_DEV_OK, H3_DEV_BAD_INDEX);
      tc_fence_before();
      mbar_arrive(smem_u32(&bar_acc_empty[acc]));
    }
    // every C store has finished before the CTA (and its shared memory) goes away
    if (leader) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

// ---------------------------------------------------------------------------
// CTA-pair form (cta_group::2), for N % 256 == 0.  A cluster of two CTAs computes one
// 256 x 256 tile: each CTA loads 128 rows of A with their scales, 128 rows of B, and the
// scales of all 256 rows of B (each CTA's tensor memory needs them); the even CTA's issuer
// copies the scales of both and multiplies.
//
// Tensor memory: two 256-column accumulators and 48 scale columns do not fit 512, so the
// accumulators share 64 columns:
//   even tiles [0, 256)   odd tiles [192, 448)   scales of A [448, 464), of B [464, 496)
// The epilogue reads the shared columns of a tile first and hands them over; the next
// tile's products start then, while the epilogue goes on with the other 192.
//
// The ring is what bounds it.  A stage's refill takes ~2,300 SM cycles from the commit that
// frees it to its bytes being seen, a k-block multiplies in 512, and a stage is 38 KB (NV)
// or 35 KB (MX): with 3, 4, 5 NV stages a k-block took 912, 714, 620 cycles (16,384 x 5,120
// x 20,480), with 5 and 6 MX stages 586 and 556.  One thread issues a stage's four copies in
// a row, each late by those before it: two producer threads (A with its scales, B with its)
// take 4 to 5 % off; four take another 5 % off MX and nothing off NV.  The scale copies from
// shared to tensor memory cost nothing that could be measured.
constexpr int kPairGroupM = 16;
constexpr uint32_t kStageC64 = 128 * 128;             // 128 rows x 64 columns of C
constexpr uint32_t kPairAcc1 = 192, kPairSfa = 448, kPairSfb = 464;

template <int FMT>
struct PairCfg {
  static constexpr int kTiles = Fp4Cfg<FMT>::kTiles;
  static constexpr uint32_t kScaleBytes = kTiles * 512;
  static constexpr uint32_t kStageBytes = 2 * kTileBytes + 3 * kScaleBytes;
  // a multiple of 1 KB, so every stage's code tiles keep the swizzle's alignment
  static constexpr uint32_t kStageStride = (kStageBytes + 1023) / 1024 * 1024;
  // all of the 227 KB: a sixth stage (MX) rather than a second staging buffer for C
  static constexpr int kStages = FMT == H3_FP4_MX ? 6 : 5;
  static constexpr int kBufs = FMT == H3_FP4_MX ? 1 : 2;
  // warps: producer 0, issuer, 4 epilogue, then the other producers
  static constexpr int kProducers = FMT == H3_FP4_MX ? 4 : 2;
  static constexpr int kThreads = 32 * (5 + kProducers);
  // NV: the factors of a tile's 256 rows of B, staged before its accumulator is ready (read
  // from global memory inside the epilogue they cost a cache miss for every 64 columns:
  // 4,096 x 6,144 x 2,048 took 38.6 us, now 24.4).  MX has no room for them and seldom any factors.
  static constexpr bool kFactors = FMT == H3_FP4_NV;
  static constexpr uint32_t kFactorAt = kStages * kStageStride + kBufs * kStageC64;   // offset
  static constexpr uint32_t kBars = kFactorAt + (kFactors ? 2 * 1024 : 0);
  static constexpr size_t kSmem = kBars + 256;
  static_assert(kSmem <= 227 * 1024, "");
};

template <int EPI, int FMT>
__global__ void __launch_bounds__(PairCfg<FMT>::kThreads, 1)
    gemm_fp4_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                         const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                         const __grid_constant__ CUtensorMap tmC, const __grid_constant__ GemmDev p) {
  using Cfg = PairCfg<FMT>;
  constexpr int S = Cfg::kStages;
  constexpr bool mx = FMT == H3_FP4_MX;
  // no static shared memory, so the dynamic part starts on its 1 KB boundary
  extern __shared__ __align__(1024) uint8_t smem_pair[];
  struct Bars {
    uint64_t full[S], empty[S], acc_full[2], shared_cols, drain;
    uint32_t tmem_base;
    int abort;
  };
  static_assert(sizeof(Bars) <= 256, "");
  Bars& bars = *reinterpret_cast<Bars*>(smem_pair + Cfg::kBars);
  uint64_t(&bar_full)[S] = bars.full;
  uint64_t(&bar_empty)[S] = bars.empty;
  uint64_t(&bar_acc_full)[2] = bars.acc_full;
  uint64_t& bar_shared_cols = bars.shared_cols;
  uint64_t& bar_drain = bars.drain;
  uint32_t& tmem_base_sh = bars.tmem_base;
  int& abort_flag = bars.abort;

  const uint32_t base = smem_u32(smem_pair);
  const int warp = warp_id();
  const uint32_t rank = cluster_ctarank();   // 0: issues the pair's products
  const bool lead = rank == 0;
  const WaitCtx wc{&abort_flag, p.status, p.wait_ns};

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&bar_full[s]), 1);    // the even CTA's: both CTAs' bytes
      mbar_init(smem_u32(&bar_empty[s]), 1);   // one multicast commit
    }
    for (int a = 0; a < 2; ++a) mbar_init(smem_u32(&bar_acc_full[a]), 1);
    mbar_init(smem_u32(&bar_shared_cols), 2);  // the even CTA's: one per CTA
    mbar_init(smem_u32(&bar_drain), 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&tmem_base_sh), kTmemCols);
    tmem_relinquish_pair();
  }
  if (warp == 0 && lane_id() == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmSA);
    tma_prefetch_desc(&tmSB);
    tma_prefetch_desc(&tmC);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers exist before any signal crosses
  tc_fence_after();
  pdl_trigger();
  pdl_wait();
  const uint32_t tmem = tmem_base_sh;

  const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;
  const int num_tiles = p.num_m * p.num_n;
  const int kblocks = (p.K + kBlockK - 1) / kBlockK;

  if (warp == 0 || warp >= 6) {
    // ---------------------------------------------------------------- producers
    if (lane_id() == 0) {
      // 0: A's codes, 1: B's, 2: A's scales, 3: B's; with two producers 0 and 1 do both
      const int role = warp == 0 ? 0 : warp - 5;
      constexpr int kP = Cfg::kProducers;
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = cid; t < num_tiles && ok; t += ncl) {
        int mb, nb;
        tile_coords(t, p.num_m, p.num_n, mb, nb, kPairGroupM);
        const int ga = mb * 2 + int(rank), gb = nb * 2;   // 128-row groups of A and of B
        for (int kb = 0; kb < kblocks; ++kb) {
          if (!mbar_wait(smem_u32(&bar_empty[stage]), phase ^ 1u, wc)) { ok = false; break; }
          const uint32_t fb = smem_u32(&bar_full[stage]);
          // the even CTA's first producer arms the barrier for the bytes of all of both CTAs
          // (columns and tiles past K read as zero and count all the same)
          if (lead && role == 0) mbar_arrive_expect_tx(fb, 2 * Cfg::kStageBytes);
          const uint32_t cfb = cluster_addr(fb, 0);
          const uint32_t sa = base + stage * Cfg::kStageStride;
          const int sx = kb * Cfg::kTiles * 64;
          if (role == 0) tma_load_2d_pair(sa, &tmA, cfb, kb * 128, ga * 128);
          if (role == 1)
            tma_load_2d_pair(sa + kTileBytes, &tmB, cfb, kb * 128, (gb + int(rank)) * 128);
          if (role == (0 + 2) % kP) tma_load_2d_pair(sa + 2 * kTileBytes, &tmSA, cfb, sx, ga);
          if (role == (1 + 2) % kP)
            tma_load_2d_pair(sa + 2 * kTileBytes + Cfg::kScaleBytes, &tmSB, cfb, sx, gb);
          if (++stage == S) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok) abort_grace();
      if (!ok && lead && role == 0) {
        // unwind: let the stages armed here land before the CTA exits (the
        // other producers' copies of a stage count on the same barrier)
        WaitCtx drain{&abort_flag, p.status, kDrainWaitNs};
        volatile int no_abort = 0;
        drain.abort = &no_abort;
        for (int s = 0; s < S; ++s) {
          const uint32_t par = (s < stage) ? phase : (phase ^ 1u);
          mbar_wait(smem_u32(&bar_full[s]), par, drain);
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (lead) {
      const bool leader = elect_one();
      const SDesc dA0 = sdesc_split(sdesc_sw128(base, 16, 1024));
      const SDesc dB0 = sdesc_split(sdesc_sw128(base + kTileBytes, 16, 1024));
      const SDesc dS0 = sdesc_split(sdesc_plain(base + 2 * kTileBytes));
      int stage = 0;
      uint32_t phase = 0;
      int it = 0;
      bool ok = true;
      for (int t = cid; t < num_tiles && ok; t += ncl, ++it) {
        if (it > 0) {   // both epilogues have read the columns this tile shares with the last
          ok = __all_sync(0xffffffffu,
                          mbar_wait_cluster(smem_u32(&bar_shared_cols), uint32_t(it - 1) & 1u, wc));
          if (!ok) break;
        }
        tc_fence_after();
        const uint32_t dtm = tmem + (it & 1) * kPairAcc1;
        for (int kb = 0; kb < kblocks; ++kb) {
          ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar_full[stage]), phase, wc));
          if (!ok) break;
          tc_fence_after();
          const uint32_t soff = stage * (Cfg::kStageStride >> 4);
          const SDesc dA{dA0.lo + soff, dA0.hi}, dB{dB0.lo + soff, dB0.hi}, dS{dS0.lo + soff, dS0.hi};
          const int steps = min(4, (p.K - kb * kBlockK) >> 6);
          if (leader) {
#pragma unroll
            for (int c = 0; c < Cfg::kTiles; ++c) {
              if (c * 4 >= steps * Cfg::kTiles) break;   // tiles past K
              tmem_cp_scales<2>(tmem + kPairSfa + 4 * c, sdesc_at(dS, c * 512));
              tmem_cp_scales<2>(tmem + kPairSfb + 8 * c, sdesc_at(dS, Cfg::kScaleBytes + c * 512));
              tmem_cp_scales<2>(tmem + kPairSfb + 8 * c + 4,
                                sdesc_at(dS, 2 * Cfg::kScaleBytes + c * 512));
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (k >= steps) break;
              const uint32_t c = uint32_t(mx ? k >> 1 : k);
              mma_f4_ss<Fp4Cfg<FMT>::kVec, 2>(dtm, sdesc_at(dA, k * 32), sdesc_at(dB, k * 32),
                                              idesc_e2m1_f32(256, 256, mx, mx ? (k & 1) * 2 : 0),
                                              tmem + kPairSfa + 4 * c, tmem + kPairSfb + 8 * c,
                                              (kb | k) != 0);
            }
            tc_commit_pair(smem_u32(&bar_empty[stage]), 0x3);
          }
          __syncwarp();
          if (++stage == S) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        if (leader) tc_commit_pair(smem_u32(&bar_acc_full[it & 1]), 0x3);
        __syncwarp();
      }
      if (leader) tc_commit_pair(smem_u32(&bar_drain), 0x3);
      __syncwarp();
    }
    // every product that writes this CTA's tensor memory has finished
    WaitCtx drain{&abort_flag, p.status, kDrainWaitNs};
    volatile int no_abort = 0;
    drain.abort = &no_abort;
    mbar_wait(smem_u32(&bar_drain), 0, drain);
  } else {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3;
    const int row_in_tile = q * 32 + lane_id();
    const bool leader = threadIdx.x == 64;
    const uint32_t sC = base + S * Cfg::kStageStride;
    const uint32_t shared_cols_c = cluster_addr(smem_u32(&bar_shared_cols), 0);
    const RopeTable rt{};
    int chunk = 0;
    int it = 0;
    for (int t = cid; t < num_tiles; t += ncl, ++it) {
      int mb, nb;
      tile_coords(t, p.num_m, p.num_n, mb, nb, kPairGroupM);
      const int row0 = mb * 256 + int(rank) * 128, grow = row0 + row_in_tile;
      const bool live = grow < p.M;
      const EpilogueRow er = epilogue_row<EPI, 2>(p, grow, live);
      float* factors = reinterpret_cast<float*>(smem_pair + Cfg::kFactorAt) + (it & 1) * 256;
      if constexpr (Cfg::kFactors) {   // the barrier below orders these before their use
        reinterpret_cast<float2*>(factors)[row_in_tile] =
            p.b_scale == nullptr
                ? make_float2(1.f, 1.f)
                : __ldg(reinterpret_cast<const float2*>(p.b_scale + nb * 256) + row_in_tile);
      }
      const bool ok = epi_bar_and(mbar_wait(smem_u32(&bar_acc_full[it & 1]), (it >> 1) & 1, wc));
      if (!ok) break;
      tc_fence_after();
      const uint32_t tacc = tmem + (it & 1) * kPairAcc1 + (uint32_t(q * 32) << 16);
#pragma unroll 1
      for (int j = 0; j < 4; ++j) {
        // 64 columns at a time, those shared with the other accumulator first
        const int c = (it & 1) ? j : (j + 3) & 3;
        uint32_t r0[32], r1[32];
        tmem_ld32(tacc + c * 64, r0);
        tmem_ld32(tacc + c * 64 + 32, r1);
        tmem_ld_wait(r0);
        tmem_ld_wait(r1);
        if (j == 0) {   // the shared columns are in registers
          tc_fence_before();
          epi_bar();
          if (leader) mbar_arrive_cluster(shared_cols_c);
        }
        if (row0 >= p.M) continue;        // uniform in the CTA: nothing to write
        uint32_t pk[32];
        epilogue_64<EPI, Cfg::kFactors ? 3 : 2>(p, rt, r0, r1, er, grow, nb * 256 + c * 64, live, pk,
                                                factors + c * 64);
        const uint32_t sb = sC + uint32_t(chunk % Cfg::kBufs) * kStageC64;
        // the store that last read this staging buffer has done so
        if (leader) {
          if constexpr (Cfg::kBufs == 1) bulk_wait_read_0();
          else bulk_wait_read_1();
        }
        epi_bar();
        const uint32_t srow = sb + uint32_t(row_in_tile) * 128, ssw = uint32_t(row_in_tile) & 7u;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                           srow + ((uint32_t(i) ^ ssw) << 4)),
                       "r"(pk[4 * i]), "r"(pk[4 * i + 1]), "r"(pk[4 * i + 2]), "r"(pk[4 * i + 3])
                       : "memory");
        fence_async_shared();
        epi_bar();
        if (leader) {
          tma_store_2d(&tmC, sb, nb * 256 + c * 64, row0);
          bulk_commit();
        }
        ++chunk;
      }
      if (er.bad) atomicCAS(p.status, H3_DEV_OK, H3_DEV_BAD_INDEX);
    }
    if (leader) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();   // neither CTA leaves while the other may still signal it
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, kTmemCols);
}

inline GemmDev gemm_dev(const GemmFp4Args& a, const DevCtx& ctx, int rows, int cols) {
  GemmDev p{};
  p.C = static_cast<__nv_bfloat16*>(a.C);
  p.M = a.M;
  p.N = a.N;
  p.K = a.K;
  p.num_m = int((int64_t(a.M) + rows - 1) / rows);
  p.num_n = a.N / cols;
  p.x_res = static_cast<const __nv_bfloat16*>(a.x_res);
  p.mod = a.mod;
  p.gate = a.gate;
  p.n_mod = a.n_mod;
  p.status = ctx.status;
  p.wait_ns = ctx.wait_ns;
  p.a_scale = a.a_s;
  p.b_scale = a.b_s;
  return p;
}

// Tensor maps of the operands: 128-row boxes of codes and of their scales (b_groups
// 128-row groups of B's).
struct OperandMaps {
  CUtensorMap A, B, SA, SB;
};
template <int FMT>
bool make_operand_maps(OperandMaps* m, const GemmFp4Args& a, int b_groups) {
  const uint64_t kbytes = uint64_t(a.K) / 2, tiles = uint64_t(a.K) / (FMT == H3_FP4_MX ? 128 : 64);
  return make_tmap_u8_2d(&m->A, a.A, a.M, kbytes, kbytes, 128) &&
         make_tmap_u8_2d(&m->B, a.B, a.N, kbytes, kbytes, 128) &&
         make_tmap_scales(&m->SA, a.a_bs, (a.M + 127ull) / 128, tiles, 1, Fp4Cfg<FMT>::kTiles) &&
         make_tmap_scales(&m->SB, a.b_bs, a.N / 128, tiles, b_groups, Fp4Cfg<FMT>::kTiles);
}

template <int EPI, int FMT>
cudaError_t launch_tiles(const GemmFp4Args& a, const DevCtx& ctx, cudaStream_t st) {
  using Cfg = Fp4Cfg<FMT>;
  OperandMaps m;
  CUtensorMap tmC;
  if (!make_operand_maps<FMT>(&m, a, 1) || !make_tmap_bf16_2d_sw64(&tmC, a.C, a.M, a.N, a.N, BM))
    return cudaErrorInvalidValue;
  const GemmDev p = gemm_dev(a, ctx, BM, BN);
  static KernelState state;
  const auto kern = gemm_fp4_kernel<EPI, FMT>;
  if (cudaError_t e = allow_smem(&state, kern, Cfg::kSmem, ctx)) return e;
  const int num = p.num_m * p.num_n;
  const Launch l(unsigned(num < ctx.num_sms ? num : ctx.num_sms), kThreads, Cfg::kSmem, st);
  if (cudaError_t e = cudaLaunchKernelEx(&l.cfg, kern, m.A, m.B, m.SA, m.SB, tmC, p)) return e;
  return cudaGetLastError();
}

template <int EPI, int FMT>
cudaError_t launch_pairs(const GemmFp4Args& a, const DevCtx& ctx, cudaStream_t st) {
  using Cfg = PairCfg<FMT>;
  OperandMaps m;
  CUtensorMap tmC;
  if (!make_operand_maps<FMT>(&m, a, 2) || !make_tmap_bf16_2d(&tmC, a.C, a.M, a.N, a.N, BM, 64))
    return cudaErrorInvalidValue;
  const GemmDev p = gemm_dev(a, ctx, 256, 256);
  static KernelState state;
  const auto kern = gemm_fp4_pair_kernel<EPI, FMT>;
  if (cudaError_t e = allow_smem(&state, kern, Cfg::kSmem, ctx)) return e;
  // how many pairs can be resident at once, asked once per device
  int nres = state.clusters[ctx.dev].load(std::memory_order_relaxed);
  if (nres <= 0) {
    const Launch all(unsigned(ctx.num_sms & ~1), Cfg::kThreads, Cfg::kSmem, st, 2);
    if (cudaError_t e = cudaOccupancyMaxActiveClusters(&nres, kern, &all.cfg)) return e;
    if (nres <= 0) return cudaErrorInvalidConfiguration;
    state.clusters[ctx.dev].store(nres, std::memory_order_relaxed);
  }
  const int num = p.num_m * p.num_n;
  const Launch l(unsigned(2 * (num < nres ? num : nres)), Cfg::kThreads, Cfg::kSmem, st, 2);
  if (cudaError_t e = cudaLaunchKernelEx(&l.cfg, kern, m.A, m.B, m.SA, m.SB, tmC, p)) return e;
  return cudaGetLastError();
}

// Which kernel (us a call at 5,120 x 5,120 or as given, among others on one GB300):
//   one or two rows, weights up to 2^25 elements   gemv, no tensor cores: 6.4 against 6.9 with
//       few (2,048 x 2,048: 3.2 against 4.7; at 20,480 x 5,120 it is the other way round,
//       17.5 against 13.3, the decoding being what bounds it)
//   up to 32 rows, or 64 where the weight tiles do not outnumber the SMs   few: 7.2 at 16 rows,
//       9.4 at 64, against 10.0 with tiles (20,480 x 5,120 at 64 rows: 27 against 18.5)
//   more   pairs of CTAs (256 x 256) unless single CTAs (128 x 128) need no more waves: 10.7
//       against 11.9 at 358 rows, but 16.5 against 12.4 at 512
template <int EPI, int FMT>
cudaError_t launch_fmt(const GemmFp4Args& a, const DevCtx& ctx, cudaStream_t st) {
  const int64_t weights = int64_t(a.N) * a.K;
  if (a.M <= 2 && weights <= (int64_t(1) << 25)) return launch_gemv_fp4(a, ctx, st);
  if (a.M <= 32 || (a.M <= 64 && a.N / 128 <= ctx.num_sms)) return launch_gemm_fp4_few(a, ctx, st);
  if (a.N % 256 == 0) {
    const int64_t m = a.M, pairs = (m + 255) / 256 * (a.N / 256), tiles = (m + 127) / 128 * (a.N / 128);
    const int64_t room = ctx.num_sms / 2;
    if ((tiles + 2 * room - 1) / (2 * room) > (pairs + room - 1) / room)
      return launch_pairs<EPI, FMT>(a, ctx, st);
  }
  return launch_tiles<EPI, FMT>(a, ctx, st);
}

template <int EPI>
cudaError_t launch_epi(const GemmFp4Args& a, const DevCtx& ctx, cudaStream_t st) {
  return a.fmt == H3_FP4_MX ? launch_fmt<EPI, H3_FP4_MX>(a, ctx, st)
                            : launch_fmt<EPI, H3_FP4_NV>(a, ctx, st);
}

}  // namespace

cudaError_t launch_gemm_fp4(const GemmFp4Args& a, const DevCtx& ctx, cudaStream_t st) {
  switch (a.epilogue) {
    case EPI_PLAIN: return launch_epi<EPI_PLAIN>(a, ctx, st);
    case EPI_GATED_RESIDUAL: return launch_epi<EPI_GATED_RESIDUAL>(a, ctx, st);
    case EPI_GELU: return launch_epi<EPI_GELU>(a, ctx, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace h3
