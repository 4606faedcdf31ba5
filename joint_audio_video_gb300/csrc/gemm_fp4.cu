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
// Persistent CTA pairs; few rows of A take other kernels (launch_fmt at the end chooses).
#include <cuda_bf16.h>

#include <type_traits>

#include "../../include/h3attn_lowp.h"
#include "gemm_epilogue.cuh"
#include "kernels.hpp"
#include "launch.hpp"
#include "ptx.cuh"
#include "tmap.hpp"

namespace h3 {
namespace {

constexpr int kBlockK = 256;                          // columns of a k-block: 128 bytes of codes
constexpr uint32_t kTileBytes = 128 * 128;            // 128 rows of a k-block
constexpr uint32_t kTmemCols = 512;

// A cluster of two CTAs (cta_group::2) computes one 256 x BN tile, BN = 256 or
// 192: each CTA loads 128 rows of A with their scales, BN / 2 rows of B, and the scales of two
// 128-row groups of B (each CTA's tensor memory needs those of all BN rows; an odd 192-row
// tile starts 64 rows, two columns, into them); the even CTA's issuer copies the scales of
// both and multiplies.
//
// Tensor memory, 512 columns.  BN = 192: two accumulators [0, 192), [192, 384), then the
// scales of A [384, 400) and of B [400, 432).  BN = 256: two accumulators and 48 scale columns
// do not fit, so the accumulators share 64 columns:
//   even tiles [0, 256)   odd tiles [192, 448)   scales of A [448, 464), of B [464, 496)
// The epilogue reads the shared columns of a tile first and hands them over; the next
// tile's products start then, ~1,500 cycles after the last ones ended, while the epilogue
// goes on with the other 192.
//
// What bounds it.  With the ring full a 256-column k-block takes ~610 SM cycles (NV; the
// scale copies are 2.4 % of it) or ~490 (MX) at BN = 256, and in long runs the power cap sets the
// clock: 58,758 x 20,480 x 5,120 NV takes 1.90 to 2.03 ms, 6.1 to 6.5 PFLOP/s, at ~1,460 of 2,070
// MHz (MX: ~1.73 ms).  In a run too short for that (4,096 x 20,480 x 5,120 NV, 125 us) the tensor
// pipe is active 76 % of the time.  The ring's depth matters because a stage's refill takes ~2,300 cycles from the
// commit that frees it to its bytes being seen: with 3, 4, 5 NV stages a k-block took 912, 714,
// 620 cycles (16,384 x 5,120 x 20,480), with 5 and 6 MX stages 586 and 556.  One thread issues a
// stage's four copies in a row, each late by those before it: two producer threads (A with its
// scales, B with its) take 4 to 5 % off; four take another 5 % off MX and nothing off NV.
// Copying the next k-block's scales between this one's products instead of ahead of its own
// made it 5 % slower.
constexpr int kPairGroupM = 16;
constexpr int kEpiGroups = 2;                         // of four epilogue warps
constexpr uint32_t kStageWarp = 32 * 64;              // staging of a warp: 32 rows x 32 columns of C

// The 128 threads of epilogue group g.
__device__ __forceinline__ void group_bar(int g) { asm volatile("bar.sync %0, 128;" ::"r"(1 + g) : "memory"); }

template <int FMT, int BN>
struct PairCfg {
  static_assert(BN == 256 || BN == 192, "");
  static constexpr bool mx = FMT == H3_FP4_MX;
  static constexpr uint32_t kAcc1 = 192;                        // columns of the odd accumulator
  static constexpr uint32_t kSfa = BN == 256 ? 448 : 384, kSfb = kSfa + 16;
  static constexpr int kTiles = mx ? 2 : 4;                     // scale tiles of a k-block
  static constexpr uint32_t kScaleBytes = kTiles * 512;
  static constexpr uint32_t kBBytes = BN / 2 * 128;
  static constexpr uint32_t kStageBytes = kTileBytes + kBBytes + 3 * kScaleBytes;
  // a multiple of 1 KB, so every stage's code tiles keep the swizzle's alignment
  static constexpr uint32_t kStageStride = (kStageBytes + 1023) / 1024 * 1024;
  // all of the 227 KB: a sixth stage rather than second staging buffers for C
  static constexpr int kStages = BN == 256 && !mx ? 5 : 6;
  static constexpr int kBufs = (BN == 256) == mx ? 1 : 2;       // of each epilogue group
  // warps: producer 0, issuer, 8 epilogue, then the other producers
  static constexpr int kProducers = mx ? 4 : 2;
  static constexpr int kThreads = 32 * (1 + 4 * kEpiGroups + kProducers);
  // NV: the factors of a tile's rows of B, staged before its accumulator is ready (read from
  // global memory inside the epilogue they cost a cache miss for every 64 columns: 4,096 x
  // 6,144 x 2,048 took 38.6 us, then 24.4).  MX has no room for them and seldom any factors: a
  // lane reads one column's a chunk ahead, and the warp has them by shuffles (with factors on
  // both sides, the same size 22.5 us; read by every thread at their use 23.0).
  static constexpr bool kFactors = !mx;
  static constexpr uint32_t kFactorAt = kStages * kStageStride + kEpiGroups * kBufs * kStageC;   // offset
  static constexpr uint32_t kBars = kFactorAt + (kFactors ? kEpiGroups * 2 * 1024 : 0);
  static constexpr size_t kSmem = kBars + 256;
  static_assert(kSmem <= 227 * 1024, "");
};

template <int EPI, int FMT, int BN>
__global__ void __launch_bounds__(PairCfg<FMT, BN>::kThreads, 1)
    gemm_fp4_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                         const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                         const __grid_constant__ CUtensorMap tmC, const __grid_constant__ GemmDev p) {
  using Cfg = PairCfg<FMT, BN>;
  constexpr int S = Cfg::kStages;
  constexpr bool mx = FMT == H3_FP4_MX;
  // no static shared memory, so the dynamic part starts on its 1 KB boundary
  extern __shared__ __align__(1024) uint8_t smem_pair[];
  struct Bars {
    uint64_t full[S], empty[S], acc_full[2], acc_free[2], drain;
    uint32_t tmem_base;
    int abort;
  };
  static_assert(sizeof(Bars) <= 256, "");
  Bars& bars = *reinterpret_cast<Bars*>(smem_pair + Cfg::kBars);
  uint64_t(&bar_full)[S] = bars.full;
  uint64_t(&bar_empty)[S] = bars.empty;
  uint64_t(&bar_acc_full)[2] = bars.acc_full;
  uint64_t(&bar_acc_free)[2] = bars.acc_free;   // BN = 256: [0], the columns both share
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
    for (int a = 0; a < 2; ++a) mbar_init(smem_u32(&bar_acc_free[a]), 2 * 4 * kEpiGroups);   // the even CTA's: one a warp
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

  if (warp == 0 || warp >= 2 + 4 * kEpiGroups) {
    // ---------------------------------------------------------------- producers
    if (lane_id() == 0) {
      // 0: A's codes, 1: B's, 2: A's scales, 3: B's; with two producers 0 and 1 do both
      const int role = warp == 0 ? 0 : warp - (1 + 4 * kEpiGroups);
      constexpr int kP = Cfg::kProducers;
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = cid; t < num_tiles && ok; t += ncl) {
        int mb, nb;
        tile_coords(t, p.num_m, p.num_n, mb, nb, kPairGroupM);
        // 128-row group of A, first 128-row group of B's scales
        const int ga = mb * 2 + int(rank), gb = nb * BN / 128;
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
            tma_load_2d_pair(sa + kTileBytes, &tmB, cfb, kb * 128, nb * BN + int(rank) * (BN / 2));
          const uint32_t ss = sa + kTileBytes + Cfg::kBBytes;
          if (role == (0 + 2) % kP) tma_load_2d_pair(ss, &tmSA, cfb, sx, ga);
          if (role == (1 + 2) % kP) tma_load_2d_pair(ss + Cfg::kScaleBytes, &tmSB, cfb, sx, gb);
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
      const SDesc dS0 = sdesc_split(sdesc_plain(base + kTileBytes + Cfg::kBBytes));
      int stage = 0;
      uint32_t phase = 0;
      int it = 0;
      bool ok = true;
      for (int t = cid; t < num_tiles && ok; t += ncl, ++it) {
        int mb, nb;
        tile_coords(t, p.num_m, p.num_n, mb, nb, kPairGroupM);
        // BN = 256: both epilogues have read the columns that this tile shares with the last;
        // BN = 192: all of the last tile but one
        constexpr int kBack = BN == 256 ? 1 : 2;
        if (it >= kBack) {
          const int last = it - kBack;
          ok = __all_sync(0xffffffffu,
                          mbar_wait_cluster(smem_u32(&bar_acc_free[BN == 256 ? 0 : it & 1]),
                                            uint32_t(BN == 256 ? last : last >> 1) & 1u, wc));
          if (!ok) break;
        }
        tc_fence_after();
        const uint32_t dtm = tmem + (it & 1) * Cfg::kAcc1;
        const uint32_t sfb = tmem + Cfg::kSfb + (BN == 192 && (nb & 1) ? 2u : 0u);
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
              tmem_cp_scales<2>(tmem + Cfg::kSfa + 4 * c, sdesc_at(dS, c * 512));
              tmem_cp_scales<2>(tmem + Cfg::kSfb + 8 * c, sdesc_at(dS, Cfg::kScaleBytes + c * 512));
              tmem_cp_scales<2>(tmem + Cfg::kSfb + 8 * c + 4,
                                sdesc_at(dS, 2 * Cfg::kScaleBytes + c * 512));
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (k >= steps) break;
              const uint32_t c = uint32_t(mx ? k >> 1 : k);
              mma_f4_ss<Cfg::kTiles, 2>(dtm, sdesc_at(dA, k * 32), sdesc_at(dB, k * 32),
                                              idesc_e2m1_f32(256, BN, mx, mx ? (k & 1) * 2 : 0),
                                              tmem + Cfg::kSfa + 4 * c, sfb + 8 * c,
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
    // Two groups of four warps take every other 32 columns each.  A warp is on its own: it
    // waits for the accumulator, stages its 32 rows and stores them without the others (with
    // barriers of a group around its chunks 58,758 x 2,048 x 128, all output, took 63.8 us
    // instead of 57.9, long sums the same).
    const int group = (warp - 2) >> 2, q = warp & 3;
    const int row_in_tile = q * 32 + lane_id();
    const uint32_t sC = base + S * Cfg::kStageStride + uint32_t((group * 4 + q) * Cfg::kBufs) * kStageWarp;
    const uint32_t srow = uint32_t(lane_id()) * 64, ssw = uint32_t(lane_id() >> 1) & 3u;
    const uint32_t free_c[2] = {cluster_addr(smem_u32(&bar_acc_free[0]), 0),
                                cluster_addr(smem_u32(&bar_acc_free[1]), 0)};
    const RopeTable rt{};
    const int32_t no_pos[3] = {0, 0, 0};
    constexpr int kEach = BN / 32 / kEpiGroups;   // chunks of 32 columns of a group
    int chunk = 0;
    int it = 0;
    for (int t = cid; t < num_tiles; t += ncl, ++it) {
      int mb, nb;
      tile_coords(t, p.num_m, p.num_n, mb, nb, kPairGroupM);
      const int row0 = mb * 256 + int(rank) * 128 + q * 32, grow = row0 + int(lane_id());
      const bool live = grow < p.M;
      const EpilogueRow er = epilogue_row<EPI, 2>(p, grow, live);
      float* factors = reinterpret_cast<float*>(smem_pair + Cfg::kFactorAt) + (group * 2 + (it & 1)) * 256;
      bool apart = false;   // NV: some product of two factors may leave fp32
      if constexpr (Cfg::kFactors) {
        const int col = nb * BN + 2 * row_in_tile;   // N is even
        if (2 * row_in_tile < BN)
          reinterpret_cast<float2*>(factors)[row_in_tile] =
              p.b_scale == nullptr || col >= p.N || !H3_IN(col >= 0 && col + 2 <= p.N, p.status)
                  ? make_float2(1.f, 1.f)
                  : ld_dep(reinterpret_cast<const float2*>(p.b_scale + col));
        group_bar(group);
        apart = far_scales<BN>(er.sa, [&](int i) { return factors[i]; });
      }
      // BN = 256: the columns shared with the other accumulator first
      const auto chunk_of = [&](int j) {
        return group + 2 * (BN == 192 || (it & 1) ? j : (j + kEach - 1) % kEach);
      };
      // MX: a lane has the factor of one column of the next chunk, read a chunk ahead
      const auto column_factor = [&](int c) {
        const int col = nb * BN + c * 32 + int(lane_id());
        return p.b_scale != nullptr && col < p.N ? ld_dep(p.b_scale + col) : 1.f;
      };
      float fb_next = Cfg::kFactors ? 1.f : column_factor(chunk_of(0));
      const bool ok =
          __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar_acc_full[it & 1]), (it >> 1) & 1, wc));
      // the others of a group may still be at their barrier: they leave by the CTA's abort flag,
      // so this warp goes on meeting them there, writing nothing
      if (!ok && !Cfg::kFactors) break;
      tc_fence_after();
      const uint32_t tacc = tmem + (it & 1) * Cfg::kAcc1 + (uint32_t(q * 32) << 16);
      // a loop of its own for far factors (one loop for both: 59.6 instead of 58.7 us for 58,758 x
      // 2,048 x 128, which has one k-block a tile)
      const auto store_tile = [&](auto far_factors) {
#pragma unroll 1
        for (int j = 0; j < kEach; ++j) {
          const int c = chunk_of(j);
          const float fb = fb_next;
          if (!Cfg::kFactors && j + 1 < kEach) fb_next = column_factor(chunk_of(j + 1));
          uint32_t r[32];
          tmem_ld32(tacc + c * 32, r);
          tmem_ld_wait(r);
          if (j == (BN == 256 ? 0 : kEach - 1)) {   // the columns to hand over are in registers
            tc_fence_before();
            __syncwarp();
            if (lane_id() == 0) mbar_arrive_cluster(free_c[BN == 256 ? 0 : it & 1]);
          }
          const int col = nb * BN + c * 32;
          if (row0 >= p.M || col >= p.N) continue;   // uniform in the warp: nothing to write
          if constexpr (!Cfg::kFactors) {   // the factors here, for the whole warp at once
            if (p.b_scale == nullptr) {
#pragma unroll
              for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * er.sa);
            } else if (__any_sync(0xffffffffu, !mid_range(er.sa) || !mid_range(fb))) {
              float v[32], b[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                v[i] = __uint_as_float(r[i]);
                b[i] = __shfl_sync(0xffffffffu, fb, i);
              }
              times_apart_n(v, 32, er.sa, b);
#pragma unroll
              for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(v[i]);
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                r[i] = __float_as_uint(__uint_as_float(r[i]) * (er.sa * __shfl_sync(0xffffffffu, fb, i)));
            }
          }
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) pk[i] = 0u;   // rows past M: clipped by the store
          if (live) {
            if (er.bad) {
#pragma unroll
              for (int i = 0; i < 32; ++i) r[i] = 0x7FC00000u;   // NaN row
            }
            epilogue_chunk<EPI, Cfg::kFactors ? 3 : 2, decltype(far_factors)::value>(
                p, rt, r, grow, col, no_pos, er.m, er.sa, pk, factors + c * 32);
          }
          const uint32_t sb = sC + uint32_t(chunk % Cfg::kBufs) * kStageWarp;
          // the store that last read this staging buffer has done so
          if (lane_id() == 0) {
            if constexpr (Cfg::kBufs == 1) bulk_wait_read_0();
            else bulk_wait_read_1();
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             sb + srow + ((uint32_t(i) ^ ssw) << 4)),
                         "r"(pk[4 * i]), "r"(pk[4 * i + 1]), "r"(pk[4 * i + 2]), "r"(pk[4 * i + 3])
                         : "memory");
          fence_async_shared();
          __syncwarp();
          if (lane_id() == 0) {
            tma_store_2d(&tmC, sb, col, row0);
            bulk_commit();
          }
          ++chunk;
        }
      };
      if (ok && !apart) store_tile(std::false_type{});
      if constexpr (Cfg::kFactors) {
        if (ok && apart) store_tile(std::true_type{});
      }
      if (er.bad && group == 0) atomicCAS(p.status, H3_DEV_OK, H3_DEV_BAD_INDEX);
    }
    if (lane_id() == 0) bulk_wait_all();
    __syncwarp();
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
  p.num_n = (a.N + cols - 1) / cols;
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

// Tensor maps of the operands: boxes of 128 rows of A and b_rows of B, and of their scales
// (b_groups 128-row groups of B's).
struct OperandMaps {
  CUtensorMap A, B, SA, SB;
};
bool make_operand_maps(OperandMaps* m, const GemmFp4Args& a, int b_rows, int b_groups) {
  const bool mx = a.fmt == H3_FP4_MX;
  const uint64_t kbytes = uint64_t(a.K) / 2, tiles = uint64_t(a.K) / (mx ? 128 : 64);
  const uint32_t box = mx ? 2 : 4;   // scale tiles of a k-block
  return make_tmap_u8_2d(&m->A, a.A, a.M, kbytes, kbytes, 128) &&
         make_tmap_u8_2d(&m->B, a.B, a.N, kbytes, kbytes, b_rows) &&
         make_tmap_scales(&m->SA, a.a_bs, (a.M + 127ull) / 128, tiles, 1, box) &&
         make_tmap_scales(&m->SB, a.b_bs, a.N / 128, tiles, b_groups, box);
}

template <int EPI, int FMT, int BN>
cudaError_t launch_pairs(const GemmFp4Args& a, const DevCtx& ctx, cudaStream_t st) {
  using Cfg = PairCfg<FMT, BN>;
  OperandMaps m;
  CUtensorMap tmC;
  if (!make_operand_maps(&m, a, BN / 2, 2) || !make_tmap_bf16_2d_sw64(&tmC, a.C, a.M, a.N, a.N, 32))
    return cudaErrorInvalidValue;
  const GemmDev p = gemm_dev(a, ctx, 256, BN);
  static KernelState state;
  const auto kern = gemm_fp4_pair_kernel<EPI, FMT, BN>;
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

// Which kernel (us a call among others on one GB300):
//   gemv, no tensor cores   one row through at most 27 x 2^20 weights, two through 12 x 2^20, in
//       one wave; against the kernel for few rows: one row 2,048 x 2,048 2.8 against 4.2 (MX; NV
//       4.5), 4,096 x 4,096 4.0 against 4.5, 5,120 x 5,120 5.2 against 5.9 (NV 5.3 against 6.3), but
//       6,144 x 5,120 7.5 against 6.1, 15,360 x 1,024 (more than one wave) 4.3 against 3.8; two
//       rows 5,120 x 2,048 3.8 against 4.3, but 2,560 x 5,120 4.6 against 4.5, 4,096 x 4,096 5.7
//       against 4.4
//   few rows, few_rows() below   against pairs: 16 rows of 5,120 x 5,120 6.2 against 8.4 (NV 6.6
//       and 8.5)
//   pairs   256 x 256 where those need at most 0.86 of the waves of 256 x 192: 358 x 20,480 x
//       5,120 (3 waves of either) 23.9 against 21.7, 700 x 5,120 x 5,120 (1 against 2) 11.2
//       against 14.4, 16,384 x 5,120 x 5,120 (17 against 23) 113 against 130; NV 25.9 and 22.3,
//       11.5 and 14.6, 125 and 141; wrong by at most 3 % over 18 sizes of either format
//
// Which row counts are few (MX; NV differs by less than 10 %).  Their cost grows with the rows,
// and with the waves of their 128-row weight tiles; that of pairs hardly does, but only few
// split K:
//   up to 16   always (40,960 x 2,048 14.6 against 15.3, 65,536 x 1,024 12.1 against 12.7)
//   up to 32   two tiles an SM at most, or long sums: 38,400 x 2,048 11.8 against 13.3, 40,960 x
//              5,120 29.0 against 32.0, but 40,960 x 2,048 16.8 against 14.7
//   up to 48   one tile an SM at most: 40 rows of 5,120 x 5,120 7.5 against 8.6, of 15,360 x
//              5,120 12.7 against 14.2; 64 rows of 20,480 x 5,120 27.0 against 16.4
//   up to 64   room for a split and long sums: 5,120 x 8,192 10.5 against 11.5, 2,048 x 12,288
//              8.9 against 14.6, but 2,048 x 2,048 6.1 against 5.7, 10,240 x 12,288 20.7 against 18.3
bool few_rows(const GemmFp4Args& a, int num_sms) {
  const int tiles = a.N / 128;
  if (a.M <= 16) return true;
  if (a.M <= 32) return tiles <= 2 * num_sms || a.K >= 4096;
  if (a.M <= 48) return tiles <= num_sms;
  return a.M <= 64 && 2 * tiles <= num_sms && a.K >= 8192;
}

template <int EPI, int FMT>
cudaError_t launch_fmt(const GemmFp4Args& a, const DevCtx& ctx, cudaStream_t st) {
  const int64_t weights = int64_t(a.N) * a.K;
  if (a.M <= 2 && weights <= (a.M == 1 ? 27 << 20 : 12 << 20) && a.N <= 80 * ctx.num_sms)
    return launch_gemv_fp4(a, ctx, st);
  if (few_rows(a, ctx.num_sms)) return launch_gemm_fp4_few(a, ctx, st);
  const int64_t rows = (int64_t(a.M) + 255) / 256, room = ctx.num_sms / 2;
  const int64_t w256 = (rows * (a.N / 256) + room - 1) / room;
  const int64_t w192 = (rows * ((int64_t(a.N) + 191) / 192) + room - 1) / room;
  if (a.N % 256 == 0 && 100 * w256 <= 86 * w192) return launch_pairs<EPI, FMT, 256>(a, ctx, st);
  return launch_pairs<EPI, FMT, 192>(a, ctx, st);
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
