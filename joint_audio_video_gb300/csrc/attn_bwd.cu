// Backward pass of joint attention on tcgen05 / TMEM.  The probabilities are computed
// again from Q, K and the saved log-sum-exp; with s = sm_scale, per head:
//
//   P  = exp(s Q K^T - lse) at the visible pairs        D = rowsum(dO * O)
//   dV = P^T dO     dS = P (dO V^T - D)     dQ = s dS K     dK = s dS^T Q
//
// Five products of 2 L^2 128 operations a head are needed, and a kernel that forms each
// block of dS once has to add its dQ into memory from every block of keys: fp32 atomics of
// 2 bytes for every 5 x 256 operations, in an order that changes the result.  Here dK, dV
// and dQ are each summed in tensor memory by one CTA pair, over a loop of its own, so S and
// dP are formed twice (seven products), nothing is added through memory, and the same call
// gives the same bits.  One launch holds both loops: CTA pairs of the first kind own 256
// keys of a head and walk over blocks of 128 queries, pairs of the second kind own 256
// queries and walk over blocks of 128 keys.
//
//   first kind  (dK, dV):  S^T = K Q^T,  dP^T = V dO^T,  dV += P^T dO,  dK += dS^T Q
//   second kind (dQ):      S = Q K^T,    dP = dO V^T,    dQ += dS K
//
// Every product is a cta_group::2 one (M = 256: 128 rows of each CTA; N = 128) of 512
// tensor-core cycles, issued by the even CTA.  P^T, dS^T and dS go back to tensor memory as
// bf16 pairs over the scores they came from and are read there as the A operand, so no
// probability passes through shared memory: that is why the first kind works on transposed
// scores.  The streamed matrices come in two forms of 16 KB for each CTA: its 64 rows of
// the block x 128 head dims (the K-major B operand of S and dP), and the block's 128 rows x
// its 64 head dims (the MN-major B operand of the sums).  A CTA's shared-memory traffic for
// one product is 48 KB or 16 KB instead of the 64 or 32 KB of a single CTA, below the
// product's 512 cycles x 128 bytes.  320 threads:
//   warp 0      TMA producer: the stationary tiles once, then the streamed tiles into a ring
//               of 16 KB slots in the order in which the products read them
//   warp 1      TMEM owner; in the even CTA the tcgen05.mma issuer
//   warps 2..9  softmax: one stationary row a thread, 64 columns of the block each
// Orders of the products (j: block), each softmax step running under the next two products:
//   first kind   dK(j-1)  dP(j)  dV(j)  S(j+1):  P(j) under the first two, dS(j) under the
//                last two; tensor memory S | dP | dK | dV, 128 columns each
//   second kind  dP(j)  dQ(j-1)  S(j+1): tensor memory S even | S odd | dP | dQ, dS(j) over S(j)
//
// Roundings: P and dS to bf16 on their way into a product (fp32 until then, and P enters
// dS unrounded); D, the sums and the softmax are fp32; each gradient is rounded once.
#include <cuda_bf16.h>

#include <cmath>

#include "f32x2.cuh"
#include "kernels.hpp"
#include "launch.hpp"
#include "ptx.cuh"
#include "tmap.hpp"

namespace h3 {
namespace {

constexpr int kThreads = 320;
constexpr int kSlots = 9;
constexpr uint32_t kBox = 128 * 64 * 2;       // 128 rows x 64 bf16: one slot, half a tile
constexpr uint32_t kHalfBox = 64 * 64 * 2;    // 64 rows x 64 bf16
constexpr uint32_t kTile = 2 * kBox;          // a stationary tile
// -lse log2(e) and -D of the 128 queries of a block (first kind).  The producer fills a
// stage again after it got the ring slot of the 16th tile on, that is once the tile kSlots
// before that one has been read: with at most 11 slots dK of the stage's block is then done.
constexpr int kAux = 4;
constexpr uint32_t kAuxBytes = 2 * 128 * 4;
static_assert(kSlots <= 11, "the stages of lse and D are freed by the ring's slots");
constexpr size_t kSmem = 2 * kTile + kSlots * kBox + kAux * kAuxBytes + 1024;

struct BwdDev {
  __nv_bfloat16* dqkv;            // [L][3d]
  const float* nlse;              // [H][Lp]  -lse log2(e), -infinity from L on
  const float* nD;                // [H][Lp]  -D, 0 from L on
  int L, H, d, Lp;
  int causal;
  float scale, scale_log2;        // sm_scale, sm_scale * log2(e)
  int quads;                      // CTA pairs a head: 256 stationary rows each
  int* status;
  uint64_t wait_ns;
  int n_seg;                      // 0: one segment [0, L)
  int32_t cu[kMaxSegments + 1];   // segment starts, cu[n_seg] = L
};

// Segment of token i: the last s with cu[s] <= i (skips empty segments).
__device__ __forceinline__ int segment_of(const BwdDev& p, int i) {
  int lo = 0, hi = p.n_seg - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.cu[mid] <= i) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// D = A B^T over the 128 head dims, both K-major (A: two boxes of 128 rows, B: two of 64).
__device__ __forceinline__ void dot_product(uint32_t d_tmem, SDesc a, SDesc b) {
  constexpr uint32_t idesc = idesc_bf16_f32(256, 128, 0, 0);
#pragma unroll
  for (int s = 0; s < 8; ++s)
    mma_bf16_ss_pair(d_tmem, sdesc_at(a, (s >> 2) * kBox + (s & 3) * 32),
                     sdesc_at(b, (s >> 2) * kHalfBox + (s & 3) * 32), idesc, s > 0);
}

// D += A B over the block's 128 rows: A (bf16 pairs) from the first 32 columns of each half
// of a 128-column score buffer, B MN-major (each CTA: its 64 head dims).
__device__ __forceinline__ void sum_product(uint32_t d_tmem, uint32_t a_tmem, SDesc b,
                                            bool accumulate) {
  constexpr uint32_t idesc = idesc_bf16_f32(256, 128, 0, 1);
#pragma unroll
  for (int s = 0; s < 8; ++s)
    mma_bf16_ts_pair(d_tmem, a_tmem + (s >> 2) * 64 + (s & 3) * 8, sdesc_at(b, s * 2048), idesc,
                     accumulate || s > 0);
}

// Four fp32 of shared memory as two pairs.
__device__ __forceinline__ void lds_f2x2(uint32_t addr, uint64_t& a, uint64_t& b) {
  asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr) : "memory");
}

// p = 2^(s c + nl) for 32 columns; nl: the columns' own (COL) or the row's.
template <bool COL>
__device__ __forceinline__ void probabilities(const uint32_t (&r)[32], uint64_t cc, uint64_t row_nl,
                                              uint32_t nl, uint64_t* p) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint64_t n0 = row_nl, n1 = row_nl;
    if constexpr (COL) {
      lds_f2x2(nl + 16 * i, n0, n1);
    }
    float a, b, c, d;
    unf2(ffma2(f2(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1])), cc, n0), a, b);
    unf2(ffma2(f2(__uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3])), cc, n1), c, d);
    p[2 * i] = f2(ex2(a), ex2(b));
    p[2 * i + 1] = f2(ex2(c), ex2(d));
  }
}

// ds = p (dp + nd) for 32 columns, as bf16 pairs.
template <bool COL>
__device__ __forceinline__ void score_gradients(const uint32_t (&r)[32], const uint64_t* p,
                                                uint64_t row_nd, uint32_t nd, uint32_t* pk) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint64_t n0 = row_nd, n1 = row_nd;
    if constexpr (COL) {
      lds_f2x2(nd + 16 * i, n0, n1);
    }
    float a, b;
    unf2(fmul2(fadd2(f2(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1])), n0), p[2 * i]), a, b);
    pk[2 * i] = pack_bf16x2(a, b);
    unf2(fmul2(fadd2(f2(__uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3])), n1), p[2 * i + 1]),
         a, b);
    pk[2 * i + 1] = pack_bf16x2(a, b);
  }
}

struct Shared {
  uint64_t bar_a;                 // the stationary tiles (the even CTA's: both CTAs' bytes)
  uint64_t bar_full[kSlots];      // likewise
  uint64_t bar_empty[kSlots];     // one multicast commit
  uint64_t bar_s[2], bar_dp;      // products done
  uint64_t bar_p, bar_ds;         // the even CTA's: 8 softmax warps per CTA
  uint64_t bar_aux[kAux];         // this CTA's own
  uint64_t bar_sum, bar_drain;
  uint32_t tmem_base;
  int abort_flag;
};

struct Maps {
  const CUtensorMap *qkv, *qkv_half, *dO, *dO_half;   // boxes of 128 and of 64 rows
};

// One CTA pair's whole loop.  DKV: its rows are keys and it walks over queries.
template <bool DKV>
__device__ __forceinline__ void run(const Maps& m, const BwdDev& p, Shared& sh, uint32_t base,
                                    uint32_t tmem, int h, int quad) {
  const int warp = warp_id();
  const uint32_t rank = cluster_ctarank();
  const bool lead = rank == 0;
  const WaitCtx wc{&sh.abort_flag, p.status, p.wait_ns};
  const uint32_t sA = base;                      // first factor of S, then of dP
  const uint32_t sRing = base + 2 * kTile;
  const uint32_t sAux = sRing + kSlots * kBox;

  const int c0 = quad * 256;                     // the pair's rows: c0 .. c0 + 255
  const int c_last = min(c0 + 255, p.L - 1);
  const int r0 = c0 + int(rank) * 128;           // this CTA's
  // the streamed rows that any of them meets
  int lo = 0, hi = p.L;
  if (p.n_seg > 0) {
    lo = p.cu[segment_of(p, c0)];
    hi = p.cu[segment_of(p, c_last) + 1];
  }
  if (p.causal) {
    if (DKV) lo = max(lo, c0); else hi = min(hi, c_last + 1);
  }
  if (DKV) lo &= ~3;                             // 16-byte boundaries in nlse and nD
  const int n = (hi - lo + 127) / 128;

  WaitCtx drain{&sh.abort_flag, p.status, kDrainWaitNs};
  volatile int no_abort = 0;
  drain.abort = &no_abort;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane_id() == 0) {
      const int xq = h * 128, xk = p.d + h * 128, xv = 2 * p.d + h * 128;
      const uint32_t ab = smem_u32(&sh.bar_a);
      const uint32_t cab = cluster_addr(ab, 0);
      if (lead) mbar_arrive_expect_tx(ab, 2 * 2 * kTile);
      const int xa = DKV ? xk : xq;
      tma_load_2d_pair(sA, m.qkv, cab, xa, r0);
      tma_load_2d_pair(sA + kBox, m.qkv, cab, xa + 64, r0);
      const CUtensorMap* second = DKV ? m.qkv : m.dO;
      const int xb = DKV ? xv : xq;
      tma_load_2d_pair(sA + kTile, second, cab, xb, r0);
      tma_load_2d_pair(sA + kTile + kBox, second, cab, xb + 64, r0);

      int cnt = 0, aux = 0;
      bool ok = true;
      // block j's 64 rows of this CTA x 128 columns (half: K-major), or its 128 rows x the
      // CTA's 64 columns
      auto put = [&](bool half, const CUtensorMap* map, int x, int j) {
        const int slot = cnt % kSlots;
        if (ok) ok = mbar_wait(smem_u32(&sh.bar_empty[slot]), ((cnt / kSlots) & 1) ^ 1u, wc);
        if (!ok) return;
        const uint32_t fb = smem_u32(&sh.bar_full[slot]);
        const uint32_t cfb = cluster_addr(fb, 0);
        const uint32_t dst = sRing + slot * kBox;
        if (lead) mbar_arrive_expect_tx(fb, 2 * kBox);
        if (half) {
          const int y = lo + j * 128 + int(rank) * 64;
          tma_load_2d_pair(dst, map, cfb, x, y);
          tma_load_2d_pair(dst + kHalfBox, map, cfb, x + 64, y);
        } else {
          tma_load_2d_pair(dst, map, cfb, x + int(rank) * 64, lo + j * 128);
        }
        ++cnt;
      };
      auto put_aux = [&](int j) {
        if (!ok) return;
        const uint32_t fb = smem_u32(&sh.bar_aux[j % kAux]);
        const uint32_t dst = sAux + (j % kAux) * kAuxBytes;
        const int at = lo + j * 128;
        if (H3_IN(h < p.H && at + 128 <= p.Lp, p.status)) {
          const size_t off = size_t(h) * p.Lp + at;
          mbar_arrive_expect_tx(fb, kAuxBytes);
          bulk_load_1d(dst, p.nlse + off, 512, fb);
          bulk_load_1d(dst + 512, p.nD + off, 512, fb);
        } else {
          mbar_arrive(fb);
        }
        aux = j + 1;
      };
      if (DKV) {
        put(true, m.qkv_half, xq, 0);
        put_aux(0);
        for (int j = 0; j < n && ok; ++j) {
          if (j > 0) put(false, m.qkv, xq, j - 1);
          put(true, m.dO_half, xq, j);
          put(false, m.dO, xq, j);
          if (j + 1 < n) {
            put(true, m.qkv_half, xq, j + 1);
            put_aux(j + 1);
          }
        }
        put(false, m.qkv, xq, n - 1);
      } else {
        put(true, m.qkv_half, xk, 0);
        for (int j = 0; j < n && ok; ++j) {
          put(true, m.qkv_half, xv, j);
          if (j > 0) put(false, m.qkv, xk, j - 1);
          if (j + 1 < n) put(true, m.qkv_half, xk, j + 1);
        }
        put(false, m.qkv, xk, n - 1);
      }
      // the even CTA lets every copy it armed land before the CTA can exit (earlier ones
      // were consumed before their slot was refilled); the odd CTA's copies count on the
      // even CTA's barriers
      if (!ok) {
        abort_grace();
        if (lead)
          for (int k = max(0, cnt - kSlots); k < cnt; ++k)
            mbar_wait(smem_u32(&sh.bar_full[k % kSlots]), (k / kSlots) & 1, drain);
        for (int k = max(0, aux - kAux); k < aux; ++k)
          mbar_wait(smem_u32(&sh.bar_aux[k % kAux]), (k / kAux) & 1, drain);
      }
      if (lead) mbar_wait(ab, 0, drain);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lead) {
      const bool leader = elect_one();
      auto wait_all = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, wc));
      };
      auto wait_warps = [&](uint64_t* bar, uint32_t parity) {   // arrivals from both CTAs
        return __all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(bar), parity, wc));
      };
      const SDesc dA = sdesc_split(sdesc_sw128(sA, 16, 1024));
      const SDesc dB = sdesc_split(sdesc_sw128(sA + kTile, 16, 1024));
      const SDesc dK0 = sdesc_split(sdesc_sw128(sRing, 16, 1024));
      const SDesc dN0 = sdesc_split(sdesc_sw128(sRing, kBox, 1024));
      int cnt = 0;   // slots used
      auto full = [&] { return wait_all(smem_u32(&sh.bar_full[cnt % kSlots]), (cnt / kSlots) & 1); };
      auto at = [&](SDesc d) { return SDesc{d.lo + uint32_t(cnt % kSlots) * (kBox >> 4), d.hi}; };
      // the slot's product is issued: signal its end, and take the next slot
      auto done = [&](uint64_t* bar) {
        if (leader) {
          if (bar != nullptr) tc_commit_pair(smem_u32(bar), 0x3);
          tc_commit_pair(smem_u32(&sh.bar_empty[cnt % kSlots]), 0x3);
        }
        __syncwarp();
        ++cnt;
      };
      auto dot = [&](uint32_t d_tmem, SDesc a, uint64_t* bar) {
        if (!full()) return false;
        tc_fence_after();
        if (leader) dot_product(d_tmem, a, at(dK0));
        done(bar);
        return true;
      };
      auto sum = [&](uint32_t d_tmem, uint32_t a_tmem, bool accumulate, uint64_t* bar) {
        if (!full()) return false;
        tc_fence_after();
        if (leader) sum_product(d_tmem, a_tmem, at(dN0), accumulate);
        done(bar);
        return true;
      };
      bool ok = wait_all(smem_u32(&sh.bar_a), 0);
      ok = ok && dot(tmem, dA, &sh.bar_s[0]);
      if (DKV) {
        const uint32_t tS = tmem, tP = tmem + 128, tK = tmem + 256, tV = tmem + 384;
        for (int j = 0; j < n && ok; ++j) {
          if (j > 0) ok = wait_warps(&sh.bar_ds, (j - 1) & 1) && sum(tK, tP, j > 1, nullptr);
          ok = ok && dot(tP, dB, &sh.bar_dp);
          ok = ok && wait_warps(&sh.bar_p, j & 1) && sum(tV, tS, j > 0, nullptr);
          if (j + 1 < n) ok = ok && dot(tS, dA, &sh.bar_s[(j + 1) & 1]);
        }
        ok = ok && wait_warps(&sh.bar_ds, (n - 1) & 1) && sum(tK, tP, n > 1, &sh.bar_sum);
      } else {
        const uint32_t tP = tmem + 256, tQ = tmem + 384;
        for (int j = 0; j < n && ok; ++j) {
          if (j > 0) ok = wait_warps(&sh.bar_ds, (j - 1) & 1);
          ok = ok && dot(tP, dB, &sh.bar_dp);
          if (j > 0) ok = ok && sum(tQ, tmem + ((j - 1) & 1) * 128, j > 1, nullptr);
          if (j + 1 < n) ok = ok && dot(tmem + ((j + 1) & 1) * 128, dA, &sh.bar_s[(j + 1) & 1]);
        }
        ok = ok && wait_warps(&sh.bar_ds, (n - 1) & 1) &&
             sum(tQ, tmem + ((n - 1) & 1) * 128, n > 1, &sh.bar_sum);
      }
      // let every product issued so far finish before either CTA frees tensor memory
      if (leader) tc_commit_pair(smem_u32(&sh.bar_drain), 0x3);
      __syncwarp();
    }
    mbar_wait(smem_u32(&sh.bar_drain), 0, drain);
  } else {
    // ------------------------------------------------------------ softmax
    const int q = warp & 3;                 // TMEM lane quarter
    const int half = (warp - 2) >> 2;       // columns 64 half .. 64 half + 63 of each block
    const int i = r0 + q * 32 + int(lane_id());   // this thread's row
    const uint32_t lane_off = uint32_t(q * 32) << 16;
    const uint32_t cp = cluster_addr(smem_u32(&sh.bar_p), 0);    // the even CTA's
    const uint32_t cds = cluster_addr(smem_u32(&sh.bar_ds), 0);
    // streamed rows that meet this one: its segment, cut at the diagonal; none past the end
    int row_lo = 0, row_hi = p.L;
    if (p.n_seg > 0) {
      const int sg = segment_of(p, min(i, p.L - 1));
      if (H3_IN(sg >= 0 && sg < p.n_seg, p.status)) {
        row_lo = p.cu[sg];
        row_hi = p.cu[sg + 1];
      }
    }
    if (p.causal) {
      if (DKV) row_lo = max(row_lo, i); else row_hi = min(row_hi, i + 1);
    }
    const bool head_ok = H3_IN(h < p.H, p.status);
    const bool live = i < p.L && head_ok;
    if (!live) row_hi = row_lo = 0;
    uint64_t nl = 0, nd = 0;                // second kind: the row's
    if (!DKV) {
      float a = -INFINITY, b = 0.f;
      if (live) {
        a = ld_dep(p.nlse + size_t(h) * p.Lp + i);
        b = ld_dep(p.nD + size_t(h) * p.Lp + i);
      }
      nl = f2(a, a);
      nd = f2(b, b);
    }
    const uint64_t cc = f2(p.scale_log2, p.scale_log2);
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const uint32_t tS = tmem + lane_off + (DKV ? 0 : (j & 1) * 128) + half * 64;
      const uint32_t tP = tmem + lane_off + (DKV ? 128 : 256) + half * 64;
      // the block's -lse log2(e), and 512 bytes on its -D (first kind)
      const uint32_t aux = sAux + (j % kAux) * kAuxBytes + half * 256;
      ok = mbar_wait(smem_u32(&sh.bar_s[j & 1]), (j >> 1) & 1, wc);
      if (DKV) ok = ok && mbar_wait(smem_u32(&sh.bar_aux[j % kAux]), (j / kAux) & 1, wc);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      uint32_t s0[32], s1[32];
      tmem_ld32(tS, s0);
      tmem_ld32(tS + 32, s1);
      tmem_ld_wait(s0);
      tmem_ld_wait(s1);
      // column c is streamed row kv0 + c; visible iff lo_rel <= c < hi_rel
      const int kv0 = lo + j * 128 + half * 64;
      const int lo_rel = row_lo - kv0, hi_rel = row_hi - kv0;
      const bool masked = __any_sync(0xffffffffu, lo_rel > 0 || hi_rel < 64);
      if (masked) {
        mask32(s0, 0, lo_rel, hi_rel);
        mask32(s1, 32, lo_rel, hi_rel);
      }
      uint64_t pr[32];
      probabilities<DKV>(s0, cc, nl, aux, pr);
      probabilities<DKV>(s1, cc, nl, aux + 128, pr + 16);
      if (DKV) {
        uint32_t pk[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          float a, b;
          unf2(pr[c], a, b);
          pk[c] = pack_bf16x2(a, b);
        }
        tmem_st32(tS, pk);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane_id() == 0) mbar_arrive_cluster(cp);
      }
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&sh.bar_dp), j & 1, wc));
      if (!ok) break;
      tc_fence_after();
      tmem_ld32(tP, s0);
      tmem_ld32(tP + 32, s1);
      tmem_ld_wait(s0);
      tmem_ld_wait(s1);
      if (masked) {   // whatever is there is not multiplied by a probability of zero
        mask32(s0, 0, lo_rel, hi_rel, 0u);
        mask32(s1, 32, lo_rel, hi_rel, 0u);
      }
      uint32_t pk[32];
      score_gradients<DKV>(s0, pr, nd, aux + 512, pk);
      score_gradients<DKV>(s1, pr + 16, nd, aux + 640, pk + 16);
      tmem_st32(DKV ? tP : tS, pk);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane_id() == 0) mbar_arrive_cluster(cds);
    }
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&sh.bar_sum), 0, wc));
    if (ok) {
      tc_fence_after();
#pragma unroll 1
      for (int part = 0; part < (DKV ? 2 : 1); ++part) {
        // dK | dV, or dQ alone
        const uint32_t tA = tmem + lane_off + (DKV ? 256 + part * 128 : 384) + half * 64;
        const float f = DKV && part == 1 ? 1.f : p.scale;
        const int col = (DKV ? 1 + part : 0) * p.d + h * 128 + half * 64;
        uint32_t o[2][32];
        tmem_ld32(tA, o[0]);
        tmem_ld32(tA + 32, o[1]);
        tmem_ld_wait(o[0]);
        tmem_ld_wait(o[1]);
        if (live && H3_IN(col + 64 <= 3 * p.d, p.status)) {
          uint4* dst = reinterpret_cast<uint4*>(p.dqkv + size_t(i) * 3 * p.d + col);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float* v = reinterpret_cast<const float*>(&o[c >> 2][8 * (c & 3)]);
            dst[c] = make_uint4(pack_bf16x2(v[0] * f, v[1] * f), pack_bf16x2(v[2] * f, v[3] * f),
                                pack_bf16x2(v[4] * f, v[5] * f), pack_bf16x2(v[6] * f, v[7] * f));
          }
        }
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    attn_bwd_kernel(const __grid_constant__ CUtensorMap tm, const __grid_constant__ CUtensorMap tm_half,
                    const __grid_constant__ CUtensorMap tmo,
                    const __grid_constant__ CUtensorMap tmo_half, const __grid_constant__ BwdDev p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int warp = warp_id();
  if (threadIdx.x == 0) {
    sh.abort_flag = 0;
    mbar_init(smem_u32(&sh.bar_a), 1);
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(smem_u32(&sh.bar_full[s]), 1);
      mbar_init(smem_u32(&sh.bar_empty[s]), 1);
    }
    for (int s = 0; s < kAux; ++s) mbar_init(smem_u32(&sh.bar_aux[s]), 1);
    mbar_init(smem_u32(&sh.bar_s[0]), 1);
    mbar_init(smem_u32(&sh.bar_s[1]), 1);
    mbar_init(smem_u32(&sh.bar_dp), 1);
    mbar_init(smem_u32(&sh.bar_p), 16);
    mbar_init(smem_u32(&sh.bar_ds), 16);
    mbar_init(smem_u32(&sh.bar_sum), 1);
    mbar_init(smem_u32(&sh.bar_drain), 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&sh.tmem_base), 512);
    tmem_relinquish_pair();
  }
  if (warp == 0 && lane_id() == 0) {
    tma_prefetch_desc(&tm);
    tma_prefetch_desc(&tm_half);
    tma_prefetch_desc(&tmo);
    tma_prefetch_desc(&tmo_half);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers exist before any signal crosses
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  pdl_wait();

  // The first kind (four products a block) ahead of the second (three): long loops first.
  // Under the causal mask the longest rows of a head go first: the first keys, the last queries.
  const Maps maps{&tm, &tm_half, &tmo, &tmo_half};
  const int pairs = p.quads * p.H;
  const int cl = int(blockIdx.x >> 1);
  if (cl < pairs) {
    run<true>(maps, p, sh, base, tmem, cl / p.quads, cl % p.quads);
  } else {
    const int r = cl - pairs, quad = r % p.quads;
    run<false>(maps, p, sh, base, tmem, r / p.quads, p.causal ? p.quads - 1 - quad : quad);
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();   // neither CTA leaves while the other may still signal it
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// nD = -rowsum(dO * O) and nlse = -lse log2(e) for each head and token, heads apart and
// padded to Lp tokens (HBM-bound: 4 bytes an element of O).  A warp takes 8 tokens of a
// head, half a warp a token of 256 bytes; the warps of a CTA take neighbouring heads.
constexpr int kPrepThreads = 256;

__global__ void __launch_bounds__(kPrepThreads)
    attn_bwd_prep_kernel(const uint4* O, const uint4* dO, const float* lse, int L, int H, int Lp,
                         float* nlse, float* nD, int* status) {
  pdl_trigger();
  pdl_wait();
  const int64_t w = int64_t(blockIdx.x) * (kPrepThreads / 32) + warp_id();
  const int h = int(w % H);
  const int64_t t0 = w / H * 8;
  if (t0 >= Lp) return;
  const int lane = int(lane_id()), hw = lane >> 4, c = lane & 15;
  uint4 o[4], g[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t t = t0 + 2 * k + hw;
    o[k] = g[k] = make_uint4(0u, 0u, 0u, 0u);
    if (t < L) {
      const size_t at = (size_t(t) * H + h) * 16 + c;
      o[k] = ld_dep(O + at);
      g[k] = ld_dep(dO + at);
    }
  }
  float mine = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t a[4] = {o[k].x, o[k].y, o[k].z, o[k].w}, b[4] = {g[k].x, g[k].y, g[k].z, g[k].w};
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s = fmaf(__uint_as_float(a[e] << 16), __uint_as_float(b[e] << 16), s);
      s = fmaf(__uint_as_float(a[e] & 0xFFFF0000u), __uint_as_float(b[e] & 0xFFFF0000u), s);
    }
#pragma unroll
    for (int x = 8; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    // token 2k of the eight sits in the lower half, 2k + 1 in the upper one
    const float v = __shfl_sync(0xffffffffu, s, (lane & 1) * 16);
    if (lane >> 1 == k) mine = v;
  }
  const int64_t t = t0 + (lane & 7);
  const size_t at = size_t(h) * Lp + t;
  if (lane >= 16 || !H3_IN(h < H && t < Lp, status)) return;
  if (lane < 8) {
    nD[at] = -mine;
  } else {
    nlse[at] = t < L ? -1.4426950408889634f * ld_dep(lse + size_t(h) * L + t) : -INFINITY;
  }
}

}  // namespace

cudaError_t launch_attention_bwd(const AttnBwdArgs& a, const DevCtx& ctx, cudaStream_t st) {
  const int d = a.H * 128;
  CUtensorMap tm, tm_half, tmo, tmo_half;
  if (!make_tmap_bf16_2d(&tm, a.qkv, a.L, 3 * d, 3 * d, 128, 64) ||
      !make_tmap_bf16_2d(&tm_half, a.qkv, a.L, 3 * d, 3 * d, 64, 64) ||
      !make_tmap_bf16_2d(&tmo, a.dO, a.L, d, d, 128, 64) ||
      !make_tmap_bf16_2d(&tmo_half, a.dO, a.L, d, d, 64, 64))
    return cudaErrorInvalidValue;
  BwdDev p{};
  p.dqkv = static_cast<__nv_bfloat16*>(a.dqkv);
  p.nlse = a.nlse;
  p.nD = a.nD;
  p.L = a.L;
  p.H = a.H;
  p.d = d;
  p.Lp = attn_bwd_padded(a.L);
  p.causal = a.causal;
  p.scale = a.sm_scale;
  p.scale_log2 = a.sm_scale * 1.4426950408889634f;
  p.quads = (a.L + 255) / 256;
  p.status = ctx.status;
  p.wait_ns = ctx.wait_ns;
  p.n_seg = a.n_seg;
  for (int i = 0; i <= a.n_seg && a.cu_seqlens; ++i) p.cu[i] = a.cu_seqlens[i];

  const int64_t warps = int64_t(p.Lp / 8) * a.H;
  const Launch prep(unsigned((warps + kPrepThreads / 32 - 1) / (kPrepThreads / 32)), kPrepThreads, 0, st);
  cudaError_t e = cudaLaunchKernelEx(&prep.cfg, attn_bwd_prep_kernel, static_cast<const uint4*>(a.O),
                                     static_cast<const uint4*>(a.dO), a.lse, a.L, a.H, p.Lp, a.nlse,
                                     a.nD, ctx.status);
  if (e != cudaSuccess) return e;
  static KernelState state;
  if ((e = allow_smem(&state, attn_bwd_kernel, kSmem, ctx)) != cudaSuccess) return e;
  const Launch main(unsigned(4LL * p.quads * a.H), kThreads, kSmem, st, 2);
  e = cudaLaunchKernelEx(&main.cfg, attn_bwd_kernel, tm, tm_half, tmo, tmo_half, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace h3
