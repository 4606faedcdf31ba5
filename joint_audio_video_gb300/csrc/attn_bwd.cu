// Backward pass of joint attention on tcgen05 / TMEM.  The probabilities are computed
// again from Q, K and the saved log-sum-exp; with s = sm_scale, per head:
//
//   P  = exp(s Q K^T - lse) at the visible pairs        D = rowsum(dO * O)
//   dV = P^T dO     dS = P (dO V^T - D)     dQ = s dS K     dK = s dS^T Q
//
// Five products of 2 L^2 128 operations a head are needed, and a kernel that forms each
// block of dS once has to add its dQ into memory from every block of keys: 64 KB of fp32
// atomics for a 128 x 128 block of 21 MFLOP, in an order that changes the result.  Here dK, dV
// and dQ are each summed in tensor memory by one CTA pair, over a loop of its own, so S and
// dP are formed twice (seven products), nothing is added through memory, and the same call
// gives the same bits.  One launch holds both loops as items: one of the first kind is 256
// keys of a head, walked over blocks of 128 queries, one of the second kind 256 queries,
// walked over blocks of 128 keys.  A resident CTA pair takes items until none is left, and
// loads and multiplies for the next one while the gradients of the last leave.
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
// product's 512 cycles x 128 bytes.  384 threads:
//   warp 0      TMA producer: the stationary tiles once, then the streamed tiles into a ring
//               in the order in which the products read them
//   warp 1      TMEM owner; in the even CTA the tcgen05.mma issuer
//   warps 2, 3  nothing (a warpgroup is what gives up registers)
//   warps 4..11 softmax: one stationary row a thread, 64 columns of the block each
// Orders of the products (j: block), each softmax step running under the next two products:
//   first kind   dK(j-1)  dP(j)  dV(j)  S(j+1):  P(j) under the first two, dS(j) under the
//                last two; tensor memory S | dP | dK | dV, 128 columns each
//   second kind  dP(j)  dQ(j-1)  S(j+1): tensor memory S even | S odd | dP | dQ, dS(j) over S(j)
// P is handed over in two chunks (32 of each warp's 64 columns), so that its product starts on
// the first while the second is on its way to tensor memory: S(j), P(j), dV(j), S(j+1) is the
// first kind's longest chain.
//
// Measured (16,384 x 40 heads): 2,110 to 2,270 cycles a block of the first kind, whose products
// take 2,048, and 1,600 to 1,690 of the second (1,536): 10.2 to 10.6 ms, 1.35 to 1.30 PFLOP/s of
// the five products, 1.89 to 1.81 of the seven, held by the power cap.  An item's way in and out
// costs ~4,000 cycles.  (Times here and below are the device's, calls in a graph; a call through
// the Python binding among others takes up to a tenth more.)
//
// Roundings: P and dS to bf16 on their way into a product (fp32 until then, and P enters
// dS unrounded); D, the sums and the softmax are fp32; each gradient is rounded once.
#include <cuda_bf16.h>

#include <climits>
#include <cmath>

#include "f32x2.cuh"
#include "kernels.hpp"
#include "launch.hpp"
#include "ptx.cuh"
#include "tmap.hpp"

namespace h3 {
namespace {

// Registers are split over the SM's four sub-partitions, three of the twelve warps on each: at
// most 168 a thread at launch, moved from the first warpgroup to the softmax warps.
constexpr int kThreads = 384;
constexpr int kRegsFew = 96, kRegsSoftmax = 200;
static_assert(kRegsFew + 2 * kRegsSoftmax <= 3 * 168, "");
constexpr uint32_t kBox = 128 * 64 * 2;       // 128 rows x 64 bf16: half a tile
constexpr uint32_t kHalfBox = 64 * 64 * 2;    // 64 rows x 64 bf16
constexpr uint32_t kTile = 2 * kBox;          // a stationary tile
// The ring's slots hold what products that follow one another read: first kind
// Q_{j-1} (128 rows x 64 dims) | dO_j (64 rows x 128 dims), then dO_j (rows) | Q_{j+1} (dims);
// second kind K_{j-1} (rows) | V_j (dims) | K_{j+1} (dims).  One wait and one release for two or
// three products: a wait costs the issuing warp, which shares its scheduler with two softmax
// warps, some 150 cycles (a slot for each product, when that was changed: 2,400 and 1,605
// cycles a block against 2,103 and 1,560).  A slot takes the next two or three of nine boxes of
// memory, so that four slots of the first kind or three of the second are in flight.
constexpr int kBoxes = 9;
constexpr int kSlots = 4;
template <bool DKV>
constexpr int kSlotBoxes = DKV ? 2 : 3;
template <bool DKV>
constexpr int kFlight = DKV ? 4 : 3;
static_assert(kFlight<true> * kSlotBoxes<true> <= kBoxes && kFlight<false> * kSlotBoxes<false> <= kBoxes &&
                  kFlight<false> <= kFlight<true> && kFlight<true> <= kSlots, "");
// -lse log2(e) and -D of the 128 queries of a block (first kind).  The stage of block j is
// filled again together with the slot that holds Q_{j+4}, five slots after the one of dK's
// product of block j: four before it, that is once a later slot has been released.
constexpr int kAux = 4;
constexpr uint32_t kAuxBytes = 2 * 128 * 4;
constexpr size_t kSmem = 2 * kTile + kBoxes * kBox + kAux * kAuxBytes + 1024;

struct BwdDev {
  __nv_bfloat16* dqkv;            // [L][3d]
  int sectors;                    // it begins on a 32-byte boundary
  int* counter;                   // items taken beyond the first of each pair
  const float* aux;               // [H][Lp / 4][2][4]: -lse log2(e), -infinity from L on; -D, 0
  int L, H, d, Lp;
  int causal;
  float scale, scale_log2;        // sm_scale, sm_scale * log2(e)
  int quads;                      // items of a kind for a head: 256 stationary rows each
  int by_rows;                    // items in order of their rows, all heads of one after another
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

// D += A B over one chunk of the block's 128 rows, 32 of each half: A (bf16 pairs) from the
// first 32 columns of each half of a 128-column score buffer, B MN-major (each CTA: its 64
// head dims).
__device__ __forceinline__ void sum_product(uint32_t d_tmem, uint32_t a_tmem, SDesc b, int chunk,
                                            bool accumulate) {
  constexpr uint32_t idesc = idesc_bf16_f32(256, 128, 0, 1);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int half = i >> 1, s = 2 * chunk + (i & 1);   // 16 rows: half, and which of its four
    mma_bf16_ts_pair(d_tmem, a_tmem + half * 64 + s * 8, sdesc_at(b, (half * 4 + s) * 2048), idesc,
                     accumulate || i > 0);
  }
}

// 16 bf16 to a 32-byte boundary (sectors), or to one of 16.
__device__ __forceinline__ void store16(__nv_bfloat16* dst, const uint32_t (&w)[8], bool sectors) {
  if (sectors) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    uint4* v = reinterpret_cast<uint4*>(dst);
    v[0] = make_uint4(w[0], w[1], w[2], w[3]);
    v[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
// Four fp32 of shared memory as two pairs.
__device__ __forceinline__ void lds_f2x2(uint32_t addr, uint64_t& a, uint64_t& b) {
  asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr) : "memory");
}

__device__ __forceinline__ void sts_f(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// One of the two values of 32 columns (four tokens in 32 bytes).
__device__ __forceinline__ void load_columns(uint32_t addr, uint64_t (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) lds_f2x2(addr + 32 * i, v[2 * i], v[2 * i + 1]);
}

// p = 2^(s c + nl) for 32 columns; nl: the columns' own (COL) or the row's.
template <bool COL>
__device__ __forceinline__ void probabilities(const uint32_t (&r)[32], uint64_t cc, uint64_t row_nl,
                                              const uint64_t (&nl)[16], uint64_t* p) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t n0 = COL ? nl[2 * i] : row_nl, n1 = COL ? nl[2 * i + 1] : row_nl;
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
      lds_f2x2(nd + 32 * i, n0, n1);
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
  uint64_t bar_a[2];              // the stationary tiles (the even CTA's: both CTAs' bytes)
  uint64_t bar_full[kSlots];      // likewise
  uint64_t bar_empty[kSlots];     // one multicast commit
  uint64_t bar_s[2], bar_dp;      // products done; S of even and odd blocks
  // the even CTA's, 8 softmax warps per CTA: chunks of P; dS, even and odd blocks (the second
  // kind's next dP is issued before dS is waited for); dP read (second kind); the sums of an
  // item read
  uint64_t bar_p[2], bar_ds[2], bar_read, bar_acc;
  uint64_t bar_sum[2], bar_drain;   // dV | dK or dQ done; everything
  uint64_t bar_aux[kAux], bar_item[2];   // this CTA's own: lse and D there; an item's number
  int item[2];
  uint32_t tmem_base;
  int abort_flag;
};

struct Maps {
  const CUtensorMap *qkv_rows, *qkv_dims;   // boxes of 128 rows x 64 columns, 64 x 128
  const CUtensorMap *dO_rows, *dO_dims;
};

// Work of a CTA pair: 256 rows of a head, and the streamed rows that any of them meets, which
// are all that it reads: a hidden pair's probability is zero, but zero times the infinity or NaN
// of a row outside would not be.  Block j takes the rows of [lo + 128 j, lo + 128 j + 128) and
// reads 128 rows from at(j) on: where that range leaves [first, last + 128), rows of a block
// beside it, which are hidden here.  Rows from L on come as zeros.
struct Item {
  bool dkv;       // the rows are keys, the streamed rows queries
  int h, c0;      // head, first row
  int lo, n;      // nominal first streamed row, blocks
  int first, last;
  __device__ __forceinline__ int at(int j) const { return min(max(lo + 128 * j, first), last); }
};
__device__ __forceinline__ Item item_of(const BwdDev& p, int idx) {
  Item it;
  const int kind = p.quads * p.H;
  // The first kind (four products a block) ahead of the second (three): long items first.  A
  // pair's numbers grow, so it never goes back from the second kind to the first, which more than
  // the time depends on; an order that mixes the kinds needs other answers for
  //   - the softmax warps' t and k, which count blocks and items of both kinds and serve for the
  //     first kind's own aux stages, bar_aux, bar_p and bar_sum[0] (the producer counts those
  //     stages, the barriers complete, in the first kind alone);
  //   - the ring: four slots in flight behind 3-box ones would not fit its nine boxes;
  //   - tensor memory: was_dkv orders dP over dK, and nothing orders the first kind's products
  //     behind the reading of the second's.
  it.dkv = idx < kind;
  if (!it.dkv) idx -= kind;
  it.h = p.by_rows ? idx % p.H : idx / p.quads;
  int quad = p.by_rows ? idx / p.H : idx % p.quads;
  // likewise under the causal mask: the first keys, the last queries
  if (p.causal && !it.dkv) quad = p.quads - 1 - quad;
  it.c0 = quad * 256;
  const int c_last = min(it.c0 + 255, p.L - 1);
  int lo = 0, hi = p.L;
  if (p.n_seg > 0) {
    lo = p.cu[segment_of(p, it.c0)];
    hi = p.cu[segment_of(p, c_last) + 1];
  }
  if (p.causal) {
    if (it.dkv) lo = max(lo, it.c0); else hi = min(hi, c_last + 1);
  }
  it.first = lo;
  // short of L, [lo, hi) holds the item's own 256 rows
  it.last = hi < p.L ? hi - 128 : INT_MAX;
  if (it.dkv) lo &= ~3;           // groups of four in aux
  it.lo = lo;
  it.n = (hi - lo + 127) / 128;
  return it;
}

// The number of item k of this CTA pair (k > 0), -1 behind the last one, -2 if the wait ran
// out.  The even CTA's producer sends it to both CTAs once it has loaded item k - 1, at the
// end of which it took slots that were released after all warps had begun item k - 1: item
// k - 2's number, in the same place, has been read.
__device__ __forceinline__ int next_item(Shared& sh, int k, const WaitCtx& wc) {
  const bool ok = mbar_wait_cluster(smem_u32(&sh.bar_item[k & 1]), ((k - 1) >> 1) & 1, wc);
  if (!__all_sync(0xffffffffu, ok)) return -2;
  return *static_cast<volatile int*>(&sh.item[k & 1]);
}
__device__ __forceinline__ void send_item(Shared& sh, int slot, uint32_t rank, int idx) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(
                   cluster_addr(smem_u32(&sh.item[slot]), rank)),
               "r"(idx), "r"(cluster_addr(smem_u32(&sh.bar_item[slot]), rank))
               : "memory");
}

// ---------------------------------------------------------------- producer (a warp of each CTA)
// The whole warp runs the loop, so that coordinates and addresses stay warp-uniform; one lane
// issues, one copy for each operand.
struct Producer {
  const Maps& m;
  const BwdDev& p;
  Shared& sh;
  const WaitCtx& wc;
  uint32_t sA, sRing, sAux;
  uint32_t rank;
  bool leader;
  int cnt = 0, aux = 0, k = 0;    // slots, lse and D stages, items so far
  int as[2] = {0, 0};             // stationary tiles
  bool ok = true;
  uint32_t cfb = 0;
  uint32_t first = 0, after = 0;  // the slot's first box, the one after it

  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t ph) {
    ok = ok && __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), ph, wc));
    return ok;
  }
  // the next slot, to be filled with `boxes` boxes
  template <bool DKV>
  __device__ __forceinline__ bool next(int boxes) {
    const int old = cnt - kFlight<DKV>;
    if (old >= 0 && !wait(&sh.bar_empty[old % kSlots], (old / kSlots) & 1)) return false;
    const uint32_t fb = smem_u32(&sh.bar_full[cnt % kSlots]);
    cfb = cluster_addr(fb, 0);
    first = after;
    after = first + kSlotBoxes<DKV>;
    if (after >= kBoxes) after -= kBoxes;
    if (rank == 0 && leader) mbar_arrive_expect_tx(fb, 2 * boxes * kBox);
    __syncwarp();
    ++cnt;
    return true;
  }
  __device__ __forceinline__ uint32_t box(uint32_t at) {
    const uint32_t b = first + at;
    return sRing + (b >= kBoxes ? b - kBoxes : b) * kBox;
  }
  // 128 rows from r on x the CTA's 64 of the columns from x on (MN-major operand)
  __device__ __forceinline__ void put_rows(int at, const CUtensorMap* map, int x, int r) {
    if (leader) tma_load_2d_pair(box(at), map, cfb, x + int(rank) * 64, r);
    __syncwarp();
  }
  // this CTA's 64 of those rows x 128 columns (K-major)
  __device__ __forceinline__ void put_dims(int at, const CUtensorMap* map, int x, int r) {
    if (leader) tma_load_3d_pair(box(at), map, cfb, 0, r + int(rank) * 64, x >> 6);
    __syncwarp();
  }
  // A stationary tile.  The first factor of S is free once the item's first slot is (the slot
  // three or four before it was released after the last S of the item before), that of dP once
  // the second slot is.
  __device__ __forceinline__ void put_a(int which, const CUtensorMap* map, int x, int r0) {
    const uint32_t ab = smem_u32(&sh.bar_a[which]);
    const uint32_t cab = cluster_addr(ab, 0), to = sA + which * kTile;
    if (leader) {
      if (rank == 0) mbar_arrive_expect_tx(ab, 2 * kTile);
      tma_load_2d_pair(to, map, cab, x, r0);
      tma_load_2d_pair(to + kBox, map, cab, x + 64, r0);
    }
    __syncwarp();
    ++as[which];
  }
  // lse and D of the 128 tokens from r on; where those begin inside a group of four (an item's
  // first or last block), the lanes put them together
  __device__ __forceinline__ void put_aux(int h, int r) {
    const uint32_t fb = smem_u32(&sh.bar_aux[aux % kAux]);
    const uint32_t to = sAux + (aux % kAux) * kAuxBytes;
    const bool in = H3_IN(h < p.H && r + 128 <= p.Lp, p.status);
    const float* from = p.aux + size_t(h) * p.Lp * 2;
    if ((r & 3) != 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = 32 * i + int(lane_id()), t = r + c;
        float nl = -INFINITY, nd = 0.f;
        if (in) {
          nl = ld_dep(from + size_t(t & ~3) * 2 + (t & 3));
          nd = ld_dep(from + size_t(t & ~3) * 2 + (t & 3) + 4);
        }
        sts_f(to + (c & ~3) * 8 + (c & 3) * 4, nl);
        sts_f(to + (c & ~3) * 8 + (c & 3) * 4 + 16, nd);
      }
      fence_async_shared();   // a later copy into this stage comes through the async proxy
      __syncwarp();
      if (leader) mbar_arrive(fb);
    } else if (leader) {
      if (in) {
        mbar_arrive_expect_tx(fb, kAuxBytes);
        bulk_load_1d(to, from + size_t(r) * 2, kAuxBytes, fb);
      } else {
        mbar_arrive(fb);
      }
    }
    __syncwarp();
    ++aux;
  }

  __device__ __forceinline__ void load(const Item& it) {
    const int n = it.n, xq = it.h * 128, xk = p.d + xq, xv = 2 * p.d + xq;
    const int r0 = it.c0 + int(rank) * 128;
    if (it.dkv) {
      if (!next<true>(1)) return;
      put_a(0, m.qkv_rows, xk, r0);
      put_dims(1, m.qkv_dims, xq, it.at(0));
      put_aux(it.h, it.at(0));
      for (int j = 0; j < n; ++j) {
        if (!next<true>(j > 0 ? 2 : 1)) return;
        if (j == 0) put_a(1, m.qkv_rows, xv, r0);
        else put_rows(0, m.qkv_rows, xq, it.at(j - 1));
        put_dims(1, m.dO_dims, xq, it.at(j));
        if (!next<true>(j + 1 < n ? 2 : 1)) return;
        put_rows(0, m.dO_rows, xq, it.at(j));
        if (j + 1 < n) {
          put_dims(1, m.qkv_dims, xq, it.at(j + 1));
          put_aux(it.h, it.at(j + 1));
        }
      }
      if (next<true>(1)) put_rows(0, m.qkv_rows, xq, it.at(n - 1));
    } else {
      if (!next<false>(1)) return;
      put_a(0, m.qkv_rows, xq, r0);
      put_dims(2, m.qkv_dims, xk, it.at(0));
      for (int j = 0; j < n; ++j) {
        if (!next<false>(1 + (j > 0) + (j + 1 < n))) return;
        if (j == 0) put_a(1, m.dO_rows, xq, r0);
        put_dims(1, m.qkv_dims, xv, it.at(j));
        if (j > 0) put_rows(0, m.qkv_rows, xk, it.at(j - 1));
        if (j + 1 < n) put_dims(2, m.qkv_dims, xk, it.at(j + 1));
      }
      if (next<false>(1)) put_rows(0, m.qkv_rows, xk, it.at(n - 1));
    }
  }
};

// ---------------------------------------------------------------- product issuer (the even CTA's warp 1)
// The whole warp runs the loop, so that slots and descriptors stay warp-uniform; one lane
// waits, issues and signals, all of a slot's work in one go (a vote after every wait, so that
// all lanes knew its end, made the warp itself the bound: some 150 cycles a wait, eleven waits
// a block).  After a wait that ran out that lane issues nothing more.
struct Issuer {
  const BwdDev& p;
  Shared& sh;
  const WaitCtx& wc;
  uint32_t tmem;
  SDesc dA, dB;                   // stationary tiles
  SDesc dDims, dRows;             // the ring's first box as either operand
  bool leader;
  bool ok = true;                 // the leader's
  int t = 0, k = 0, reads = 0;    // blocks, items, blocks of the second kind so far
  bool was_dkv = false;
  uint32_t slot = 0, parity = 0, box = 0;   // the next slot: its number, its phase, its first box
  uint32_t full = 0, empty = 0, ph = 0;     // the slot at work: its barriers, its phase,
  SDesc rows{0, 0}, dims{0, 0}, last{0, 0}; // its boxes: rows, the K-major one, the one after that

  __device__ __forceinline__ SDesc at_box(SDesc d, uint32_t b) {
    return SDesc{d.lo + (b >= kBoxes ? b - kBoxes : b) * (kBox >> 4), d.hi};
  }
  template <bool DKV, int AT = 1>
  __device__ __forceinline__ void take() {
    full = smem_u32(&sh.bar_full[slot]);
    empty = smem_u32(&sh.bar_empty[slot]);
    ph = parity;
    rows = at_box(dRows, box);
    dims = at_box(dDims, box + AT);
    last = at_box(dDims, box + AT + 1);
    box += kSlotBoxes<DKV>;
    if (box >= kBoxes) box -= kBoxes;
    slot = (slot + 1) % kSlots;
    parity ^= uint32_t(slot == 0);
  }
  // By the leader:
  __device__ __forceinline__ void wait(uint32_t bar, uint32_t phase) {
    ok = ok && mbar_wait(bar, phase, wc);
  }
  __device__ __forceinline__ void wait(uint64_t* bar, uint32_t phase) { wait(smem_u32(bar), phase); }
  __device__ __forceinline__ void commit(uint32_t bar) {
    if (ok) tc_commit_pair(bar, 0x3);
  }
  __device__ __forceinline__ void commit(uint64_t* bar) { commit(smem_u32(bar)); }
  __device__ __forceinline__ void dot(uint32_t d_tmem, SDesc a, SDesc b, uint64_t* bar) {
    if (!ok) return;
    tc_fence_after();
    dot_product(d_tmem, a, b);
    tc_commit_pair(smem_u32(bar), 0x3);
  }
  __device__ __forceinline__ void sum(uint32_t d_tmem, uint32_t a_tmem, int chunk, bool accumulate) {
    if (!ok) return;
    tc_fence_after();
    sum_product(d_tmem, a_tmem, rows, chunk, accumulate);
  }
  // dS of block b of all
  __device__ __forceinline__ void sum_ds(uint32_t d_tmem, uint32_t a_tmem, int b, bool accumulate) {
    wait(&sh.bar_ds[b & 1], (b >> 1) & 1);
    sum(d_tmem, a_tmem, 0, accumulate);
    sum(d_tmem, a_tmem, 1, true);
  }

  // S of an item's first block goes where products that come before it read last.
  __device__ __forceinline__ void issue_dkv(int n) {
    const uint32_t tS = tmem, tP = tmem + 128, tK = tmem + 256, tV = tmem + 384;
    take<true>();
    if (leader) {
      wait(&sh.bar_a[0], k & 1);
      wait(full, ph);
      dot(tS, dA, dims, &sh.bar_s[t & 1]);
      commit(empty);
      wait(&sh.bar_a[1], k & 1);
    }
    __syncwarp();
    for (int j = 0; j < n; ++j, ++t) {
      take<true>();   // Q_{j-1} | dO_j
      if (leader) {
        wait(full, ph);
        if (j > 0) sum_ds(tK, tP, t - 1, j > 1);
        dot(tP, dB, dims, &sh.bar_dp);
        commit(empty);
      }
      __syncwarp();
      // dO_j | Q_{j+1}; P of the first block comes after the warps have read the sums of the
      // item before
      take<true>();
      if (leader) {
        wait(full, ph);
        wait(&sh.bar_p[0], t & 1);
        sum(tV, tS, 0, j > 0);
        wait(&sh.bar_p[1], t & 1);
        sum(tV, tS, 1, true);
        if (j + 1 < n) dot(tS, dA, dims, &sh.bar_s[(t + 1) & 1]);
        else commit(&sh.bar_sum[0]);
        commit(empty);
      }
      __syncwarp();
    }
    take<true>();
    if (leader) {
      wait(full, ph);
      sum_ds(tK, tP, t - 1, n > 1);
    }
  }
  // S even | S odd | dP | dQ; a block's dP comes after the one before has been read.
  __device__ __forceinline__ void issue_dq(int n) {
    const uint32_t tP = tmem + 256, tQ = tmem + 384;
    take<false, 2>();
    if (leader) {
      wait(&sh.bar_a[0], k & 1);
      wait(full, ph);
      dot(tmem + (t & 1) * 128, dA, dims, &sh.bar_s[t & 1]);
      commit(empty);
      if (was_dkv) wait(&sh.bar_acc, (k - 1) & 1);   // dP's place held dK
      wait(&sh.bar_a[1], k & 1);
    }
    __syncwarp();
    for (int j = 0; j < n; ++j, ++t, ++reads) {
      take<false>();   // K_{j-1} | V_j | K_{j+1}
      if (leader) {
        wait(full, ph);
        if (j > 0) wait(&sh.bar_read, (reads - 1) & 1);
        dot(tP, dB, dims, &sh.bar_dp);
        if (j > 0) sum_ds(tQ, tmem + ((t - 1) & 1) * 128, t - 1, j > 1);
        if (j + 1 < n) dot(tmem + ((t + 1) & 1) * 128, dA, last, &sh.bar_s[(t + 1) & 1]);
        commit(empty);
      }
      __syncwarp();
    }
    take<false>();
    if (leader) {
      wait(full, ph);
      sum_ds(tQ, tmem + ((t - 1) & 1) * 128, t - 1, n > 1);
    }
  }
  __device__ __forceinline__ bool issue(const Item& it) {
    if (it.dkv) issue_dkv(it.n);
    else issue_dq(it.n);
    if (leader) {
      commit(&sh.bar_sum[1]);
      commit(empty);
    }
    was_dkv = it.dkv;
    ++k;
    return __all_sync(0xffffffffu, ok);
  }
};

// ---------------------------------------------------------------- softmax (8 warps a CTA)
// A block's softmax is a chain of latencies that has to fit under the products beside it
// (1,024 cycles for each step of the first kind, 1,536 for both of the second), so what can be
// known for a whole item, or loaded ahead of the scores, is.
struct Softmax {
  const BwdDev& p;
  Shared& sh;
  const WaitCtx& wc;
  uint32_t tmem, sAux, rank;
  uint32_t even;                  // what to add to an address in here for the even CTA's
  int t = 0, k = 0;               // blocks, items so far

  // A wait that ran out, by a lane: the warp goes on to the end of the item's blocks (further
  // waits are left out) and stops before it writes.
  bool ok = true;
  __device__ __forceinline__ void wait(uint64_t* bar, uint32_t phase) {
    ok = ok && mbar_wait(smem_u32(bar), phase, wc);
  }
  // one arrival a warp at the even CTA's barrier, tensor memory read and written before
  __device__ __forceinline__ void arrive(uint64_t* bar) {
    tc_fence_before();
    __syncwarp();
    if (lane_id() == 0) mbar_arrive_cluster(smem_u32(bar) + even);
  }

  template <bool DKV>
  __device__ __forceinline__ bool run(const Item& it) {
    const int warp = warp_id();
    const int q = warp & 3;                 // TMEM lane quarter
    const int half = (warp - 4) >> 2;       // columns 64 half .. 64 half + 63 of each block
    const int r0 = it.c0 + int(rank) * 128 + q * 32;
    const int i = r0 + int(lane_id());      // this thread's row
    const int h = it.h;
    const uint32_t lane_off = uint32_t(q * 32) << 16;
    // streamed rows that meet this one: its segment, cut at the diagonal.  A row past the end
    // needs no mask: what it computes stays in its row, which is not written.
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
    if (i >= p.L) {
      row_lo = 0;
      row_hi = 1 << 30;
    }
    uint64_t nl = 0, nd = 0;                // second kind: the row's
    if (!DKV) {
      float a = -INFINITY, b = 0.f;
      if (live) {
        const float* at = p.aux + (size_t(h) * p.Lp + (i & ~3)) * 2 + (i & 3);
        a = ld_dep(at);
        b = ld_dep(at + 4);
      }
      nl = f2(a, a);
      nd = f2(b, b);
    }
    const uint64_t cc = f2(p.scale_log2, p.scale_log2);
    // streamed rows that all of the warp's rows meet
    int all_lo = row_lo, all_hi = row_hi;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      all_lo = max(all_lo, __shfl_xor_sync(0xffffffffu, all_lo, o));
      all_hi = min(all_hi, __shfl_xor_sync(0xffffffffu, all_hi, o));
    }
    uint32_t s0[32], s1[32];
    int take = it.lo;                       // first row that the block takes
    for (int j = 0; j < it.n; ++j, ++t, take += 128) {
      const int at = it.at(j);
      const int kv0 = at + half * 64;       // streamed row of the warp's first column
      const uint32_t tS = tmem + lane_off + (DKV ? 0 : (t & 1) * 128) + half * 64;
      const uint32_t tP = tmem + lane_off + (DKV ? 128 : 256) + half * 64;
      // the block's -lse log2(e), four tokens in 32 bytes, and 16 bytes on its -D (first kind)
      const uint32_t aux = sAux + (t % kAux) * kAuxBytes + half * 512;
      uint64_t col_nl[16];                  // first kind: of the first chunk
      if constexpr (DKV) {
        wait(&sh.bar_aux[t % kAux], (t / kAux) & 1);
        load_columns(aux, col_nl);
      }
      wait(&sh.bar_s[t & 1], (t >> 1) & 1);
      __syncwarp();
      tc_fence_after();
      tmem_ld32(tS, s0);
      tmem_ld_wait(s0);
      tmem_ld32(tS + 32, s1);   // lands under the first chunk's exponentials
      // of the warp
      const bool masked = kv0 < all_lo || kv0 + 64 > all_hi || at != take;
      const int lo = max(row_lo, take), hi = min(row_hi, take + 128);
      uint64_t pr[32];
      uint32_t pk[16];
      auto pack = [&](int c) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float a, b;
          unf2(pr[16 * c + e], a, b);
          pk[e] = pack_bf16x2(a, b);
        }
      };
      // bit c of a chunk: streamed row kv0 (+ 32) + c meets this one
      if (__builtin_expect(masked, 0)) keep32(s0, bits32(lo - kv0, hi - kv0), kNegInf);
      probabilities<DKV>(s0, cc, nl, col_nl, pr);
      if constexpr (DKV) {
        pack(0);
        tmem_st16(tS, pk);      // waited for once the second chunk is computed
        load_columns(aux + 256, col_nl);
      }
      tmem_ld_wait(s1);
      if (__builtin_expect(masked, 0)) keep32(s1, bits32(lo - kv0 - 32, hi - kv0 - 32), kNegInf);
      probabilities<DKV>(s1, cc, nl, col_nl, pr + 16);
      if constexpr (DKV) {
        pack(1);
        tmem_st_wait();
        arrive(&sh.bar_p[0]);
        tmem_st16(tS + 16, pk);
        tmem_st_wait();
        arrive(&sh.bar_p[1]);
      }

      wait(&sh.bar_dp, t & 1);
      __syncwarp();
      tc_fence_after();
      tmem_ld32(tP, s0);
      tmem_ld32(tP + 32, s1);
      tmem_ld_wait(s0);
      tmem_ld_wait(s1);
      if (!DKV) arrive(&sh.bar_read);
      if (__builtin_expect(masked, 0)) {   // whatever stands at a hidden pair is not multiplied by its probability of zero
        keep32(s0, bits32(lo - kv0, hi - kv0), 0u);
        keep32(s1, bits32(lo - kv0 - 32, hi - kv0 - 32), 0u);
      }
      score_gradients<DKV>(s0, pr, nd, aux + 16, pk);
      tmem_st16(DKV ? tP : tS, pk);
      score_gradients<DKV>(s1, pr + 16, nd, aux + 272, pk);
      tmem_st16((DKV ? tP : tS) + 16, pk);
      tmem_st_wait();
      arrive(&sh.bar_ds[t & 1]);
    }
    // The sums leave straight from the registers, 128 bytes of a row a thread in whole sectors:
    // the warps need not wait for the stores (through shared memory and the TMA, with the next
    // item's tile waiting for the stage, was no faster; 16 bytes at a time took 5,700 and 3,000
    // cycles an item).
#pragma unroll 1
    for (int part = DKV ? 0 : 1; part < 2; ++part) {   // dV, dK | dQ
      wait(&sh.bar_sum[part], k & 1);
      if (!__all_sync(0xffffffffu, ok)) return false;
      tc_fence_after();
      const uint32_t tA = tmem + lane_off + (DKV ? 384 - part * 128 : 384) + half * 64;
      const float f = part == 0 ? 1.f : p.scale;
      const int col = (DKV ? 2 - part : 0) * p.d + h * 128 + half * 64;
      tmem_ld32(tA, s0);
      tmem_ld32(tA + 32, s1);
      tmem_ld_wait(s0);
      tmem_ld_wait(s1);
      if (part == 1) arrive(&sh.bar_acc);
      if (live && H3_IN(col + 64 <= 3 * p.d, p.status)) {
        __nv_bfloat16* dst = p.dqkv + size_t(i) * 3 * p.d + col;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int at = 16 * (c & 1) + 2 * e;
            w[e] = pack_bf16x2(__uint_as_float(c < 2 ? s0[at] : s1[at]) * f,
                               __uint_as_float(c < 2 ? s0[at + 1] : s1[at + 1]) * f);
          }
          store16(dst + 16 * c, w, p.sectors);
        }
      }
    }
    ++k;
    return true;
  }
};

__global__ void __launch_bounds__(kThreads, 1)
    attn_bwd_kernel(const __grid_constant__ CUtensorMap tm_rows, const __grid_constant__ CUtensorMap tm_dims,
                    const __grid_constant__ CUtensorMap tmo_rows,
                    const __grid_constant__ CUtensorMap tmo_dims, const __grid_constant__ BwdDev p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sA = base;                  // first factors of S and of dP
  const uint32_t sRing = base + 2 * kTile;
  const uint32_t sAux = sRing + kBoxes * kBox;
  const int warp = warp_id();
  const uint32_t rank = cluster_ctarank();   // 0: issues the pair's products
  if (threadIdx.x == 0) {
    sh.abort_flag = 0;
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&sh.bar_a[s]), 1);
      mbar_init(smem_u32(&sh.bar_s[s]), 1);
      mbar_init(smem_u32(&sh.bar_p[s]), 16);
      mbar_init(smem_u32(&sh.bar_ds[s]), 16);
      mbar_init(smem_u32(&sh.bar_sum[s]), 1);
      mbar_init(smem_u32(&sh.bar_item[s]), 1);
    }
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(smem_u32(&sh.bar_full[s]), 1);
      mbar_init(smem_u32(&sh.bar_empty[s]), 1);
    }
    for (int s = 0; s < kAux; ++s) mbar_init(smem_u32(&sh.bar_aux[s]), 1);
    mbar_init(smem_u32(&sh.bar_dp), 1);
    mbar_init(smem_u32(&sh.bar_read), 16);
    mbar_init(smem_u32(&sh.bar_acc), 16);
    mbar_init(smem_u32(&sh.bar_drain), 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&sh.tmem_base), 512);
    tmem_relinquish_pair();
  }
  if (warp == 0 && lane_id() == 0) {
    tma_prefetch_desc(&tm_rows);
    tma_prefetch_desc(&tm_dims);
    tma_prefetch_desc(&tmo_rows);
    tma_prefetch_desc(&tmo_dims);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers exist before any signal crosses
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  pdl_wait();

  const Maps maps{&tm_rows, &tm_dims, &tmo_rows, &tmo_dims};
  const WaitCtx wc{&sh.abort_flag, p.status, p.wait_ns};
  WaitCtx drain{&sh.abort_flag, p.status, kDrainWaitNs};
  volatile int no_abort = 0;
  drain.abort = &no_abort;
  int idx = int(blockIdx.x >> 1);
  if (warp >= 4) {
    set_max_registers<true, kRegsSoftmax>();
    Softmax sm{p, sh, wc, tmem, sAux, rank, cluster_addr(smem_u32(&sh), 0) - smem_u32(&sh)};
    while (idx >= 0) {
      const Item it = item_of(p, idx);
      if (!(it.dkv ? sm.run<true>(it) : sm.run<false>(it))) break;
      idx = next_item(sh, sm.k, wc);
    }
  } else {
    set_max_registers<false, kRegsFew>();
    if (warp == 0) {
      const bool leader = elect_one();
      Producer pr{maps, p, sh, wc, sA, sRing, sAux, rank, leader};
      while (idx >= 0) {
        // the number of the next item, on its way while this one is loaded
        int next = 0;
        if (rank == 0 && leader) next = int(gridDim.x >> 1) + atomicAdd(p.counter, 1);
        pr.load(item_of(p, idx));
        if (!pr.ok) break;
        const int slot = ++pr.k & 1;
        if (leader) {
          mbar_arrive_expect_tx(smem_u32(&sh.bar_item[slot]), 4);
          if (rank == 0) {
            if (next >= 2 * p.quads * p.H) next = -1;
            send_item(sh, slot, 0, next);
            send_item(sh, slot, 1, next);
          }
        }
        __syncwarp();
        idx = next_item(sh, pr.k, wc);
        if (idx == -2) pr.ok = false;
      }
      // the even CTA lets every copy it armed land before the CTA can exit (earlier ones were
      // consumed before their slot was refilled); the odd CTA's copies count on the even CTA's
      // barriers
      if (!pr.ok) {
        abort_grace();
        if (rank == 0) {
          for (int s = max(0, pr.cnt - kSlots); s < pr.cnt; ++s)
            mbar_wait(smem_u32(&sh.bar_full[s % kSlots]), (s / kSlots) & 1, drain);
          for (int a = 0; a < 2; ++a)
            if (pr.as[a] > 0) mbar_wait(smem_u32(&sh.bar_a[a]), (pr.as[a] - 1) & 1, drain);
        }
        for (int s = max(0, pr.aux - kAux); s < pr.aux; ++s)
          mbar_wait(smem_u32(&sh.bar_aux[s % kAux]), (s / kAux) & 1, drain);
      }
    } else if (warp == 1) {
      if (rank == 0) {
        Issuer is{p, sh, wc, tmem,
                  sdesc_split(sdesc_sw128(sA, 16, 1024)), sdesc_split(sdesc_sw128(sA + kTile, 16, 1024)),
                  sdesc_split(sdesc_sw128(sRing, 16, 1024)), sdesc_split(sdesc_sw128(sRing, kBox, 1024)),
                  elect_one()};
        while (idx >= 0) {
          if (!is.issue(item_of(p, idx))) break;
          idx = next_item(sh, is.k, wc);
        }
        // let every product issued so far finish before either CTA frees tensor memory
        if (is.leader) tc_commit_pair(smem_u32(&sh.bar_drain), 0x3);
        __syncwarp();
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    mbar_wait(smem_u32(&sh.bar_drain), 0, drain);
    __syncwarp();
  }
  cluster_sync();   // neither CTA leaves while the other may still signal it
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// aux: -lse log2(e) and -D = -rowsum(dO * O) for each head and token, heads apart and padded
// to Lp tokens (HBM-bound: 4 bytes an element of O); the count of items starts at 0.  A warp
// takes 8 tokens of a head, half a warp a token of 256 bytes; the warps of a CTA take
// neighbouring heads.
constexpr int kPrepThreads = 256;

__global__ void __launch_bounds__(kPrepThreads)
    attn_bwd_prep_kernel(const uint4* O, const uint4* dO, const float* lse, int L, int H, int Lp,
                         float* aux, int* counter, int* status) {
  pdl_trigger();
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *counter = 0;
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
    if ((lane & 7) >> 1 == k) mine = v;
  }
  // lanes 0 .. 7 write -lse log2(e), 8 .. 15 -D: two groups of four tokens, 64 bytes
  const int64_t t = t0 + (lane & 7);
  const float v = (lane & 8) ? -mine : t < L ? -1.4426950408889634f * ld_dep(lse + size_t(h) * L + t) : -INFINITY;
  if (lane < 16 && H3_IN(h < H && t < Lp, status))
    aux[(size_t(h) * Lp + (t & ~3)) * 2 + ((lane & 8) >> 1) + (lane & 3)] = v;
}

}  // namespace

cudaError_t launch_attention_bwd(const AttnBwdArgs& a, const DevCtx& ctx, cudaStream_t st) {
  const int d = a.H * 128;
  CUtensorMap tm_rows, tm_dims, tmo_rows, tmo_dims;
  if (!make_tmap_bf16_2d(&tm_rows, a.qkv, a.L, 3 * d, 3 * d, 128, 64) ||
      !make_tmap_bf16_halves(&tm_dims, a.qkv, a.L, 3 * d, 64) ||
      !make_tmap_bf16_2d(&tmo_rows, a.dO, a.L, d, d, 128, 64) ||
      !make_tmap_bf16_halves(&tmo_dims, a.dO, a.L, d, 64))
    return cudaErrorInvalidValue;
  BwdDev p{};
  p.dqkv = static_cast<__nv_bfloat16*>(a.dqkv);
  p.sectors = (reinterpret_cast<uintptr_t>(a.dqkv) & 31u) == 0;
  p.counter = a.counter;
  p.aux = a.aux;
  p.L = a.L;
  p.H = a.H;
  p.d = d;
  p.Lp = attn_bwd_padded(a.L);
  p.causal = a.causal;
  p.scale = a.sm_scale;
  p.scale_log2 = a.sm_scale * 1.4426950408889634f;
  p.quads = (a.L + 255) / 256;
  // Under the causal mask items differ in length.  The longest rows of all heads go first while
  // what the heads stream (1 KB a token and head) about fits L2 together: 4,099 x 16 heads 163
  // against 181 us head by head, 8,192 x 16 (134 MB) 519 against 551, 4,096 x 40 (168 MB) 378
  // against 387-410; beyond, a head's items follow one another and share its stream: 16,384 x
  // 16 (268 MB) 2,090-2,150 against 2,180-2,190.
  p.by_rows = a.causal && int64_t(a.L) * a.H * 1024 <= int64_t(192) << 20;
  p.status = ctx.status;
  p.wait_ns = ctx.wait_ns;
  p.n_seg = a.n_seg;
  for (int i = 0; i <= a.n_seg && a.cu_seqlens; ++i) p.cu[i] = a.cu_seqlens[i];

  const int64_t warps = int64_t(p.Lp / 8) * a.H;
  const Launch prep(unsigned((warps + kPrepThreads / 32 - 1) / (kPrepThreads / 32)), kPrepThreads, 0, st);
  cudaError_t e = cudaLaunchKernelEx(&prep.cfg, attn_bwd_prep_kernel, static_cast<const uint4*>(a.O),
                                     static_cast<const uint4*>(a.dO), a.lse, a.L, a.H, p.Lp, a.aux,
                                     a.counter, ctx.status);
  if (e != cudaSuccess) return e;
  static KernelState state;
  if ((e = allow_smem(&state, attn_bwd_kernel, kSmem, ctx)) != cudaSuccess) return e;
  const int64_t items = 2LL * p.quads * a.H, most = ctx.num_sms > 1 ? ctx.num_sms / 2 : 1;
  const Launch main(unsigned(2 * (items < most ? items : most)), kThreads, kSmem, st, 2);
  e = cudaLaunchKernelEx(&main.cfg, attn_bwd_kernel, tm_rows, tm_dims, tmo_rows, tmo_dims, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace h3
