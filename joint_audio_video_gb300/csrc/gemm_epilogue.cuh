// What the tcgen05 GEMMs share: the tile order and the fused epilogues that turn a
// finished fp32 accumulator tile into rows of C (see gemm.cu for the list).
#pragma once

#include <cuda_bf16.h>

#include "factors.cuh"
#include "kernels.hpp"
#include "ptx.cuh"

namespace h3 {
namespace {

constexpr int BM = 128;

struct GemmDev {
  __nv_bfloat16* C;
  int M, N, K;
  int num_m, num_n;
  const int32_t* pos;
  int d;
  const __nv_bfloat16* x_res;
  const uint8_t* mod;
  const float* gate;
  int n_mod;
  int* status;
  uint64_t wait_ns;
  const float* a_scale;
  const float* b_scale;
};

__device__ __forceinline__ void tile_coords(int t, int num_m, int num_n, int& mb, int& nb,
                                            int group_m) {
  const int per_group = group_m * num_n;
  const int g = t / per_group;
  const int first_m = g * group_m;
  const int gsz = min(num_m - first_m, group_m);
  const int r = t - g * per_group;
  mb = first_m + r % gsz;
  nb = r / gsz;
}

// Whether, for some row of this warp and column of a tile BN wide, the product of the two
// scales may leave fp32: a lane looks at its row's scale and at every 32nd column's, b(i) for
// column i of the tile.  Asked before the accumulator is waited for (asked in every chunk
// 4,096 x 8,192 x 256 in E4M3 took 41.0 us instead of 34.9).
template <int BN, class Scale>
__device__ __forceinline__ bool far_scales(float sa, Scale b) {
  bool far = !mid_range(sa);
#pragma unroll
  for (int c = 0; c < BN; c += 32) far |= !mid_range(b(c + int(lane_id())));
  return __any_sync(0xffffffffu, far);
}

// Epilogue of one 32-column chunk held in r[] (fp32 bits) for row `grow`,
// global columns gc .. gc+31.  SC: 0 no scales, 1 a_scale[row] * b_scale[col],
// 2 scales that the caller has applied, 3 as 1 with the columns' scales at b_shared in shared
// memory (2 and 3: kernels that may start before the work ahead of them is done).  FAR: some
// product of two scales may leave fp32.
template <int EPI, int SC, bool FAR>
__device__ __forceinline__ void epilogue_chunk(const GemmDev& p, const RopeTable& rt,
                                               uint32_t (&r)[32], int grow, int gc,
                                               const int32_t (&pr)[3], int m, float sa,
                                               uint32_t (&pk)[16],
                                               const float* b_shared = nullptr) {
  // row grow, columns gc .. gc + 31 of C and x_res, columns of gate (row m) and b_scale
  if (!H3_IN(gc >= 0 && gc + 32 <= p.N && grow >= 0 && grow < p.M && (EPI != EPI_GATED_RESIDUAL || m < p.n_mod),
             p.status))
    return;
  float v[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
  if constexpr ((SC == 1 || SC == 3) && FAR) {
    float t[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) t[i] = v[i];
    times_apart_n(t, 32, sa, SC == 3 ? b_shared : p.b_scale + gc);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = t[i];
  } else if constexpr (SC == 3) {
    const float4* sb = reinterpret_cast<const float4*>(b_shared);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 b = sb[i];
      v[4 * i + 0] *= sa * b.x;
      v[4 * i + 1] *= sa * b.y;
      v[4 * i + 2] *= sa * b.z;
      v[4 * i + 3] *= sa * b.w;
    }
  } else if constexpr (SC == 1) {   // row scale of A times column scale of B
    const float4* sb = reinterpret_cast<const float4*>(p.b_scale + gc);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 b = __ldg(sb + i);
      v[4 * i + 0] *= sa * b.x;
      v[4 * i + 1] *= sa * b.y;
      v[4 * i + 2] *= sa * b.z;
      v[4 * i + 3] *= sa * b.w;
    }
  }
  if constexpr (EPI == EPI_ROPE) {
    if (gc < 2 * p.d) {   // Q or K block: rotate pairs (2k, 2k+1) of the head
      const int k0 = (gc & 127) >> 1;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int k = k0 + j;
        const int ax = rt.axis[k];
        const int pa = ax == 0 ? pr[0] : (ax == 1 ? pr[1] : pr[2]);
        const float ang = float(pa) * rt.inv_freq[k];
        float s, c;
        sincosf(ang, &s, &c);
        const float a = v[2 * j], b = v[2 * j + 1];
        v[2 * j] = a * c - b * s;
        v[2 * j + 1] = a * s + b * c;
      }
    }
  }
  if constexpr (EPI == EPI_GELU) {
    // 0.5 u (1 + tanh(sqrt(2/pi) (u + 0.044715 u^3))), tanh by the MUFU
    // instruction (relative error ~2^-11, below the bf16 rounding of the result)
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float u = v[i];
      float t;
      asm("tanh.approx.f32 %0, %1;" : "=f"(t) : "f"(0.7978845608028654f * fmaf(0.044715f * u, u * u, u)));
      v[i] = 0.5f * u * (1.f + t);
    }
  }
  if constexpr (EPI == EPI_GATED_RESIDUAL) {
    const uint4* xr = reinterpret_cast<const uint4*>(p.x_res + size_t(grow) * p.N + gc);
    const float4* gr = reinterpret_cast<const float4*>(p.gate + size_t(m) * p.N + gc);
    uint4 xv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) xv[i] = xr[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 g = SC < 2 ? __ldg(gr + i) : ld_dep(gr + i);
      const uint32_t w0 = (&xv[i >> 1].x)[(i & 1) * 2];
      const uint32_t w1 = (&xv[i >> 1].x)[(i & 1) * 2 + 1];
      v[4 * i + 0] = fmaf(g.x, v[4 * i + 0], __uint_as_float(w0 << 16));
      v[4 * i + 1] = fmaf(g.y, v[4 * i + 1], __uint_as_float(w0 & 0xFFFF0000u));
      v[4 * i + 2] = fmaf(g.z, v[4 * i + 2], __uint_as_float(w1 << 16));
      v[4 * i + 3] = fmaf(g.w, v[4 * i + 3], __uint_as_float(w1 & 0xFFFF0000u));
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) pk[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
}

// The epilogue hands C to the TMA in 128-row x 32-column chunks staged in shared
// memory (64-byte rows with the 64-byte swizzle: 16-byte chunk c of row r at
// c ^ ((r / 2) % 4)), two staging buffers; each chunk is one bulk tensor store,
// so C leaves the SM as whole lines instead of one 16-byte piece per row.
constexpr uint32_t kStageC = BM * 64;   // bytes of one staging buffer
__device__ __forceinline__ void epi_bar() {   // the 128 epilogue threads
  asm volatile("bar.sync 1, 128;" ::: "memory");
}
__device__ __forceinline__ bool epi_bar_and(bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred q, a;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "bar.red.and.pred a, 1, 128, q;\n\tselp.u32 %0, 1, 0, a;\n\t}"
      : "=r"(r)
      : "r"(uint32_t(pred))
      : "memory");
  return r != 0;
}

// Epilogue of one finished accumulator: 128 rows (this thread's row is
// row_in_tile) x BN columns at tensor-memory address tacc, written as C rows
// row0 .. row0 + 127, columns col0 .. col0 + BN - 1.  Returns true if the
// row's modality id was out of range (the row is written as NaN).
template <int BN, int EPI, int SC, bool FAR>
__device__ __forceinline__ bool epilogue_tile(const GemmDev& p, const RopeTable& rt,
                                              const CUtensorMap* tmC, uint32_t tacc, int row0,
                                              int col0, int row_in_tile, bool leader, uint32_t sC,
                                              int& chunk) {
  const uint32_t srow = uint32_t(row_in_tile) * 64;
  const uint32_t ssw = uint32_t(row_in_tile >> 1) & 3u;
  const int grow = row0 + row_in_tile;
  const bool live = grow < p.M;
  int32_t pr[3] = {0, 0, 0};
  int m = 0;
  if constexpr (EPI == EPI_ROPE) {
    if (live) {
      pr[0] = p.pos[size_t(grow) * 3 + 0];
      pr[1] = p.pos[size_t(grow) * 3 + 1];
      pr[2] = p.pos[size_t(grow) * 3 + 2];
    }
  }
  float sa = 1.f;
  if constexpr (SC != 0) {
    if (live) sa = __ldg(p.a_scale + grow);
  }
  bool bad = false;
  if constexpr (EPI == EPI_GATED_RESIDUAL) {
    if (live) {
      m = p.mod[grow];
      if (m >= p.n_mod) { bad = true; m = 0; }
    }
  }
#pragma unroll 1
  for (int c = 0; c < BN / 32; ++c) {
    uint32_t r[32];
    tmem_ld32(tacc + c * 32, r);
    tmem_ld_wait(r);
    uint32_t pk[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) pk[i] = 0u;   // rows past M: clipped by the store
    if (live) {
      if (bad) {
#pragma unroll
        for (int i = 0; i < 32; ++i) r[i] = 0x7FC00000u;   // NaN row
      }
      epilogue_chunk<EPI, SC, FAR>(p, rt, r, grow, col0 + c * 32, pr, m, sa, pk);
    }
    // the store that last read this buffer (two chunks ago) has read it
    const uint32_t sb = sC + uint32_t(chunk & 1) * kStageC;
    if (leader) bulk_wait_read_1();
    epi_bar();
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(sb + srow + ((uint32_t(i) ^ ssw) << 4)),
                   "r"(pk[4 * i]), "r"(pk[4 * i + 1]), "r"(pk[4 * i + 2]), "r"(pk[4 * i + 3])
                   : "memory");
    fence_async_shared();
    epi_bar();
    if (leader) {
      tma_store_2d(tmC, sb, col0 + c * 32, row0);
      bulk_commit();
    }
    ++chunk;
  }
  return bad;
}

// What the epilogue of one row needs beside its accumulator.
struct EpilogueRow {
  float sa;     // a_scale of the row
  int m;        // its modality
  bool bad;     // the modality id was out of range: the row is written as NaN
};
template <int EPI, int SC>
__device__ __forceinline__ EpilogueRow epilogue_row(const GemmDev& p, int grow, bool live) {
  EpilogueRow e{1.f, 0, false};
  if constexpr (SC != 0) {
    if (live && p.a_scale != nullptr) e.sa = ld_dep(p.a_scale + grow);
  }
  if constexpr (EPI == EPI_GATED_RESIDUAL) {
    if (live) {
      e.m = p.mod[grow];
      if (e.m >= p.n_mod) { e.bad = true; e.m = 0; }
    }
  }
  return e;
}

}  // namespace
}  // namespace h3
