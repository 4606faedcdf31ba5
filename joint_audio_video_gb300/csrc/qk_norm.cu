// RMS norm of each head's queries and keys with the 3D rotary embedding in the same pass,
// and its gradient (both HBM-bound).
//
//   y = R(pos) (x r w),  r = 1 / sqrt(mean x^2 + eps) over the head's 128 values
//   with g = R(pos)^T dy:  dw += g x r,   dx = r (g w - x r^2 mean(x g w))
//
// R turns pair (2j, 2j + 1) of section a by pos[a] base^(-2j / n_a).  Half a warp holds a
// head of a token, 8 values (4 pairs) a lane, so the norm is a sum over 16 lanes, the rotation
// stays in the lane, and a lane's four cosines and sines serve all heads of its token.  The
// angles are exact: a frequency is a 64-bit fraction of a turn for each position, the product
// with the position keeps its fraction (integer arithmetic drops whole turns), and only the
// reduced angle is rounded to fp32, however far the position.
// A warp takes a token: a head's query in its lower half and its key in the upper one, head after
// head, four steps of 512 bytes in flight, then (where the output is another array) the values,
// which are copied.  A lane reads its weights and works out its four angles once for all of that,
// which is what bounds the kernels besides the bytes: with 16 pairs of heads a warp instead of all
// 58,758 x 40 heads took 617 us against 559, and one head, whose angles serve a single step, takes
// 31 us for 13 of bytes.  Seven CTAs of 128 threads an SM keep the reads going (three of 256: 559
// against 541 us); the gradient has registers for five (four: 834 us, six spill in the loop: 1,155).
// What spills as it is (24 bytes a thread; the gradient 52) are registers around the call of
// far_inverse, and 8 bytes of the gradient besides: 11 and 32 of some 4,800 and 7,300
// instructions that a warp executes for a token of 40 heads.
// Algorithmic traffic an element of Q or K: 4 bytes, and 4 of V if copied; the gradient 6, 4.
// 58,758 x 40 heads, out of place: 537 us, 6.7 TB/s; the gradient 769 us, 6.3 TB/s.  In place 376 us,
// 6.4 TB/s, and 602 us, 6.0 TB/s.  (Times here and below are the device's, calls in a graph.)
#include <cmath>
#include <cstring>

#include "f32x2.cuh"
#include "kernels.hpp"
#include "launch.hpp"
#include "ptx.cuh"

namespace h3 {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 4;    // pairs of heads in flight

struct QkNormDev {
  const uint4* qkv;
  const uint4* dout;       // gradient only
  const int32_t* pos;
  const float* wq;
  const float* wk;
  uint4* out;
  int L, H;
  int copy_v;              // the output is another array
  int s0, s01;             // head dims before the h and the w section
  int shares;              // of a token's heads
  float eps;
  int tiny_eps;            // eps below 2^-60: rows of small values need care
  float* partial;          // gradient: [gridDim.x][256] sums of dw, or nullptr
  int* status;
  alignas(16) uint64_t turn[64];   // of pair k: fraction of a turn for each position, times 2^64
};

// Eight bf16 values as four pairs of fp32, and back.
__device__ __forceinline__ void unpack8(const uint4& v, uint64_t (&f)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ uint4 pack8(const uint64_t (&f)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    unf2(f[i], a, b);
    w[i] = pack_bf16x2(a, b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// sum of a b over the lane's eight values
__device__ __forceinline__ float dot8(const uint64_t (&a)[4], const uint64_t (&b)[4]) {
  const uint64_t s = fadd2(ffma2(a[0], b[0], fmul2(a[1], b[1])), ffma2(a[2], b[2], fmul2(a[3], b[3])));
  float lo, hi;
  unf2(s, lo, hi);
  return lo + hi;
}
// The pair (u, v) turned by (cos, sin); the sines and cosines as pairs would take eight more
// registers than the two instructions are worth.
__device__ __forceinline__ uint64_t turn(uint64_t uv, float cs, float sn) {
  float u, v;
  unf2(uv, u, v);
  return f2(fmaf(u, cs, -v * sn), fmaf(u, sn, v * cs));
}
__device__ __forceinline__ void st_cs(uint4* p, const uint4& v) { __stcs(p, v); }   // written once
// Over the 16 lanes of a head; every lane gets the result.
__device__ __forceinline__ float sum16(float v) {
#pragma unroll
  for (int x = 8; x > 0; x >>= 1) v += __shfl_xor_sync(0xffffffffu, v, x);
  return v;
}

// The lane's four rotations (BACK: the other way).
template <bool BACK>
__device__ __forceinline__ void rotations(const QkNormDev& p, int n, int c, float (&cs)[4], float (&sn)[4]) {
  // The lanes' table entries differ: through the constant bank, where arguments lie, they come
  // one after the other, as generic loads of 16 bytes together (some 10 us of 45 at 58,758 x 1
  // head).  The gradient, whose resident warps go from token to token, is better off with the
  // former from a few heads on (58,758 x 40 768 us against 788, x 5 112 against 117, x 4 95
  // against 98, 4,096 x 16 26.8 against 27.4, but 58,758 x 1 49 against 44).
  uint64_t turn[2];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (BACK)
      turn[j % 2] = p.turn[4 * c + j];
    else if (j % 2 == 0)
      asm volatile("ld.v2.u64 {%0, %1}, [%2];" : "=l"(turn[0]), "=l"(turn[1]) : "l"(p.turn + 4 * c + j));
    const int k = 4 * c + j;                                    // pair: dims 2k, 2k + 1
    const int axis = (2 * k >= p.s0) + (2 * k >= p.s01);
    const int64_t at = ld_dep(p.pos + size_t(n) * 3 + axis);
    // The fraction as a signed number of half turns, to fp32 however small: where u is little or
    // nothing, u cos a - v sin a is no better than the sine, whose own error counts then.  (With the
    // hardware's functions, off by some 2^-21 and so by percents of a small sine,
    // 58,758 x 1 head takes 27 us against 31, x 4 62 against 64, x 40 535 both, the gradient the
    // same.)
    const uint64_t frac = uint64_t(at) * turn[j % 2];
    const float half = fmaf(float(uint32_t(frac)), 0x1p-63f, float(int32_t(frac >> 32)) * 0x1p-31f);
    sincospif(BACK ? -half : half, &sn[j], &cs[j]);
  }
}

// 1 / sqrt(mean x^2 + eps) of a head whose squares leave fp32 or, beside an eps that does not
// hide them, vanish: x times 2^-e, and the same power of two to be taken off the factor.
// All lanes of the warp are here; without an eps a head of zeros gets a factor of zero.
__device__ __noinline__ float far_inverse(uint64_t (&pairs)[4], float eps, int* e) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) unf2(pairs[i], x[2 * i], x[2 * i + 1]);
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  bool bad = false;   // an infinity or a NaN: the formula's zeros and NaN
#pragma unroll
  for (int i = 0; i < 8; ++i) bad |= !(fabsf(x[i]) <= 3.4e38f);
  bad = sum16(bad ? 1.f : 0.f) > 0.f;
  *e = bad || top == 0.f ? 0 : max(ilogbf(top), -90);
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = ldexpf(x[i], -*e);
    ss = fmaf(x[i], x[i], ss);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) pairs[i] = f2(x[2 * i], x[2 * i + 1]);
  ss = sum16(ss);
  if (top == 0.f && !bad && eps == 0.f) return 0.f;
  return rsqrtf(ss * (1.f / 128.f) + ldexpf(eps, -2 * *e));
}

template <bool GRAD>
__global__ void __launch_bounds__(kThreads, GRAD ? 5 : 7)
    qk_norm_kernel(const __grid_constant__ QkNormDev p) {
  __shared__ float red[GRAD ? kWarps : 1][256];
  pdl_trigger();
  pdl_wait();
  const int lane = int(lane_id()), hw = lane >> 4, c = lane & 15;
  const float* weight = hw ? p.wk : p.wq;            // half a warp has queries, the other keys
  uint64_t w[4], dw[4];
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    float4 v = make_float4(1.f, 1.f, 1.f, 1.f);
    if (weight != nullptr) v = ld_dep(reinterpret_cast<const float4*>(weight + 8 * c + 2 * i));
    w[i] = f2(v.x, v.y);
    w[i + 1] = f2(v.z, v.w);
    dw[i] = dw[i + 1] = 0;
  }
  // steps of a token: a head's query and key each, then two heads of V each
  const int norms = p.H, all = norms + (p.copy_v ? (p.H + 1) / 2 : 0);
  const size_t row = size_t(3) * p.H * 16;
  const int64_t items = int64_t(p.L) * p.shares;
  for (int64_t it = int64_t(blockIdx.x) * kWarps + warp_id(); it < items;
       it += int64_t(gridDim.x) * kWarps) {
    const int n = int(it / p.shares), share = int(it - int64_t(n) * p.shares);
    const size_t base = size_t(n) * row + c;
    float cs[4], sn[4];
    bool turned = false;
    for (int i0 = share; i0 < all; i0 += kBatch * p.shares) {
      uint4 xv[kBatch], gv[kBatch];
      uint32_t at[kBatch];   // of this half warp's head in the row, none: past it
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int i = i0 + b * p.shares;
        const bool norm = i < norms;
        const int head = norm ? hw * p.H + i : 2 * (p.H + i - norms) + hw;   // of the row's 3 H
        const bool in = i < all && head < 3 * p.H;
        at[b] = in ? uint32_t(head) * 16 : ~0u;
        xv[b] = gv[b] = make_uint4(0u, 0u, 0u, 0u);
        if (in && H3_IN(n < p.L && at[b] + 16 <= row, p.status)) {
          if (!GRAD || norm) xv[b] = ld_dep_cs(p.qkv + base + at[b]);
          if (GRAD) gv[b] = ld_dep_cs(p.dout + base + at[b]);
        }
      }
      if (!turned && i0 < norms) {   // under the first loads
        rotations<GRAD>(p, n, c, cs, sn);
        turned = true;
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int i = i0 + b * p.shares;
        if (i >= all) break;   // both halves of the warp
        uint4 o = GRAD ? gv[b] : xv[b];
        if (i < norms) {
          uint64_t x[4], g[4];
          unpack8(xv[b], x);
          float sq = dot8(x, x);
          if constexpr (GRAD) {
            unpack8(gv[b], g);
#pragma unroll
            for (int j = 0; j < 4; ++j) g[j] = turn(g[j], cs[j], sn[j]);
          }
          sq = sum16(sq);
          float r = rsqrtf(sq * (1.f / 128.f) + p.eps);
          int ex = 0;
          // squares out of fp32's range (or, with next to no eps, below it), infinities, NaN
          const bool far = !(sq < 0x1p120f) || (p.tiny_eps && sq < 0x1p-80f);
          if (__any_sync(0xffffffffu, far)) {
            uint64_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = x[e];
            int fe;
            const float fr = far_inverse(y, p.eps, &fe);
            if (far) {
              r = fr;
              ex = fe;
#pragma unroll
              for (int e = 0; e < 4; ++e) x[e] = y[e];
            }
          }
          const uint64_t rr = f2(r, r);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = fmul2(x[e], rr);   // normalised
          if constexpr (!GRAD) {
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = turn(fmul2(x[j], w[j]), cs[j], sn[j]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              dw[e] = ffma2(g[e], x[e], dw[e]);
              g[e] = fmul2(g[e], w[e]);
            }
            const float sg = sum16(dot8(g, x)) * (-1.f / 128.f);
            const uint64_t mm = f2(sg, sg);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = fmul2(rr, ffma2(x[e], mm, g[e]));
            if (__any_sync(0xffffffffu, ex != 0)) {   // the factor of a head taken times 2^-ex
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float a, b2;
                unf2(x[e], a, b2);
                x[e] = f2(ldexpf(a, -ex), ldexpf(b2, -ex));
              }
            }
          }
          o = pack8(x);
        }
        if (at[b] != ~0u && H3_IN(n < p.L && at[b] + 16 <= row, p.status)) st_cs(p.out + base + at[b], o);
      }
    }
  }
  if constexpr (GRAD) {
    if (p.partial == nullptr) return;
    // the CTA's sums, in a fixed order
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      unf2(dw[i], a, b);
      red[warp_id()][128 * hw + 8 * c + 2 * i] = a;
      red[warp_id()][128 * hw + 8 * c + 2 * i + 1] = b;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < 256; k += kThreads) {
      float s = 0.f;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) s += red[v][k];
      if (H3_IN(blockIdx.x < kQkNormPartials, p.status)) p.partial[size_t(blockIdx.x) * 256 + k] = s;
    }
  }
}

// dw from the CTAs' sums: 32 columns a CTA, 32 threads a column, in a fixed order.
__global__ void __launch_bounds__(1024)
    qk_norm_dw_kernel(const float* partial, int rows, float* dwq, float* dwk, int* status) {
  __shared__ float red[32][33];
  pdl_wait();
  const int x = int(threadIdx.x & 31), y = int(threadIdx.x >> 5);
  const int col = int(blockIdx.x) * 32 + x;
  float s = 0.f;
  for (int r0 = y; r0 < rows; r0 += 256) {   // eight loads in flight
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = r0 + 32 * i;
      v[i] = 0.f;
      if (r < rows && H3_IN(r < kQkNormPartials && col < 256, status))
        v[i] = ld_dep(partial + size_t(r) * 256 + col);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s += v[i];
  }
  red[y][x] = s;
  __syncthreads();
  // warp y now has column y of the CTA: lane x its x-th thread's sum
  s = red[x][y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int mine = int(blockIdx.x) * 32 + y;
  float* dw = mine < 128 ? dwq : dwk;
  if (x == 0 && dw != nullptr && H3_IN(mine < 256, status)) dw[mine & 127] = s;
}

// Turns for each position of the 64 pairs, times 2^64; whole turns (a base below 1 / 2 pi) do
// not matter.  64 powers take 1.7 us, so a thread keeps the last sections' and base's.
struct Turns {
  int32_t sec[3] = {-1, -1, -1};
  float base = 0.f;
  uint64_t turn[64];
};
const uint64_t* turns(const int32_t (&sec)[3], float base) {
  static thread_local Turns last;
  if (last.base == base && std::memcmp(last.sec, sec, sizeof sec) == 0) return last.turn;
  int k = 0;
  for (int s = 0; s < 3; ++s)
    for (int j = 0; j < sec[s] / 2; ++j, ++k) {
      const double t = std::pow(double(base), -2.0 * j / sec[s]) / 6.283185307179586476925;
      last.turn[k] = uint64_t(std::ldexp(t - std::floor(t), 64));
    }
  last.base = base;
  std::memcpy(last.sec, sec, sizeof sec);
  return last.turn;
}

QkNormDev device_args(const QkNormArgs& a, const DevCtx& ctx) {
  QkNormDev p{};
  p.qkv = static_cast<const uint4*>(a.qkv);
  p.dout = static_cast<const uint4*>(a.dout);
  p.pos = a.pos;
  p.wq = a.wq;
  p.wk = a.wk;
  p.out = static_cast<uint4*>(a.out);
  p.L = a.L;
  p.H = a.H;
  p.copy_v = a.out != (a.dout != nullptr ? a.dout : a.qkv);
  p.s0 = a.sec[0];
  p.s01 = a.sec[0] + a.sec[1];
  p.eps = a.eps;
  p.tiny_eps = a.eps < 0x1p-60f;
  p.status = ctx.status;
  std::memcpy(p.turn, turns(a.sec, a.base), sizeof p.turn);
  return p;
}

}  // namespace

// Warps of a token: as many as fill every SM once (kWanted warps), of at least kBatch steps each.
// For 56 warps 2,048 or 4,099 x 16 heads take 9.8 or 16.8 us instead of 8.4 or 15.9: every warp
// works out the angles again.
constexpr int kWanted = 28;
static int shares_of(const QkNormDev& p, const DevCtx& ctx) {
  const int all = p.H + (p.copy_v ? (p.H + 1) / 2 : 0);
  const int fine = (all + kBatch - 1) / kBatch;
  const int64_t wanted = (int64_t(ctx.num_sms) * kWanted + p.L - 1) / p.L;
  return wanted < fine ? int(wanted) : fine;
}

cudaError_t launch_qk_norm(const QkNormArgs& a, const DevCtx& ctx, cudaStream_t st) {
  QkNormDev p = device_args(a, ctx);
  p.shares = shares_of(p, ctx);
  const int64_t grid = (int64_t(a.L) * p.shares + kWarps - 1) / kWarps;
  const Launch l(unsigned(grid < INT32_MAX ? grid : INT32_MAX), kThreads, 0, st);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, qk_norm_kernel<false>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_qk_norm_bwd(const QkNormArgs& a, const DevCtx& ctx, cudaStream_t st) {
  QkNormDev p = device_args(a, ctx);
  p.shares = shares_of(p, ctx);
  p.partial = a.dwq != nullptr || a.dwk != nullptr ? a.partial : nullptr;
  static KernelState state;
  int per_sm = 1;
  if (cudaError_t e = ctas_per_sm(&state, qk_norm_kernel<true>, kThreads, 0, ctx, &per_sm)) return e;
  // as many CTAs as are resident at once: each leaves one row of sums
  int64_t grid = (int64_t(a.L) * p.shares + kWarps - 1) / kWarps;
  const int64_t most = int64_t(ctx.num_sms) * per_sm;
  grid = grid < most ? grid : most;
  if (grid > kQkNormPartials) grid = kQkNormPartials;
  const Launch l(unsigned(grid), kThreads, 0, st);
  cudaError_t e = cudaLaunchKernelEx(&l.cfg, qk_norm_kernel<true>, p);
  if (e != cudaSuccess || p.partial == nullptr) return e != cudaSuccess ? e : cudaGetLastError();
  const Launch sum(8, 1024, 0, st);
  e = cudaLaunchKernelEx(&sum.cfg, qk_norm_dw_kernel, static_cast<const float*>(a.partial), int(grid),
                         a.dwq, a.dwk, ctx.status);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace h3
