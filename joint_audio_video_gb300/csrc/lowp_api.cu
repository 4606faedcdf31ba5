// C ABI of the 4-bit projections and the quantising norms (include/h3attn_lowp.h).
// As in h3attn_api.cu, every entry point checks its arguments on the host and returns
// a status before anything is launched.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/h3attn_lowp.h"
#include "api_common.hpp"
#include "kernels.hpp"

namespace h3 {
namespace {

bool valid_fmt(int32_t fmt) { return fmt == H3_FP4_MX || fmt == H3_FP4_NV; }
bool valid_k(int32_t K) { return K >= 128 && K <= 65536 && K % 128 == 0; }
bool aligned4(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
// an optional array: absent, or aligned
bool optional16(const void* p) { return p == nullptr || aligned16(p); }

size_t scale_bytes(int32_t fmt, size_t R, size_t K) {
  return (R + 127) / 128 * 128 * (K / (fmt == H3_FP4_MX ? 32 : 16));
}

struct Span {
  const void* p;
  size_t n;
};
// No two of the spans overlap (absent ones aside).
template <int N>
bool disjoint(const Span (&s)[N]) {
  for (int i = 0; i < N; ++i)
    for (int j = i + 1; j < N; ++j)
      if (s[i].p != nullptr && s[j].p != nullptr && overlap(s[i].p, s[i].n, s[j].p, s[j].n))
        return false;
  return true;
}
// `o` overlaps none of the spans.
template <int N>
bool apart(const Span& o, const Span (&s)[N]) {
  for (int i = 0; i < N; ++i)
    if (o.p != nullptr && s[i].p != nullptr && overlap(o.p, o.n, s[i].p, s[i].n)) return false;
  return true;
}

h3_status rms_norm(const RmsNormArgs& a, size_t q_bytes, size_t bs_bytes, bool has_scale,
                   h3_stream_t stream) {
  if (a.L < 1 || !valid_d(a.d)) return H3_ERR_INVALID_ARG;
  if (!(a.eps >= 0.f) || !std::isfinite(a.eps)) return H3_ERR_INVALID_ARG;
  if (!aligned16(a.x) || !optional16(a.res) || !aligned16(a.weight) || !optional16(a.sum) ||
      !aligned16(a.q))
    return H3_ERR_INVALID_ARG;
  const size_t n = size_t(a.L) * a.d * 2;
  const Span in[3] = {{a.x, n}, {a.res, n}, {a.weight, size_t(a.d) * 4}};
  const Span q{a.q, q_bytes}, bs{a.bs, bs_bytes},
      scale{has_scale ? a.scale : nullptr, size_t(a.L) * 4};
  if (!apart(q, in) || !apart(bs, in) || !apart(scale, in)) return H3_ERR_INVALID_ARG;
  const Span out[4] = {q, bs, scale, {a.sum, n}};
  if (!disjoint(out)) return H3_ERR_INVALID_ARG;
  if (a.sum != nullptr)   // may be x or res itself, else apart from both
    for (int i = 0; i < 3; ++i)
      if (in[i].p != nullptr && !(i < 2 && in[i].p == a.sum) &&
          overlap(a.sum, n, in[i].p, in[i].n))
        return H3_ERR_INVALID_ARG;
  DevCtx ctx;
  if (h3_status s = dev_ctx(&ctx)) return s;
  return finish(launched(launch_rms_norm(a, ctx, reinterpret_cast<cudaStream_t>(stream))), stream);
}

}  // namespace
}  // namespace h3

using namespace h3;

extern "C" {

h3_status h3_fp4_scale_bytes(int32_t fmt, int32_t R, int32_t K, size_t* bytes) {
  if (bytes == nullptr || !valid_fmt(fmt) || R < 1 || !valid_k(K)) return H3_ERR_INVALID_ARG;
  *bytes = scale_bytes(fmt, size_t(R), size_t(K));
  return H3_OK;
}

h3_status h3_quantize_rows_fp4(const uint16_t* x, int32_t fmt, int32_t R, int32_t K, uint8_t* q,
                               uint8_t* bs, float* s, h3_stream_t stream) {
  const Trace trace_("h3_quantize_rows_fp4");
  if (!valid_fmt(fmt) || R < 1 || !valid_k(K)) return H3_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(q) || !aligned16(bs)) return H3_ERR_INVALID_ARG;
  if (fmt == H3_FP4_NV && !aligned4(s)) return H3_ERR_INVALID_ARG;
  const size_t r = size_t(R), k = size_t(K);
  const Span all[4] = {{x, r * k * 2},
                       {q, r * k / 2},
                       {bs, scale_bytes(fmt, r, k)},
                       {fmt == H3_FP4_NV ? s : nullptr, r * 4}};
  if (!disjoint(all)) return H3_ERR_INVALID_ARG;
  DevCtx ctx;
  if (h3_status e = dev_ctx(&ctx)) return e;
  return finish(launched(launch_quantize_fp4(x, fmt, R, K, q, bs, s, ctx,
                                             reinterpret_cast<cudaStream_t>(stream))), stream);
}

h3_status h3_dequantize_rows_fp4(const uint8_t* q, const uint8_t* bs, const float* s, int32_t fmt,
                                 int32_t R, int32_t K, uint16_t* y, h3_stream_t stream) {
  const Trace trace_("h3_dequantize_rows_fp4");
  if (!valid_fmt(fmt) || R < 1 || !valid_k(K)) return H3_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(bs) || !aligned16(y) || (s != nullptr && !aligned4(s)))
    return H3_ERR_INVALID_ARG;
  const size_t r = size_t(R), k = size_t(K);
  const Span in[3] = {{q, r * k / 2}, {bs, scale_bytes(fmt, r, k)}, {s, r * 4}};
  if (!apart(Span{y, r * k * 2}, in)) return H3_ERR_INVALID_ARG;
  DevCtx ctx;
  if (h3_status e = dev_ctx(&ctx)) return e;
  return finish(launched(launch_dequantize_fp4(q, bs, s, fmt, R, K, y, ctx,
                                               reinterpret_cast<cudaStream_t>(stream))), stream);
}

h3_status h3_gemm_fp4(const uint8_t* A, const uint8_t* a_bs, const float* a_s, const uint8_t* B,
                      const uint8_t* b_bs, const float* b_s, int32_t fmt, int32_t M, int32_t N,
                      int32_t K, uint16_t* C, h3_stream_t stream) {
  const Trace trace_("h3_gemm_fp4");
  if (!valid_fmt(fmt) || M < 1 || N < 128 || N % 128 != 0 || !valid_k(K)) return H3_ERR_INVALID_ARG;
  // the kernels count output tiles (at least 128 x 128) in 32-bit integers
  if ((int64_t(M) + 127) / 128 * (int64_t(N) / 128) > INT32_MAX) return H3_ERR_INVALID_ARG;
  if (!aligned16(A) || !aligned16(a_bs) || !optional16(a_s) || !aligned16(B) || !aligned16(b_bs) ||
      !optional16(b_s) || !aligned16(C))
    return H3_ERR_INVALID_ARG;
  const size_t m = size_t(M), n = size_t(N), k = size_t(K);
  const Span in[6] = {{A, m * k / 2}, {a_bs, scale_bytes(fmt, m, k)}, {a_s, m * 4},
                      {B, n * k / 2}, {b_bs, scale_bytes(fmt, n, k)}, {b_s, n * 4}};
  if (!apart(Span{C, m * n * 2}, in)) return H3_ERR_INVALID_ARG;
  DevCtx ctx;
  if (h3_status s = dev_ctx(&ctx)) return s;
  GemmFp4Args g{};
  g.A = A;
  g.a_bs = a_bs;
  g.a_s = a_s;
  g.B = B;
  g.b_bs = b_bs;
  g.b_s = b_s;
  g.fmt = fmt;
  g.M = M;
  g.N = N;
  g.K = K;
  g.C = C;
  g.epilogue = EPI_PLAIN;
  return finish(launched(launch_gemm_fp4(g, ctx, reinterpret_cast<cudaStream_t>(stream))), stream);
}

h3_status h3_rms_norm_fp8(const uint16_t* x, const uint16_t* res, const float* weight, int32_t L,
                          int32_t d, float eps, uint16_t* sum, uint8_t* q, float* scale,
                          h3_stream_t stream) {
  const Trace trace_("h3_rms_norm_fp8");
  if (L < 1 || !valid_d(d) || !aligned4(scale)) return H3_ERR_INVALID_ARG;
  const RmsNormArgs a{x, res, weight, L, d, eps, 0, sum, q, nullptr, scale};
  return rms_norm(a, size_t(L) * d, 0, true, stream);
}

h3_status h3_rms_norm_fp4(const uint16_t* x, const uint16_t* res, const float* weight, int32_t L,
                          int32_t d, float eps, int32_t fmt, uint16_t* sum, uint8_t* q,
                          uint8_t* bs, float* s, h3_stream_t stream) {
  const Trace trace_("h3_rms_norm_fp4");
  if (!valid_fmt(fmt) || L < 1 || !valid_d(d) || !aligned16(bs)) return H3_ERR_INVALID_ARG;
  if (fmt == H3_FP4_NV && !aligned4(s)) return H3_ERR_INVALID_ARG;
  const RmsNormArgs a{x, res, weight, L, d, eps, fmt, sum, q, bs, s};
  return rms_norm(a, size_t(L) * d / 2, scale_bytes(fmt, size_t(L), size_t(d)), fmt == H3_FP4_NV,
                  stream);
}

// Workspace of the 4-bit MLP: y [L][d] | h [L][hidden] bf16 | the codes, block scales and
// row factors of y, then of h.
h3_status h3_mlp_workspace_size_fp4(const h3_mlp_desc* desc, int32_t fmt, size_t* bytes) {
  if (bytes == nullptr || !valid_fmt(fmt)) return H3_ERR_INVALID_ARG;
  size_t base = 0;
  if (h3_status s = h3_mlp_workspace_size(desc, &base)) return s;
  const size_t L = size_t(desc->L);
  const size_t wide = size_t(desc->d > desc->hidden ? desc->d : desc->hidden);
  *bytes = base + round256(L * wide / 2) + round256(scale_bytes(fmt, L, wide)) + round256(L * 4);
  return H3_OK;
}

h3_status h3_mlp_block_fwd_fp4(const h3_mlp_desc* desc, int32_t fmt, const uint16_t* x,
                               const uint8_t* mod, const float* shift, const float* scale,
                               const float* gate, const uint8_t* W1_q, const uint8_t* W1_bs,
                               const float* W1_s, const uint8_t* W2_q, const uint8_t* W2_bs,
                               const float* W2_s, void* workspace, size_t workspace_bytes,
                               uint16_t* out, h3_stream_t stream) {
  const Trace trace_("h3_mlp_block_fwd_fp4");
  size_t need = 0;
  if (h3_status s = h3_mlp_workspace_size_fp4(desc, fmt, &need)) return s;
  if (!aligned16(x) || mod == nullptr || !aligned16(shift) || !aligned16(scale) ||
      !aligned16(gate) || !aligned16(W1_q) || !aligned16(W1_bs) || !optional16(W1_s) ||
      !aligned16(W2_q) || !aligned16(W2_bs) || !optional16(W2_s) || !aligned16(out) ||
      workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return H3_ERR_INVALID_ARG;
  if (workspace_bytes < need) return H3_ERR_WORKSPACE;
  const size_t L = size_t(desc->L), d = size_t(desc->d), hid = size_t(desc->hidden);
  const size_t nm = size_t(desc->n_mod) * d * 4;
  const Span in[10] = {{mod, L},
                       {shift, nm},
                       {scale, nm},
                       {gate, nm},
                       {W1_q, hid * d / 2},
                       {W1_bs, scale_bytes(fmt, hid, d)},
                       {W1_s, hid * 4},
                       {W2_q, d * hid / 2},
                       {W2_bs, scale_bytes(fmt, d, hid)},
                       {W2_s, d * 4}};
  const Span ws_span{workspace, need}, out_span{out, L * d * 2};
  if (x != out && overlap(x, L * d * 2, out, L * d * 2)) return H3_ERR_INVALID_ARG;
  if (overlap(workspace, need, x, L * d * 2) || overlap(workspace, need, out, L * d * 2) ||
      !apart(ws_span, in) || !apart(out_span, in))
    return H3_ERR_INVALID_ARG;
  DevCtx ctx;
  if (h3_status s = dev_ctx(&ctx)) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint8_t* y = ws;
  uint8_t* h = y + round256(L * d * 2);
  uint8_t* q4 = h + round256(L * hid * 2);
  const size_t wide = d > hid ? d : hid;
  uint8_t* bs = q4 + round256(L * wide / 2);
  float* s4 = reinterpret_cast<float*>(bs + round256(scale_bytes(fmt, L, wide)));
  const float* as = fmt == H3_FP4_NV ? s4 : nullptr;
  if (launch_adaln_modulate(x, mod, shift, scale, desc->L, desc->d, desc->n_mod, desc->ln_eps, y,
                            ctx, st) != cudaSuccess ||
      launch_quantize_fp4(y, fmt, desc->L, desc->d, q4, bs, s4, ctx, st) != cudaSuccess)
    return H3_ERR_CUDA;
  GemmFp4Args up{};
  up.A = q4;
  up.a_bs = bs;
  up.a_s = as;
  up.B = W1_q;
  up.b_bs = W1_bs;
  up.b_s = W1_s;
  up.fmt = fmt;
  up.M = desc->L;
  up.N = desc->hidden;
  up.K = desc->d;
  up.C = h;
  up.epilogue = EPI_GELU;
  if (launch_gemm_fp4(up, ctx, st) != cudaSuccess ||
      launch_quantize_fp4(h, fmt, desc->L, desc->hidden, q4, bs, s4, ctx, st) != cudaSuccess)
    return H3_ERR_CUDA;
  GemmFp4Args down = up;
  down.B = W2_q;
  down.b_bs = W2_bs;
  down.b_s = W2_s;
  down.N = desc->d;
  down.K = desc->hidden;
  down.C = out;
  down.epilogue = EPI_GATED_RESIDUAL;
  down.x_res = x;
  down.mod = mod;
  down.gate = gate;
  down.n_mod = desc->n_mod;
  return finish(launched(launch_gemm_fp4(down, ctx, st)), stream);
}

}  // extern "C"
