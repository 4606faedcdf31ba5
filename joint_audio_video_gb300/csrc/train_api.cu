// C ABI of the norm of queries and keys and of the gradients (include/h3attn_train.h).
// As in h3attn_api.cu, every entry point checks its arguments on the host and returns a
// status before anything is launched.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/h3attn_train.h"
#include "api_common.hpp"
#include "kernels.hpp"

namespace h3 {
namespace {

bool aligned256(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }

// L tokens of n_heads heads of head_dim.
h3_status check_shape(int32_t L, int32_t n_heads, int32_t head_dim) {
  if (L < 1 || n_heads < 1) return H3_ERR_INVALID_ARG;
  if (head_dim != 128) return H3_ERR_UNSUPPORTED;
  return valid_heads(n_heads) ? H3_OK : H3_ERR_INVALID_ARG;
}

h3_status check_norm(const QkNormArgs& a, int32_t head_dim) {
  if (h3_status s = check_shape(a.L, a.H, head_dim)) return s;
  if (h3_status s = check_rope(a.sec, head_dim, a.base)) return s;
  if (!(a.eps >= 0.f) || !std::isfinite(a.eps)) return H3_ERR_INVALID_ARG;
  if (!aligned16(a.qkv) || !aligned4(a.pos) || !optional16(a.wq) || !optional16(a.wk) ||
      !aligned16(a.out))
    return H3_ERR_INVALID_ARG;
  return H3_OK;
}

size_t qkv_bytes(int32_t L, int32_t H) { return size_t(L) * H * 128 * 3 * 2; }

QkNormArgs norm_args(const uint16_t* qkv, const int32_t* pos, const float* wq, const float* wk,
                     int32_t L, int32_t n_heads, const int32_t* sec, float base, float eps,
                     uint16_t* out) {
  QkNormArgs a{};
  a.qkv = qkv;
  a.pos = pos;
  a.wq = wq;
  a.wk = wk;
  a.L = L;
  a.H = n_heads;
  if (sec != nullptr)
    for (int i = 0; i < 3; ++i) a.sec[i] = sec[i];
  a.base = base;
  a.eps = eps;
  a.out = out;
  return a;
}

h3_status attention_bwd(AttnBwdArgs a, int32_t head_dim, void* workspace, size_t workspace_bytes,
                        h3_stream_t stream) {
  size_t need = 0;
  if (h3_status s = h3_attn_bwd_workspace_size(a.L, a.H, head_dim, &need)) return s;
  if (a.causal != 0 && a.causal != 1) return H3_ERR_INVALID_ARG;
  if (!(a.sm_scale > 0.f) || !std::isfinite(a.sm_scale)) return H3_ERR_INVALID_ARG;
  if (a.n_seg != 0)
    if (h3_status s = check_segments(a.cu_seqlens, a.n_seg, a.L)) return s;
  if (!aligned16(a.qkv) || !aligned16(a.O) || !aligned4(a.lse) || !aligned16(a.dO) ||
      !aligned16(a.dqkv) || !aligned256(workspace))
    return H3_ERR_INVALID_ARG;
  if (workspace_bytes < need) return H3_ERR_WORKSPACE;
  const size_t n = qkv_bytes(a.L, a.H);
  const Span in[4] = {{a.qkv, n}, {a.O, n / 3}, {a.lse, size_t(a.L) * a.H * 4}, {a.dO, n / 3}};
  const Span ws{workspace, need}, out{a.dqkv, n};
  if (!apart(ws, in) || !apart(out, in) || overlap(ws.p, ws.n, out.p, out.n)) return H3_ERR_INVALID_ARG;
  DevCtx ctx;
  if (h3_status s = dev_ctx(&ctx)) return s;
  // a counter, then -lse log2(e) and -D of every head and token
  uint8_t* w = static_cast<uint8_t*>(workspace);
  a.counter = reinterpret_cast<int*>(w);
  a.aux = reinterpret_cast<float*>(w + 256);
  return finish(launched(launch_attention_bwd(a, ctx, reinterpret_cast<cudaStream_t>(stream))), stream);
}

}  // namespace
}  // namespace h3

using namespace h3;

extern "C" {

h3_status h3_qk_norm_mrope(const uint16_t* qkv, const int32_t* pos, const float* wq,
                           const float* wk, int32_t L, int32_t n_heads, int32_t head_dim,
                           const int32_t sec[3], float base, float eps, uint16_t* out,
                           h3_stream_t stream) {
  const Trace trace_("h3_qk_norm_mrope");
  if (sec == nullptr) return H3_ERR_INVALID_ARG;
  const QkNormArgs a = norm_args(qkv, pos, wq, wk, L, n_heads, sec, base, eps, out);
  if (h3_status s = check_norm(a, head_dim)) return s;
  const size_t n = qkv_bytes(L, n_heads);
  const Span in[3] = {{pos, size_t(L) * 12}, {wq, 512}, {wk, 512}};
  if (!apart(Span{out, n}, in) || (out != qkv && overlap(out, n, qkv, n))) return H3_ERR_INVALID_ARG;
  DevCtx ctx;
  if (h3_status s = dev_ctx(&ctx)) return s;
  return finish(launched(launch_qk_norm(a, ctx, reinterpret_cast<cudaStream_t>(stream))), stream);
}

h3_status h3_qk_norm_mrope_bwd_workspace_size(int32_t L, int32_t n_heads, int32_t head_dim,
                                              size_t* bytes) {
  if (bytes == nullptr) return H3_ERR_INVALID_ARG;
  if (h3_status s = check_shape(L, n_heads, head_dim)) return s;
  *bytes = size_t(kQkNormPartials) * 256 * 4;
  return H3_OK;
}

h3_status h3_qk_norm_mrope_bwd(const uint16_t* qkv, const int32_t* pos, const float* wq,
                               const float* wk, const uint16_t* dout, int32_t L, int32_t n_heads,
                               int32_t head_dim, const int32_t sec[3], float base, float eps,
                               void* workspace, size_t workspace_bytes, uint16_t* dqkv, float* dwq,
                               float* dwk, h3_stream_t stream) {
  const Trace trace_("h3_qk_norm_mrope_bwd");
  if (sec == nullptr) return H3_ERR_INVALID_ARG;
  QkNormArgs a = norm_args(qkv, pos, wq, wk, L, n_heads, sec, base, eps, dqkv);
  if (h3_status s = check_norm(a, head_dim)) return s;
  if (!aligned16(dout) || (dwq != nullptr && !aligned4(dwq)) || (dwk != nullptr && !aligned4(dwk)))
    return H3_ERR_INVALID_ARG;
  const bool sums = dwq != nullptr || dwk != nullptr;
  size_t need = 0;
  if (h3_status s = h3_qk_norm_mrope_bwd_workspace_size(L, n_heads, head_dim, &need)) return s;
  if (sums && !aligned256(workspace)) return H3_ERR_INVALID_ARG;
  if (sums && workspace_bytes < need) return H3_ERR_WORKSPACE;
  const size_t n = qkv_bytes(L, n_heads);
  const Span in[5] = {{qkv, n}, {pos, size_t(L) * 12}, {wq, 512}, {wk, 512}, {dout, n}};
  const Span ws{sums ? workspace : nullptr, need}, q{dwq, 512}, k{dwk, 512}, out{dqkv, n};
  if (!apart(ws, in) || !apart(q, in) || !apart(k, in)) return H3_ERR_INVALID_ARG;
  const Span outs[4] = {ws, q, k, out};
  if (!disjoint(outs)) return H3_ERR_INVALID_ARG;
  for (int i = 0; i < 5; ++i)   // dqkv may be dout itself
    if (in[i].p != nullptr && !(i == 4 && dqkv == dout) && overlap(dqkv, n, in[i].p, in[i].n))
      return H3_ERR_INVALID_ARG;
  DevCtx ctx;
  if (h3_status s = dev_ctx(&ctx)) return s;
  a.dout = dout;
  a.dwq = dwq;
  a.dwk = dwk;
  a.partial = static_cast<float*>(workspace);
  return finish(launched(launch_qk_norm_bwd(a, ctx, reinterpret_cast<cudaStream_t>(stream))), stream);
}

h3_status h3_attn_bwd_workspace_size(int32_t L, int32_t n_heads, int32_t head_dim, size_t* bytes) {
  if (bytes == nullptr) return H3_ERR_INVALID_ARG;
  if (h3_status s = check_shape(L, n_heads, head_dim)) return s;
  // tokens and CTAs (four for 256 tokens of a head) are counted in 31 bits
  if (L > (1 << 30) || 4 * ((int64_t(L) + 255) / 256) * n_heads > INT32_MAX) return H3_ERR_INVALID_ARG;
  *bytes = 256 + round256(size_t(n_heads) * size_t(attn_bwd_padded(L)) * 8);
  return H3_OK;
}

h3_status h3_joint_attn_bwd(const uint16_t* qkv, const uint16_t* O, const float* lse,
                            const uint16_t* dO, int32_t L, int32_t n_heads, int32_t head_dim,
                            int32_t causal, float sm_scale, void* workspace,
                            size_t workspace_bytes, uint16_t* dqkv, h3_stream_t stream) {
  const Trace trace_("h3_joint_attn_bwd");
  const AttnBwdArgs a{qkv, O, lse, dO, L, n_heads, causal, sm_scale, 0, nullptr, nullptr, nullptr,
                      dqkv};
  return attention_bwd(a, head_dim, workspace, workspace_bytes, stream);
}

h3_status h3_joint_attn_varlen_bwd(const uint16_t* qkv, const uint16_t* O, const float* lse,
                                   const uint16_t* dO, const int32_t* cu_seqlens, int32_t n_seg,
                                   int32_t L, int32_t n_heads, int32_t head_dim, int32_t causal,
                                   float sm_scale, void* workspace, size_t workspace_bytes,
                                   uint16_t* dqkv, h3_stream_t stream) {
  const Trace trace_("h3_joint_attn_varlen_bwd");
  if (n_seg < 1) return H3_ERR_INVALID_ARG;
  const AttnBwdArgs a{qkv, O, lse, dO, L, n_heads, causal, sm_scale, n_seg, cu_seqlens,
                      nullptr, nullptr, dqkv};
  return attention_bwd(a, head_dim, workspace, workspace_bytes, stream);
}

}  // extern "C"
