/*
 * h3attn — the attention sub-block's norm of queries and keys, and the gradients that train
 * it: a third header beside h3attn.h, whose conventions hold here too.
 *
 *   qkv  = y Wqkv^T                                         h3_qkv_proj
 *   Q,K <- norm of each head, then the 3D rotary embedding  h3_qk_norm_mrope
 *   O    = softmax(s Q K^T) V, with its log-sum-exp         h3_joint_attn_fwd, _varlen_fwd
 *   dQ, dK, dV from dO                                      h3_joint_attn_bwd, _varlen_bwd
 *   gradients back through the norm and the rotation        h3_qk_norm_mrope_bwd
 *
 * h3_attn_block_fwd keeps none of qkv, O and lse for the caller: a training step takes the
 * block apart into its single calls, as above.  Without the norm the rotation is
 * h3_mrope_apply, and its gradient (in place, the V block not touched) the same call on
 * dqkv with every position negated.
 *
 * Every gradient is a sum in a fixed order: the same call gives the same bits (on the same
 * model of GPU; the same sums in place, or over other tokens or heads, may be split in another
 * way).  Nothing is added to what an output held before.  No call keeps anything of its
 * arrays for another (a host thread keeps the rotation's last 64 frequencies, a function of sec
 * and base alone); what the forward pass saves for the backward pass is qkv before the norm,
 * qkv after it, O and lse, all the caller's.
 *
 * Calls may start before the work ahead of them in the stream is done, but touch no memory
 * before.  Workspaces are read only after they are written; calls that may overlap (on two
 * streams, or in two graphs replayed together) need one each.
 */
#ifndef H3ATTN_TRAIN_H_
#define H3ATTN_TRAIN_H_

#include "h3attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * RMS norm of each head's queries and keys, and the rotary embedding of h3_mrope_apply, in
 * one pass:
 *   x[n, h] -> R(pos[n]) (x[n, h] / sqrt(mean x[n, h]^2 + eps) * w),   w = wq for Q, wk for K
 * with the mean over the head's 128 values.  fp32 arithmetic, one rounding to bf16; angles
 * are right to fp32 for every position (h3_mrope_apply rounds position x frequency to fp32
 * first, so far positions differ there by up to |angle| 2^-24).
 *   qkv [L][3*H*128] bf16, columns [Q | K | V]; pos [L][3] int32 (4-byte aligned);
 *   wq, wk [128] fp32, each shared by all heads, or NULL for ones; eps >= 0;
 *   sec, base as in h3_mrope_apply.
 *   out [L][3*H*128] bf16: qkv itself (V is not touched), or an array apart from it (V is
 *   copied).
 * A head of zeros gives zeros; heads whose squares leave fp32's range are normalised all the
 * same; an infinity or a NaN gives the formula's zeros and NaN in its own head.
 */
h3_status h3_qk_norm_mrope(const uint16_t* qkv, const int32_t* pos, const float* wq,
                           const float* wk, int32_t L, int32_t n_heads, int32_t head_dim,
                           const int32_t sec[3], float base, float eps, uint16_t* out,
                           h3_stream_t stream);

/*
 * The gradient of h3_qk_norm_mrope.  With r = 1 / sqrt(mean x^2 + eps), g = R(pos)^T dout:
 *   dw  = sum over tokens and heads of g x r         (separately for Q and K)
 *   dx  = r (g w - x r^2 mean(x g w))
 *   qkv: what the forward call read (its input, before the norm).
 *   dout [L][3*H*128] bf16: the gradient of its output.
 *   dqkv [L][3*H*128] bf16: dout itself (the V block is not touched), or an array apart from
 *   it (the V block is copied); never qkv.  A head of zeros with eps = 0 gets zeros.
 *   dwq, dwk [128] fp32, 4-byte aligned, each or both NULL if not wanted.  With both NULL the
 *   workspace is not used and may be NULL.
 *   workspace >= h3_qk_norm_mrope_bwd_workspace_size() bytes, 256-byte aligned.
 */
h3_status h3_qk_norm_mrope_bwd_workspace_size(int32_t L, int32_t n_heads, int32_t head_dim,
                                              size_t* bytes);
h3_status h3_qk_norm_mrope_bwd(const uint16_t* qkv, const int32_t* pos, const float* wq,
                               const float* wk, const uint16_t* dout, int32_t L, int32_t n_heads,
                               int32_t head_dim, const int32_t sec[3], float base, float eps,
                               void* workspace, size_t workspace_bytes, uint16_t* dqkv, float* dwq,
                               float* dwk, h3_stream_t stream);

/*
 * The gradient of h3_joint_attn_fwd (and, with segments, of h3_joint_attn_varlen_fwd) by
 * recomputing the probabilities.  Per head, at the visible pairs (i, j), with s = sm_scale:
 *   P_ij = exp(s q_i . k_j - lse_i)       dV_j = sum_i P_ij dO_i
 *   dS_ij = P_ij (dO_i . v_j - dO_i . O_i)
 *   dQ_i = s sum_j dS_ij k_j              dK_j = s sum_i dS_ij q_i
 * bf16 tensor-core products with P and dS rounded to bf16, all sums in fp32, each gradient
 * rounded once.
 *   qkv, causal, sm_scale, cu_seqlens, n_seg: as the forward call had them; O, lse: what it
 *   wrote (lse [n_heads][L] fp32); dO [L][n_heads*128] bf16: the gradient of O.
 *   dqkv [L][3*n_heads*128] bf16, columns [dQ | dK | dV] as in qkv; apart from every input.
 *   L at most 2^30, and ceil(L / 256) n_heads below 2^29.
 *   workspace >= h3_attn_bwd_workspace_size() bytes, 256-byte aligned, apart from the rest.
 * An infinity or a NaN in an input, at a token t, may reach the gradients of its head in the
 * blocks of 256 tokens (from token 0 on) that hold a token of t's segment, tokens of other
 * segments in such a block included, and reaches nothing else.  A segment whose values may be
 * anything, as padding's, therefore begins on a multiple of 256.
 */
h3_status h3_attn_bwd_workspace_size(int32_t L, int32_t n_heads, int32_t head_dim, size_t* bytes);
h3_status h3_joint_attn_bwd(const uint16_t* qkv, const uint16_t* O, const float* lse,
                            const uint16_t* dO, int32_t L, int32_t n_heads, int32_t head_dim,
                            int32_t causal, float sm_scale, void* workspace,
                            size_t workspace_bytes, uint16_t* dqkv, h3_stream_t stream);
h3_status h3_joint_attn_varlen_bwd(const uint16_t* qkv, const uint16_t* O, const float* lse,
                                   const uint16_t* dO, const int32_t* cu_seqlens, int32_t n_seg,
                                   int32_t L, int32_t n_heads, int32_t head_dim, int32_t causal,
                                   float sm_scale, void* workspace, size_t workspace_bytes,
                                   uint16_t* dqkv, h3_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* H3ATTN_TRAIN_H_ */
