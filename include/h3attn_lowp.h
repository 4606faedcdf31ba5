/*
 * h3attn_lowp — 4-bit projections and the norms that feed quantised projections.
 *
 * Next to the E4M3 projections of h3attn.h (h3_quantize_rows_fp8, h3_gemm_fp8,
 * h3_mlp_block_fwd_fp8), part of the same library and under the same conventions
 * (row-major matrices, bf16 as uint16_t, 16-byte aligned device pointers, work on
 * the caller's stream and the current device, argument errors found on the host
 * before anything is launched, kernel errors through h3_sync_status()):
 *
 *   microscaled 4-bit rows and back      h3_quantize_rows_fp4, h3_dequantize_rows_fp4
 *   4-bit product                        h3_gemm_fp4
 *   RMS norm of x + res, output in E4M3  h3_rms_norm_fp8   (for h3_gemm_fp8)
 *   the same with 4-bit output           h3_rms_norm_fp4   (for h3_gemm_fp4)
 *   MLP sub-block on 4-bit products      h3_mlp_block_fwd_fp4
 *
 * Forward only, like the rest of the library.  No call allocates device memory.
 *
 * A 4-bit matrix [R][K] (K % 128 == 0, 128 <= K <= 65536) is three arrays:
 *   q  [R][K/2] bytes: E2M1 codes (sign, then 0 .5 1 1.5 2 3 4 6), column 2j in
 *      the low half of byte j, column 2j + 1 in the high half.
 *   bs h3_fp4_scale_bytes(fmt, R, K) bytes: the scale of every block of columns.
 *      H3_FP4_MX: blocks of 32, E8M0 (2^(byte - 127); 255 is NaN).
 *      H3_FP4_NV: blocks of 16, E4M3 (unsigned; 0x7F is NaN).
 *      Layout: tiles of 128 rows x 4 blocks, 512 bytes each, the tiles of one
 *      128-row group consecutive along K; with S = K / block, block b of row r is
 *      byte  ((r / 128) * (S / 4) + b / 4) * 512 + (r % 32) * 16
 *            + (r % 128 / 32) * 4 + b % 4,
 *      the order in which the tensor cores take scales.  Rows are counted up to
 *      the next multiple of 128; the bytes of rows >= R are neither written nor
 *      do they reach any result.
 *   s  [R] fp32: one more factor for each row, or NULL for ones.
 * and stands for  E2M1(q[r][k]) * scale(bs, r, k / block) * s[r].
 */
#ifndef H3ATTN_LOWP_H_
#define H3ATTN_LOWP_H_

#include "h3attn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define H3_FP4_MX 1 /* one E8M0 scale for 32 columns */
#define H3_FP4_NV 2 /* one E4M3 scale for 16 columns, and one factor for each row */

/* Bytes of the block-scale array of a 4-bit matrix [R][K], R >= 1. */
h3_status h3_fp4_scale_bytes(int32_t fmt, int32_t R, int32_t K, size_t* bytes);

/*
 * Row-wise 4-bit quantisation of x [R][K] bf16.  With a = max |x| over a block:
 *   MX: scale 2^k, k the smallest integer with a <= 6 * 2^k (at least -127), so
 *       nothing is clipped; s is not used and may be NULL.
 *   NV: s[r] = 2^e, e the smallest integer >= -117 with max |x[r]| <= 2688 * 2^e
 *       (448 * 6: the largest scale times the largest code; 1 for an all-zero
 *       row); scale = E4M3(a / (6 * s[r])), to nearest, ties to even.
 * q = E2M1(x / (scale * s[r])), to nearest, ties to the even code, 6 at most.  A
 * power of two for the row keeps every step but the two roundings exact, so the
 * codes are those of real arithmetic.  A block that holds an infinity or a NaN
 * gets a NaN scale (and counts as zero in the row's maximum): it stands for NaN.
 * No array may overlap another.
 */
h3_status h3_quantize_rows_fp4(const uint16_t* x, int32_t fmt, int32_t R, int32_t K, uint8_t* q,
                               uint8_t* bs, float* s, h3_stream_t stream);

/* y [R][K] bf16 = what a 4-bit matrix stands for (s NULL: ones), rounded to bf16:
 * exact for the output of h3_quantize_rows_fp4 inside bf16's normal range (a value that
 * was rounded up past its largest becomes infinite).  y may not overlap q, bs or s. */
h3_status h3_dequantize_rows_fp4(const uint8_t* q, const uint8_t* bs, const float* s, int32_t fmt,
                                 int32_t R, int32_t K, uint16_t* y, h3_stream_t stream);

/*
 * C[m][n] = sum_k A[m][k] B[n][k] over two 4-bit matrices of one format, A [M][K]
 * (activations) and B [N][K] (a weight in nn.Linear layout) -> C [M][N] bf16.  The sum
 * of codes times block scales is held in fp32 (one below 2^-126 may lose bits); its
 * product with the factors is right wherever it is in range, whatever a_s[m] b_s[n]
 * alone would be.  a_s [M] and b_s [N] fp32 row factors, each 16-byte aligned or NULL
 * for ones.  N % 128 == 0; C may not overlap any input.
 */
h3_status h3_gemm_fp4(const uint8_t* A, const uint8_t* a_bs, const float* a_s, const uint8_t* B,
                      const uint8_t* b_bs, const float* b_s, int32_t fmt, int32_t M, int32_t N,
                      int32_t K, uint16_t* C, h3_stream_t stream);

/*
 * RMS norm with the residual's addition and an E4M3 output (the row format of
 * h3_quantize_rows_fp8, for h3_gemm_fp8):
 *   sum[n] = bf16(x[n] + res[n])
 *   y[n]   = sum[n] * weight / sqrt(mean_k sum[n][k]^2 + eps)       (fp32)
 *   scale[n] = max |y[n]| / 448, at least 2^-126 (1 for an all-zero row),
 *   q[n] = E4M3(y[n] / scale[n])
 *   x [L][d] bf16, weight [d] fp32 -> q [L][d] bytes, scale [L] fp32.
 *   res [L][d] bf16 or NULL (then sum[n] = x[n]); sum [L][d] bf16 or NULL (then it
 *   is not written).  sum may be res or x (each part of a row is read before it
 *   is written); otherwise no output may overlap an input or another output.
 * The norm is of the sum as it is stored, so a later norm of `sum` sees the same
 * values.  It is right for finite rows of any size, also where their squares leave
 * fp32 or eps is 0; a row of zeros gives zeros.
 * d % 128 == 0, 128 <= d <= 16384, eps >= 0.
 */
h3_status h3_rms_norm_fp8(const uint16_t* x, const uint16_t* res, const float* weight, int32_t L,
                          int32_t d, float eps, uint16_t* sum, uint8_t* q, float* scale,
                          h3_stream_t stream);

/* The same with y quantised to 4 bits as by h3_quantize_rows_fp4, taking its
 * decisions on the fp32 y: q [L][d/2], bs h3_fp4_scale_bytes(fmt, L, d) bytes, s [L]
 * (MX: not used, may be NULL). */
h3_status h3_rms_norm_fp4(const uint16_t* x, const uint16_t* res, const float* weight, int32_t L,
                          int32_t d, float eps, int32_t fmt, uint16_t* sum, uint8_t* q,
                          uint8_t* bs, float* s, h3_stream_t stream);

/*
 * h3_mlp_block_fwd with both feed-forward products in 4 bits (y and h quantised per
 * token; W1 [hidden][d] and W2 [d][hidden] as 4-bit matrices with row factors W1_s
 * [hidden], W2_s [d], 16-byte aligned or NULL).  workspace >=
 * h3_mlp_workspace_size_fp4(desc, fmt) bytes, 256-byte aligned; out may be x.
 */
h3_status h3_mlp_workspace_size_fp4(const h3_mlp_desc* desc, int32_t fmt, size_t* bytes);
h3_status h3_mlp_block_fwd_fp4(const h3_mlp_desc* desc, int32_t fmt, const uint16_t* x,
                               const uint8_t* mod, const float* shift, const float* scale,
                               const float* gate, const uint8_t* W1_q, const uint8_t* W1_bs,
                               const float* W1_s, const uint8_t* W2_q, const uint8_t* W2_bs,
                               const float* W2_s, void* workspace, size_t workspace_bytes,
                               uint16_t* out, h3_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* H3ATTN_LOWP_H_ */
