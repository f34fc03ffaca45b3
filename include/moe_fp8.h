/*
 * moe_fp8.h -- C ABI of the block-scaled FP8 (E4M3) operators: activation
 * quantisation, the dense product, and the grouped expert FFN.  They stand beside
 * the MXFP4 layer of moe_mxfp4.h, share its status codes and conventions (device
 * pointers, stream, host checks, no allocation, no state, deterministic results)
 * and take the same routing outputs; moe_combine sums their expert rows.
 *
 * Format.  Elements are OCP E4M3 (4 exponent bits of bias 7, 3 mantissa bits,
 * largest value 448, 0x7F and 0xFF NaN).  A row of K elements is cut into
 * ceil(K / 128) runs of 128 (the last may be shorter).
 *   activations  e4m3 [rows][K], scales fp32 [rows][ceil(K/128)]: one per run
 *   weights      e4m3 [N][K], scales fp32 [ceil(N/128)][ceil(K/128)]: one per
 *                block of 128 rows and one run
 * A value is element * scale.  Scales may be any finite fp32 whose products are finite: a
 * product of matrices multiplies each run's sum by x_scale * w_scale, rounded to fp32 first, so
 * one that overflows gives an infinity (NaN beside a sum of 0), and one below 2^-126 keeps its
 * bits down to 2^-149 only.  Scales that moe_quantize_fp8 makes are between 2^-109 and 2^120.
 */
#ifndef MOE_FP8_H
#define MOE_FP8_H

#include "moe_mxfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * moe_quantize_fp8 -- bf16 rows to E4M3 elements with one scale per run of 128.
 *
 * Per row and run, with a = max(max_i |x_i|, 2^-100):
 *   scale = a / 448 rounded to fp32,  q_i = 448 x_i / a rounded once to E4M3
 * (nearest, ties to even).  A run that holds an infinity or a NaN gets a NaN scale
 * and NaN elements (0x7F); a run of zeros gets zeros.
 *
 *   x      bf16 [rows][K]              16-byte aligned
 *   q      e4m3 [rows][K]              out; 16-byte aligned
 *   scale  fp32 [rows][ceil(K/128)]    out
 * K is a positive multiple of 16, at most 65536.  rows = 0 enqueues nothing.
 */
moe_status moe_quantize_fp8(const uint16_t* x, int64_t rows, int32_t K, uint8_t* q, float* scale,
                            void* stream);

/*
 * moe_gemm_fp8 -- the dense product y = X W^T of block-scaled FP8 matrices.
 *
 *   y[m][n] = sum_b x_scale[m][b] * w_scale[n/128][b] * sum_{i in run b} xq[m][i] * w[n][i]
 * Sums are fp32; y is rounded once to its type.  A bf16 result is made by the FP8 matrix
 * instruction, which aligns each 16 products to the largest of them and keeps 13 bits under
 * it: within 2^-9 of the sum of the terms' magnitudes, about 1.4e-5 of y on normal data.  An
 * fp32 result is made with fp32 products throughout, at about half the rate.
 *
 *   xq       e4m3 [M][K]                         16-byte aligned
 *   x_scale  fp32 [M][ceil(K/128)]
 *   w        e4m3 [N][K]                         16-byte aligned
 *   w_scale  fp32 [ceil(N/128)][ceil(K/128)]
 *   y        bf16 or fp32 [M][N], by y_type      out; 16-byte aligned
 *   ws       workspace of moe_gemm_fp8_workspace_bytes(M, N, K) bytes, 16-byte aligned.  That
 *            is 0 at every size: no tile of the product uses any, and NULL with 0 bytes will do
 * K is a positive multiple of 16, at most 65536; N >= 1, at most 2^24; M * N at most
 * 2^38.  M = 0 enqueues nothing.
 */
moe_status moe_gemm_fp8(const uint8_t* xq, const float* x_scale, int64_t M, int32_t N, int32_t K,
                        const uint8_t* w, const float* w_scale, int32_t y_type, void* y, void* ws,
                        size_t ws_bytes, void* stream);

/* Workspace bytes of moe_gemm_fp8: 0. */
size_t moe_gemm_fp8_workspace_bytes(int64_t M, int32_t N, int32_t K);

/*
 * moe_grouped_ffn_fp8 -- every expert's FFN on its rows, in expert-major order, over
 * block-scaled FP8 weights: moe_grouped_ffn_mxfp4's contract in the format above.
 *
 * For expert e and each row p in [offsets[e], offsets[e+1]), token t = gather[p] / k:
 *   x[t] is quantised as by moe_quantize_fp8;
 *   g = x[t] . W1[e][i],  u = x[t] . W1[e][I+i]           (moe_gemm_fp8's product: as for fp32
 *                          up to 90 rows per expert on average, above that as for bf16)
 *   h[i] = SiLU(min(g, limit)) * clamp(u, -limit, limit)  (fp32)
 *   h is quantised from fp32 by moe_quantize_fp8's rule, the quotient 448 h / a being within
 *   2^-22 of itself before it is rounded to E4M3;
 *   y_sorted[p][n] = h . W2[e][n] (as for bf16), rounded once to bf16.
 * A limit <= 0 or not finite disables the clamp.
 *
 *   x         bf16  [T][H]                   16-byte aligned
 *   w1        e4m3  [E][2I][H]               rows 0..I-1 gate, I..2I-1 up; 16-byte aligned
 *   w1_scale  fp32  [E][2I/128][H/128]
 *   w2        e4m3  [E][H][I]                16-byte aligned
 *   w2_scale  fp32  [E][H/128][I/128]
 *   counts, offsets, gather                  as written by moe_expert_offsets
 *   y_sorted  bf16  [T*k][H]                 out; 16-byte aligned
 *   ws        workspace of at least moe_fp8_workspace_bytes(T, E, k, H, I) bytes,
 *             16-byte aligned; contents on entry are ignored.
 * H and I are multiples of 128, at most 65536, with H * I at most 2^31 - 2^20 (32-bit
 * offsets within an expert's W1); activations fit as for moe_grouped_ffn_mxfp4.  T = 0 enqueues
 * nothing.  Rows of y_sorted behind the last expert's rows are left as they were.
 */
moe_status moe_grouped_ffn_fp8(const uint16_t* x, int64_t T, int32_t H, int32_t I, int32_t E,
                               int32_t k, const uint8_t* w1, const float* w1_scale,
                               const uint8_t* w2, const float* w2_scale, const int32_t* counts,
                               const int32_t* offsets, const int32_t* gather, float swiglu_limit,
                               uint16_t* y_sorted, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes of moe_grouped_ffn_fp8, also enough for moe_expert_offsets and the
 * routing calls at these sizes.  It does not shrink as T grows, so a workspace for the largest
 * batch serves the smaller ones.  0 for invalid sizes. */
size_t moe_fp8_workspace_bytes(int64_t T, int32_t E, int32_t k, int32_t H, int32_t I);

#ifdef __cplusplus
}
#endif

#endif /* MOE_FP8_H */
