/*
 * moe_block.h -- C ABI of the operators around the routed layer in a model's block: the RMS norm
 * that makes its inputs (with the residual's addition, in bf16 and in block-scaled FP8) and its
 * gradient, the loss that balances the router's load and its gradient, and the low-rank adapters of
 * many requests beside a shared projection.  They share the status codes and conventions of
 * moe_mxfp4.h (device pointers, stream, host checks before anything is enqueued, no allocation, no
 * state, deterministic results) and the FP8 format of moe_fp8.h.
 *
 * Strides count elements from one row to the next.
 */
#ifndef MOE_BLOCK_H
#define MOE_BLOCK_H

#include "moe_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * moe_rms_norm -- addition of the residual stream, RMS norm, and the layer's inputs.
 *
 * Per row:
 *   s_i = bf16(x_i + residual_i)   (residual NULL: s = x)
 *   y_i = s_i * w_i / sqrt(mean_j s_j^2 + eps)
 * with statistics and products in fp32, at any magnitude of bf16 rows and with elements of any other
 * magnitude beside them; only a product s_i w_i under 2^-126 keeps fewer digits than y may have.  y is
 * infinite where it is itself past its type, not where s_i w_i is.  y is rounded once to bf16;
 * q and scale are moe_quantize_fp8's format and rule on the fp32 values of y, not on their bf16
 * rounding: per run of 128 and with a = max(max_i |y_i|, 2^-100), scale = a / 448 and q_i =
 * E4M3(448 y_i / a).  A run of y that holds an infinity or a NaN gets a NaN scale and NaN elements.
 * A row whose mean square and eps are both 0 gives NaN.
 *
 *   x         bf16 [rows][H], x_stride between rows   16-byte aligned
 *   residual  bf16 [rows][H] or NULL                  16-byte aligned
 *   weight    fp32 or bf16 [H], by weight_type        16-byte aligned
 *   sum       bf16 [rows][H] or NULL                  out; s, only with a residual; 16-byte aligned
 *   y         bf16 [rows][H] or NULL                  out; 16-byte aligned
 *   q         e4m3 [rows][H] or NULL                  out; 16-byte aligned
 *   scale     fp32 [rows][ceil(H/128)]                out; with q, NULL without
 * y or q is given, or both.  H is a positive multiple of 8 (with q, of 16), at most 65536; x_stride
 * is a multiple of 8 and at least H; eps is finite and not negative.  sum and y may each be the
 * buffer of residual, or that of x if x_stride is H.  rows = 0 enqueues nothing.
 */
moe_status moe_rms_norm(const uint16_t* x, int64_t x_stride, const uint16_t* residual, int64_t rows,
                        int32_t H, int32_t weight_type, const void* weight, float eps,
                        uint16_t* sum, uint16_t* y, uint8_t* q, float* scale, void* stream);

/*
 * moe_rms_norm_grad -- the gradient of y by s and by the weight.
 *
 * Per row, with r = 1 / sqrt(mean_j s_j^2 + eps), u = s r and z = dy w:
 *   dx_i = r (z_i - u_i mean_j(z_j u_j)) + dsum_i      (dsum NULL: without it)
 *   dweight_i = sum over rows of dy_i u_i
 * in fp32, at any magnitude of bf16 rows as for moe_rms_norm (where r itself is past fp32's range, too);
 * dx is rounded once.  s is moe_rms_norm's sum, or its x where there was no residual; dx is
 * then the gradient of x and of residual alike (roundings count as the identity).  dsum is
 * the gradient that reaches sum beside the norm.  The rows' order of summation in dweight depends on
 * the sizes alone.
 *
 *   s         bf16 [rows][H], s_stride between rows   16-byte aligned
 *   weight    fp32 or bf16 [H], by weight_type        16-byte aligned
 *   dy        bf16 [rows][H]                          16-byte aligned
 *   dsum      bf16 [rows][H] or NULL                  16-byte aligned
 *   dx        bf16 [rows][H] or NULL                  out; 16-byte aligned; may be dy's or dsum's buffer
 *   dweight   fp32 [H] or NULL                        out; 16-byte aligned
 *   ws        moe_rms_norm_grad_workspace_bytes(rows, H) bytes, 16-byte aligned; NULL with 0 bytes
 *             will do without dweight.  Contents on entry are ignored
 * dx or dweight is given, or both (dsum needs dx).  H, s_stride and eps as for moe_rms_norm.  rows = 0
 * writes zeros to dweight.  A row whose mean square and eps are both 0 gives NaN.
 */
moe_status moe_rms_norm_grad(const uint16_t* s, int64_t s_stride, int64_t rows, int32_t H,
                             int32_t weight_type, const void* weight, float eps,
                             const uint16_t* dy, const uint16_t* dsum, uint16_t* dx, float* dweight,
                             void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes of moe_rms_norm_grad.  It does not shrink as rows grow.  0 for invalid sizes. */
size_t moe_rms_norm_grad_workspace_bytes(int64_t rows, int32_t H);

/*
 * moe_balance_loss -- the loss that balances the router's load over packed sequences, the experts'
 * counts, and in the same pass the loss's gradient.
 *
 * For a sequence of tokens t in [seq_offsets[s], seq_offsets[s+1]), n of them, and with
 *   p_te = softmax(l_t)_e                                        (MOE_SCORE_SOFTMAX)
 *   p_te = sigmoid(l_te) / sum_i sigmoid(l_ti)                   (MOE_SCORE_SIGMOID)
 *   counts[s][e] = (token, slot) pairs of the sequence whose topk_ids is e
 * it is
 *   loss[s] = sum_e (E / (k n) counts[s][e]) (1/n sum_t p_te)
 * which is 1 where the load is even; 0 if n = 0.  With dlogits, and counts taken as constants:
 *   dlogits_te = dloss[s] E / (k n^2) p_te (c_e - sum_i p_ti c_i) [sigmoid: times 1 - sigmoid(l_te)]
 *                + add_to_te                                     (add_to NULL: without it)
 * c being counts[s].  Rows of no sequence are padding: they count nowhere, and their gradient is 0 +
 * add_to.  A logit of -inf or NaN excludes its expert, as for moe_route_scored: p 0, gradient 0;
 * a token whose experts are all excluded has p = 0.  A logit of +inf has score 1 (softmax: the
 * +inf logits share 1 equally).  Sigmoid scores are divided at any magnitude (logits of -1000 too).
 * Ids outside 0 .. E-1 are counted nowhere.  p and the gradient are fp32, sums over tokens fp64; each
 * output is rounded once.
 *
 *   logits       fp32 or bf16 [T][E], by logits_type; aligned to its elements
 *   topk_ids     int32 [T][k]
 *   seq_offsets  int32 [n_seqs+1], not decreasing, from 0 or more to T or less; NULL: one
 *                sequence of all T tokens (n_seqs = 1)
 *   loss         fp32  [n_seqs]      out
 *   counts       int32 [n_seqs][E]   out
 *   dloss        fp32  [n_seqs]      the gradient that reaches loss; with dlogits
 *   add_to       [T][E] of the logits' type, or NULL
 *   dlogits      [T][E] of the logits' type, or NULL    out; may be add_to's or logits' buffer
 *   ws           moe_balance_loss_workspace_bytes(T, E, n_seqs) bytes, 16-byte aligned; contents on
 *                entry are ignored
 * E <= 1024, k <= 8 and k <= E, n_seqs <= 2^20.  T = 0 writes zeros to loss and counts.
 */
moe_status moe_balance_loss(const void* logits, int32_t logits_type, int64_t T, int32_t E, int32_t k,
                            int32_t score, const int32_t* topk_ids, const int32_t* seq_offsets,
                            int32_t n_seqs, float* loss, int32_t* counts, const float* dloss,
                            const void* add_to, void* dlogits, void* ws, size_t ws_bytes,
                            void* stream);

/* Workspace bytes of moe_balance_loss.  It does not shrink as T grows.  0 for invalid sizes. */
size_t moe_balance_loss_workspace_bytes(int64_t T, int32_t E, int32_t n_seqs);

/*
 * moe_balance_loss_grad -- moe_balance_loss's dlogits alone, from its counts: for a backward pass
 * apart from the forward pass.  Exactly the bits that moe_balance_loss writes.  T = 0 enqueues nothing.
 */
moe_status moe_balance_loss_grad(const void* logits, int32_t logits_type, int64_t T, int32_t E,
                                 int32_t k, int32_t score, const int32_t* seq_offsets,
                                 int32_t n_seqs, const int32_t* counts, const float* dloss,
                                 const void* add_to, void* dlogits, void* stream);

/*
 * moe_lora_group -- the rows of a batch in their adapters' order.
 *
 *   adapter  int32 [M]      each row's adapter; outside 0 .. L-1 (say -1): none
 *   offsets  int32 [L+1]    out; adapter a's rows are rows[offsets[a]] .. rows[offsets[a+1] - 1]
 *   rows     int32 [M]      out; row indices, ascending within an adapter; the rows without an
 *                           adapter, ascending, are behind offsets[L]
 * 1 <= L <= 1024; no two of the three overlap.  M = 0 writes zeros to offsets.  One call serves
 * every moe_lora_add of the batch.
 */
moe_status moe_lora_group(const int32_t* adapter, int64_t M, int32_t L, int32_t* offsets,
                          int32_t* rows, void* stream);

/*
 * moe_lora_add -- low-rank adapters of many requests beside one shared projection.
 *
 * For each row m of adapter a:
 *   y[m][n] = base[m][n] + scaling[a] * sum_r (sum_i x[m][i] A[a][r][i]) B[a][n][r]
 * and y[m] = base[m] for a row without an adapter (base NULL: 0 in its place).  base is the shared
 * projection's result, moe_gemm_fp8's y for one.  Inner sums are fp32 of exact products; they enter
 * the second product whole for an fp32 y, within 2^-17 of themselves for a bf16 one; y is rounded
 * once.  An infinite weight makes an infinity or a NaN as the formula does, of no other row.
 *
 *   x        bf16 [M][K], x_stride between rows    16-byte aligned
 *   a        bf16 [L][R][K]                        16-byte aligned
 *   b        bf16 [L][N][R]                        16-byte aligned
 *   scaling  fp32 [L], or NULL for 1
 *   offsets, rows    as written by moe_lora_group for these M rows and L adapters
 *   base     bf16 or fp32 [M][N], by y_type, base_stride between rows, or NULL; 16-byte aligned
 *   y        bf16 or fp32 [M][N], by y_type, y_stride between rows   out; 16-byte aligned; may be
 *            base's buffer if the strides agree (rows without an adapter are then not touched), and
 *            overlaps nothing else
 *   ws       moe_lora_add_workspace_bytes(M, N, K, R, L) bytes, 16-byte aligned; contents on entry
 *            are ignored
 * K is a positive multiple of 8, at most 65536; R a positive multiple of 8, at most 256 (an adapter of
 * a smaller rank has zeros in the rows of A that it lacks); 1 <= N <= 2^24; 1 <= L <= 1024.
 * x_stride is a multiple of 8 and at least K; base_stride and y_stride are at least N.  M = 0 enqueues
 * nothing.
 */
moe_status moe_lora_add(const uint16_t* x, int64_t x_stride, int64_t M, int32_t K, int32_t N,
                        int32_t R, int32_t L, const uint16_t* a, const uint16_t* b,
                        const float* scaling, const int32_t* offsets, const int32_t* rows,
                        int32_t y_type, const void* base, int64_t base_stride, void* y,
                        int64_t y_stride, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes of moe_lora_add.  It does not shrink as M grows.  0 for invalid sizes. */
size_t moe_lora_add_workspace_bytes(int64_t M, int32_t N, int32_t K, int32_t R, int32_t L);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_H */
