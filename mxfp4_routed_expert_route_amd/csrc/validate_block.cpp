// Host-side checks and workspace sizes of the operators around the routed layer (no HIP calls).
#include "validate_block.h"

#include <climits>

#include "block_plan.h"

namespace moe {
namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// Whether m and n 4-byte elements share any.
bool overlap(const void* a, int64_t m, const void* b, int64_t n) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
  return p < q ? q - p < static_cast<uintptr_t>(m) * 4 : p - q < static_cast<uintptr_t>(n) * 4;
}

moe_status check_rows(int64_t rows, int32_t H, int32_t multiple) {
  if (rows < 0 || H < 1) return MOE_ERR_INVALID_ARGUMENT;
  if (H % multiple != 0 || H > kMaxDim || rows > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// A row stride that keeps rows on 16 bytes of 2-byte elements, and offsets within 2^62.
moe_status check_stride(int64_t stride, int64_t least, int64_t multiple) {
  if (stride < least) return MOE_ERR_INVALID_ARGUMENT;
  if (stride % multiple != 0 || stride > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool is_type(int32_t t) { return t == MOE_F32 || t == MOE_BF16; }
bool is_eps(float eps) { return eps >= 0.f && eps <= 3.402823466e38f; }   // false for NaN

moe_status check_routing(int32_t logits_type, int64_t T, int32_t E, int32_t k, int32_t score,
                         const void* seq_offsets, int32_t n_seqs) {
  if (T < 0 || E < 1 || k < 1 || k > E || n_seqs < 1) return MOE_ERR_INVALID_ARGUMENT;
  if (!is_type(logits_type)) return MOE_ERR_INVALID_ARGUMENT;
  if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARGUMENT;
  if (seq_offsets == nullptr && n_seqs != 1) return MOE_ERR_INVALID_ARGUMENT;
  if (E > kMaxE || k > kMaxK || T > INT32_MAX / k || n_seqs > kMaxSequences) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

moe_status check_rms_norm(const void* x, int64_t x_stride, const void* residual, int64_t rows, int32_t H,
                          int32_t weight_type, const void* weight, float eps, const void* sum,
                          const void* y, const void* q, const void* scale) {
  if (!is_type(weight_type) || !is_eps(eps)) return MOE_ERR_INVALID_ARGUMENT;
  moe_status s = check_rows(rows, H, q ? 16 : 8);
  if (s == MOE_OK) s = check_stride(x_stride, H, 8);
  if (s != MOE_OK || rows == 0) return s;
  if (!x || !weight || (!y && !q) || (!q != !scale) || (sum && !residual)) return MOE_ERR_INVALID_ARGUMENT;
  // an output in x's place: rows of one buffer would overlap the next rows of the other
  if (x_stride != H && (sum == x || y == x)) return MOE_ERR_INVALID_ARGUMENT;
  if (sum && sum == y) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(sum, 16) ||
      !aligned(y, 16) || !aligned(q, 16) || !aligned(scale, 4))
    return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

moe_status norm_grad_workspace(int64_t rows, int32_t H, size_t* bytes) {
  const moe_status s = check_rows(rows, H, 8);
  if (s != MOE_OK) return s;
  *bytes = align_up(static_cast<size_t>(norm_grad_groups(rows, H)) * static_cast<size_t>(H) * sizeof(float), 256);
  return MOE_OK;
}

moe_status check_rms_norm_grad(const void* s, int64_t s_stride, int64_t rows, int32_t H,
                               int32_t weight_type, const void* weight, float eps, const void* dy,
                               const void* dsum, const void* dx, const void* dweight, const void* ws,
                               size_t ws_bytes) {
  if (!is_type(weight_type) || !is_eps(eps)) return MOE_ERR_INVALID_ARGUMENT;
  moe_status st = check_rows(rows, H, 8);
  if (st == MOE_OK) st = check_stride(s_stride, H, 8);
  if (st != MOE_OK) return st;
  if ((!dx && !dweight) || (dsum && !dx)) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(dweight, 16)) return MOE_ERR_MISALIGNED;
  if (rows == 0) return MOE_OK;
  if (!s || !weight || !dy || (dweight && !ws)) return MOE_ERR_INVALID_ARGUMENT;
  if (dx == s) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(s, 16) || !aligned(weight, 16) || !aligned(dy, 16) || !aligned(dsum, 16) ||
      !aligned(dx, 16) || !aligned(ws, 16))
    return MOE_ERR_MISALIGNED;
  size_t need = 0;
  st = norm_grad_workspace(rows, H, &need);
  if (st != MOE_OK) return st;
  if (dweight && ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  return MOE_OK;
}

moe_status balance_workspace(int64_t T, int32_t E, int32_t n_seqs, size_t* bytes) {
  if (T < 0 || E < 1 || n_seqs < 1) return MOE_ERR_INVALID_ARGUMENT;
  if (E > kMaxE || T > INT32_MAX || n_seqs > kMaxSequences) return MOE_ERR_UNSUPPORTED;
  *bytes = align_up(static_cast<size_t>(balance_slots(T, n_seqs)) * sizeof(double), 256) +
           align_up(static_cast<size_t>(balance_count_slots(T)) * static_cast<size_t>(E) * sizeof(int32_t), 256);
  return MOE_OK;
}

moe_status check_balance(const void* logits, int32_t logits_type, int64_t T, int32_t E, int32_t k,
                         int32_t score, const void* ids, const void* seq_offsets, int32_t n_seqs,
                         const void* loss, const void* counts, const void* dloss, const void* add_to,
                         const void* dlogits, const void* ws, size_t ws_bytes) {
  moe_status s = check_routing(logits_type, T, E, k, score, seq_offsets, n_seqs);
  if (s != MOE_OK) return s;
  if (!loss || !counts) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(loss, 4) || !aligned(counts, 4)) return MOE_ERR_MISALIGNED;
  if (T == 0) return MOE_OK;
  if (!logits || !ids || !ws) return MOE_ERR_INVALID_ARGUMENT;
  if (!dlogits != !dloss || (add_to && !dlogits)) return MOE_ERR_INVALID_ARGUMENT;
  const uintptr_t size = logits_type == MOE_BF16 ? 2 : 4;
  if (!aligned(logits, size) || !aligned(ids, 4) || !aligned(seq_offsets, 4) || !aligned(dloss, 4) ||
      !aligned(add_to, size) || !aligned(dlogits, size) || !aligned(ws, 16))
    return MOE_ERR_MISALIGNED;
  size_t need = 0;
  s = balance_workspace(T, E, n_seqs, &need);
  if (s != MOE_OK) return s;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  return MOE_OK;
}

moe_status check_balance_grad(const void* logits, int32_t logits_type, int64_t T, int32_t E, int32_t k,
                              int32_t score, const void* seq_offsets, int32_t n_seqs,
                              const void* counts, const void* dloss, const void* add_to,
                              const void* dlogits) {
  const moe_status s = check_routing(logits_type, T, E, k, score, seq_offsets, n_seqs);
  if (s != MOE_OK || T == 0) return s;
  if (!logits || !counts || !dloss || !dlogits) return MOE_ERR_INVALID_ARGUMENT;
  const uintptr_t size = logits_type == MOE_BF16 ? 2 : 4;
  if (!aligned(logits, size) || !aligned(seq_offsets, 4) || !aligned(counts, 4) || !aligned(dloss, 4) ||
      !aligned(add_to, size) || !aligned(dlogits, size))
    return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

moe_status check_lora_group(const void* adapter, int64_t M, int32_t L, const void* offsets,
                            const void* rows) {
  if (M < 0 || L < 1) return MOE_ERR_INVALID_ARGUMENT;
  if (M > INT32_MAX || L > kMaxAdapters) return MOE_ERR_UNSUPPORTED;
  if (!offsets) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(offsets, 4)) return MOE_ERR_MISALIGNED;
  if (M == 0) return MOE_OK;
  if (!adapter || !rows) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(adapter, 4) || !aligned(rows, 4)) return MOE_ERR_MISALIGNED;
  // rows are dealt out by counts of adapter: it has to stay as it was
  if (overlap(adapter, M, rows, M) || overlap(adapter, M, offsets, L + 1) || overlap(rows, M, offsets, L + 1))
    return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

moe_status lora_workspace(int64_t M, int32_t N, int32_t K, int32_t R, int32_t L, size_t* bytes) {
  if (M < 0 || N < 1 || K < 1 || R < 1 || L < 1) return MOE_ERR_INVALID_ARGUMENT;
  if (K % 8 != 0 || K > kMaxDim || R % 8 != 0 || R > kMaxRank || N > kLoraMaxN || L > kMaxAdapters ||
      M > INT32_MAX)
    return MOE_ERR_UNSUPPORTED;
  *bytes = align_up(lora_partial_rows(M) * static_cast<size_t>(R) * sizeof(float), 256);
  return MOE_OK;
}

moe_status check_lora_add(const void* x, int64_t x_stride, int64_t M, int32_t K, int32_t N, int32_t R,
                          int32_t L, const void* a, const void* b, const void* scaling,
                          const void* offsets, const void* rows, int32_t y_type, const void* base,
                          int64_t base_stride, const void* y, int64_t y_stride, const void* ws,
                          size_t ws_bytes) {
  size_t need = 0;
  moe_status s = lora_workspace(M, N, K, R, L, &need);
  if (s != MOE_OK) return s;
  if (!is_type(y_type)) return MOE_ERR_INVALID_ARGUMENT;
  s = check_stride(x_stride, K, 8);
  if (s == MOE_OK) s = check_stride(y_stride, N, 1);
  if (s == MOE_OK && base) s = check_stride(base_stride, N, 1);
  if (s != MOE_OK || M == 0) return s;
  if (!x || !a || !b || !offsets || !rows || !y || !ws) return MOE_ERR_INVALID_ARGUMENT;
  if (base == y && base_stride != y_stride) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(x, 16) || !aligned(a, 16) || !aligned(b, 16) || !aligned(scaling, 4) ||
      !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(base, 16) || !aligned(y, 16) || !aligned(ws, 16))
    return MOE_ERR_MISALIGNED;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  return MOE_OK;
}

}  // namespace moe
