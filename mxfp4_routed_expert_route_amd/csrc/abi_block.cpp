// extern "C" entry points of the operators around the routed layer: host-side checks, then
// launches.
#include <hip/hip_runtime.h>

#include "../../include/moe_block.h"
#include "block.h"
#include "block_plan.h"
#include "validate_block.h"

namespace {

moe_status from_hip(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }
hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

}  // namespace

extern "C" {

moe_status moe_rms_norm(const uint16_t* x, int64_t x_stride, const uint16_t* residual, int64_t rows,
                        int32_t H, int32_t weight_type, const void* weight, float eps,
                        uint16_t* sum, uint16_t* y, uint8_t* q, float* scale, void* stream) {
  const moe_status s = moe::check_rms_norm(x, x_stride, residual, rows, H, weight_type, weight, eps, sum,
                                           y, q, scale);
  if (s != MOE_OK || rows == 0) return s;
  const moe::NormArgs a{x, x_stride, residual, rows, H, weight, weight_type == MOE_F32, eps, sum, y, q, scale};
  return from_hip(moe::launch_rms_norm(a, as_stream(stream)));
}

moe_status moe_rms_norm_grad(const uint16_t* s, int64_t s_stride, int64_t rows, int32_t H,
                             int32_t weight_type, const void* weight, float eps,
                             const uint16_t* dy, const uint16_t* dsum, uint16_t* dx, float* dweight,
                             void* ws, size_t ws_bytes, void* stream) {
  const moe_status st = moe::check_rms_norm_grad(s, s_stride, rows, H, weight_type, weight, eps, dy, dsum,
                                                 dx, dweight, ws, ws_bytes);
  if (st != MOE_OK) return st;
  const moe::NormGradArgs a{s, s_stride, rows, H, weight, weight_type == MOE_F32, eps, dy, dsum, dx, dweight,
                            static_cast<float*>(ws)};
  return from_hip(moe::launch_rms_norm_grad(a, as_stream(stream)));
}

size_t moe_rms_norm_grad_workspace_bytes(int64_t rows, int32_t H) {
  size_t bytes = 0;
  return moe::norm_grad_workspace(rows, H, &bytes) == MOE_OK ? bytes : 0;
}

moe_status moe_balance_loss(const void* logits, int32_t logits_type, int64_t T, int32_t E, int32_t k,
                            int32_t score, const int32_t* topk_ids, const int32_t* seq_offsets,
                            int32_t n_seqs, float* loss, int32_t* counts, const float* dloss,
                            const void* add_to, void* dlogits, void* ws, size_t ws_bytes,
                            void* stream) {
  const moe_status s = moe::check_balance(logits, logits_type, T, E, k, score, topk_ids, seq_offsets, n_seqs,
                                          loss, counts, dloss, add_to, dlogits, ws, ws_bytes);
  if (s != MOE_OK) return s;
  const size_t sums = (static_cast<size_t>(moe::balance_slots(T, n_seqs)) * sizeof(double) + 255) / 256 * 256;
  const moe::BalanceArgs a{logits, T, E, k, score == MOE_SCORE_SIGMOID, topk_ids, seq_offsets, n_seqs,
                           loss, counts, dloss, add_to, dlogits, static_cast<double*>(ws),
                           T == 0 ? nullptr : reinterpret_cast<int32_t*>(static_cast<char*>(ws) + sums)};
  return from_hip(moe::launch_balance(a, logits_type == MOE_BF16, as_stream(stream)));
}

size_t moe_balance_loss_workspace_bytes(int64_t T, int32_t E, int32_t n_seqs) {
  size_t bytes = 0;
  return moe::balance_workspace(T, E, n_seqs, &bytes) == MOE_OK ? bytes : 0;
}

moe_status moe_balance_loss_grad(const void* logits, int32_t logits_type, int64_t T, int32_t E,
                                 int32_t k, int32_t score, const int32_t* seq_offsets,
                                 int32_t n_seqs, const int32_t* counts, const float* dloss,
                                 const void* add_to, void* dlogits, void* stream) {
  const moe_status s = moe::check_balance_grad(logits, logits_type, T, E, k, score, seq_offsets, n_seqs,
                                               counts, dloss, add_to, dlogits);
  if (s != MOE_OK || T == 0) return s;
  const moe::BalanceArgs a{logits, T, E, k, score == MOE_SCORE_SIGMOID, nullptr, seq_offsets, n_seqs,
                           nullptr, const_cast<int32_t*>(counts), dloss, add_to, dlogits, nullptr, nullptr};
  return from_hip(moe::launch_balance(a, logits_type == MOE_BF16, as_stream(stream)));
}

moe_status moe_lora_group(const int32_t* adapter, int64_t M, int32_t L, int32_t* offsets,
                          int32_t* rows, void* stream) {
  const moe_status s = moe::check_lora_group(adapter, M, L, offsets, rows);
  if (s != MOE_OK) return s;
  return from_hip(moe::launch_lora_group(adapter, M, L, offsets, rows, as_stream(stream)));
}

moe_status moe_lora_add(const uint16_t* x, int64_t x_stride, int64_t M, int32_t K, int32_t N,
                        int32_t R, int32_t L, const uint16_t* a, const uint16_t* b,
                        const float* scaling, const int32_t* offsets, const int32_t* rows,
                        int32_t y_type, const void* base, int64_t base_stride, void* y,
                        int64_t y_stride, void* ws, size_t ws_bytes, void* stream) {
  const moe_status s = moe::check_lora_add(x, x_stride, M, K, N, R, L, a, b, scaling, offsets, rows, y_type,
                                           base, base_stride, y, y_stride, ws, ws_bytes);
  if (s != MOE_OK || M == 0) return s;
  const moe::LoraArgs l{x, x_stride, M, K, N, R, L, a, b, scaling, offsets, rows, base, base_stride, y,
                        y_stride, static_cast<float*>(ws)};
  return from_hip(moe::launch_lora_add(l, y_type == MOE_F32, as_stream(stream)));
}

size_t moe_lora_add_workspace_bytes(int64_t M, int32_t N, int32_t K, int32_t R, int32_t L) {
  size_t bytes = 0;
  return moe::lora_workspace(M, N, K, R, L, &bytes) == MOE_OK ? bytes : 0;
}

}  // extern "C"
