// Host-side checks of the operators around the routed layer (no HIP calls).
#pragma once
#include <cstddef>
#include <cstdint>

#include "../../include/moe_block.h"

namespace moe {

moe_status check_rms_norm(const void* x, int64_t x_stride, const void* residual, int64_t rows, int32_t H,
                          int32_t weight_type, const void* weight, float eps, const void* sum,
                          const void* y, const void* q, const void* scale);
moe_status check_rms_norm_grad(const void* s, int64_t s_stride, int64_t rows, int32_t H,
                               int32_t weight_type, const void* weight, float eps, const void* dy,
                               const void* dsum, const void* dx, const void* dweight, const void* ws,
                               size_t ws_bytes);
moe_status norm_grad_workspace(int64_t rows, int32_t H, size_t* bytes);
moe_status check_balance(const void* logits, int32_t logits_type, int64_t T, int32_t E, int32_t k,
                         int32_t score, const void* ids, const void* seq_offsets, int32_t n_seqs,
                         const void* loss, const void* counts, const void* dloss, const void* add_to,
                         const void* dlogits, const void* ws, size_t ws_bytes);
moe_status check_balance_grad(const void* logits, int32_t logits_type, int64_t T, int32_t E, int32_t k,
                              int32_t score, const void* seq_offsets, int32_t n_seqs,
                              const void* counts, const void* dloss, const void* add_to,
                              const void* dlogits);
moe_status balance_workspace(int64_t T, int32_t E, int32_t n_seqs, size_t* bytes);
moe_status check_lora_group(const void* adapter, int64_t M, int32_t L, const void* offsets,
                            const void* rows);
moe_status check_lora_add(const void* x, int64_t x_stride, int64_t M, int32_t K, int32_t N, int32_t R,
                          int32_t L, const void* a, const void* b, const void* scaling,
                          const void* offsets, const void* rows, int32_t y_type, const void* base,
                          int64_t base_stride, const void* y, int64_t y_stride, const void* ws,
                          size_t ws_bytes);
moe_status lora_workspace(int64_t M, int32_t N, int32_t K, int32_t R, int32_t L, size_t* bytes);

}  // namespace moe
