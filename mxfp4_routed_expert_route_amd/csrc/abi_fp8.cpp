// extern "C" entry points of scored routing and the block-scaled FP8 operators: host-side
// checks, then launches.
#include <hip/hip_runtime.h>

#include "../../include/moe_fp8.h"
#include "fp8.h"
#include "launch.h"
#include "validate_fp8.h"

namespace {

moe_status from_hip(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }
hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

}  // namespace

extern "C" {

moe_status moe_route_scored(const void* logits, int32_t logits_type, int64_t T, int32_t E,
                            int32_t k, int32_t score, const float* bias, int32_t groups,
                            int32_t topk_groups, int32_t group_top, int32_t renormalize,
                            float scale, int32_t* topk_ids, float* topk_weights, void* stream) {
  const moe_status s = moe::check_route_scored(logits, logits_type, T, E, k, score, bias, groups,
                                               topk_groups, group_top, topk_ids, topk_weights);
  if (s != MOE_OK || T == 0) return s;
  const moe::ScoredRouting r{score, bias, groups, topk_groups, group_top, renormalize, scale};
  return from_hip(moe::launch_route_scored(logits, logits_type == MOE_BF16, T, E, k, r, topk_ids,
                                           topk_weights, nullptr, as_stream(stream)));
}

moe_status moe_route_scored_and_group(const void* logits, int32_t logits_type, int64_t T,
                                      int32_t E, int32_t k, int32_t score, const float* bias,
                                      int32_t groups, int32_t topk_groups, int32_t group_top,
                                      int32_t renormalize, float scale, int32_t* topk_ids,
                                      float* topk_weights, uint32_t* bitmatrix, int32_t* counts,
                                      int32_t* offsets, int32_t* gather, int32_t* scatter,
                                      void* ws, size_t ws_bytes, void* stream) {
  moe_status s = moe::check_route_scored(logits, logits_type, T, E, k, score, bias, groups,
                                         topk_groups, group_top, topk_ids, topk_weights);
  if (s != MOE_OK) return s;
  s = moe::check_bitmatrix(topk_ids, T, E, k, bitmatrix);
  if (s != MOE_OK) return s;
  s = moe::check_offsets(bitmatrix, topk_ids, T, E, k, counts, offsets, gather, scatter, ws,
                         ws_bytes);
  if (s != MOE_OK) return s;
  if (T == 0)
    return from_hip(moe::launch_offsets(nullptr, nullptr, 0, E, k, counts, offsets, nullptr,
                                        nullptr, nullptr, as_stream(stream)));
  const moe::ScoredRouting r{score, bias, groups, topk_groups, group_top, renormalize, scale};
  return from_hip(moe::launch_route_scored_and_group(
      logits, logits_type == MOE_BF16, T, E, k, r, topk_ids, topk_weights, bitmatrix, counts,
      offsets, gather, scatter, ws, as_stream(stream)));
}

moe_status moe_quantize_fp8(const uint16_t* x, int64_t rows, int32_t K, uint8_t* q, float* scale,
                            void* stream) {
  const moe_status s = moe::check_quantize_fp8(x, rows, K, q, scale);
  if (s != MOE_OK || rows == 0) return s;
  return from_hip(moe::launch_quantize_fp8(x, rows, K, q, scale, (K + 127) / 128, 1, as_stream(stream)));
}

moe_status moe_gemm_fp8(const uint8_t* xq, const float* x_scale, int64_t M, int32_t N, int32_t K,
                        const uint8_t* w, const float* w_scale, int32_t y_type, void* y, void* ws,
                        size_t, void* stream) {
  const moe_status s = moe::check_gemm_fp8(xq, x_scale, M, N, K, w, w_scale, y_type, y, ws);
  if (s != MOE_OK || M == 0) return s;
  return from_hip(moe::launch_gemm_fp8(xq, x_scale, M, N, K, w, w_scale, y_type == MOE_F32, y,
                                       as_stream(stream)));
}

size_t moe_gemm_fp8_workspace_bytes(int64_t, int32_t, int32_t) { return 0; }

moe_status moe_grouped_ffn_fp8(const uint16_t* x, int64_t T, int32_t H, int32_t I, int32_t E,
                               int32_t k, const uint8_t* w1, const float* w1_scale,
                               const uint8_t* w2, const float* w2_scale, const int32_t* counts,
                               const int32_t* offsets, const int32_t* gather, float swiglu_limit,
                               uint16_t* y_sorted, void* ws, size_t ws_bytes, void* stream) {
  moe_status s = moe::check_ffn_fp8(x, T, H, I, E, k, w1, w1_scale, w2, w2_scale, counts, offsets,
                                    gather, y_sorted, ws, ws_bytes);
  if (s != MOE_OK || T == 0) return s;
  moe::Fp8WsLayout L;
  s = moe::fp8_workspace_layout(T, E, k, H, I, &L);
  if (s != MOE_OK) return s;
  return from_hip(moe::launch_ffn_fp8(x, T, H, I, E, k, w1, w1_scale, w2, w2_scale, counts, offsets,
                                      gather, swiglu_limit, y_sorted, ws, L, as_stream(stream)));
}

size_t moe_fp8_workspace_bytes(int64_t T, int32_t E, int32_t k, int32_t H, int32_t I) {
  moe::Fp8WsLayout L;
  if (moe::fp8_workspace_layout(T, E, k, H, I, &L) != MOE_OK) return 0;
  return L.total;
}

}  // extern "C"
