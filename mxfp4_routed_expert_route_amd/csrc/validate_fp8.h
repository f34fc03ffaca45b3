// Host-side checks and workspace layout of scored routing and the block-scaled FP8
// operators.  Pure C++, like validate.h.
#pragma once
#include "../../include/moe_fp8.h"
#include "validate.h"

namespace moe {

struct Fp8WsLayout {
  size_t xq, xs;     // [T][H] codes, [T][H/128] scales
  size_t hq, hs;     // [T*k][I] codes, [T*k][I/128] scales
  size_t plan;       // row-tile count, then the RowTile list
  size_t total;
  int64_t tile_bound;
  int tile_rows;
};

moe_status fp8_workspace_layout(int64_t T, int32_t E, int32_t k, int32_t H, int32_t I,
                                Fp8WsLayout* out);

moe_status check_route_scored(const void* logits, int32_t logits_type, int64_t T, int32_t E,
                              int32_t k, int32_t score, const void* bias, int32_t groups,
                              int32_t topk_groups, int32_t group_top, const void* ids,
                              const void* weights);
moe_status check_quantize_fp8(const void* x, int64_t rows, int32_t K, const void* q,
                              const void* scale);
moe_status check_gemm_fp8(const void* xq, const void* xs, int64_t M, int32_t N, int32_t K,
                          const void* w, const void* ws, int32_t y_type, const void* y,
                          const void* work);
moe_status check_ffn_fp8(const void* x, int64_t T, int32_t H, int32_t I, int32_t E, int32_t k,
                         const void* w1, const void* w1s, const void* w2, const void* w2s,
                         const void* counts, const void* offsets, const void* gather,
                         const void* y_sorted, const void* ws, size_t ws_bytes);

}  // namespace moe
