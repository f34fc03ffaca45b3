// Host-side checks and workspace layout of scored routing and the block-scaled FP8
// operators (no HIP calls).
#include "validate_fp8.h"

#include <climits>

#include "config.h"
#include "fp8_plan.h"

namespace moe {
namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

moe_status check_sizes(int64_t T, int32_t E, int32_t k) {
  if (T < 0 || E < 1 || k < 1 || k > E) return MOE_ERR_INVALID_ARGUMENT;
  if (E > kMaxE || k > kMaxK || T > INT32_MAX / k) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_dims(int64_t T, int32_t k, int32_t H, int32_t I) {
  if (H <= 0 || I <= 0) return MOE_ERR_INVALID_ARGUMENT;
  if (H % 128 != 0 || I % 128 != 0 || H > kMaxDim || I > kMaxDim) return MOE_ERR_UNSUPPORTED;
  // an expert's W1 (2 I rows of H bytes) is addressed with 32-bit offsets, below
  // kRsrcOutOfRange (0xFFF00000)
  if (static_cast<int64_t>(H) * I > kFp8MaxExpert) return MOE_ERR_UNSUPPORTED;
  const int64_t lim = kMaxActivationBytes;
  if (T * H * 2 > lim || T * k * static_cast<int64_t>(I) * 2 > lim ||
      T * k * static_cast<int64_t>(H) * 2 > lim)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

moe_status fp8_workspace_layout(int64_t T, int32_t E, int32_t k, int32_t H, int32_t I,
                                Fp8WsLayout* out) {
  moe_status s = check_sizes(T, E, k);
  if (s != MOE_OK) return s;
  s = check_dims(T, k, H, I);
  if (s != MOE_OK) return s;
  WsLayout routing;
  s = workspace_layout(T, E, k, 0, 0, &routing);
  if (s != MOE_OK) return s;
  const size_t t = static_cast<size_t>(T), slots = t * static_cast<size_t>(k);
  Fp8WsLayout L{};
  L.tile_rows = fp8_tile_rows(T, E, k, I);
  L.tile_bound = ffn_tile_bound(static_cast<int64_t>(slots), E, L.tile_rows);
  size_t end = 0;
  auto take = [&end](size_t bytes) {
    const size_t at = end;
    end = align_up(end + bytes, 256);
    return at;
  };
  L.xq = take(t * H);
  L.xs = take(t * (H / 128) * sizeof(float));
  L.hq = take(slots * I);
  L.hs = take(slots * (I / 128) * sizeof(float));
  // room for the smallest tiles, whatever the rule takes: the size then never shrinks as T grows
  L.plan = take(256 + static_cast<size_t>(ffn_tile_bound(static_cast<int64_t>(slots), E, kFfnMinTileRows)) *
                          sizeof(RowTile));
  L.total = end > routing.offsets_bytes ? end : routing.offsets_bytes;
  *out = L;
  return MOE_OK;
}

moe_status check_route_scored(const void* logits, int32_t logits_type, int64_t T, int32_t E,
                              int32_t k, int32_t score, const void* bias, int32_t groups,
                              int32_t topk_groups, int32_t group_top, const void* ids,
                              const void* weights) {
  const moe_status s = check_sizes(T, E, k);
  if (s != MOE_OK) return s;
  if (logits_type != MOE_F32 && logits_type != MOE_BF16) return MOE_ERR_INVALID_ARGUMENT;
  if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARGUMENT;
  if (groups < 1 || E % groups != 0 || topk_groups < 1 || topk_groups > groups)
    return MOE_ERR_INVALID_ARGUMENT;
  if (group_top != 1 && group_top != 2) return MOE_ERR_INVALID_ARGUMENT;
  if (k > topk_groups * (E / groups)) return MOE_ERR_INVALID_ARGUMENT;
  if (groups > kWave) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!logits || !ids || !weights) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(logits, logits_type == MOE_BF16 ? 2 : 4) || !aligned(bias, 4) || !aligned(ids, 4) ||
      !aligned(weights, 4))
    return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

moe_status check_quantize_fp8(const void* x, int64_t rows, int32_t K, const void* q,
                              const void* scale) {
  if (rows < 0 || K < 1) return MOE_ERR_INVALID_ARGUMENT;
  if (K % 16 != 0 || K > kMaxDim || rows > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!x || !q || !scale) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scale, 4)) return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

moe_status check_gemm_fp8(const void* xq, const void* xs, int64_t M, int32_t N, int32_t K,
                          const void* w, const void* ws, int32_t y_type, const void* y,
                          const void* work) {
  if (M < 0 || N < 1 || K < 1) return MOE_ERR_INVALID_ARGUMENT;
  if (y_type != MOE_F32 && y_type != MOE_BF16) return MOE_ERR_INVALID_ARGUMENT;
  if (K % 16 != 0 || K > kMaxDim || N > kFp8MaxN || M > INT32_MAX ||
      M * static_cast<int64_t>(N) > kFp8MaxOut)
    return MOE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_OK;
  if (!xq || !xs || !w || !ws || !y) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(xq, 16) || !aligned(w, 16) || !aligned(y, 16) || !aligned(xs, 4) ||
      !aligned(ws, 4) || !aligned(work, 16))
    return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

moe_status check_ffn_fp8(const void* x, int64_t T, int32_t H, int32_t I, int32_t E, int32_t k,
                         const void* w1, const void* w1s, const void* w2, const void* w2s,
                         const void* counts, const void* offsets, const void* gather,
                         const void* y_sorted, const void* ws, size_t ws_bytes) {
  moe_status s = check_sizes(T, E, k);
  if (s != MOE_OK) return s;
  s = check_dims(T, k, H, I);
  if (s != MOE_OK || T == 0) return s;
  if (!x || !w1 || !w1s || !w2 || !w2s || !counts || !offsets || !gather || !y_sorted || !ws)
    return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(x, 16) || !aligned(w1, 16) || !aligned(w2, 16) || !aligned(y_sorted, 16) ||
      !aligned(ws, 16) || !aligned(w1s, 4) || !aligned(w2s, 4) || !aligned(counts, 4) ||
      !aligned(offsets, 4) || !aligned(gather, 4))
    return MOE_ERR_MISALIGNED;
  Fp8WsLayout L;
  s = fp8_workspace_layout(T, E, k, H, I, &L);
  if (s != MOE_OK) return s;
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  return MOE_OK;
}

}  // namespace moe
