// Host-only driver for the argument checks (built with g++ and sanitizers, no GPU).
// Forces every status code of every entry point's check from the host and checks
// the workspace layout; exits non-zero on the first mismatch.
#include <climits>
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#include "../block_plan.h"
#include "../config.h"
#include "../fp8_plan.h"
#include "../validate.h"
#include "../validate_block.h"
#include "../validate_fp8.h"

using namespace moe;

static int failures = 0;
static void expect(const char* what, moe_status got, moe_status want) {
  if (got != want) {
    std::printf("FAIL %s: got %d want %d\n", what, static_cast<int>(got), static_cast<int>(want));
    ++failures;
  }
}

int main() {
  alignas(256) static unsigned char buf[4096];
  const void* p = buf;                 // 256-aligned stand-in pointer
  const void* odd = buf + 1;           // misaligned
  const void* p4 = buf + 4;            // 4- but not 16-aligned

  // route
  expect("route ok", check_route(p, 16, 256, 6, p, p), MOE_OK);
  expect("route T=0 nulls", check_route(nullptr, 0, 256, 6, nullptr, nullptr), MOE_OK);
  expect("route T<0", check_route(p, -1, 256, 6, p, p), MOE_ERR_INVALID_ARGUMENT);
  expect("route k=0", check_route(p, 16, 256, 0, p, p), MOE_ERR_INVALID_ARGUMENT);
  expect("route k>E", check_route(p, 16, 4, 5, p, p), MOE_ERR_INVALID_ARGUMENT);
  expect("route E=0", check_route(p, 16, 0, 1, p, p), MOE_ERR_INVALID_ARGUMENT);
  expect("route E>1024", check_route(p, 16, 1025, 6, p, p), MOE_ERR_UNSUPPORTED);
  expect("route k>8", check_route(p, 16, 256, 9, p, p), MOE_ERR_UNSUPPORTED);
  expect("route T*k overflow", check_route(p, (int64_t)1 << 31, 256, 6, p, p), MOE_ERR_UNSUPPORTED);
  expect("route null logits", check_route(nullptr, 16, 256, 6, p, p), MOE_ERR_INVALID_ARGUMENT);
  expect("route null ids", check_route(p, 16, 256, 6, nullptr, p), MOE_ERR_INVALID_ARGUMENT);
  expect("route misaligned", check_route(odd, 16, 256, 6, p, p), MOE_ERR_MISALIGNED);

  // bitmatrix
  expect("bm ok", check_bitmatrix(p, 16, 256, 6, p), MOE_OK);
  expect("bm null", check_bitmatrix(p, 16, 256, 6, nullptr), MOE_ERR_INVALID_ARGUMENT);
  expect("bm misaligned", check_bitmatrix(p, 16, 256, 6, odd), MOE_ERR_MISALIGNED);
  expect("bm T=0", check_bitmatrix(nullptr, 0, 256, 6, nullptr), MOE_OK);

  // offsets
  WsLayout L;
  expect("layout", workspace_layout(8191, 256, 6, 4096, 2048, &L), MOE_OK);
  if (L.n_blocks != 16 || L.offsets_bytes != 16 * 256 * 4) { std::printf("FAIL offsets layout\n"); ++failures; }
  if (L.tile_bound != (49146 + (kFfnMinTileRows - 1) * 256) / kFfnMinTileRows) {
    std::printf("FAIL tile bound\n"); ++failures;
  }
  // decode sizes (T k < E, K of 2048 / 4096): 1-row tiles on the GEMV kernels
  WsLayout G;
  expect("layout gemv", workspace_layout(8, 256, 6, 4096, 2048, &G), MOE_OK);
  if (ffn_tile_rows(8, 256, 6, 4096, 2048) != kFfnGemvTileRows || G.tile_bound != 48) {
    std::printf("FAIL gemv tile rule / bound\n"); ++failures;
  }
  if (ffn_tile_rows(8, 256, 6, 256, 128) != 16 || ffn_tile_rows(43, 256, 6, 4096, 2048) != 16) {
    std::printf("FAIL gemv tile rule limits\n"); ++failures;
  }
  // ffn_tile_bound against the exact tile count of random and extreme row counts
  {
    unsigned rng = 12345u;
    auto next = [&]() { rng = rng * 1664525u + 1013904223u; return rng >> 8; };
    const int sizes[] = {2, 16, 32, 80, 128};
    for (int trial = 0; trial < 2000; ++trial) {
      const int E = 1 + static_cast<int>(next() % 300);
      const int R = sizes[trial % 5];
      static int c[300];
      int64_t n = 0, tiles = 0;
      for (int e = 0; e < E; ++e) {
        const unsigned kind = trial % 4;   // sparse, 1 mod R, skewed, uniform
        c[e] = kind == 0 ? (next() % 5 == 0 ? static_cast<int>(next() % 4) : 0)
             : kind == 1 ? static_cast<int>(R * (next() % 3) + 1)
             : kind == 2 ? (e == 0 ? static_cast<int>(next() % 5000) : static_cast<int>(next() % 3))
                         : static_cast<int>(next() % 200);
        n += c[e];
        tiles += (c[e] + R - 1) / R;
      }
      if (tiles > ffn_tile_bound(n, E, R)) {
        std::printf("FAIL tile bound trial %d: %lld tiles > %lld\n", trial,
                    static_cast<long long>(tiles), static_cast<long long>(ffn_tile_bound(n, E, R)));
        ++failures;
        break;
      }
    }
  }
  if (L.ffn_plan_offset < (size_t)49146 * 2048 * 2 || L.total < L.ffn_bytes || L.total < L.offsets_bytes) {
    std::printf("FAIL ffn layout\n"); ++failures;
  }
  expect("offs ok", check_offsets(p, p, 16, 256, 6, p, p, p, p, p, L.total), MOE_OK);
  expect("offs small ws", check_offsets(p, p, 1025, 256, 6, p, p, p, p, p, 256 * 4), MOE_ERR_WORKSPACE_TOO_SMALL);
  expect("offs ws misaligned", check_offsets(p, p, 16, 256, 6, p, p, p, p, p4, 1 << 20), MOE_ERR_MISALIGNED);
  expect("offs null gather", check_offsets(p, p, 16, 256, 6, p, p, nullptr, p, p, 1 << 20), MOE_ERR_INVALID_ARGUMENT);
  expect("offs T=0", check_offsets(nullptr, nullptr, 0, 256, 6, p, p, nullptr, nullptr, nullptr, 0), MOE_OK);
  expect("offs T=0 null counts", check_offsets(nullptr, nullptr, 0, 256, 6, nullptr, p, nullptr, nullptr, nullptr, 0), MOE_ERR_INVALID_ARGUMENT);

  // ffn
  WsLayout F;
  workspace_layout(16, 256, 6, 256, 128, &F);
  expect("ffn ok", check_ffn(p, 16, 256, 128, 256, 6, p, p, p, p, p, p, p, p, p, F.ffn_bytes), MOE_OK);
  expect("ffn H%128", check_ffn(p, 16, 192, 128, 256, 6, p, p, p, p, p, p, p, p, p, 1 << 30), MOE_ERR_UNSUPPORTED);
  expect("ffn I%128", check_ffn(p, 16, 256, 64, 256, 6, p, p, p, p, p, p, p, p, p, 1 << 30), MOE_ERR_UNSUPPORTED);
  expect("ffn H=0", check_ffn(p, 16, 0, 128, 256, 6, p, p, p, p, p, p, p, p, p, 1 << 30), MOE_ERR_INVALID_ARGUMENT);
  expect("ffn small ws", check_ffn(p, 16, 256, 128, 256, 6, p, p, p, p, p, p, p, p, p, F.ffn_bytes - 1), MOE_ERR_WORKSPACE_TOO_SMALL);
  expect("ffn x misaligned", check_ffn(p4, 16, 256, 128, 256, 6, p, p, p, p, p, p, p, p, p, F.ffn_bytes), MOE_ERR_MISALIGNED);
  expect("ffn w1 misaligned", check_ffn(p, 16, 256, 128, 256, 6, p4, p, p, p, p, p, p, p, p, F.ffn_bytes), MOE_ERR_MISALIGNED);
  expect("ffn w1 scales misaligned", check_ffn(p, 16, 256, 128, 256, 6, p, p4, p, p, p, p, p, p, p, F.ffn_bytes), MOE_ERR_MISALIGNED);
  expect("ffn w2 scales misaligned", check_ffn(p, 16, 256, 128, 256, 6, p, p, p, p4, p, p, p, p, p, F.ffn_bytes), MOE_ERR_MISALIGNED);
  expect("ffn null w2s", check_ffn(p, 16, 256, 128, 256, 6, p, p, p, nullptr, p, p, p, p, p, F.ffn_bytes), MOE_ERR_INVALID_ARGUMENT);
  expect("ffn T=0", check_ffn(nullptr, 0, 256, 128, 256, 6, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0), MOE_OK);

  // combine
  expect("comb ok", check_combine(p, p, p, 16, 256, 6, p), MOE_OK);
  expect("comb H%8", check_combine(p, p, p, 16, 260, 6, p), MOE_ERR_UNSUPPORTED);
  expect("comb k=0", check_combine(p, p, p, 16, 256, 0, p), MOE_ERR_INVALID_ARGUMENT);
  expect("comb y misaligned", check_combine(p, p, p, 16, 256, 6, p4), MOE_ERR_MISALIGNED);
  expect("comb null", check_combine(p, nullptr, p, 16, 256, 6, p), MOE_ERR_INVALID_ARGUMENT);
  expect("comb T=0", check_combine(nullptr, nullptr, nullptr, 0, 256, 6, nullptr), MOE_OK);

  // scored routing
  auto scored = [&](int64_t T, int32_t E, int32_t k, int32_t groups, int32_t topk, int32_t top) {
    return check_route_scored(p, MOE_F32, T, E, k, MOE_SCORE_SIGMOID, p, groups, topk, top, p, p);
  };
  expect("scored ok", scored(16, 256, 6, 8, 4, 2), MOE_OK);
  expect("scored largest T", scored(INT32_MAX / 8, 1024, 8, 64, 64, 1), MOE_OK);
  expect("scored T*k overflow", scored(INT32_MAX / 8 + 1, 1024, 8, 64, 64, 1), MOE_ERR_UNSUPPORTED);
  expect("scored largest int64 T", scored(INT64_MAX, 256, 6, 8, 4, 2), MOE_ERR_UNSUPPORTED);
  expect("scored least int64 T", scored(INT64_MIN, 256, 6, 8, 4, 2), MOE_ERR_INVALID_ARGUMENT);
  expect("scored largest groups", scored(16, 256, 6, INT32_MAX, INT32_MAX, 2), MOE_ERR_INVALID_ARGUMENT);
  expect("scored least groups", scored(16, 256, 6, INT32_MIN, INT32_MIN, 2), MOE_ERR_INVALID_ARGUMENT);
  expect("scored largest topk_groups", scored(16, 256, 6, 8, INT32_MAX, 2), MOE_ERR_INVALID_ARGUMENT);
  expect("scored largest E and k", scored(16, INT32_MAX, INT32_MAX, 1, 1, 2), MOE_ERR_UNSUPPORTED);
  expect("scored misaligned", check_route_scored(odd, MOE_BF16, 16, 256, 6, MOE_SCORE_SOFTMAX, p, 1, 1, 1, p, p), MOE_ERR_MISALIGNED);

  // quantisation
  expect("quantise ok", check_quantize_fp8(p, INT32_MAX, kMaxDim, p, p), MOE_OK);
  expect("quantise rows", check_quantize_fp8(p, INT64_MAX, kMaxDim, p, p), MOE_ERR_UNSUPPORTED);
  expect("quantise K", check_quantize_fp8(p, 1, INT32_MAX, p, p), MOE_ERR_UNSUPPORTED);
  expect("quantise least K", check_quantize_fp8(p, 1, INT32_MIN, p, p), MOE_ERR_INVALID_ARGUMENT);
  expect("quantise misaligned", check_quantize_fp8(p, 1, 256, p4, p), MOE_ERR_MISALIGNED);

  // dense product
  auto dense = [&](int64_t M, int32_t N, int32_t K) {
    return check_gemm_fp8(p, p, M, N, K, p, p, MOE_BF16, p, nullptr);
  };
  expect("dense ok", dense(16, 256, 128), MOE_OK);
  expect("dense largest M", dense(INT32_MAX, 128, kMaxDim), MOE_OK);
  expect("dense M * N", dense(INT32_MAX, 129, kMaxDim), MOE_ERR_UNSUPPORTED);
  expect("dense largest N", dense(1 << 14, kFp8MaxN, kMaxDim), MOE_OK);
  expect("dense N", dense(1, kFp8MaxN + 1, 128), MOE_ERR_UNSUPPORTED);
  expect("dense largest int64 M", dense(INT64_MAX, INT32_MAX, 128), MOE_ERR_UNSUPPORTED);
  expect("dense misaligned", check_gemm_fp8(p, p, 16, 256, 128, p, p, MOE_F32, p4, nullptr), MOE_ERR_MISALIGNED);

  // grouped FP8 FFN: the largest activations and experts, and one step past them
  auto ffn8 = [&](int64_t T, int32_t E, int32_t k, int32_t H, int32_t I, size_t ws_bytes) {
    return check_ffn_fp8(p, T, H, I, E, k, p, p, p, p, p, p, p, p, p, ws_bytes);
  };
  struct { int64_t T; int32_t E, k, H, I; } sizes[] = {
      {1, 1, 1, 128, 128}, {8, 256, 6, 4096, 2048}, {8191, 256, 6, 4096, 2048}, {kMaxActivationBytes / 256, 1024, 1, 128, 128},
      {kMaxActivationBytes / 2 / 8 / 65536, 8, 8, 65536, 128}, {16, 2, 1, 65536, 32752 / 128 * 128}, {16, 2, 1, 128, 65536}};
  for (const auto& z : sizes) {
    Fp8WsLayout L8;
    expect("fp8 layout", fp8_workspace_layout(z.T, z.E, z.k, z.H, z.I, &L8), MOE_OK);
    const int64_t slots = z.T * z.k;
    const size_t ends[] = {L8.xs, L8.hq, L8.hs, L8.plan, L8.total};
    const size_t need[] = {L8.xq + static_cast<size_t>(z.T) * z.H, L8.xs + static_cast<size_t>(z.T) * (z.H / 128) * 4,
                           L8.hq + static_cast<size_t>(slots) * z.I, L8.hs + static_cast<size_t>(slots) * (z.I / 128) * 4,
                           L8.plan + 256 + static_cast<size_t>(L8.tile_bound) * sizeof(RowTile)};
    for (int i = 0; i < 5; ++i)
      if (ends[i] < need[i]) { std::printf("FAIL fp8 layout part %d, T = %lld\n", i, static_cast<long long>(z.T)); ++failures; }
    if (L8.tile_bound < 1 || L8.tile_bound > INT32_MAX) { std::printf("FAIL fp8 tile bound\n"); ++failures; }
    expect("fp8 ffn ok", ffn8(z.T, z.E, z.k, z.H, z.I, L8.total), MOE_OK);
    expect("fp8 ffn small ws", ffn8(z.T, z.E, z.k, z.H, z.I, L8.total - 1), MOE_ERR_WORKSPACE_TOO_SMALL);
  }
  expect("fp8 ffn activations", ffn8(kMaxActivationBytes / 256 + 1, 1024, 1, 128, 128, SIZE_MAX), MOE_ERR_UNSUPPORTED);
  expect("fp8 ffn expert", ffn8(1, 2, 1, 65536, 32768, SIZE_MAX), MOE_ERR_UNSUPPORTED);
  expect("fp8 ffn largest H and I", ffn8(1, 2, 1, 65536, 65536, SIZE_MAX), MOE_ERR_UNSUPPORTED);
  expect("fp8 ffn int32 H and I", ffn8(1, 2, 1, INT32_MAX / 128 * 128, INT32_MAX / 128 * 128, SIZE_MAX), MOE_ERR_UNSUPPORTED);
  expect("fp8 ffn largest int64 T", ffn8(INT64_MAX, 1024, 8, 65536, 128, SIZE_MAX), MOE_ERR_UNSUPPORTED);
  expect("fp8 ffn T * k", ffn8(INT32_MAX, 1024, 1, 65536, 128, SIZE_MAX), MOE_ERR_UNSUPPORTED);
  expect("fp8 ffn misaligned", check_ffn_fp8(p4, 16, 128, 128, 4, 2, p, p, p, p, p, p, p, p, p, 1 << 20), MOE_ERR_MISALIGNED);
  if (failures == 0) std::printf("scored routing and fp8 checks ok\n");

  // the operators around the layer, at the ends of their ranges
  auto norm = [&](int64_t rows, int32_t H, int64_t stride, float eps) {
    return check_rms_norm(p, stride, p, rows, H, MOE_BF16, p, eps, p, nullptr, p, p);
  };
  expect("norm ok", norm(INT32_MAX, kMaxDim, kMaxDim, 1e-6f), MOE_OK);
  expect("norm largest int64 rows", norm(INT64_MAX, 16, 16, 0.f), MOE_ERR_UNSUPPORTED);
  expect("norm least int64 rows", norm(INT64_MIN, 16, 16, 0.f), MOE_ERR_INVALID_ARGUMENT);
  expect("norm largest H", norm(1, INT32_MAX, INT32_MAX, 0.f), MOE_ERR_UNSUPPORTED);
  expect("norm largest stride", norm(1, 16, INT64_MAX, 0.f), MOE_ERR_UNSUPPORTED);
  expect("norm least stride", norm(1, 16, INT64_MIN, 0.f), MOE_ERR_INVALID_ARGUMENT);
  size_t bytes = 0;
  expect("norm grad ws", norm_grad_workspace(INT32_MAX, kMaxDim, &bytes), MOE_OK);
  if (bytes < static_cast<size_t>(norm_grad_groups(INT32_MAX, kMaxDim)) * kMaxDim * 4) { std::printf("FAIL norm grad ws\n"); ++failures; }
  expect("norm grad small ws", check_rms_norm_grad(p, kMaxDim, INT32_MAX, kMaxDim, MOE_F32, p, 0.f, p, nullptr, nullptr, p, p, bytes - 1), MOE_ERR_WORKSPACE_TOO_SMALL);
  auto balance = [&](int64_t T, int32_t E, int32_t k, int32_t seqs) {
    return check_balance(p, MOE_F32, T, E, k, MOE_SCORE_SIGMOID, p, p, seqs, p, p, p, p, p, p, SIZE_MAX);
  };
  expect("balance ok", balance(INT32_MAX / 8, kMaxE, 8, kMaxSequences), MOE_OK);
  expect("balance T * k", balance(INT32_MAX / 8 + 1, kMaxE, 8, 1), MOE_ERR_UNSUPPORTED);
  expect("balance largest int64 T", balance(INT64_MAX, kMaxE, 1, 1), MOE_ERR_UNSUPPORTED);
  expect("balance sequences", balance(1, 2, 1, INT32_MAX), MOE_ERR_UNSUPPORTED);
  expect("balance ws", balance_workspace(INT32_MAX, kMaxE, kMaxSequences, &bytes), MOE_OK);
  auto at = [](uintptr_t v) { return reinterpret_cast<const void*>(v); };
  const uintptr_t far = uintptr_t{1} << 40;
  expect("lora group ok", check_lora_group(at(far), INT32_MAX, kMaxAdapters, at(2 * far), at(3 * far)), MOE_OK);
  expect("lora group last row shared", check_lora_group(at(far), INT32_MAX, 2, at(far + (uintptr_t{1} << 33) - 8), at(3 * far)), MOE_ERR_INVALID_ARGUMENT);
  expect("lora group beside", check_lora_group(at(far), INT32_MAX, 2, at(far + (uintptr_t{1} << 33) - 4), at(3 * far)), MOE_OK);
  expect("lora group in place", check_lora_group(at(far), 4, 2, at(2 * far), at(far)), MOE_ERR_INVALID_ARGUMENT);
  auto lora = [&](int64_t M, int32_t N, int32_t K, int32_t R, int32_t L) {
    return check_lora_add(p, K, M, K, N, R, L, p, p, p, p, p, MOE_BF16, p, N, p, N, p, SIZE_MAX);
  };
  expect("lora ok", lora(INT32_MAX, kLoraMaxN, kMaxDim, kMaxRank, kMaxAdapters), MOE_OK);
  expect("lora largest int64 M", lora(INT64_MAX, 16, 16, 8, 1), MOE_ERR_UNSUPPORTED);
  expect("lora least int64 M", lora(INT64_MIN, 16, 16, 8, 1), MOE_ERR_INVALID_ARGUMENT);
  expect("lora largest sizes", lora(1, INT32_MAX, INT32_MAX, INT32_MAX, INT32_MAX), MOE_ERR_UNSUPPORTED);
  for (int64_t M : {int64_t{1}, int64_t{300}, kLoraPartialRows, kLoraPartialRows + 1, int64_t{INT32_MAX}})
    if (static_cast<size_t>(lora_max_splits(M)) * static_cast<size_t>(M) > lora_partial_rows(M) || lora_max_splits(M) < 1) {
      std::printf("FAIL lora splits\n");
      ++failures;
    }

  if (failures) return 1;
  std::printf("validate_check ok\n");
  return 0;
}
