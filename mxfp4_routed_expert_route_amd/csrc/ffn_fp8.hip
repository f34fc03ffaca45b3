// The grouped FFN over block-scaled FP8 weights and the dense product: dispatch.
#include "fp8.h"
#include "fp8_common.h"
#include "validate_fp8.h"

namespace moe {

hipError_t launch_gemm_fp8(const uint8_t* xq, const float* x_scale, int64_t M, int N, int K,
                           const uint8_t* w, const float* w_scale, bool f32, void* y,
                           hipStream_t stream) {
  Fp8Product p{};
  p.act = xq;
  p.act_scale = x_scale;
  p.w = w;
  p.w_scale = w_scale;
  p.K = K;
  p.n = N;
  p.rows = M;
  p.k_top = 1;
  p.out_kind = f32 ? kFp8OutF32 : kFp8OutBf16;
  p.out = y;
  p.ld_out = N;
  p.act_rows = M;
  p.scale_row = (K + kFp8Block - 1) / kFp8Block;
  p.scale_k = 1;
  bool done = false;
  const hipError_t err = launch_fp8_rows(p, stream, &done);
  return done || err != hipSuccess ? err : launch_fp8_dense(p, stream);
}

hipError_t launch_ffn_fp8(const uint16_t* x, int64_t T, int H, int I, int E, int k,
                          const uint8_t* w1, const float* w1s, const uint8_t* w2, const float* w2s,
                          const int32_t* counts, const int32_t* offsets, const int32_t* gather,
                          float limit, uint16_t* y_sorted, void* ws, const Fp8WsLayout& L,
                          hipStream_t stream) {
  char* wsb = static_cast<char*>(ws);
  uint8_t* xq = reinterpret_cast<uint8_t*>(wsb + L.xq);
  float* xs = reinterpret_cast<float*>(wsb + L.xs);
  uint8_t* hq = reinterpret_cast<uint8_t*>(wsb + L.hq);
  float* hs = reinterpret_cast<float*>(wsb + L.hs);
  int32_t* n_tiles = reinterpret_cast<int32_t*>(wsb + L.plan);
  RowTile* tiles = reinterpret_cast<RowTile*>(wsb + L.plan + 256);
  const int64_t slots = T * k;
  hipError_t err = launch_plan(counts, offsets, E, L.tile_rows, slots, L.tile_bound, n_tiles, tiles,
                               stream);
  if (err != hipSuccess) return err;
  // scales of x and h are kept run by run, [K/128][rows]: a tile's are contiguous in a step
  err = launch_quantize_fp8(x, T, H, xq, xs, 1, T, stream);
  if (err != hipSuccess) return err;

  Fp8Product p{};
  p.rows = slots;
  p.tiles = tiles;
  p.n_tiles = n_tiles;
  p.tile_bound = L.tile_bound;
  p.k_top = k;
  p.limit = limit;
  p.clamp = limit > 0.f && limit <= 3.402823466e38f ? 1 : 0;   // finite and positive
  p.act = xq;
  p.act_scale = xs;
  p.act_rows = T;
  p.scale_row = 1;
  p.scale_k = T;
  p.w = w1;
  p.w_scale = w1s;
  p.K = H;
  p.n = 2 * I;
  p.gather = gather;
  p.out_kind = kFp8OutSwiglu;
  p.out = hq;
  p.out_scale = hs;
  p.ld_out = I;
  err = launch_fp8_grouped(L.tile_rows, p, stream);
  if (err != hipSuccess) return err;
  p.act = hq;
  p.act_scale = hs;
  p.act_rows = slots;
  p.scale_k = slots;
  p.w = w2;
  p.w_scale = w2s;
  p.K = I;
  p.n = H;
  p.gather = nullptr;
  p.out_kind = kFp8OutBf16;
  p.out = y_sorted;
  p.ld_out = H;
  return launch_fp8_grouped(L.tile_rows, p, stream);
}

}  // namespace moe
