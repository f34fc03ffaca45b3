// Internal launchers of the block-scaled FP8 operators (arguments are already checked).
#pragma once
#include <hip/hip_runtime.h>
#include <cstdint>

#include "fp8_plan.h"

namespace moe {

// The scale of row r, run b goes to scale[r * scale_row + b * scale_k].
hipError_t launch_quantize_fp8(const uint16_t* x, int64_t rows, int K, uint8_t* q, float* scale,
                               int64_t scale_row, int64_t scale_k, hipStream_t stream);

// What a product's epilogue writes.
enum Fp8Out : int {
  kFp8OutBf16 = 0,   // bf16 [rows][n]
  kFp8OutF32 = 1,    // fp32 [rows][n]
  kFp8OutSwiglu = 2  // h from the gate and up halves of n: E4M3 codes [rows][n / 2], with scales
                     // [n / 256][rows] in out_scale (grouped only)
};

// One product, dense or grouped.  Rows p of the activations (grouped: p in a tile of the
// plan, read at row gather[p] / k_top if gather is set, else p) times the n weight rows of
// the tile's expert (dense: expert 0, rows 0 .. rows - 1).
struct Fp8Product {
  const uint8_t* act;        // [.][K]
  const float* act_scale;    // of row r, run b at [r * scale_row + b * scale_k]
  int64_t act_rows, scale_row, scale_k;
  const uint8_t* w;          // [E][n][K]
  const float* w_scale;      // [E][ceil(n/128)][ceil(K/128)]
  int K, n;
  int64_t rows;              // dense rows, or the grouped slots T*k
  const RowTile* tiles;      // nullptr: dense
  const int32_t* n_tiles;
  int64_t tile_bound;
  const int32_t* gather;
  int k_top;
  float limit;
  int clamp;
  int out_kind;              // Fp8Out
  void* out;
  float* out_scale;
  int ld_out;
};

// Dense, few tiles (fp8_rows.hip): sets *done, or leaves larger outputs to launch_fp8_dense.
hipError_t launch_fp8_rows(const Fp8Product& p, hipStream_t stream, bool* done);
// LDS tiles (fp8_tile.hip).  tile_rows: as the plan was cut (fp8_tile_rows).
hipError_t launch_fp8_dense(const Fp8Product& p, hipStream_t stream);
hipError_t launch_fp8_grouped(int tile_rows, const Fp8Product& p, hipStream_t stream);

hipError_t launch_gemm_fp8(const uint8_t* xq, const float* x_scale, int64_t M, int N, int K,
                           const uint8_t* w, const float* w_scale, bool f32, void* y,
                           hipStream_t stream);

struct Fp8WsLayout;
hipError_t launch_ffn_fp8(const uint16_t* x, int64_t T, int H, int I, int E, int k,
                          const uint8_t* w1, const float* w1s, const uint8_t* w2, const float* w2s,
                          const int32_t* counts, const int32_t* offsets, const int32_t* gather,
                          float limit, uint16_t* y_sorted, void* ws, const Fp8WsLayout& L,
                          hipStream_t stream);

// ffn.hip: the row-tile plan of the grouped FFN.
hipError_t launch_plan(const int32_t* counts, const int32_t* offsets, int E, int tile_rows,
                       int64_t n_slots, int64_t tile_bound, int32_t* n_tiles, RowTile* tiles,
                       hipStream_t stream);

}  // namespace moe
