// Tiling rules and limits of the block-scaled FP8 operators, shared by the host checks and
// the launch code.  Pure C++.
#pragma once
#include <cstdint>

#include "config.h"

namespace moe {

constexpr int32_t kFp8MaxN = 1 << 24;
constexpr int64_t kFp8MaxExpert = (int64_t{1} << 31) - (1 << 20);   // H * I
constexpr int64_t kFp8MaxOut = int64_t{1} << 38;   // M * N of the dense product

// Rows per row tile of the grouped FP8 FFN.
inline int fp8_tile_rows(int64_t T, int E, int k) {
  const int64_t avg_rows = T * k / E;
  if (T <= 16 || avg_rows < 4) return 16;
  if (avg_rows <= 24) return 32;
  return avg_rows <= 64 ? 64 : 256;
}
// Rows a tile of the dense product takes.
inline int fp8_gemm_tile_rows(int64_t M) { return M <= 32 ? 16 : M <= 512 ? 64 : 256; }

}  // namespace moe
