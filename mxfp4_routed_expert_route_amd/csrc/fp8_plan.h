// Tiling rules and limits of the block-scaled FP8 operators, shared by the host checks and
// the launch code.  Pure C++.
#pragma once
#include <cstdint>

#include "config.h"

namespace moe {

constexpr int32_t kFp8MaxN = 1 << 24;
constexpr int64_t kFp8MaxExpert = (int64_t{1} << 31) - (1 << 20);   // H * I
constexpr int64_t kFp8MaxOut = int64_t{1} << 38;   // M * N of the dense product

constexpr int kFp8Cus = 256;   // CUs of an MI355X: how far tiles are cut to give each one work

// Rows per row tile of the grouped FP8 FFN, from the mean rows per expert: 16, 32 and 96 rows
// while the batch is bound by the weights (each expert's are read about once: its rows fit one
// tile up to about three standard deviations over the mean), then 256, bound by the products.
inline int fp8_tile_rows(int64_t T, int E, int k) {
  const int64_t avg_rows = T * k / E;
  if (T <= 16 || avg_rows <= 6) return 16;
  if (avg_rows <= 20) return 32;
  return avg_rows <= 72 ? 96 : 256;
}

}  // namespace moe
