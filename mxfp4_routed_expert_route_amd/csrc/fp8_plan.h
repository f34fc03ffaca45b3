// Tiling rules and limits of the block-scaled FP8 operators, shared by the host checks and
// the launch code.  Pure C++.
#pragma once
#include <cstdint>

#include "config.h"

namespace moe {

constexpr int kFp8Block = 128;   // K elements per scale, and weight rows per scale
constexpr int32_t kFp8MaxN = 1 << 24;
constexpr int64_t kFp8MaxExpert = (int64_t{1} << 31) - (1 << 20);   // H * I
constexpr int64_t kFp8MaxOut = int64_t{1} << 38;   // M * N of the dense product

constexpr int kFp8Cus = 256;   // CUs of an MI355X: how far tiles are cut to give each one work

// Rows per row tile of the grouped FP8 FFN, from the mean rows per expert.  While the batch is
// bound by the weights, an expert's rows are to fit one tile (each weight is then read once) and
// all CUs are to have a workgroup; from 90 rows on it is bound by the products and takes 256.
// Measured (us; H = 4096, I = 2048, k = 6 unless said; random routing):
//   96 / 256 rows: 256 experts 84 rows on average 1325 / 1637, 96 1680 / 1662, 128 2341 / 1729;
//     64 experts 80 364 / 445, 96 448 / 453, 128 602 / 469.
//   32 / 96 rows: 256 experts 20 1042 / 1059, 24 1101 / 1068; 64 experts 20 266 / 292, 24 316 / 296.
//   16 / 32 rows: 256 experts 2 845 / 854, 6 1009 / 970, 12 1143 / 991; 64 experts 3 270 / 251, 12
//     314 / 259.  Few tokens leave no second workgroup for a CU, and 16-row tiles keep more copies
//     on their way: 256 experts, 1 token 50 / 68, 2 70 / 76, 6 164 / 179, 8 186 / 190, 12 255 / 252.
//   Fewer first-product workgroups than CUs (8 experts, k = 2), 16 / 32 / 96: 4 rows 57 / 71, 12 61
//     / 72, 16 - / 72 / 60; at 256 workgroups (16 experts) 12 rows 115 / 88 / 88.
inline int fp8_tile_rows(int64_t T, int E, int k, int I) {
  const int64_t slots = T * k, avg_rows = slots / E;
  if (avg_rows > 90) return 256;
  if (avg_rows > 20) return 96;
  if (T <= 8) return 16;
  const int64_t workgroups = (slots < E ? slots : E) * (I / kFp8Block);
  if (workgroups < kFp8Cus) return avg_rows <= 12 ? 16 : 96;
  return 32;
}

}  // namespace moe
