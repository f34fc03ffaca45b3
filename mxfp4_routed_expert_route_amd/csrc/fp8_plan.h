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
//   96 / 256 rows: 256 experts 84 rows on average 1522 / 1706, 96 2004 / 1694, 128 2659 / 1745;
//     64 experts 80 423 / 441, 90 437 / 462, 96 509 / 453, 128 678 / 474.
//   32 / 96 rows: 256 experts 20 1070 / 1065, 24 1116 / 1075; 64 experts 20 277 / 296, 24 319 / 306.
//   16 / 32 rows: 256 experts 2 849 / 888, 6 1046 / 1012, 12 1143 / 1032; 64 experts 3 272 / 255, 12
//     325 / 270.  Few tokens leave no second workgroup for a CU, and 16-row tiles keep more copies
//     on their way: 256 experts, 1 token 57 / 66, 2 63 / 77, 6 172 / 187, 8 186 / 201, 12 259 / 262.
//   Fewer first-product workgroups than CUs (k = 2), 16 / 32 / 96: 8 experts 2 rows 53 / 67 / 55, 12
//     56 / 69 / 59, 20 57 / 69 / 60; 16 experts of I = 1024 8 50 / 60 / 51, 12 56 / 60 / 54, 20 56 /
//     61 / 55; at 256 workgroups (16 experts) 12 rows 117 / 92 / 92.
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
