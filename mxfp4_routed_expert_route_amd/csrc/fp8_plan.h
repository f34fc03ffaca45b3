// Tiling rules and limits of the block-scaled FP8 operators, shared by the host checks and
// the launch code.  Pure C++.
#pragma once
#include <cstdint>

#include "config.h"

namespace moe {

constexpr int32_t kFp8MaxN = 1 << 24;
constexpr int64_t kFp8MaxOut = int64_t{1} << 38;   // M * N of the dense product

// Rows per row tile of the grouped FP8 FFN.
inline int fp8_tile_rows(int64_t, int, int) { return 16; }

}  // namespace moe
