// Sizes of the operators around the routed layer that the host checks and the launches share.
#pragma once
#include <cstddef>
#include <cstdint>

#include "config.h"

namespace moe {

constexpr int kMaxAdapters = 1024;
constexpr int kMaxRank = 256;
constexpr int kMaxSequences = 1 << 20;
constexpr int kLoraMaxN = 1 << 24;

// moe_rms_norm_grad: most workgroups, each of which leaves one partial row of dweight: 2^18 threads, were a
// row's as many as here.  The launch gives a row of 520 to 1024 elements 64 or 128 threads and one of up to 8192 512,
// so that fewer run there.  The partial rows are 4 H bytes a workgroup: up to 8.4 MB to H = 8192, then 256 of them,
// 16.8 MB at 16384 and 67 at 65536.  2^17 / 2^18 / 2^19, us: 8191 x 4096 with dsum 71.2 / 55.5 / 59.5, 1000 x 4096
// 12.9 / 12.9 / 16.1, 65536 x 128 15.0 / 14.8 / 16.6, 2048 x 16384 68.2 / 52.2 / 59.5.
inline int64_t norm_grad_groups(int64_t rows, int H) {
  int64_t threads = 256;   // of a row, or of several short ones
  while (threads < 1024 && threads * 8 < H) threads *= 2;
  const int64_t most = (1 << 18) / threads;
  return rows < most ? rows : most;
}

// moe_balance_loss: tokens per workgroup at least, and the sums that the workgroups leave.
constexpr int kBalanceMinChunk = 16;
inline int64_t balance_slots(int64_t T, int n_seqs) {
  return (T + kBalanceMinChunk - 1) / kBalanceMinChunk + n_seqs;
}
// A sequence of more (token, slot) pairs is counted by a launch of its own, in chunks of at least
// kCountChunk tokens, and has more than kLongTokens tokens: chunk c's counts of the sequence that
// begins at token t are at slot c + t / kLongTokens, no two at one.  A border of 4096 / 8192 / 16384 pairs, us:
// 65536 tokens of 256 experts, k = 8, in 64 sequences 42.2 / 42.5 / 47.1, 8191 tokens in 16 19.9 / 19.2 / 19.0.
constexpr int kShortPairs = 8192, kLongTokens = kShortPairs / kMaxK, kCountChunk = 256;
inline int64_t balance_count_slots(int64_t T) { return T / kCountChunk + T / kLongTokens + 2; }

// moe_lora_add: rows of partial inner sums, [splits of K][M], and the splits that fit them.
constexpr int64_t kLoraPartialRows = 8192;
constexpr int kLoraMaxSplits = 16;
inline size_t lora_partial_rows(int64_t M) {   // two splits at least
  return static_cast<size_t>(2 * M > kLoraPartialRows ? 2 * M : kLoraPartialRows);
}
inline int lora_max_splits(int64_t M) {
  const int64_t s = static_cast<int64_t>(lora_partial_rows(M)) / M;   // M >= 1
  return static_cast<int>(s < kLoraMaxSplits ? s : kLoraMaxSplits);
}

}  // namespace moe
