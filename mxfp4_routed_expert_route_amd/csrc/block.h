// Internal launchers of the operators around the routed layer (arguments are already checked).
#pragma once
#include <hip/hip_runtime.h>
#include <cstddef>
#include <cstdint>

namespace moe {

struct NormArgs {
  const uint16_t* x;
  int64_t x_stride;
  const uint16_t* residual;
  int64_t rows;
  int H;
  const void* w;
  int w_f32;
  float eps;
  uint16_t* sum;
  uint16_t* y;
  uint8_t* q;
  float* scale;
};
hipError_t launch_rms_norm(const NormArgs& a, hipStream_t stream);

struct NormGradArgs {
  const uint16_t* s;
  int64_t s_stride;
  int64_t rows;
  int H;
  const void* w;
  int w_f32;
  float eps;
  const uint16_t* dy;
  const uint16_t* dsum;
  uint16_t* dx;
  float* dw;
  float* part;   // [norm_grad_groups(rows, H)][H]
};
hipError_t launch_rms_norm_grad(const NormGradArgs& a, hipStream_t stream);

struct BalanceArgs {
  const void* logits;
  int64_t T;
  int E, k, sigmoid;
  const int32_t* ids;       // nullptr: counts are given
  const int32_t* offsets;   // nullptr: one sequence
  int n_seqs;
  float* loss;
  int32_t* counts;
  const float* dloss;
  const void* add;
  void* dlogits;            // nullptr: no gradient
  double* slots;            // sums over a chunk's tokens of a sequence, at [chunk + sequence]
  int32_t* partial;         // counts of long sequences by chunk: block_plan.h
};
hipError_t launch_balance(const BalanceArgs& a, bool bf16, hipStream_t stream);

hipError_t launch_lora_group(const int32_t* adapter, int64_t M, int L, int32_t* offsets, int32_t* rows,
                             hipStream_t stream);

struct LoraArgs {
  const uint16_t* x;
  int64_t x_stride, M;
  int K, N, R, L;
  const uint16_t* a;
  const uint16_t* b;
  const float* scaling;
  const int32_t* offsets;
  const int32_t* rows;
  const void* base;
  int64_t base_stride;
  void* y;
  int64_t y_stride;
  float* v;                 // inner sums in the grouped order, [splits of K][M][R]
};
hipError_t launch_lora_add(const LoraArgs& a, bool f32, hipStream_t stream);
// lora_tall.hip: sets *done, or leaves the call to others (few rows, R > 64).
hipError_t launch_lora_tall(const LoraArgs& a, bool f32, int wide, hipStream_t stream, bool* done);

}  // namespace moe
