// A row's statistics for the RMS norm and its gradient.
//
// Layout.  T lanes take a row; lane t holds elements 8 (t + T i) .. + 7 of chunk i, so a load is 16
// bytes a lane and a run of 128 elements lies in 16 neighbouring lanes of one chunk.
//
// Range.  Squares of bf16 values leave fp32 beyond about 2^63 and below 2^-63.  A row whose sum of
// squares is outside [2^-80, 2^100] is multiplied by a power of two and summed again; eps
// goes with it.  Rows below, of zeros say, need that only if eps is as small.  Its price is one
// comparison a row.
#pragma once
#include "block_common.h"

namespace moe {

constexpr int kNormPower = 100;

struct RowFactor {
  float f;       // the row is multiplied by this power of two
  double f2;
};

// What a row with the sum of squares `ss` is multiplied by; 1 for all but extreme rows.
__device__ __forceinline__ float row_factor(float ss, float mean_eps_floor) {
  if (!(ss <= 0x1p100f)) return 0x1p-100f;
  return ss < 0x1p-80f && mean_eps_floor < 0x1p-60f ? 0x1p100f : 1.0f;
}

// 1 / sqrt(ss / H + eps f^2) of a row multiplied by f.
__device__ __forceinline__ float row_rstd(float ss, int H, float eps, float f) {
  const double mean = static_cast<double>(ss) / H + static_cast<double>(eps) * f * f;
  return static_cast<float>(1.0 / sqrt(mean));
}

// Sum over a row's T lanes (one wavefront or a workgroup), in all of them.  `lds` holds T / 64
// floats that no other sum since the last barrier has used.
template <int T>
__device__ __forceinline__ float row_sum(float v, float* lds) {
  v = run_sum<64>(v);
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < T / 64; ++i) v += lds[i];
  }
  return v;
}

// Eight weights from element `at` on.
__device__ __forceinline__ void load_weight8(const void* w, bool f32, int at, float (&v)[8]) {
  if (f32) {   // uniform
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + at);
    const float4 a = p[0], b = p[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    unpack_bf16x8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + at), v);
  }
}

}  // namespace moe
