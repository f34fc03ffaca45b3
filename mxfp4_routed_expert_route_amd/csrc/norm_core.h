// A row's statistics for the RMS norm and its gradient.
//
// Layout.  T threads take a row, thread t elements 8 (t + T i) .. + 7 of chunk i, so a load is 16
// bytes a thread and a run of 128 elements lies in 16 neighbouring lanes of one chunk.  Rows of up
// to 512 elements take 16, 32 or 64 lanes of a wavefront (kLanes) and need no barrier; longer
// ones a workgroup of whole wavefronts (kLanes 0), as few threads as hold them.
//
// Range.  Squares of bf16 values leave fp32 beyond about 2^63 and below 2^-63.  A row whose sum of
// squares is outside [2^-80, 2^100] is multiplied by 2^100 or 2^-74 and summed again; eps
// goes with it.  Rows below, of zeros say, need that only if eps is as small.  Its price is one
// comparison a row.
#pragma once
#include "block_common.h"

namespace moe {

// What a row with the sum of squares `ss` is multiplied by; 1 for all but extreme rows.  2^-74 is the
// largest that keeps the squares of 65536 elements in range, so that the least is lost of small ones.
__device__ __forceinline__ float row_factor(float ss, float eps) {
  if (!(ss <= 0x1p100f)) return 0x1p-74f;
  return ss < 0x1p-80f && eps < 0x1p-60f ? 0x1p100f : 1.0f;
}

// 1 / sqrt(ss / H + eps f^2) of a row multiplied by f.
__device__ __forceinline__ float row_rstd(float ss, int H, float eps, float f) {
  const double mean = static_cast<double>(ss) / H + static_cast<double>(eps) * f * f;
  return static_cast<float>(1.0 / sqrt(mean));
}

constexpr int kMaxWaves = 16;   // of a workgroup

// Sums of two values over a row's threads, in all of them.  A workgroup's go through `lds`, which no
// thread may still be reading from for another sum.
template <int kLanes>
__device__ __forceinline__ float2 row_sum(float2 v, float2* lds) {
  constexpr int L = kLanes ? kLanes : 64;
  v.x = run_sum<L>(v.x);
  v.y = run_sum<L>(v.y);
  if constexpr (kLanes == 0) {
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    const int waves = blockDim.x >> 6;
    v = lds[0];
    for (int i = 1; i < waves; ++i) {
      const float2 o = lds[i];
      v.x += o.x;
      v.y += o.y;
    }
  }
  return v;
}

// Lanes of a wavefront for a row of H <= 512 elements.
inline int norm_lanes(int H) { return H <= 128 ? 16 : H <= 256 ? 32 : 64; }
// Threads for a row of H elements in chunks of 8 C.
inline int norm_threads(int H, int C) { return (H + 8 * 64 * C - 1) / (8 * 64 * C) * 64; }

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
