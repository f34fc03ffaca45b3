// Shared pieces of the kernels around the routed layer (norm, balance loss, adapters).
#pragma once
#include "config.h"
#include "device.h"

namespace moe {

template <int kCtrl>
__device__ __forceinline__ float dpp_f32(float v) {
  const int u = __float_as_int(v);
  return __int_as_float(__builtin_amdgcn_update_dpp(u, u, kCtrl, 0xF, 0xF, false));
}

// Sum and maximum over aligned runs of `L` lanes (16, 32 or 64), in every lane of the run: rotations
// of the 16-lane rows, then swaps of rows and of halves.  Every lane adds the same two values at
// each step, in either order, so all of them hold the same bits.
template <int L, class Op>
__device__ __forceinline__ float run_reduce(float v, Op op) {
  static_assert(L == 16 || L == 32 || L == 64);
  v = op(v, dpp_f32<0x128>(v));
  v = op(v, dpp_f32<0x124>(v));
  v = op(v, dpp_f32<0x122>(v));
  v = op(v, dpp_f32<0x121>(v));
  if constexpr (L >= 32) {
    const uint32_t u = __float_as_uint(v);
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  if constexpr (L == 64) {
    const uint32_t u = __float_as_uint(v);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    v = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  return v;
}
template <int L>
__device__ __forceinline__ float run_sum(float v) {
  return run_reduce<L>(v, [](float a, float b) { return a + b; });
}
template <int L>
__device__ __forceinline__ float run_max(float v) {
  return run_reduce<L>(v, [](float a, float b) { return fmaxf(a, b); });
}

__device__ __forceinline__ void unpack_bf16x8(uint4 d, float (&v)[8]) {
  const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_bits_to_f32(w[i] & 0xFFFFu);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack_bf16x8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

}  // namespace moe
