// Shared pieces of the block-scaled FP8 (OCP E4M3) kernels.
#pragma once
#include "config.h"
#include "device.h"
#include "fp8_plan.h"

namespace moe {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

// ---- quantisation of one run of 128 elements
//
// a = max(max |x|, 2^-100); scale = a / 448; q = E4M3(448 x / a), one rounding.  With
// a = m 2^e, 1 <= m < 2, the quotient is t / m for t = x * (448 2^-e) (for bf16 x exact:
// 8 + 3 significant bits).  r = RN(1 / m), q0 = t r, and one correction by the exact
// remainder fma(-q0, m, t) give the correctly rounded quotient; a quotient of an 11-bit
// by an 8-bit number that is not on a border of E4M3 is further from it than fp32's
// rounding, so rounding it again to E4M3 is one rounding of the true quotient.
// Five operations an element, where an IEEE division takes about ten.  For fp32 x (the FFN's
// h) t is rounded as well: the quotient is off by at most 2^-23 and its own rounding, under
// 2^-22, so a code is the neighbour of the nearest one where 448 x / a is that close to the
// border between them.
struct RunScale {
  float scale, c, m, r;
};

__device__ __forceinline__ RunScale run_scale(float amax) {   // amax finite
  const float a = fmaxf(amax, 0x1p-100f);
  const uint32_t bits = __float_as_uint(a), be = bits >> 23;   // be in 27 .. 254
  RunScale s;
  s.scale = a / 448.0f;
  s.c = __uint_as_float(((262u - be) << 23) | 0x600000u);      // 1.75 * 2^(8 - e)
  s.m = __uint_as_float((bits & 0x7FFFFFu) | 0x3F800000u);
  s.r = 1.0f / s.m;
  return s;
}
__device__ __forceinline__ float run_quotient(float x, const RunScale& s) {
  const float t = x * s.c;
  const float q0 = t * s.r;
  return copysignf(fmaf(fmaf(-q0, s.m, t), s.r, q0), x);   // a -0 stays one
}
// Four values to four E4M3 bytes (gfx950's converts: OCP, nearest, ties to even).
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true));
}
constexpr uint32_t kNanCodes = 0x7F7F7F7Fu;

// Maximum over the 16 lanes of a DPP row (lanes 16i .. 16i + 15), in every lane: four
// rotations of the row.
__device__ __forceinline__ uint32_t row16_max_u32(uint32_t v) {
#define MOE_ROW_ROR(CTRL)                                                                    \
  {                                                                                          \
    const uint32_t o = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(                    \
        static_cast<int>(v), static_cast<int>(v), CTRL, 0xF, 0xF, false));                   \
    v = o > v ? o : v;                                                                       \
  }
  MOE_ROW_ROR(0x128) MOE_ROW_ROR(0x124) MOE_ROW_ROR(0x122) MOE_ROW_ROR(0x121)
#undef MOE_ROW_ROR
  return v;
}

// One 128-element run of E4M3 rows, from zero: D = A . B.  Lane l holds row l % 16 of each
// operand; which 32 of the 128 elements lane group l / 16 holds does not matter as long as
// both operands agree.  D: lane l has A rows 4 (l / 16) .. + 3 of B row l % 16.
//
// kFull false (bf16 results, and h in 256-row tiles): the FP8 MFMA.  It aligns the
// products of 16 consecutive elements to the largest of them and drops what lies under
// 2^-13 of that one's power of two (measured with single pairs of products at every
// distance; the groups are then summed in fp32), so a sum is off by at most 15 2^-13 of the
// sum of its terms' magnitudes; on normal data by 1.4e-5 of its size, against bf16's 2e-3.
// kFull true (fp32 results, which would show it, and h in smaller tiles): four bf16 MFMAs on
// operands converted exactly; products and sums keep fp32's 24 bits, at about half the rate.
//
// h shows the cut too: a gate off by 1.4e-5 moves one code of h in some thousands by a step, and
// the FFN's error against 64 bits is 0.0018 to 0.0021 of y's 2-norm, with full products 0.00166,
// which is bf16's rounding.  They cost 256 experts (H = 4096, I = 2048, k = 6) 174 -> 176 us for 8 tokens
// (16-row tiles), 1028 -> 1030 for 512 (32) and 1190 -> 1219 for 2048 (96), but 1490 -> 2550 for
// 8191 skewed ones (256).  W2's product, whose result is only rounded, gains nothing by them.
__device__ __forceinline__ bf16x8 e4m3_to_bf16(int lo, int hi) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
template <bool kFull>
__device__ __forceinline__ floatx4 mfma_e4m3(i32x8 a, i32x8 b) {
  floatx4 d = {0.f, 0.f, 0.f, 0.f};
  if constexpr (kFull) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(e4m3_to_bf16(a[2 * i], a[2 * i + 1]),
                                                  e4m3_to_bf16(b[2 * i], b[2 * i + 1]), d, 0, 0, 0);
    return d;
  } else {
    // zero scale operands select the form without scales
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, d, 0, 0, 0, 0, 0, 0);
  }
}

// SiLU(min(g, L)) * clamp(u, -L, L) in fp32 (NaN passes through).
__device__ __forceinline__ float swiglu_fp8(float g, float u, float limit, bool clamp) {
  if (clamp) {
    g = g > limit ? limit : g;
    u = u > limit ? limit : (u < -limit ? -limit : u);
  }
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

}  // namespace moe
