// Dense block-scaled FP8 product on small tiles, K shared out among a workgroup's wavefronts.
//
// A workgroup takes 16 MS activation rows x 16 NF weight rows.  Wavefront w takes the
// 128-element runs w, w + W, ... of K, straight to registers and kDepth runs ahead, adds up
// multiplier * partial product in fp32, and the W sums are added in wavefront order through
// LDS.  A load takes 16 rows x 64 contiguous bytes, the operand's own shape.
//
// For outputs of few tiles, which are bound by latency: the LDS-tiled kernel meets a barrier a
// step, this one none before the end.  Measured (us in a graph, N = K = 4096): 1 row 5.5, 16 rows
// 7.1 (16 x 16 LDS tiles do not exist; 32 x 32 with K in 4: 7.9).  A smaller tile than the rule's
// reads the operands more often (16 x 16 tiles, 128 rows: 37.9), a larger one leaves CUs idle
// (32 x 64 tiles, 16 rows: 14.0).  All tiles together get about 8 TB/s out of the L2s and the
// memory behind them (128 rows: 101 MB in 15.6 us less 3), which is why the LDS tiles, whose
// copies take whole lines, pass it at a long K.  More runs ahead (kDepth 4) change nothing.  A
// single row of N = K = 4096 takes 5.2 us by the kernel trace: its 16.8 MB of weights need 2.5, a
// launch's start and end about 2.
#include "fp8.h"
#include "fp8_common.h"

namespace moe {
namespace {

template <int MS, int NF, int W, int kDepth, int kOut>
__global__ __launch_bounds__(64 * W) void rows_kernel(Fp8Product p, int col_blocks) {
  constexpr bool kFull = kOut == kFp8OutF32;
  constexpr int TM = 16 * MS, cols = 16 * NF;
  extern __shared__ __attribute__((aligned(16))) unsigned char rows_lds[];
  floatx4* part = reinterpret_cast<floatx4*>(rows_lds);            // [W][MS][NF][64]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int tile = blockIdx.x / col_blocks;
  const int n0 = (blockIdx.x - tile * col_blocks) * cols;
  const int64_t p_begin = static_cast<int64_t>(tile) * TM, left = p.rows - p_begin;
  const int rows = left < TM ? static_cast<int>(left) : TM;
  const int K = p.K, nk = (K + kFp8Block - 1) / kFp8Block;
  const int n_blk = (p.n + kFp8Block - 1) / kFp8Block;

  // weights and activations: a resource on this tile's rows
  const int w_rows = p.n - n0 < cols ? p.n - n0 : cols;
  const __amdgpu_buffer_rsrc_t wrs = make_rsrc(p.w + static_cast<int64_t>(n0) * K,
                                               static_cast<uint32_t>(w_rows) * static_cast<uint32_t>(K));
  const __amdgpu_buffer_rsrc_t ars = make_rsrc(p.act + p_begin * K,
                                               static_cast<uint32_t>(rows) * static_cast<uint32_t>(K));
  uint32_t woff[NF], aoff[MS];
  const float* wscale[NF];
  const float* ascale[MS];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int n = 16 * f + r16, b = (n0 + 16 * f) / kFp8Block;
    woff[f] = n < w_rows ? static_cast<uint32_t>(n) * static_cast<uint32_t>(K) + 16u * g : kRsrcOutOfRange;
    wscale[f] = p.w_scale + static_cast<int64_t>(b < n_blk ? b : n_blk - 1) * nk;   // past n: any
  }
#pragma unroll
  for (int m = 0; m < MS; ++m) {
    const int r = 16 * m + r16;
    aoff[m] = r < rows ? static_cast<uint32_t>(r) * static_cast<uint32_t>(K) + 16u * g : kRsrcOutOfRange;
    ascale[m] = p.act_scale + (p_begin + (r < rows ? r : 0)) * p.scale_row;
  }

  struct Run {
    i32x8 a[NF], b[MS];
    float x[MS], w[NF];
  };
  auto load = [&](Run& r, int kb) {
    const int k0 = kb * kFp8Block;
    // past K (a short last run): zeros
    const bool in0 = k0 + 16 * g < K, in1 = k0 + 64 + 16 * g < K;
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const i32x4 lo = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(
          wrs, in0 ? woff[f] + k0 : kRsrcOutOfRange, 0, 0));
      const i32x4 hi = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(
          wrs, in1 ? woff[f] + k0 + 64 : kRsrcOutOfRange, 0, 0));
      r.a[f] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
#pragma unroll
    for (int m = 0; m < MS; ++m) {
      const i32x4 lo = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(
          ars, in0 ? aoff[m] + k0 : kRsrcOutOfRange, 0, 0));
      const i32x4 hi = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(
          ars, in1 ? aoff[m] + k0 + 64 : kRsrcOutOfRange, 0, 0));
      r.b[m] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
#pragma unroll
    for (int m = 0; m < MS; ++m) r.x[m] = ascale[m][kb];
#pragma unroll
    for (int f = 0; f < NF; ++f) r.w[f] = wscale[f][kb];
  };
  floatx4 acc[MS][NF];
#pragma unroll
  for (int m = 0; m < MS; ++m)
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[m][f] = floatx4{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const Run& r) {
#pragma unroll
    for (int m = 0; m < MS; ++m)
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const floatx4 d = mfma_e4m3<kFull>(r.a[f], r.b[m]);
        const float s = r.x[m] * r.w[f];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][f][i] = fmaf(d[i], s, acc[m][f][i]);
      }
  };
  Run ring[kDepth];
#pragma unroll
  for (int d = 0; d < kDepth; ++d)
    if (wave + d * W < nk) load(ring[d], wave + d * W);   // uniform
  for (int kb = wave; kb < nk; kb += kDepth * W) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      if (kb + d * W < nk) multiply(ring[d]);
      if (kb + (kDepth + d) * W < nk) load(ring[d], kb + (kDepth + d) * W);
    }
  }
#pragma unroll
  for (int m = 0; m < MS; ++m)
#pragma unroll
    for (int f = 0; f < NF; ++f) part[((wave * MS + m) * NF + f) * 64 + lane] = acc[m][f];
  __syncthreads();

  // the fragments' sums are shared out among the wavefronts
  for (int u = wave; u < MS * NF; u += W) {
    const int m = u / NF, f = u - m * NF;
    floatx4 s = part[u * 64 + lane];
#pragma unroll
    for (int w = 1; w < W; ++w) s += part[(w * MS * NF + u) * 64 + lane];
    if (16 * m + r16 >= rows) continue;
    const int c = n0 + 16 * f + 4 * g;
    const int64_t at = (p_begin + 16 * m + r16) * p.ld_out + c;
    const bool wide = p.n % 4 == 0;   // columns come in whole fours, on 8 or 16 bytes
    if constexpr (kOut == kFp8OutF32) {
      float* dst = static_cast<float*>(p.out) + at;
      if (wide && c < p.n) {
        *reinterpret_cast<floatx4*>(dst) = s;
      } else {
        for (int i = 0; i < 4; ++i)
          if (c + i < p.n) dst[i] = s[i];
      }
    } else {
      uint16_t* dst = static_cast<uint16_t*>(p.out) + at;
      if (wide && c < p.n) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
      } else {
        for (int i = 0; i < 4; ++i)
          if (c + i < p.n) dst[i] = f32_to_bf16_bits(s[i]);
      }
    }
  }
}

template <int MS, int NF, int W, int kDepth, int kOut>
hipError_t launch(const Fp8Product& p, hipStream_t stream) {
  constexpr int lds = W * MS * NF * 64 * 16;
  static_assert(lds <= 64 * 1024, "no attribute needed");
  const int col_blocks = (p.n + 16 * NF - 1) / (16 * NF);
  const int64_t tiles = (p.rows + 16 * MS - 1) / (16 * MS);
  rows_kernel<MS, NF, W, kDepth, kOut>
      <<<dim3(static_cast<unsigned>(tiles * col_blocks)), dim3(64 * W), lds, stream>>>(p, col_blocks);
  return hipGetLastError();
}

// The smallest tile of which the output has at most one per CU; nothing for larger outputs and
// for a long K.  Over a long K the LDS tiles' reads of whole lines are worth their barriers
// (launch_fp8_dense has the figures), but not against 32 x 16 tiles that leave CUs idle: this
// kernel / the 32 x 32 LDS tile, us, K = 4096: 64x1024 (128 tiles) 7.0 / 8.5, 128x1024 (256) 9.8 / 8.5.
template <int kOut>
hipError_t launch_fitting(const Fp8Product& p, hipStream_t stream, bool* done) {
  *done = true;
  auto fits = [&](int tm, int tn, int most = kFp8Cus) {
    return (p.rows + tm - 1) / tm * ((p.n + tn - 1) / tn) <= most;
  };
  if (fits(16, 16)) return launch<1, 1, 8, 2, kOut>(p, stream);
  const bool tall = p.K <= 2048, wide = p.K <= 1024;
  if (fits(32, 16, tall ? kFp8Cus : kFp8Cus * 3 / 4)) return launch<2, 1, 8, 2, kOut>(p, stream);
  if (tall && fits(32, 32)) return launch<2, 2, 8, 2, kOut>(p, stream);
  if (wide && fits(32, 64)) return launch<2, 4, 8, 1, kOut>(p, stream);
  *done = false;
  return hipSuccess;
}

}  // namespace

hipError_t launch_fp8_rows(const Fp8Product& p, hipStream_t stream, bool* done) {
  return p.out_kind == kFp8OutF32 ? launch_fitting<kFp8OutF32>(p, stream, done)
                                  : launch_fitting<kFp8OutBf16>(p, stream, done);
}

}  // namespace moe
