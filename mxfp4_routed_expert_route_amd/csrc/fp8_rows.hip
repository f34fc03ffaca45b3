// Block-scaled FP8 product for few rows: tiles of up to 16 activation rows.
//
// A workgroup takes one tile and 16 weight rows (SwiGLU: 16 gate rows and their 16 up
// rows); its wavefronts share out the 128-element runs of K, each adds up scale * partial
// product in fp32 over its runs, and the partial sums are added in wavefront order in LDS.
// The weights are the MFMA's A operand and go straight to registers, 16 rows x 64
// contiguous bytes per load.
#include "fp8.h"
#include "fp8_common.h"

namespace moe {
namespace {

constexpr int kWaves = 4;

template <int kOut>
__global__ __launch_bounds__(64 * kWaves) void rows_kernel(Fp8Product p, int n_groups) {
  constexpr bool kSwiglu = kOut == kFp8OutSwiglu;
  constexpr int kFrag = kSwiglu ? 2 : 1;
  __shared__ floatx4 part[kWaves][kFrag][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r16 = lane & 15, g = lane >> 4;
  const int64_t tile = blockIdx.x / n_groups;
  const int ng = static_cast<int>(blockIdx.x - tile * n_groups);
  int expert = 0;
  int64_t p_begin = tile * 16, p_end = p_begin + 16 < p.rows ? p_begin + 16 : p.rows;
  if (p.tiles != nullptr) {
    if (tile >= *p.n_tiles) return;   // uniform
    const RowTile rt = p.tiles[tile];
    expert = rt.expert;
    p_begin = rt.p_begin;
    p_end = rt.p_end;
  }
  // this lane's activation row
  int64_t row = p_begin + r16;
  bool valid = row < p_end;
  if (valid && p.gather != nullptr) {
    const int slot = p.gather[row];
    valid = slot >= 0 && slot < p.rows;
    row = valid ? slot / p.k_top : 0;
  }
  const int nb = (p.K + kFp8Block - 1) / kFp8Block;
  const int half = p.n / 2;
  const uint8_t* arow = p.act + (valid ? row : 0) * static_cast<int64_t>(p.K);
  const float* ascale = p.act_scale + (valid ? row : 0) * p.scale_row;
  const int64_t e_rows = static_cast<int64_t>(expert) * p.n;
  const int n_blocks = (p.n + kFp8Block - 1) / kFp8Block;
  int n0[kFrag];
  const uint8_t* wrow[kFrag];
  const float* wscale[kFrag];
  bool wvalid[kFrag];
#pragma unroll
  for (int f = 0; f < kFrag; ++f) {
    n0[f] = ng * 16 + f * half;
    const int n = n0[f] + r16;
    wvalid[f] = n < p.n;
    wrow[f] = p.w + (e_rows + (wvalid[f] ? n : 0)) * p.K;
    wscale[f] = p.w_scale + (static_cast<int64_t>(expert) * n_blocks + n0[f] / kFp8Block) * nb;
  }
  floatx4 acc[kFrag];
#pragma unroll
  for (int f = 0; f < kFrag; ++f) acc[f] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
  for (int kb = wave; kb < nb; kb += kWaves) {
    const int k0 = kb * kFp8Block + 16 * g;   // lane group g: elements 16g.. and 64 + 16g..
    const bool in0 = k0 < p.K, in1 = k0 + 64 < p.K;
    const i32x4 z = {0, 0, 0, 0};
    const i32x4 b0 = valid && in0 ? *reinterpret_cast<const i32x4*>(arow + k0) : z;
    const i32x4 b1 = valid && in1 ? *reinterpret_cast<const i32x4*>(arow + k0 + 64) : z;
    const i32x8 b = __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7);
    const float xs = valid ? ascale[kb * p.scale_k] : 0.f;
#pragma unroll
    for (int f = 0; f < kFrag; ++f) {
      const i32x4 a0 = wvalid[f] && in0 ? *reinterpret_cast<const i32x4*>(wrow[f] + k0) : z;
      const i32x4 a1 = wvalid[f] && in1 ? *reinterpret_cast<const i32x4*>(wrow[f] + k0 + 64) : z;
      const i32x8 a = __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7);
      const floatx4 d = mfma_e4m3<kOut == kFp8OutF32>(a, b);
      const float s = xs * wscale[f][kb];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[f][i] = fmaf(d[i], s, acc[f][i]);
    }
  }
#pragma unroll
  for (int f = 0; f < kFrag; ++f) part[wave][f][lane] = acc[f];
  __syncthreads();
  if (wave != 0) return;
  floatx4 sum[kFrag];
#pragma unroll
  for (int f = 0; f < kFrag; ++f) {
    sum[f] = part[0][f][lane];
    for (int w = 1; w < kWaves; ++w) sum[f] += part[w][f][lane];
  }
  if (p_begin + r16 >= p_end) return;
  const int64_t out_row = (p_begin + r16) * p.ld_out;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = ng * 16 + 4 * g + i;
    if (n >= (kSwiglu ? half : p.n)) break;
    if constexpr (kSwiglu)
      static_cast<float*>(p.out)[out_row + n] = swiglu_fp8(sum[0][i], sum[1][i], p.limit, p.clamp != 0);
    else if constexpr (kOut == kFp8OutF32)
      static_cast<float*>(p.out)[out_row + n] = sum[0][i];
    else
      static_cast<uint16_t*>(p.out)[out_row + n] = f32_to_bf16_bits(sum[0][i]);
  }
}

}  // namespace

hipError_t launch_fp8_rows(const Fp8Product& p, hipStream_t stream) {
  const int cols = p.out_kind == kFp8OutSwiglu ? p.n / 2 : p.n;
  const int n_groups = (cols + 15) / 16;
  const int64_t tiles = p.tiles ? p.tile_bound : (p.rows + 15) / 16;
  const dim3 grid(static_cast<unsigned>(tiles * n_groups)), block(64 * kWaves);
  if (p.out_kind == kFp8OutSwiglu)
    rows_kernel<kFp8OutSwiglu><<<grid, block, 0, stream>>>(p, n_groups);
  else if (p.out_kind == kFp8OutF32)
    rows_kernel<kFp8OutF32><<<grid, block, 0, stream>>>(p, n_groups);
  else
    rows_kernel<kFp8OutBf16><<<grid, block, 0, stream>>>(p, n_groups);
  return hipGetLastError();
}

}  // namespace moe
