// Gradient of the RMS norm by its rows and by its weight.
//
// With u = s r and z = dy w: dx = r (z - u mean(z u)) + dsum, dweight = sum over rows of dy u.  A row
// is read once; its two sums, of s^2 and of z s, are reduced together.  A workgroup goes over many
// rows, keeps its part of dweight in registers and leaves one partial row of it, in an order that
// the sizes alone set; a second kernel adds the partial rows.
#include "block.h"
#include "block_plan.h"
#include "norm_core.h"

namespace moe {
namespace {

template <int T, int C, int W>
__global__ __launch_bounds__(T * W) void norm_grad_kernel(NormGradArgs a) {
  static_assert(T == 64 || W == 1, "a barrier is for one row");
  __shared__ float sums[4][T / 64];
  __shared__ float part[W > 1 ? W * 64 * 8 : 1];
  const int t = threadIdx.x % T, wave = threadIdx.x / T;
  float acc[C][8];
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
  const int64_t step = static_cast<int64_t>(gridDim.x) * W;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * W + wave; row < a.rows; row += step) {
    const uint16_t* s_row = a.s + row * a.s_stride;
    const int64_t at = row * a.H;
    uint4 s[C], g[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int col = 8 * (t + T * i);
      s[i] = g[i] = make_uint4(0u, 0u, 0u, 0u);
      if (col < a.H) {
        s[i] = *reinterpret_cast<const uint4*>(s_row + col);
        g[i] = *reinterpret_cast<const uint4*>(a.dy + at + col);
      }
    }
    auto both = [&](float f, float& ss, float& dot) {
      ss = dot = 0.f;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int col = 8 * (t + T * i);
        float u[8], d[8], w[8];
        unpack_bf16x8(s[i], u);
        unpack_bf16x8(g[i], d);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = 0.f;
        if (col < a.H) load_weight8(a.w, a.w_f32, col, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          u[j] *= f;
          ss = fmaf(u[j], u[j], ss);
          dot = fmaf(d[j] * w[j], u[j], dot);
        }
      }
    };
    float ss, dot;
    both(1.0f, ss, dot);
    ss = row_sum<T>(ss, sums[0]);
    dot = row_sum<T>(dot, sums[1]);
    const float f = row_factor(ss, a.eps);
    if (f != 1.0f) {   // uniform per row
      both(f, ss, dot);
      ss = row_sum<T>(ss, sums[2]);
      dot = row_sum<T>(dot, sums[3]);
    }
    if constexpr (T > 64) __syncthreads();   // the next row's sums
    const float r = row_rstd(ss, a.H, a.eps, f);
    const float c = r * dot / static_cast<float>(a.H);   // mean(z u)
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int col = 8 * (t + T * i);
      if (col >= a.H) continue;
      float u[8], d[8], w[8];
      unpack_bf16x8(s[i], u);
      unpack_bf16x8(g[i], d);
      load_weight8(a.w, a.w_f32, col, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u[j] = u[j] * f * r;
        acc[i][j] = fmaf(d[j], u[j], acc[i][j]);
        d[j] = f * r * fmaf(-u[j], c, d[j] * w[j]);
      }
      if (a.dx != nullptr) {   // uniform
        if (a.dsum != nullptr) {
          float e[8];
          unpack_bf16x8(*reinterpret_cast<const uint4*>(a.dsum + at + col), e);
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] += e[j];
        }
        *reinterpret_cast<uint4*>(a.dx + at + col) = pack_bf16x8(d);
      }
    }
  }
  if (a.dw == nullptr) return;
  float* out = a.part + static_cast<int64_t>(blockIdx.x) * a.H;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int col = 8 * (t + T * i);
    if constexpr (W == 1) {
      if (col < a.H) {
        *reinterpret_cast<float4*>(out + col) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
        *reinterpret_cast<float4*>(out + col + 4) = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
      }
    } else {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) part[(wave * 8 + j) * 64 + t] = acc[i][j];
      __syncthreads();
      for (int e = threadIdx.x; e < 512; e += T * W) {   // element 8 (e % 64) + e / 64 of the chunk
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) v += part[k * 512 + e];
        const int to = 8 * ((e & 63) + 64 * i) + (e >> 6);
        if (to < a.H) out[to] = v;
      }
    }
  }
}

// dweight: 64 columns a workgroup, the partial rows dealt to 16 groups of 16 lanes.
__global__ __launch_bounds__(256) void norm_grad_sum_kernel(const float* __restrict__ part, int groups, int H,
                                                            float* __restrict__ dw) {
  __shared__ float4 lds[16][16];
  const int lane = threadIdx.x & 15, group = threadIdx.x >> 4;
  const int col = 64 * blockIdx.x + 4 * lane;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < H)   // H is a multiple of 8
    for (int p = group; p < groups; p += 16) {
      const float4 o = *reinterpret_cast<const float4*>(part + static_cast<int64_t>(p) * H + col);
      v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
    }
  lds[group][lane] = v;
  __syncthreads();
  if (group != 0 || col >= H) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) {
    const float4 o = lds[i][lane];
    v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
  }
  *reinterpret_cast<float4*>(dw + col) = v;
}

template <int T, int C, int W>
hipError_t launch(const NormGradArgs& a, hipStream_t stream) {
  const int64_t need = (a.rows + W - 1) / W;
  const int groups = static_cast<int>(need < kNormGradGroups ? need : kNormGradGroups);
  if (groups > 0) {
    norm_grad_kernel<T, C, W><<<dim3(groups), dim3(T * W), 0, stream>>>(a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || a.dw == nullptr) return err;
  }
  norm_grad_sum_kernel<<<dim3((a.H + 63) / 64), dim3(256), 0, stream>>>(a.part, groups, a.H, a.dw);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm_grad(const NormGradArgs& a, hipStream_t stream) {
  if (a.rows == 0 && a.dw == nullptr) return hipSuccess;
  if (a.H <= 512) return launch<64, 1, 4>(a, stream);
  if (a.H <= 1024) return launch<64, 2, 4>(a, stream);
  if (a.H <= 2048) return launch<64, 4, 4>(a, stream);
  if (a.H <= 4096) return launch<64, 8, 4>(a, stream);
  if (a.H <= 8192) return launch<256, 4, 1>(a, stream);
  if (a.H <= 16384) return launch<1024, 2, 1>(a, stream);
  if (a.H <= 32768) return launch<1024, 4, 1>(a, stream);
  return launch<1024, 8, 1>(a, stream);
}

}  // namespace moe
