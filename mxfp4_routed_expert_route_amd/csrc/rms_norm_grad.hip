// Gradient of the RMS norm by its rows and by its weight.
//
// With u = s r and z = dy w: dx = r (z - u mean(z u)) + dsum, dweight = sum over rows of dy u.  A row
// is read once; its two sums, of s^2 and of z s, are reduced together.  A workgroup goes over many
// rows, keeps its part of dweight in registers and leaves one partial row of it, in an order that
// the sizes alone set; a second kernel adds the partial rows.
//
// Bound by memory: 8191 x 4096 with dsum moves 268 MB in 55 us (4.9 TB/s; the rows 51.0, the partial rows'
// sum 4.2).  77 x 2064 is two launches in a chain, 3.4 and 2.6 us.  Beyond H = 16384 the row's parts of
// dweight alone take the 128 registers of a lane: 33 of them spill (88 beyond 32768), and the row is read
// twice: 1024 x 32768 with dsum 106 us for 268 MB.  At H = 1024 a row is two wavefronts, a chunk a lane, and
// waits for its barrier: 8191 rows 19.5 us for 67 MB.
#include "block.h"
#include "block_plan.h"
#include "norm_core.h"

namespace moe {
namespace {

// What a thread holds of a row; from C = 4 on a row is read twice instead, the second time from cache.
template <int C>
struct GradRow {
  uint4 s[C], g[C], e[C];   // s, dy, dsum
};

template <int kLanes, int C>
__global__ __launch_bounds__(kLanes ? 256 : 1024) void norm_grad_kernel(NormGradArgs a) {
  constexpr int kRows = kLanes ? 256 / kLanes : 1;   // of a workgroup at a time
  constexpr bool kKeep = C <= 2;   // the row, and the weights
  __shared__ float2 sums[3][kMaxWaves];
  __shared__ float part[kLanes ? 256 * 8 : 1];
  const int T = kLanes ? kLanes : blockDim.x;
  const int t = kLanes ? threadIdx.x % kLanes : threadIdx.x;
  const int sub = kLanes ? threadIdx.x / kLanes : 0;
  float weights[kKeep ? C : 1][8], acc[C][8];
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
  auto load_weights = [&](int i, float (&w)[8]) {
    const int col = 8 * (t + T * i);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 0.f;
    if (col < a.H) load_weight8(a.w, a.w_f32, col, w);
  };
  auto load_all_weights = [&]() {
    if constexpr (kKeep)
#pragma unroll
      for (int i = 0; i < C; ++i) load_weights(i, weights[i]);
  };
  auto scale_weights = [&](float by) {
    if constexpr (kKeep)
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) weights[i][j] *= by;
  };
  load_all_weights();
  auto load = [&](int64_t row, int i, uint4& s, uint4& g, uint4& e) {
    const int col = 8 * (t + T * i);
    s = g = e = make_uint4(0u, 0u, 0u, 0u);
    if (row < a.rows && col < a.H) {
      s = *reinterpret_cast<const uint4*>(a.s + row * a.s_stride + col);
      g = *reinterpret_cast<const uint4*>(a.dy + row * a.H + col);
      if (a.dsum != nullptr) e = *reinterpret_cast<const uint4*>(a.dsum + row * a.H + col);
    }
  };
  // chunk i of the row: s, dy, dsum, w
  auto chunk = [&](const GradRow<C>& r, int64_t row, int i, float (&u)[8], float (&d)[8], float (&e)[8], float (&w)[8]) {
    if constexpr (kKeep) {
      unpack_bf16x8(r.s[i], u);
      unpack_bf16x8(r.g[i], d);
      unpack_bf16x8(r.e[i], e);
    } else {
      uint4 s4, g4, e4;
      load(row, i, s4, g4, e4);
      unpack_bf16x8(s4, u);
      unpack_bf16x8(g4, d);
      unpack_bf16x8(e4, e);
    }
    if constexpr (kKeep) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = weights[i][j];
    } else {
      load_weights(i, w);
    }
  };
  auto both = [&](const GradRow<C>& r, int64_t row, float f) {
    float2 v = make_float2(0.f, 0.f);   // of s^2, of z s
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float u[8], d[8], e[8], w[8];
      chunk(r, row, i, u, d, e, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u[j] *= f;
        v.x = fmaf(u[j], u[j], v.x);
        v.y = fmaf(d[j] * w[j], u[j], v.y);
      }
    }
    return v;
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  int turn = 0;
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * kRows; row0 < a.rows; row0 += step) {   // uniform
    const int64_t row = row0 + sub;
    GradRow<C> r;
    if constexpr (kKeep)
#pragma unroll
      for (int i = 0; i < C; ++i) load(row, i, r.s[i], r.g[i], r.e[i]);
    float2 v = row_sum<kLanes>(both(r, row, 1.0f), sums[turn]);   // two in turn: one barrier a row
    turn ^= 1;
    const float f = row_factor(v.x, a.eps);
    if (f != 1.0f) {   // uniform over the threads of a row
      v = row_sum<kLanes>(both(r, row, f), sums[2]);
      if constexpr (kLanes == 0) __syncthreads();   // sums[2] may be next in line too
    }
    // a row that is not there adds zeros (its zeros with an eps of 0 would be NaN)
    const float rstd = row < a.rows ? row_rstd(v.x, a.H, a.eps, f) : 0.f;
    // u = s p r, dx = r (p z - u c) + dsum: c is p mean(z u).  p is 1 but where 1 / rms is past fp32's largest
    // value, in subnormal rows without eps.
    float p = 1.0f, r1 = f * rstd, c = rstd * v.y / static_cast<float>(a.H);
    const bool large = r1 >= 0x1p120f;
    if (__builtin_expect(large, false)) {   // uniform over the threads of a row
      p = 0x1p24f;   // 1 / rms is 2^141 at most
      r1 = f * 0x1p-24f * rstd;
      c *= p;
      scale_weights(p);
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int col = 8 * (t + T * i);
      float u[8], d[8], e[8], w[8];
      chunk(r, row, i, u, d, e, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u[j] = u[j] * p * r1;
        acc[i][j] = fmaf(d[j], u[j], acc[i][j]);
        if (!kKeep) w[j] *= p;
        d[j] = fmaf(r1, fmaf(-u[j], c, d[j] * w[j]), e[j]);
      }
      if (a.dx != nullptr && row < a.rows && col < a.H)
        *reinterpret_cast<uint4*>(a.dx + row * a.H + col) = pack_bf16x8(d);
    }
    if (__builtin_expect(large, false)) load_all_weights();
  }
  if (a.dw == nullptr) return;
  float* out = a.part + static_cast<int64_t>(blockIdx.x) * a.H;
  if constexpr (kLanes == 0) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int col = 8 * (t + T * i);
      if (col < a.H) {
        *reinterpret_cast<float4*>(out + col) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
        *reinterpret_cast<float4*>(out + col + 4) = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
      }
    }
  } else {   // the rows' sums at element 8 t + j: [row][j][t]
#pragma unroll
    for (int j = 0; j < 8; ++j) part[(sub * 8 + j) * kLanes + t] = acc[0][j];
    __syncthreads();
    for (int e = threadIdx.x; e < 8 * kLanes; e += 256) {
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < kRows; ++k) v += part[k * 8 * kLanes + e];
      const int to = 8 * (e % kLanes) + e / kLanes;
      if (to < a.H) out[to] = v;
    }
  }
}

// dweight: 32 columns a workgroup, the partial rows dealt to 128 groups of 8 lanes.
__global__ __launch_bounds__(1024) void norm_grad_sum_kernel(const float* __restrict__ part, int groups, int H,
                                                             float* __restrict__ dw) {
  __shared__ float4 lds[128][8];
  const int lane = threadIdx.x & 7, group = threadIdx.x >> 3;
  const int col = 32 * blockIdx.x + 4 * lane;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float4 o) { v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w; };
  if (col < H) {   // H is a multiple of 8
    const float* p = part + col;
    int i = group;
    for (; i + 384 < groups; i += 512) {   // four loads on their way at once
      float4 o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = *reinterpret_cast<const float4*>(p + static_cast<int64_t>(i + 128 * k) * H);
#pragma unroll
      for (int k = 0; k < 4; ++k) add(o[k]);
    }
    for (; i < groups; i += 128) add(*reinterpret_cast<const float4*>(p + static_cast<int64_t>(i) * H));
  }
  lds[group][lane] = v;
  __syncthreads();
  if (threadIdx.x >= 64) return;   // one wavefront: groups 0 .. 7
#pragma unroll
  for (int i = 1; i < 16; ++i) add(lds[group + 8 * i][lane]);
#pragma unroll
  for (int d = 8; d <= 32; d *= 2)
    add(make_float4(__shfl_xor(v.x, d, 64), __shfl_xor(v.y, d, 64), __shfl_xor(v.z, d, 64), __shfl_xor(v.w, d, 64)));
  if (group == 0 && col < H) *reinterpret_cast<float4*>(dw + col) = v;
}

template <int kLanes, int C>
hipError_t launch(const NormGradArgs& a, hipStream_t stream) {
  const int threads = kLanes ? 256 : norm_threads(a.H, C), per = kLanes ? 256 / kLanes : 1;
  const int64_t need = (a.rows + per - 1) / per, most = norm_grad_groups(a.rows, a.H);
  const int groups = static_cast<int>(need < most ? need : most);
  if (groups > 0) {
    norm_grad_kernel<kLanes, C><<<dim3(groups), dim3(threads), 0, stream>>>(a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || a.dw == nullptr) return err;
  }
  norm_grad_sum_kernel<<<dim3((a.H + 31) / 32), dim3(1024), 0, stream>>>(a.part, groups, a.H, a.dw);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm_grad(const NormGradArgs& a, hipStream_t stream) {
  if (a.rows == 0 && a.dw == nullptr) return hipSuccess;
  if (a.H <= 512) {
    switch (norm_lanes(a.H)) {
      case 16: return launch<16, 1>(a, stream);
      case 32: return launch<32, 1>(a, stream);
      default: return launch<64, 1>(a, stream);
    }
  }
  // chunks a thread, 1 / 2, with dsum: 8191 x 1024 20.1 us / 20.3, 8191 x 2048 33.3 / 34.1, 8191 x 4096 55.5 / 54.9,
  // 4096 x 8192 62.1 / 61.2; the next row on its way while one is worked on gains nothing (57.4 / 56.2)
  if (a.H <= 4096) return launch<0, 1>(a, stream);
  if (a.H <= 16384) return launch<0, 2>(a, stream);
  if (a.H <= 32768) return launch<0, 4>(a, stream);
  return launch<0, 8>(a, stream);
}

}  // namespace moe
