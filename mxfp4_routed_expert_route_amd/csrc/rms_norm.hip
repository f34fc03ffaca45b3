// RMS norm with the residual's addition; outputs in bf16, in E4M3 with run scales, or both.
//
// A row stays in registers from its one load to the stores.  With z = s w (exact in fp32 for
// bf16 weights) and y = z rstd, rstd is the same for a whole run of 128, so the codes are
// E4M3(448 z / max |z|): they do not wait for rstd and carry none of its rounding.  Only a run
// whose y, or z, lies below the format's floor of 2^-100 is quantised from y.  A row whose squares are
// too large for fp32 is multiplied by 2^-74 (norm_core.h), which its small elements must not be before
// they meet rstd: its y are s rstd 2^-74 w, in this order.  Where s w overflows (weights of 2^78 or more),
// what was stored is stored again, from s rstd w.  Other rows pay 0.6 to 0.9 us of 27 to 58 for it at
// 8191 x 4096: their elements stay until the results are seen.
//
// Bound by memory: with the residual and both outputs an element moves 9 bytes, 8191 x 4096 302 MB
// in 58 us (5.2 TB/s, a large copy 5.1; counters show no byte read or written twice).  A single row is
// its launch and one chain of load, sum and store: kernel 3.4 us, the host's call 5.6.
#include <type_traits>

#include "block.h"
#include "fp8_common.h"
#include "norm_core.h"

namespace moe {
namespace {

__device__ __forceinline__ uint32_t max_magnitude(uint32_t m, float v) {
  const uint32_t b = __float_as_uint(v) & 0x7FFFFFFFu;
  return b > m ? b : m;
}

template <int kLanes, int C>
__global__ __launch_bounds__(kLanes ? 256 : 1024) void rms_norm_kernel(NormArgs a) {
  __shared__ float2 lds[2][kMaxWaves];
  const int T = kLanes ? kLanes : blockDim.x;
  const int t = kLanes ? threadIdx.x % kLanes : threadIdx.x;
  const int64_t row = kLanes ? static_cast<int64_t>(blockIdx.x) * (256 / kLanes) + threadIdx.x / kLanes : blockIdx.x;
  const bool live = row < a.rows;   // lanes without a row keep the others company
  const int H = live ? a.H : 0;
  const uint16_t* x = a.x + row * a.x_stride;
  const int64_t at = row * a.H;
  uint4 s[C];
  float2 ss = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int col = 8 * (t + T * i);
    s[i] = make_uint4(0u, 0u, 0u, 0u);
    if (col < H) s[i] = *reinterpret_cast<const uint4*>(x + col);
  }
  if (a.residual != nullptr) {   // uniform
    uint4 r[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int col = 8 * (t + T * i);
      r[i] = make_uint4(0u, 0u, 0u, 0u);
      if (col < H) r[i] = *reinterpret_cast<const uint4*>(a.residual + at + col);
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int col = 8 * (t + T * i);
      float u[8], v[8];
      unpack_bf16x8(s[i], u);
      unpack_bf16x8(r[i], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] += v[j];
      s[i] = pack_bf16x8(u);
      if (a.sum != nullptr && col < H) *reinterpret_cast<uint4*>(a.sum + at + col) = s[i];
    }
  }
#pragma unroll
  for (int i = 0; i < C; ++i) {
    float u[8];
    unpack_bf16x8(s[i], u);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss.x = fmaf(u[j], u[j], ss.x);
  }
  ss = row_sum<kLanes>(ss, lds[0]);
  const float f = row_factor(ss.x, a.eps);
  if (__builtin_expect(f != 1.0f, false)) {   // uniform over the threads of a row
    ss.x = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float u[8];
      unpack_bf16x8(s[i], u);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss.x = fmaf(u[j] * f, u[j] * f, ss.x);
    }
    ss = row_sum<kLanes>(ss, lds[1]);
  }
  // Returns whether s w overflowed, in any of the thread's runs (without q, elements).
  auto finish = [&](auto in_range) {
    constexpr bool kInRange = decltype(in_range)::value;   // f is 1, and s w expected below an infinity
    const float rstd = row_rstd(ss.x, a.H, a.eps, kInRange ? 1.0f : f);
    uint32_t largest = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int col = 8 * (t + T * i);
      const bool here = col < H;
      float z[8], y[8], w[8];
      // without this the compiler keeps the elements unpacked from the sum of squares on, in twice the registers
      asm("" : "+v"(s[i].x), "+v"(s[i].y), "+v"(s[i].z), "+v"(s[i].w));
      unpack_bf16x8(s[i], z);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = 0.f;
      if (here) load_weight8(a.w, a.w_f32, col, w);
      uint32_t m = 0;   // largest |z|, on the bits
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float u = z[j];
        z[j] = (kInRange ? u : u * f) * w[j];
        y[j] = z[j] * rstd;
        if (!kInRange && (f < 1.0f || !(fabsf(z[j]) < __builtin_inff())))
          y[j] = (f < 1.0f ? u * rstd * f : u * f * rstd) * w[j];
        m = max_magnitude(m, z[j]);
      }
      if (a.y != nullptr && here) *reinterpret_cast<uint4*>(a.y + at + col) = pack_bf16x8(y);
      if (a.q != nullptr) {   // uniform
        m = row16_max_u32(m);
        const float zmax = __uint_as_float(m);
        float amax = zmax * rstd;
        const bool direct = zmax >= 0x1p-100f && amax >= 0x1p-100f && zmax < __builtin_inff();
        if (!kInRange && !direct) {   // uniform over the run
          uint32_t top = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) top = max_magnitude(top, y[j]);
          amax = __uint_as_float(row16_max_u32(top));
        }
        const bool finite = amax < __builtin_inff();   // false for NaN
        amax = finite ? fmaxf(amax, 0x1p-100f) : 1.0f;
        const RunScale r = run_scale(direct ? zmax : amax);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = run_quotient(direct ? z[j] : y[j], r);
        uint2 o = make_uint2(pack_e4m3(y[0], y[1], y[2], y[3]), pack_e4m3(y[4], y[5], y[6], y[7]));
        if (!finite) o.x = o.y = kNanCodes;
        if (here) {
          *reinterpret_cast<uint2*>(a.q + at + col) = o;
          if ((t & 15) == 0)
            a.scale[row * ((a.H + kFp8Block - 1) / kFp8Block) + col / kFp8Block] =
                finite ? amax / 448.0f : __uint_as_float(0x7FC00000u);
        }
      }
      largest = m > largest ? m : largest;
    }
    return largest >= 0x7F800000u;
  };
  bool out_of_range = f != 1.0f;   // uniform over the threads of a row
  if (__builtin_expect(!out_of_range, true)) out_of_range = finish(std::true_type{});
  if (__builtin_expect(out_of_range, false)) finish(std::false_type{});
}

template <int kLanes, int C>
hipError_t launch(NormArgs a, hipStream_t stream) {
  const int per = kLanes ? 256 / kLanes : 1;   // rows of a workgroup
  const int threads = kLanes ? 256 : norm_threads(a.H, C);
  // a launch has fewer than 2^32 threads
  const int64_t most = 1 << 21, rows = a.rows;
  const int64_t runs = (a.H + kFp8Block - 1) / kFp8Block;
  for (int64_t r = 0; r < rows; r += most) {
    a.rows = rows - r < most ? rows - r : most;
    rms_norm_kernel<kLanes, C>
        <<<dim3(static_cast<unsigned>((a.rows + per - 1) / per)), dim3(threads), 0, stream>>>(a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    a.x += most * a.x_stride;
    if (a.residual) a.residual += most * a.H;
    if (a.sum) a.sum += most * a.H;
    if (a.y) a.y += most * a.H;
    if (a.q) a.q += most * a.H, a.scale += most * runs;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t stream) {
  if (a.H <= 512) {
    switch (norm_lanes(a.H)) {
      case 16: return launch<16, 1>(a, stream);
      case 32: return launch<32, 1>(a, stream);
      default: return launch<64, 1>(a, stream);
    }
  }
  // chunks a thread, 1 / 2, residual and both outputs: 8191 x 1024 15.7 us / 15.6, 8191 x 2048 31.0 / 33.4, 8191 x
  // 4096 56.2 / 58.7 (y alone 30.8 / 28.0, E4M3 alone 34.5 / 28.4), 4096 x 8192 58.8 / 59.3 (32.5 / 29.0, 38.2 /
  // 29.7); 4 are slower (62.2 at 8191 x 4096)
  if (a.H <= 2048) return launch<0, 1>(a, stream);
  if (a.H <= 16384) return launch<0, 2>(a, stream);
  if (a.H <= 32768) return launch<0, 4>(a, stream);
  return launch<0, 8>(a, stream);
}

}  // namespace moe
