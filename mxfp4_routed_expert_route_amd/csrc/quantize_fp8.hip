// Rows to E4M3 elements with one scale per run of 128 (the rule: fp8_common.h).
//
// Sixteen lanes take a run, eight elements each: one 16-byte load,
// the run's maximum by four rotations of the 16-lane row, one 8-byte store; a wavefront
// does four runs at a time.  Bound by the traffic, 3 bytes an element: 8191 rows of 4096 (101
// MB) take 18.9 to 22.3 us by the kernel trace, 4.5 to 5.3 TB/s, where a plain copy gets 5.1; 8
// rows take 2.1 us, a launch's own time.
#include "fp8.h"
#include "fp8_common.h"

namespace moe {
namespace {

__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const uint4 d = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_bits_to_f32(w[i] & 0xFFFFu);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__global__ __launch_bounds__(256) void quantize_kernel(const uint16_t* __restrict__ x, int64_t runs, int K,
                                                       int nb, uint8_t* __restrict__ q,
                                                       float* __restrict__ scale, int64_t scale_row,
                                                       int64_t scale_k) {
  const int64_t run = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
  const int64_t row = run / nb;
  const int64_t b = run - row * nb;
  const int col = static_cast<int>(b) * kFp8Block + 8 * (threadIdx.x & 15);
  const bool here = run < runs && col < K;   // K is a multiple of 16: all eight or none
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.f;
  if (here) load8(x + row * K + col, v);
  uint32_t m = 0;   // on magnitudes as integers: NaN sorts above infinity
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = __float_as_uint(v[i]) & 0x7FFFFFFFu;
    m = a > m ? a : m;
  }
  m = row16_max_u32(m);
  const bool finite = m < 0x7F800000u;   // uniform over the run
  const RunScale s = run_scale(finite ? __uint_as_float(m) : 1.0f);
  uint2 o;
  o.x = pack_e4m3(run_quotient(v[0], s), run_quotient(v[1], s), run_quotient(v[2], s), run_quotient(v[3], s));
  o.y = pack_e4m3(run_quotient(v[4], s), run_quotient(v[5], s), run_quotient(v[6], s), run_quotient(v[7], s));
  if (!finite) o.x = o.y = kNanCodes;
  if (!here) return;
  *reinterpret_cast<uint2*>(q + row * K + col) = o;
  if ((threadIdx.x & 15) == 0) scale[row * scale_row + b * scale_k] = finite ? s.scale : __uint_as_float(0x7FC00000u);
}

}  // namespace

hipError_t launch_quantize_fp8(const uint16_t* x, int64_t rows, int K, uint8_t* q, float* scale,
                               int64_t scale_row, int64_t scale_k, hipStream_t stream) {
  const int nb = (K + kFp8Block - 1) / kFp8Block;
  // a launch has fewer than 2^32 threads: 2^24 runs at a time
  const int64_t most = (1 << 24) / nb;   // at least 2^15: K is at most 65536
  for (int64_t r = 0; r < rows; r += most) {
    const int64_t runs = (rows - r < most ? rows - r : most) * nb;
    quantize_kernel<<<dim3(static_cast<unsigned>((runs + 15) / 16)), dim3(256), 0, stream>>>(
        x + r * K, runs, K, nb, q + r * K, scale + r * scale_row, scale_row, scale_k);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace moe
