// The rows of a batch in their adapters' order.
#include "block.h"
#include "block_plan.h"
#include "lora_core.h"

namespace moe {
namespace {

// A stable counting sort by one workgroup.  Each wavefront counts its own stretch of rows, the counts
// become first positions, and each wavefront then deals its rows out, 64 at a time: rows of the
// same adapter find one another by a ballot for each bit of it.
template <int W>
__global__ __launch_bounds__(64 * W) void group_kernel(const int32_t* __restrict__ adapter, int M, int L,
                                                       int32_t* __restrict__ offsets, int32_t* __restrict__ rows) {
  extern __shared__ int place[];   // [W][L + 1]; bin L: no adapter
  __shared__ int wave_sums[W];
  __shared__ int carry;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int bins = L + 1;
  for (int i = threadIdx.x; i < W * bins; i += 64 * W) place[i] = 0;
  if (threadIdx.x == 0) carry = 0;
  __syncthreads();
  const int64_t each = ((static_cast<int64_t>(M) + W - 1) / W + 63) / 64 * 64;
  const int64_t begin = wave * each < M ? wave * each : M;
  const int64_t end = begin + each < M ? begin + each : M;
  int* mine = place + wave * bins;
  auto bin_of = [&](int64_t i) {
    const int id = adapter[i];
    return static_cast<unsigned>(id) < static_cast<unsigned>(L) ? id : L;
  };
  const int first_bin = begin + lane < end ? bin_of(begin + lane) : -1;   // of the first 64 rows
  for (int64_t i = begin + lane; i < end; i += 64) atomicAdd(&mine[i < begin + 64 ? first_bin : bin_of(i)], 1);
  __syncthreads();
  // exclusive sums over (bin, wavefront), 64 W bins at a time
  for (int b0 = 0; b0 < bins; b0 += 64 * W) {
    const int b = b0 + threadIdx.x;
    int n = 0;
    if (b < bins)
      for (int w = 0; w < W; ++w) n += place[w * bins + b];
    int upto = n;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int o = __shfl_up(upto, d, 64);
      if (lane >= d) upto += o;
    }
    if (lane == 63) wave_sums[wave] = upto;
    __syncthreads();
    int first = carry + upto - n;
    for (int w = 0; w < wave; ++w) first += wave_sums[w];
    __syncthreads();
    if (threadIdx.x == 64 * W - 1) carry = first + n;
    if (b < bins) {
      offsets[b] = first;   // bin L: the rows that have one end here
      for (int w = 0; w < W; ++w) {
        const int c = place[w * bins + b];
        place[w * bins + b] = first;
        first += c;
      }
    }
    __syncthreads();
  }
  for (int64_t i0 = begin; i0 < end; i0 += 64) {   // uniform per wavefront
    const int64_t i = i0 + lane;
    const bool here = i < end;
    const int bin = i0 == begin ? first_bin : here ? bin_of(i) : -1;
    uint64_t same = __builtin_amdgcn_ballot_w64(here);
#pragma unroll
    for (int bit = 0; bit < 11; ++bit) {   // bins number at most 1025
      const uint64_t set = __builtin_amdgcn_ballot_w64((bin >> bit) & 1);
      same &= (bin >> bit) & 1 ? set : ~set;
    }
    if (here) {
      const int rank = __popcll(same & ((1ull << lane) - 1));
      const int at = mine[bin];
      rows[at + rank] = static_cast<int32_t>(i);
      // the lowest lane moves the bin on; a wavefront's LDS accesses are in order, the read is before
      if (rank == 0) mine[bin] = at + __popcll(same);
    }
    wave_sync_lds();
  }
}

}  // namespace

hipError_t launch_lora_group(const int32_t* adapter, int64_t M, int L, int32_t* offsets, int32_t* rows,
                             hipStream_t stream) {
  // 16 wavefronts where their counts fit 48 KB of LDS, else 8
  const int m = static_cast<int>(M);
  const size_t lds = static_cast<size_t>(L + 1) * sizeof(int);
  if (16 * lds <= 48 * 1024)
    group_kernel<16><<<dim3(1), dim3(1024), 16 * lds, stream>>>(adapter, m, L, offsets, rows);
  else
    group_kernel<8><<<dim3(1), dim3(512), 8 * lds, stream>>>(adapter, m, L, offsets, rows);
  return hipGetLastError();
}

}  // namespace moe
