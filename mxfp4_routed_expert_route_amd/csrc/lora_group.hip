// The rows of a batch in their adapters' order.
#include "block.h"
#include "block_plan.h"
#include "lora_core.h"

namespace moe {
namespace {

// Rows of a wavefront, at least.  64 / 128 / 512, us: 512 rows and 64 adapters 3.9 / 4.9 / 7.2, 8191 and 8 6.7 /
// 8.2 / 8.6, 65536 and 64 14.3 / 15.9 / 17.1.  One workgroup for all of them takes 12.6 and 79 for the last two.
constexpr int kGroupRows = 64;

// A stable counting sort.  A workgroup deals out a stretch of rows, each of its wavefronts a part of that:
// the wavefronts count their parts, the counts become first positions, and the rows follow, 64 at
// a time; rows of the same adapter find one another by a ballot for each bit of it.  Of the other
// stretches a workgroup counts all rows by itself, which spares a launch between counting and dealing.
//
// Bound by latency: a serving step's few hundred rows take little more than an empty kernel.
template <int W>
__global__ __launch_bounds__(64 * W) void group_kernel(const int32_t* __restrict__ adapter, int M, int L, int each,
                                                       int32_t* __restrict__ offsets, int32_t* __restrict__ rows) {
  constexpr int kAhead = 8;        // rounds of 64 rows whose ids are on their way at once
  extern __shared__ int place[];   // [W][L + 1], in front of this stretch [L + 1], behind it [L + 1]; bin L: no adapter
  __shared__ int wave_sums[W];
  __shared__ int carry;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int bins = L + 1;
  int* mine = place + wave * bins;
  int* front = place + W * bins;
  int* behind = front + bins;
  // `each` rows a wavefront, a multiple of 64
  const int64_t stretch = static_cast<int64_t>(each) * W * blockIdx.x, stretch_end = stretch + each * W;
  const int64_t begin = stretch + wave * each < M ? stretch + wave * each : M;
  const int64_t end = begin + each < M ? begin + each : M;
  auto bin_of = [&](int id) { return static_cast<unsigned>(id) < static_cast<unsigned>(L) ? id : L; };
  // Counts rows i0 + 64 step j + lane < i1, for all j.
  auto count = [&](int* to, int64_t i0, int64_t i1, int step) {
    for (; i0 < i1; i0 += 64 * kAhead * step) {   // uniform per wavefront
      int bin[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int64_t i = i0 + 64 * step * j + lane;
        bin[j] = adapter[i < i1 ? i : i0];
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int64_t at = i0 + 64 * step * j;
        const int b = bin_of(bin[j]), b0 = __builtin_amdgcn_readfirstlane(b);
        const uint64_t here = __builtin_amdgcn_ballot_w64(at + lane < i1);
        if (__builtin_amdgcn_ballot_w64(at + lane < i1 && b != b0) == 0) {   // one adapter's, as in a prompt
          if (lane == 0 && here != 0) atomicAdd(&to[b0], __popcll(here));
        } else if (at + lane < i1) {
          atomicAdd(&to[b], 1);
        }
      }
    }
  };
  const int first_bin = begin + lane < end ? bin_of(adapter[begin + lane]) : -1;   // of the first 64 rows
  for (int i = threadIdx.x; i < (W + 2) * bins; i += 64 * W) place[i] = 0;
  if (threadIdx.x == 0) carry = 0;
  __syncthreads();
  if (first_bin >= 0) atomicAdd(&mine[first_bin], 1);
  count(mine, begin + 64, end, 1);
  if (gridDim.x > 1) {   // uniform
    count(front, 64 * wave, stretch < M ? stretch : M, W);
    count(behind, stretch_end + 64 * wave, M, W);
  }
  __syncthreads();
  // exclusive sums over bins, 64 W of them at a time
  for (int b0 = 0; b0 < bins; b0 += 64 * W) {
    const int b = b0 + threadIdx.x;
    int n = 0;
    if (b < bins)
      for (int w = 0; w < W + 2; ++w) n += place[w * bins + b];
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
      if (blockIdx.x == 0) offsets[b] = first;   // bin L: the rows that have one end here
      first += front[b];
      for (int w = 0; w < W; ++w) {
        const int c = place[w * bins + b];
        place[w * bins + b] = first;
        first += c;
      }
    }
    __syncthreads();
  }
  const int bits = 32 - __builtin_clz(static_cast<unsigned>(L));   // of a bin
  int next = first_bin;
  for (int64_t i0 = begin; i0 < end; i0 += 64) {   // uniform per wavefront
    const int64_t i = i0 + lane;
    const bool here = i < end;
    const int bin = next;
    if (i0 + 64 < end) next = bin_of(adapter[i + 64 < end ? i + 64 : i0]);
    uint64_t same = __builtin_amdgcn_ballot_w64(here);
    for (int bit = 0; bit < bits; ++bit) {   // uniform
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
  // 16 wavefronts where their counts fit 64 KB of LDS, else 8
  const size_t lds = static_cast<size_t>(L + 1) * sizeof(int);
  const int waves = 18 * lds <= 64 * 1024 - 1024 ? 16 : 8;
  // up to 256 workgroups
  const int64_t unit = 64 * waves;
  int64_t each = (M + 256 * unit - 1) / (256 * unit) * 64;
  if (each < kGroupRows) each = kGroupRows;
  int64_t groups = (M + each * waves - 1) / (each * waves);
  if (groups < 1) groups = 1;
  const dim3 grid(static_cast<unsigned>(groups));
  if (waves == 16)
    group_kernel<16><<<grid, dim3(1024), 18 * lds, stream>>>(adapter, static_cast<int>(M), L, static_cast<int>(each),
                                                             offsets, rows);
  else
    group_kernel<8><<<grid, dim3(512), 10 * lds, stream>>>(adapter, static_cast<int>(M), L, static_cast<int>(each),
                                                           offsets, rows);
  return hipGetLastError();
}

}  // namespace moe
