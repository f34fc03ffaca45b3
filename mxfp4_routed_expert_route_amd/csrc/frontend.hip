// The routing front-end in one launch for small batches: top-k routing, the
// token x expert bit matrix and the expert offsets / permutations, with exactly
// the outputs of moe_route, moe_build_bitmatrix and moe_expert_offsets.
//
// One workgroup of 16 wavefronts, for T <= 64 tokens:
//   1. wavefront w routes tokens w, w+16, w+32, w+48 (route_token);
//   2. the bit matrix is built in LDS: thread i owns entry i = t*k + j; the logical
//      block is the T*k entries, and threads past it (padding) stay inactive
//      (txtmix.com article, §3; aihot.vn README translation, "Định tuyến MXFP4");
//   3. every wavefront takes the column masks of 64 experts over the T rows
//      (lane = token); wavefront 0 scans their popcounts into counts and offsets
//      and writes each slot's row p = offsets[e] + rank of the token within e.
// With a plan buffer, wavefront 0 also writes the grouped FFN's row-tile plan
// (moe_forward_mxfp4), which saves the FFN its plan launch.  Larger batches run
// the routing kernel, which then also writes the bit matrix, and the offsets
// kernels of the separate call.
#include "group_core.h"
#include "launch.h"

namespace moe {
namespace {

template <int EPL>
__global__ __launch_bounds__(1024) void frontend_small_kernel(
    const float* __restrict__ logits, int T, int E, int k, int words, int32_t* __restrict__ ids,
    float* __restrict__ weights, uint32_t* __restrict__ bm, int32_t* __restrict__ counts,
    int32_t* __restrict__ offsets, int32_t* __restrict__ gather, int32_t* __restrict__ scatter,
    int tile_rows, int tile_bound, int32_t* __restrict__ n_tiles, RowTile* __restrict__ tiles) {
  __shared__ FrontLds lds;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n_waves = blockDim.x >> 6;

  // 1. routing
  for (int t = wave; t < T; t += n_waves) {
    int id;
    float w;
    route_token<EPL>(logits + static_cast<int64_t>(t) * E, E, k, lane, id, w);
    if (lane < k) {
      ids[t * k + lane] = id;
      weights[t * k + lane] = w;
      lds.ids[t * k + lane] = id;
    }
  }
  group_small<EPL>(lds, T, E, k, words, bm, counts, offsets, gather, scatter, tile_rows, tile_bound,
                   n_tiles, tiles);
}

}  // namespace

hipError_t launch_route_and_group(const float* logits, int64_t T, int E, int k, int32_t* ids,
                                  float* weights, uint32_t* bm, int32_t* counts, int32_t* offsets,
                                  int32_t* gather, int32_t* scatter, void* ws, hipStream_t stream,
                                  const PlanOut* plan, bool* plan_written,
                                  const SplitArgs* split, bool* split_done) {
  if (plan_written) *plan_written = false;
  if (split_done) *split_done = false;
  if (T > kFrontMaxTokens) {
    hipError_t err = launch_route(logits, T, E, k, ids, weights, stream, bm, split);
    if (err != hipSuccess) return err;
    if (split_done) *split_done = split != nullptr;
    return launch_offsets(bm, ids, T, E, k, counts, offsets, gather, scatter, ws, stream, plan,
                          plan_written);
  }
  const int words = (E + 31) / 32;
  const int epl = (E + 63) / 64;
  const int t = static_cast<int>(T);
  const int tile_rows = plan ? plan->tile_rows : 1;
  const int tile_bound = plan ? static_cast<int>(plan->tile_bound) : 0;
  int32_t* n_tiles = plan ? plan->n_tiles : nullptr;
  RowTile* tiles = plan ? static_cast<RowTile*>(plan->tiles) : nullptr;
  if (epl <= 1)
    frontend_small_kernel<1><<<1, 1024, 0, stream>>>(logits, t, E, k, words, ids, weights, bm,
                                                     counts, offsets, gather, scatter,
                                                     tile_rows, tile_bound, n_tiles, tiles);
  else if (epl <= 2)
    frontend_small_kernel<2><<<1, 1024, 0, stream>>>(logits, t, E, k, words, ids, weights, bm,
                                                     counts, offsets, gather, scatter,
                                                     tile_rows, tile_bound, n_tiles, tiles);
  else if (epl <= 4)
    frontend_small_kernel<4><<<1, 1024, 0, stream>>>(logits, t, E, k, words, ids, weights, bm,
                                                     counts, offsets, gather, scatter,
                                                     tile_rows, tile_bound, n_tiles, tiles);
  else if (epl <= 8)
    frontend_small_kernel<8><<<1, 1024, 0, stream>>>(logits, t, E, k, words, ids, weights, bm,
                                                     counts, offsets, gather, scatter,
                                                     tile_rows, tile_bound, n_tiles, tiles);
  else
    frontend_small_kernel<16><<<1, 1024, 0, stream>>>(logits, t, E, k, words, ids, weights, bm,
                                                      counts, offsets, gather, scatter,
                                                      tile_rows, tile_bound, n_tiles, tiles);
  const hipError_t err = hipGetLastError();
  if (err == hipSuccess && plan_written) *plan_written = tiles != nullptr;
  return err;
}

}  // namespace moe
