// Grouping of a small batch's rows by expert in one workgroup, shared by the one-launch
// front-ends (frontend.hip: plain top-k; route_scored.hip: scored routing): the token x
// expert bit matrix, the expert counts and offsets and the gather / scatter
// permutations of T <= 64 routed tokens, and optionally the grouped FFN's row-tile plan.
#pragma once
#include "config.h"
#include "routing_core.h"

namespace moe {

constexpr int kFrontMaxTokens = 64;

struct FrontLds {
  int ids[kFrontMaxTokens * kMaxK];              // the routed ids, written by the caller
  uint32_t rows[kFrontMaxTokens * (kMaxE / 32)];
  uint64_t masks[kMaxE];
  int off[kMaxE];
};

__device__ __forceinline__ void wave_sync_lds() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Every thread of a 1024-thread workgroup calls this once its wavefront has written
// its tokens' ids to lds.ids.  EPL: experts per lane, ceil(E / 64) or more.
template <int EPL>
__device__ __forceinline__ void group_small(
    FrontLds& lds, int T, int E, int k, int words, uint32_t* __restrict__ bm,
    int32_t* __restrict__ counts, int32_t* __restrict__ offsets, int32_t* __restrict__ gather,
    int32_t* __restrict__ scatter, int tile_rows, int tile_bound, int32_t* __restrict__ n_tiles,
    RowTile* __restrict__ tiles) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n_waves = blockDim.x >> 6;
  for (int i = threadIdx.x; i < T * words; i += blockDim.x) lds.rows[i] = 0u;
  __syncthreads();

  // 2. bit matrix: entries past T*k are padding lanes of the logical block
  const int n_entries = T * k;
  if (static_cast<int>(threadIdx.x) < n_entries) {
    const int e = lds.ids[threadIdx.x];
    if (static_cast<unsigned>(e) < static_cast<unsigned>(E))
      atomicOr(&lds.rows[(threadIdx.x / k) * words + (e >> 5)], 1u << (e & 31));
  }
  __syncthreads();
  for (int i = threadIdx.x; i < T * words; i += blockDim.x) bm[i] = lds.rows[i];

  // 3. expert column masks, 64 experts per wavefront (lane = token), then counts,
  // offsets and permutations in wavefront 0
  for (int w0 = 2 * wave; w0 < words; w0 += 2 * n_waves)
    column_masks_64(lds.rows, lane, lane < T, E, words, lane, lds.masks, w0);
  __syncthreads();
  if (wave != 0) return;
  int c[EPL];
  int sum = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane * EPL + i;
    c[i] = e < E ? __popcll(lds.masks[e]) : 0;
    sum += c[i];
  }
  int incl = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(incl, d, 64);
    if (lane >= d) incl += o;
  }
  int run = incl - sum;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane * EPL + i;
    if (e < E) {
      counts[e] = c[i];
      offsets[e] = run;
      lds.off[e] = run;
    }
    run += c[i];
  }
  if (lane == 63) offsets[E] = incl;
  if (tiles != nullptr) {
    // the FFN's row-tile plan (same tiles and order as its plan kernel): expert e
    // cut into ceil(count / tile_rows) tiles, experts in index order
    int nt[EPL], tsum = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      nt[i] = (c[i] + tile_rows - 1) / tile_rows;
      tsum += nt[i];
    }
    int tincl = tsum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(tincl, d, 64);
      if (lane >= d) tincl += o;
    }
    int slot = tincl - tsum;
    int off = incl - sum;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      for (int t = 0; t < nt[i] && slot < tile_bound; ++t, ++slot) {
        RowTile rt;
        rt.expert = lane * EPL + i;
        rt.p_begin = off + t * tile_rows;
        rt.p_end = (t + 1) * tile_rows < c[i] ? off + (t + 1) * tile_rows : off + c[i];
        rt.multi = c[i] > tile_rows ? 1 : 0;
        tiles[slot] = rt;
      }
      off += c[i];
    }
    if (lane == 63) *n_tiles = tincl < tile_bound ? tincl : tile_bound;
  }
  wave_sync_lds();
  // one lane per (token, choice) entry: its row is the expert's offset plus the
  // earlier tokens that chose the same expert (bits below the token in its mask)
  for (int s = lane; s < n_entries; s += 64) {
    const int e = lds.ids[s];
    if (static_cast<unsigned>(e) >= static_cast<unsigned>(E)) continue;
    const int p = lds.off[e] + __popcll(lds.masks[e] & ((1ull << (s / k)) - 1ull));
    if (p < 0 || p >= n_entries) continue;
    gather[p] = s;
    scatter[s] = p;
  }
}

}  // namespace moe
