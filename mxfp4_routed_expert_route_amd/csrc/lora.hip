// Low-rank adapters of many requests beside a shared projection.
//
// v = x A_a^T (K long, R wide), then y = base + scaling_a v B_a^T, for the rows of each adapter a in
// the order that moe_lora_group gives them.  A workgroup takes 16 rows of one adapter and finds
// them from the offsets.  Both products are bf16 MFMAs with the weights as the A operand, so that
// a lane holds neighbouring results of one row.
#include "block.h"
#include "block_common.h"
#include "block_plan.h"

namespace moe {
namespace {

constexpr int kTile = 16;   // rows
constexpr int64_t kMaxGroups = 1 << 23;   // of 256 threads: a launch has fewer than 2^32

// ---------------------------------------------------------------- grouping

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
  for (int64_t i = begin + lane; i < end; i += 64) atomicAdd(&mine[bin_of(i)], 1);
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
    const int bin = here ? bin_of(i) : -1;
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
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
}

// ---------------------------------------------------------------- tiles

struct Tile {
  int adapter;       // L: rows without an adapter; -1: none
  int begin, rows;   // positions in the grouped order
};

// Tile number `tile` of the batch, found by one wavefront: each lane counts the tiles of a few
// neighbouring adapters.  Behind them come the tiles of the rows without an adapter.
__device__ __forceinline__ Tile find_tile(const int32_t* offsets, int L, int M, int tile) {
  const int lane = threadIdx.x & 63;
  const int per = (L + 63) / 64;
  auto clamp = [&](int v) { return v < 0 ? 0 : v > M ? M : v; };
  int n = 0;
  for (int i = 0; i < per; ++i) {
    const int a = lane * per + i;
    if (a < L) {
      const int rows = clamp(offsets[a + 1]) - clamp(offsets[a]);
      n += rows > 0 ? (rows + kTile - 1) / kTile : 0;
    }
  }
  int upto = n;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(upto, d, 64);
    if (lane >= d) upto += o;
  }
  const uint64_t behind = __builtin_amdgcn_ballot_w64(upto > tile);
  if (behind == 0ull) {
    const int total = __shfl(upto, 63, 64);
    const int begin = clamp(offsets[L]);
    const int64_t at = begin + static_cast<int64_t>(tile - total) * kTile;
    if (at >= M) return Tile{-1, 0, 0};
    return Tile{L, static_cast<int>(at), M - at < kTile ? static_cast<int>(M - at) : kTile};
  }
  const int owner = static_cast<int>(__builtin_ctzll(behind));
  int left = tile - __shfl(upto - n, owner, 64);
  Tile r{-1, 0, 0};
  for (int i = 0; i < per; ++i) {
    const int a = owner * per + i;
    if (a >= L) break;
    const int from = clamp(offsets[a]), rows = clamp(offsets[a + 1]) - from;
    const int tiles = rows > 0 ? (rows + kTile - 1) / kTile : 0;
    if (left < tiles) {
      const int rest = rows - left * kTile;
      r = Tile{a, from + left * kTile, rest < kTile ? rest : kTile};
      break;
    }
    left -= tiles;
  }
  return Tile{__builtin_amdgcn_readfirstlane(r.adapter), __builtin_amdgcn_readfirstlane(r.begin),
              __builtin_amdgcn_readfirstlane(r.rows)};
}

__device__ __forceinline__ bf16x8 load_bf16x8(const uint16_t* p, bool here) {
  uint4 d = make_uint4(0u, 0u, 0u, 0u);
  if (here) d = *reinterpret_cast<const uint4*>(p);
  return __builtin_bit_cast(bf16x8, d);
}

// ---------------------------------------------------------------- x A^T

// NF fragments of 16 ranks.  The wavefronts share K out in steps of 64.
template <int NF>
__global__ __launch_bounds__(256) void shrink_kernel(LoraArgs a, int tile0) {
  __shared__ floatx4 part[4][NF][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const Tile tile = find_tile(a.offsets, a.L, static_cast<int>(a.M), tile0 + blockIdx.x);
  if (tile.adapter < 0 || tile.adapter >= a.L) return;   // uniform over the workgroup
  const int p = tile.begin + (r16 < tile.rows ? r16 : 0);
  const int row = a.rows[p];
  const bool live = static_cast<unsigned>(row) < static_cast<unsigned>(a.M);
  const uint16_t* x = a.x + (live ? row : 0) * a.x_stride;
  const uint16_t* w[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int r = 16 * f + r16;
    w[f] = a.a + (static_cast<int64_t>(tile.adapter) * a.R + (r < a.R ? r : 0)) * a.K;
  }
  floatx4 acc[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) acc[f] = floatx4{0.f, 0.f, 0.f, 0.f};
  for (int k0 = 64 * wave; k0 < a.K; k0 += 256) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = k0 + 16 * g + 8 * h;
      const bool here = k < a.K;
      const bf16x8 v = load_bf16x8(x + k, here);
#pragma unroll
      for (int f = 0; f < NF; ++f)
        acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(load_bf16x8(w[f] + k, here), v, acc[f], 0, 0, 0);
    }
  }
#pragma unroll
  for (int f = 0; f < NF; ++f) part[wave][f][lane] = acc[f];
  __syncthreads();
  for (int f = wave; f < NF; f += 4) {
    floatx4 s = part[0][f][lane];
#pragma unroll
    for (int i = 1; i < 4; ++i) s += part[i][f][lane];
    const int r = 16 * f + 4 * g;
    if (r16 < tile.rows && r < a.R)
      *reinterpret_cast<floatx4*>(a.v + static_cast<int64_t>(tile.begin + r16) * a.R + r) = s;
  }
}

// ---------------------------------------------------------------- base + v B^T

__device__ __forceinline__ void load_row8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// v in kParts bf16 parts: the upper bits of what is left each time, the last part rounded.  Three
// hold all 24 bits, for fp32 results; two leave 2^-17 of v, far under a bf16 result's step.
template <int kParts>
__device__ __forceinline__ void split(const float (&v)[8], bf16x8 (&part)[kParts]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float left = v[j];
#pragma unroll
    for (int i = 0; i < kParts - 1; ++i) {
      const float h = __uint_as_float(__float_as_uint(left) & 0xFFFF0000u);
      part[i][j] = static_cast<__bf16>(h);
      left = fabsf(h) < __builtin_inff() ? left - h : 0.f;   // an infinity stays one
    }
    part[kParts - 1][j] = static_cast<__bf16>(left);
  }
}

// A wavefront takes 64 columns: lane (r16, g) has columns 16 g .. + 15 of row r16, so the weights'
// fragment f holds, as its row 4 g + j, column 16 g + 4 f + j.
template <class Out>
__global__ __launch_bounds__(256) void expand_kernel(LoraArgs a, int tile0, int col_blocks, int wide) {
  constexpr int kParts = sizeof(Out) == 4 ? 3 : 2;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int tile_no = blockIdx.x / col_blocks;
  const int n0 = (blockIdx.x - tile_no * col_blocks) * 256 + 64 * wave;
  const Tile tile = find_tile(a.offsets, a.L, static_cast<int>(a.M), tile0 + tile_no);
  if (tile.adapter < 0 || n0 >= a.N) return;   // uniform per wavefront
  const Out* base = static_cast<const Out*>(a.base);
  Out* y = static_cast<Out*>(a.y);
  if (tile.adapter == a.L && a.base == a.y) return;
  const int p = tile.begin + (r16 < tile.rows ? r16 : 0);
  floatx4 acc[4];
#pragma unroll
  for (int f = 0; f < 4; ++f) acc[f] = floatx4{0.f, 0.f, 0.f, 0.f};
  float scaling = 0.f;
  if (tile.adapter < a.L) {   // uniform
    scaling = a.scaling ? a.scaling[tile.adapter] : 1.0f;
    const uint16_t* w[4];
    bool in[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const int n = n0 + 16 * (r16 >> 2) + 4 * f + (r16 & 3);
      in[f] = n < a.N;
      w[f] = a.b + (static_cast<int64_t>(tile.adapter) * a.N + (in[f] ? n : 0)) * a.R;
    }
    for (int k0 = 0; k0 < a.R; k0 += 32) {
      const int k = k0 + 8 * g;
      const bool here = k < a.R;
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (here) load_row8(a.v + static_cast<int64_t>(p) * a.R + k, v);
      bf16x8 part[kParts];
      split<kParts>(v, part);
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const bf16x8 b = load_bf16x8(w[f] + k, here && in[f]);
#pragma unroll
        for (int i = 0; i < kParts; ++i)
          acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, part[i], acc[f], 0, 0, 0);
      }
    }
  }
  if (r16 >= tile.rows) return;
  const int row = a.rows[p];
  if (static_cast<unsigned>(row) >= static_cast<unsigned>(a.M)) return;
  const int c0 = n0 + 16 * g;
  if (c0 >= a.N) return;
  const Out* from = base ? base + row * a.base_stride + c0 : nullptr;
  Out* to = y + row * a.y_stride + c0;
  const bool whole = wide && c0 + 16 <= a.N;
  float o[16];
  if constexpr (sizeof(Out) == 4) {
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      if (from == nullptr) {
#pragma unroll
        for (int j = 0; j < 4; ++j) o[4 * f + j] = 0.f;
      } else if (whole) {
        const float4 d = *reinterpret_cast<const float4*>(from + 4 * f);
        o[4 * f] = d.x; o[4 * f + 1] = d.y; o[4 * f + 2] = d.z; o[4 * f + 3] = d.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) o[4 * f + j] = c0 + 4 * f + j < a.N ? from[4 * f + j] : 0.f;
      }
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float d[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (from != nullptr) {
        if (whole) {
          unpack_bf16x8(*reinterpret_cast<const uint4*>(from + 8 * h), d);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (c0 + 8 * h + j < a.N) d[j] = bf16_bits_to_f32(from[8 * h + j]);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) o[8 * h + j] = d[j];
    }
  }
  if (tile.adapter < a.L) {
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[4 * f + j] = fmaf(scaling, acc[f][j], o[4 * f + j]);
  }
  if constexpr (sizeof(Out) == 4) {
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      if (whole) {
        *reinterpret_cast<float4*>(to + 4 * f) = make_float4(o[4 * f], o[4 * f + 1], o[4 * f + 2], o[4 * f + 3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (c0 + 4 * f + j < a.N) to[4 * f + j] = o[4 * f + j];
      }
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float d[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = o[8 * h + j];
      if (whole) {
        *reinterpret_cast<uint4*>(to + 8 * h) = pack_bf16x8(d);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c0 + 8 * h + j < a.N) to[8 * h + j] = f32_to_bf16_bits(d[j]);
      }
    }
  }
}

template <int NF>
hipError_t launch_shrink(const LoraArgs& a, int64_t tiles, hipStream_t stream) {
  for (int64_t at = 0; at < tiles; at += kMaxGroups) {
    const int64_t n = tiles - at < kMaxGroups ? tiles - at : kMaxGroups;
    shrink_kernel<NF><<<dim3(static_cast<unsigned>(n)), dim3(256), 0, stream>>>(a, static_cast<int>(at));
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

template <class Out>
hipError_t launch_expand(const LoraArgs& a, int64_t tiles, int wide, hipStream_t stream) {
  const int col_blocks = (a.N + 255) / 256;
  const int64_t most = kMaxGroups / col_blocks;   // 2^7 at least: N is at most 2^24
  for (int64_t at = 0; at < tiles; at += most) {
    const int64_t n = tiles - at < most ? tiles - at : most;
    expand_kernel<Out><<<dim3(static_cast<unsigned>(n * col_blocks)), dim3(256), 0, stream>>>(
        a, static_cast<int>(at), col_blocks, wide);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
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

hipError_t launch_lora_add(const LoraArgs& a, bool f32, hipStream_t stream) {
  // tiles: an adapter's last one may be short
  const int64_t touched = a.M < a.L ? a.M : a.L;
  const int64_t tiles = (a.M + (kTile - 1) * touched) / kTile;
  hipError_t err;
  if (a.R <= 16) err = launch_shrink<1>(a, tiles, stream);
  else if (a.R <= 32) err = launch_shrink<2>(a, tiles, stream);
  else if (a.R <= 64) err = launch_shrink<4>(a, tiles, stream);
  else if (a.R <= 128) err = launch_shrink<8>(a, tiles, stream);
  else err = launch_shrink<16>(a, tiles, stream);
  if (err != hipSuccess) return err;
  const int64_t unit = f32 ? 4 : 8;
  const int wide = a.y_stride % unit == 0 && (a.base == nullptr || a.base_stride % unit == 0);
  // one more for the rows without an adapter
  const int64_t all = (a.M + (kTile - 1) * (touched + 1)) / kTile;
  return f32 ? launch_expand<float>(a, all, wide, stream) : launch_expand<uint16_t>(a, all, wide, stream);
}

}  // namespace moe
