// Low-rank adapters of many requests beside a shared projection: few rows, or ranks above 64.
//
// v = x A_a^T (K long, R wide), then y = base + scaling_a v B_a^T, for the rows of each adapter a in
// the order that moe_lora_group gives them.  A tile is some rows of one adapter; a wavefront finds
// its tile from the offsets.  Both products are bf16 MFMAs with the weights as the A operand, so
// that a lane holds neighbouring results of one row.  The inner sums stay fp32; the second product takes
// them in bf16 parts (split).
//
// Bound by latency at these sizes: 1x4096x4096 rank 16 reads 0.3 MB in one launch of 8.0 us, of which the
// chain of offsets, rows and first loads takes about 4; 512 rows of 64 adapters read 23 MB and write 4 in
// 7.1 and 6.6 us for the two products, whose floor at a copy's rate is 5.8 together.  Ranks above 64 are
// bound by x, read once for each 64 ranks, and by fp32 inner sums that each block of columns reads and
// splits again: 8191x4096x4096 105 us at rank 128, 162 at 256.  Registers spill in small_kernel at 64
// ranks (5 to 7) and in expand_kernel with fp32 results beyond 32 (3 to 19).
#include "block.h"
#include "block_plan.h"
#include "lds_copy.h"
#include "lora_core.h"

namespace moe {
namespace {

constexpr int64_t kMaxThreads = int64_t{1} << 31;   // of a launch: fewer than 2^32

// ---------------------------------------------------------------- x A^T

// One wavefront's share of 16 rows times NF x 16 ranks: chunks of 64 elements of K, c0, c0 + step, ...,
// kDepth of them on their way.  A chunk is a 128-byte line of a row.
template <int NF, int kDepth>
__device__ __forceinline__ void inner_products(const uint16_t* x, const uint16_t* const (&w)[NF], int K, int c0,
                                               int step, floatx4 (&acc)[NF]) {
  const int g = (threadIdx.x & 63) >> 4;
  const int chunks = (K + 63) / 64;
  struct Chunk {
    bf16x8 x[2], w[NF][2];
  };
  auto load = [&](Chunk& d, int c) {
    const int k0 = 64 * c + 8 * g;
    if (64 * c + 64 <= K) {   // uniform
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int f = 0; f < NF; ++f) d.w[f][h] = load_bf16x8(w[f] + k0 + 32 * h, true);
        d.x[h] = load_bf16x8(x + k0 + 32 * h, true);
      }
    } else {   // zeros past K
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool here = k0 + 32 * h < K;
#pragma unroll
        for (int f = 0; f < NF; ++f) d.w[f][h] = load_bf16x8(w[f] + k0 + 32 * h, here);
        d.x[h] = load_bf16x8(x + k0 + 32 * h, here);
      }
    }
  };
  Chunk ring[kDepth];
#pragma unroll
  for (int d = 0; d < kDepth; ++d)
    if (c0 + d * step < chunks) load(ring[d], c0 + d * step);   // uniform
#pragma unroll
  for (int f = 0; f < NF; ++f) acc[f] = floatx4{0.f, 0.f, 0.f, 0.f};
  for (int c = c0; c < chunks; c += kDepth * step) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      if (c + d * step < chunks) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int f = 0; f < NF; ++f)
            acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ring[d].w[f][h], ring[d].x[h], acc[f], 0, 0, 0);
        if (c + (kDepth + d) * step < chunks) load(ring[d], c + (kDepth + d) * step);
      }
    }
  }
}

// The inner sums of up to 16 rows and NF x 16 ranks, K shared out among a workgroup's eight wavefronts and
// `splits` workgroups, whose sums the second product adds up.  Operands go straight to registers: with
// few rows an adapter nothing is read twice, and a ring in LDS only adds a wait (512 rows of 4 adapters, rank
// 16, both products: 11.1 us against 14.6 by way of LDS).
template <int NF>
__global__ __launch_bounds__(512) void shrink_kernel(LoraArgs a, int tile0, int rank_blocks, int splits) {
  constexpr int W = 8;
  __shared__ floatx4 part[W][NF][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int per = rank_blocks * splits, of = blockIdx.x / per;
  const int split_no = (blockIdx.x - of * per) / rank_blocks;
  const int rank0 = (blockIdx.x - of * per - split_no * rank_blocks) * 16 * NF;
  const Tiles<16> tiles(a.offsets, a.L, static_cast<int>(a.M));
  if (tile0 + of >= tiles.total) return;   // uniform over the workgroup
  const Tile tile = tiles.find(tile0 + of);
  if (tile.adapter >= a.L) return;
  const uint16_t *x, *w[NF];
  const int row = a.rows[tile.begin + (r16 < tile.rows ? r16 : 0)];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int r = rank0 + 16 * f + r16;
    w[f] = a.a + (static_cast<int64_t>(tile.adapter) * a.R + (r < a.R ? r : 0)) * a.K;
  }
  x = a.x + (static_cast<unsigned>(row) < static_cast<unsigned>(a.M) ? row : 0) * a.x_stride;
  floatx4 acc[NF];
  inner_products<NF, NF == 4 ? 2 : 4>(x, w, a.K, split_no * W + wave, splits * W, acc);
#pragma unroll
  for (int f = 0; f < NF; ++f) part[wave][f][lane] = acc[f];
  __syncthreads();
  for (int f = wave; f < NF; f += W) {
    floatx4 s = part[0][f][lane];
#pragma unroll
    for (int i = 1; i < W; ++i) s += part[i][f][lane];
    const int r = rank0 + 16 * f + 4 * g;
    if (r16 < tile.rows && r < a.R)
      *reinterpret_cast<floatx4*>(a.v + (static_cast<int64_t>(split_no) * a.M + tile.begin + r16) * a.R + r) = s;
  }
}

// The same for up to 64 rows of an adapter with many: both operands go to LDS by loads that write it
// themselves, in whole lines (8 rows x 128 bytes a copy), four chunks of K deep; a wavefront takes 16
// of the rows.  Piece c (16 bytes) of LDS row r sits at place c ^ ((r >> 1) & 7), so that operand
// reads meet no bank conflict.
__global__ __launch_bounds__(256) void shrink_stream_kernel(LoraArgs a, int tile0, int rank_blocks, int splits) {
  constexpr int NF = 4, kRows = 64, kLines = kRows + 16 * NF, kStages = 4, W = 4;
  constexpr int kEach = kLines / 8 / W;   // copies of a chunk
  __shared__ __attribute__((aligned(16))) unsigned char lds[kStages][kLines * 128];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int per = rank_blocks * splits, of = blockIdx.x / per;
  const int split_no = (blockIdx.x - of * per) / rank_blocks;
  const int rank0 = (blockIdx.x - of * per - split_no * rank_blocks) * 16 * NF;
  const Tiles<kRows> tiles(a.offsets, a.L, static_cast<int>(a.M));
  if (tile0 + of >= tiles.total) return;   // uniform over the workgroup
  const Tile tile = tiles.find(tile0 + of);
  if (tile.adapter >= a.L) return;
  const int K = a.K, chunks = (K + 63) / 64;
  const int begin = static_cast<int>(static_cast<int64_t>(chunks) * split_no / splits);
  const int end = static_cast<int>(static_cast<int64_t>(chunks) * (split_no + 1) / splits);

  // copy i of this wavefront: LDS rows 8 (wave + W i) + lane / 8, of the same parity of eights
  const int piece = (lane & 7) ^ (4 * (wave & 1) + (lane >> 4));
  const uint16_t* from[kEach];   // the row's first element
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int r = 8 * (wave + W * i) + (lane >> 3);
    if (r < kRows) {
      const int row = a.rows[tile.begin + (r < tile.rows ? r : 0)];
      from[i] = a.x + (static_cast<unsigned>(row) < static_cast<unsigned>(a.M) ? row : 0) * a.x_stride;
    } else {
      const int rank = rank0 + r - kRows;
      from[i] = a.a + (static_cast<int64_t>(tile.adapter) * a.R + (rank < a.R ? rank : 0)) * K;
    }
  }
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) unsigned char*)&lds[0][0]));
  auto copy = [&](int c) {
    const int at = 64 * c + 8 * piece;
    const int k = at < K ? at : 0;   // past K: any, the operands are zeroed
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      copy16_global(from[i] + k, lds0 + (c - begin) % kStages * (kLines * 128) + 1024 * (wave + W * i));
  };
  floatx4 acc[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) acc[f] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s)
    if (begin + s < end) copy(begin + s);
  const int place = r16 * 128 + 16 * (g ^ ((r16 >> 1) & 7));   // piece g; piece g + 4 is at ^ 64
  for (int c = begin; c < end; ++c) {
    if (c + kStages - 1 < end)   // uniform: this chunk's copies are the oldest
      wait_copies<(kStages - 2) * kEach>();
    else
      wait_copies<0>();
    wait_lds();
    barrier();   // all wavefronts' copies of it are there, and the chunk before it has been read
    if (c + kStages - 1 < end) copy(c + kStages - 1);
    const unsigned char* stage = lds[(c - begin) % kStages];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const unsigned char* at = stage + (h ? place ^ 64 : place);
      bf16x8 v = *reinterpret_cast<const bf16x8*>(at + wave * 16 * 128);
      const bool here = 64 * c + 32 * h + 8 * g < K;
      if (!here) v = bf16x8{0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        bf16x8 w = *reinterpret_cast<const bf16x8*>(at + (kRows + 16 * f) * 128);
        if (!here) w = bf16x8{0, 0, 0, 0, 0, 0, 0, 0};
        acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, v, acc[f], 0, 0, 0);
      }
    }
  }
  const int p = 16 * wave + r16;
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int r = rank0 + 16 * f + 4 * g;
    if (p < tile.rows && r < a.R)
      *reinterpret_cast<floatx4*>(a.v + (static_cast<int64_t>(split_no) * a.M + tile.begin + p) * a.R + r) = acc[f];
  }
}

// ---------------------------------------------------------------- base + v B^T

// Workgroups go through (block of 256 columns, 16 rows of one adapter) pairs, a run of neighbouring ones
// each, 64 columns a wavefront, which keeps its weights in registers until the adapter or the block
// changes.  The next pair's inner sums and base are on their way while one is worked on, and the
// row numbers of the one behind it.  Results go through LDS, so that base is read and y written in
// whole lines: 8 (fp32: 16) lanes a row.
// XCD x takes the blocks x, x + 8, ... where they number a multiple of 8: each L2 then holds its own
// part of the weights.
template <class Out, int KS>
__global__ __launch_bounds__(256, KS <= 2 ? 4 : KS == 4 ? 3 : 2) void expand_kernel(LoraArgs a, int col_blocks,
                                                                                    int wide, int splits) {
  constexpr int kParts = kPartsOf<Out>, kAheadKS = KS * sizeof(Out) <= 4 ? KS : 0;   // inner sums on their way, where registers allow
  constexpr int kPiece = 16 / sizeof(Out), kLanes = 64 / kPiece;       // columns of a lane, lanes of a row
  constexpr int kRows = 64 / kLanes, kGoes = 16 / kRows;               // rows of an access, accesses
  constexpr int kPitch = 68;                                           // floats of a row in LDS
  __shared__ __attribute__((aligned(16))) float lds[4][16 * kPitch];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const Out* base = static_cast<const Out*>(a.base);
  Out* y = static_cast<Out*>(a.y);
  const Tiles<16> tiles(a.offsets, a.L, static_cast<int>(a.M));
  const int n_tiles = a.base == a.y ? lane_value(tiles.upto, 63) : tiles.total;   // in place: adapters' rows alone

  // this workgroup's run of pairs, block-major
  const bool by_xcd = col_blocks % 8 == 0;   // and the grid is a multiple of 8
  const int mine = by_xcd ? col_blocks / 8 : col_blocks;
  const int groups = by_xcd ? gridDim.x / 8 : gridDim.x, group = by_xcd ? blockIdx.x / 8 : blockIdx.x;
  const int64_t pairs = static_cast<int64_t>(mine) * n_tiles;
  const int64_t first = pairs * group / groups, end = pairs * (group + 1) / groups;

  struct Pair {
    Tile tile;
    int n0;   // this wavefront's first column
  };
  int block = 0, tile_no = 0;   // of the next pair to look up
  auto next_pair = [&]() {
    const Pair p{tiles.find(tile_no),
                 (by_xcd ? block * 8 + static_cast<int>(blockIdx.x % 8) : block) * 256 + 64 * wave};
    if (++tile_no == n_tiles) {
      tile_no = 0;
      ++block;
    }
    return p;
  };
  struct Ids {
    int row[kGoes];   // -1: none
  };
  auto load_ids = [&](const Pair& p) {
    Ids d;
#pragma unroll
    for (int i = 0; i < kGoes; ++i) {
      const int r = kRows * i + lane / kLanes;
      const int row = a.rows[p.tile.begin + (r < p.tile.rows ? r : 0)];
      d.row[i] = r < p.tile.rows && static_cast<unsigned>(row) < static_cast<unsigned>(a.M) ? row : -1;
    }
    return d;
  };
  auto load_v = [&](const Tile& t, int s, float (&v)[8]) {
    const int k = 32 * s + 8 * g;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
    if (k < a.R) {
      const float* from = a.v + static_cast<int64_t>(t.begin + (r16 < t.rows ? r16 : 0)) * a.R + k;
      load_f32x8(from, v);
      for (int q = 1; q < splits; ++q) {
        float o[8];
        load_f32x8(from + static_cast<int64_t>(q) * a.M * a.R, o);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += o[j];
      }
    }
  };
  struct In {
    Cols<Out, kPiece> base[kGoes];
    float v[kAheadKS ? kAheadKS : 1][8];
  };
  const int my_col = kPiece * (lane % kLanes);
  auto load_in = [&](const Pair& p, const Ids& ids) {
    In d;
    const int left = a.N - p.n0 - my_col;
    const bool whole = wide && p.n0 + 64 <= a.N;   // uniform
#pragma unroll
    for (int i = 0; i < kGoes; ++i) {
      d.base[i].zero();
      if (base != nullptr && ids.row[i] >= 0)
        d.base[i].load(base + ids.row[i] * a.base_stride + p.n0 + my_col, left, whole);
    }
    if constexpr (kAheadKS != 0)
      if (p.tile.adapter < a.L)
#pragma unroll
        for (int s = 0; s < KS; ++s) load_v(p.tile, s, d.v[s]);
    return d;
  };

  if (first >= end) return;   // uniform over the workgroup
  block = static_cast<int>(first / n_tiles);
  tile_no = static_cast<int>(first - static_cast<int64_t>(block) * n_tiles);
  bf16x8 w[KS][4];
  float scaling = 1.0f;
  int w_adapter = -1, w_n0 = -1;
  Pair cur = next_pair();
  Ids ids = load_ids(cur);
  In in = load_in(cur, ids);
  Pair nxt = cur;
  Ids next_ids = ids;
  if (first + 1 < end) {
    nxt = next_pair();
    next_ids = load_ids(nxt);
  }
  for (int64_t u = first; u < end; ++u) {
    const bool with = cur.tile.adapter < a.L;   // uniform
    if (with && (cur.tile.adapter != w_adapter || cur.n0 != w_n0)) {
      w_adapter = cur.tile.adapter;
      w_n0 = cur.n0;
      if (a.scaling != nullptr) scaling = a.scaling[w_adapter];
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const int n = w_n0 + 16 * f + r16;
        const uint16_t* from = a.b + (static_cast<int64_t>(w_adapter) * a.N + (n < a.N ? n : 0)) * a.R;
#pragma unroll
        for (int s = 0; s < KS; ++s) w[s][f] = load_bf16x8(from + 32 * s + 8 * g, 32 * s + 8 * g < a.R && n < a.N);
      }
    }
    In next;
    Pair after = nxt;
    Ids after_ids = next_ids;
    if (u + 1 < end) next = load_in(nxt, next_ids);
    if (u + 2 < end) {
      after = next_pair();
      after_ids = load_ids(after);
    }
    if (with) {
      floatx4 acc[4];
#pragma unroll
      for (int f = 0; f < 4; ++f) acc[f] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        float v[8];
        if constexpr (kAheadKS != 0) {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = in.v[s][j];
        } else {
          load_v(cur.tile, s, v);
        }
        bf16x8 part[kParts];
        split<kParts>(v, part);
#pragma unroll
        for (int q = 0; q < kParts; ++q)
#pragma unroll
          for (int f = 0; f < 4; ++f)
            acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[s][f], part[q], acc[f], 0, 0, 0);
      }
      float* mine = lds[wave];
      wave_sync_lds();   // the last pair's have been read
#pragma unroll
      for (int f = 0; f < 4; ++f) *reinterpret_cast<floatx4*>(mine + r16 * kPitch + 16 * f + 4 * g) = acc[f];
      wave_sync_lds();
      if (__builtin_expect(any_nan(acc, true), false)) {   // uniform
        const int n = cur.n0 + lane;
#pragma unroll 1
        for (int r = 0; r < cur.tile.rows; ++r) {
          float* at = mine + r * kPitch + lane;
          const float* v = a.v + static_cast<int64_t>(cur.tile.begin + r) * a.R;
          auto inner = [&](int k) {
            float s = 0.f;
            for (int q = 0; q < splits; ++q) s += v[static_cast<int64_t>(q) * a.M * a.R + k];
            return s;
          };
          if (n < a.N && *at != *at) *at = whole_product(inner, a.b + (static_cast<int64_t>(w_adapter) * a.N + n) * a.R, a.R);
        }
        wave_sync_lds();
      }
#pragma unroll
      for (int i = 0; i < kGoes; ++i) {
        const float* from = mine + (kRows * i + lane / kLanes) * kPitch + my_col;
#pragma unroll
        for (int j = 0; j < kPiece; j += 4) {
          const floatx4 d = *reinterpret_cast<const floatx4*>(from + j);
          Cols<Out, kPiece>& o = in.base[i];
          o.put4(j, fmaf(scaling, d[0], o.get(j)), fmaf(scaling, d[1], o.get(j + 1)),
                 fmaf(scaling, d[2], o.get(j + 2)), fmaf(scaling, d[3], o.get(j + 3)));
        }
      }
    }
    const int left = a.N - cur.n0 - my_col;
    const bool whole = wide && cur.n0 + 64 <= a.N;
#pragma unroll
    for (int i = 0; i < kGoes; ++i)
      if (ids.row[i] >= 0) in.base[i].store(y + ids.row[i] * a.y_stride + cur.n0 + my_col, left, whole);
    cur = nxt;
    ids = next_ids;
    in = next;
    nxt = after;
    next_ids = after_ids;
  }
}

// ---------------------------------------------------------------- both in one launch

// For a few tiles: a workgroup makes all inner sums of its 16 rows, K over its 16 wavefronts, and then 16
// columns a wavefront.  A is read once for each block of 256 columns, from L2, which costs less than
// a second launch.
template <class Out, int NF>
__global__ __launch_bounds__(1024) void small_kernel(LoraArgs a, int col_blocks, int wide) {
  constexpr int W = 16, KS = (NF + 1) / 2, kParts = kPartsOf<Out>;
  constexpr int kPitch = 32 * KS + 4;   // floats of a row of inner sums
  __shared__ floatx4 part[W][NF][64];
  __shared__ __attribute__((aligned(16))) float own_sums[NF < 4 ? 16 * kPitch : 4];
  float* sums = NF < 4 ? own_sums : reinterpret_cast<float*>(part);   // with four fragments, LDS is full
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int tile_no = blockIdx.x / col_blocks;
  const int n0 = (blockIdx.x - tile_no * col_blocks) * 256 + 16 * wave;
  // up to 64 rows: their numbers come with the offsets, not after them
  const bool few = a.M <= 64;   // uniform
  const int first_rows = few ? a.rows[lane < a.M ? lane : 0] : 0;
  const Tiles<16> tiles(a.offsets, a.L, static_cast<int>(a.M));
  if (tile_no >= tiles.total) return;   // uniform over the workgroup
  const Tile tile = tiles.find(tile_no);
  const bool none = tile.adapter == a.L;
  if (none && a.base == a.y) return;
  const Out* base = static_cast<const Out*>(a.base);
  Out* y = static_cast<Out*>(a.y);
  const int c0 = n0 + 4 * g, left = a.N - c0;
  const bool whole = wide && left >= 4;
  const int p = tile.begin + (r16 < tile.rows ? r16 : 0);
  const int row = few ? __shfl(first_rows, p, 64) : a.rows[p];
  const bool live = r16 < tile.rows && static_cast<unsigned>(row) < static_cast<unsigned>(a.M);
  const bool out = live && left > 0;
  Cols<Out, 4> cols;
  cols.zero();
  if (base != nullptr && out) cols.load(base + row * a.base_stride + c0, left, whole);
  if (!none) {
    const float scaling = a.scaling != nullptr ? a.scaling[tile.adapter] : 1.0f;
    const int n = n0 + r16;
    const uint16_t* from = a.b + (static_cast<int64_t>(tile.adapter) * a.N + (n < a.N ? n : 0)) * a.R;
    bf16x8 b[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) b[s] = load_bf16x8(from + 32 * s + 8 * g, 32 * s + 8 * g < a.R && n < a.N);
    const uint16_t *x, *w[NF];
    x = a.x + (static_cast<unsigned>(row) < static_cast<unsigned>(a.M) ? row : 0) * a.x_stride;
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const int r = 16 * f + r16;
      w[f] = a.a + (static_cast<int64_t>(tile.adapter) * a.R + (r < a.R ? r : 0)) * a.K;
    }
    floatx4 acc[NF];
    inner_products<NF, NF == 1 ? 4 : 2>(x, w, a.K, wave, W, acc);
#pragma unroll
    for (int f = 0; f < NF; ++f) part[wave][f][lane] = acc[f];
    __syncthreads();
    floatx4 total = {0.f, 0.f, 0.f, 0.f};   // ranks past NF x 16 and past R are zeros
    if (wave < NF && 16 * wave + 4 * g < a.R) {
#pragma unroll
      for (int i = 0; i < W; ++i) total += part[i][wave][lane];
    }
    if constexpr (NF == 4) __syncthreads();
    if (wave < 2 * KS) *reinterpret_cast<floatx4*>(&sums[r16 * kPitch + 16 * wave + 4 * g]) = total;
    __syncthreads();
    floatx4 d[1] = {floatx4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      float v[8];
      load_f32x8(&sums[r16 * kPitch + 32 * s + 8 * g], v);
      bf16x8 q[kParts];
      split<kParts>(v, q);
#pragma unroll
      for (int i = 0; i < kParts; ++i) d[0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[s], q[i], d[0], 0, 0, 0);
    }
    if (__builtin_expect(any_nan(d, true), false)) {   // uniform
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < left && d[0][j] != d[0][j])
          d[0][j] = whole_product([&](int r) { return sums[r16 * kPitch + r]; },
                                  a.b + (static_cast<int64_t>(tile.adapter) * a.N + c0 + j) * a.R, a.R);
    }
    cols.put4(0, fmaf(scaling, d[0][0], cols.get(0)), fmaf(scaling, d[0][1], cols.get(1)),
              fmaf(scaling, d[0][2], cols.get(2)), fmaf(scaling, d[0][3], cols.get(3)));
  }
  if (out) cols.store(y + row * a.y_stride + c0, left, whole);
}

// ---------------------------------------------------------------- launches

// Tiles of `rows` rows, at most, of M rows over `groups` adapters: each one's last tile may be short.
int64_t tile_bound(int64_t M, int64_t groups, int64_t rows) { return (M + (rows - 1) * groups) / rows; }

template <int NF>
hipError_t launch_shrink(const LoraArgs& a, hipStream_t stream, int* splits) {
  const int64_t touched = a.M < a.L ? a.M : a.L;
  const int rank_blocks = (a.R + 16 * NF - 1) / (16 * NF), chunks = (a.K + 63) / 64;
  // Tiles of 64 rows need some fifty of them to fill the GPU without more splits of K than the second product
  // reads at ease.  16 rows / 64 rows, us, 4096x4096 with 8 adapters: rank 128 2048 rows 43 / 54, 3000 67 / 57,
  // 4096 76 / 68, 8191 139 / 105; rank 256 2048 rows 73 / 84, 4096 132 / 98.
  const bool stream_rows = NF == 4 && rank_blocks > 1 && tile_bound(a.M, touched, 64) >= 48;
  const int64_t tiles = tile_bound(a.M, touched, stream_rows ? 64 : 16);
  // workgroups to fill the GPU, with four chunks of K or two a wavefront at least
  const int64_t fill = (stream_rows ? 512 : 256) / (tiles * rank_blocks), most_splits = chunks / (stream_rows ? 4 : 16);
  int64_t s = fill < most_splits ? fill : most_splits;
  if (s > lora_max_splits(a.M)) s = lora_max_splits(a.M);
  *splits = s < 1 ? 1 : static_cast<int>(s);
  const int per = rank_blocks * *splits;
  const int64_t most = kMaxThreads / 512 / per;
  for (int64_t at = 0; at < tiles; at += most) {
    const dim3 grid(static_cast<unsigned>((tiles - at < most ? tiles - at : most) * per));
    if (stream_rows)
      shrink_stream_kernel<<<grid, dim3(256), 0, stream>>>(a, static_cast<int>(at), rank_blocks, *splits);
    else
      shrink_kernel<NF><<<grid, dim3(512), 0, stream>>>(a, static_cast<int>(at), rank_blocks, *splits);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

template <class Out, int KS>
hipError_t launch_expand(const LoraArgs& a, int wide, int splits, hipStream_t stream) {
  const int col_blocks = (a.N + 255) / 256;
  const int64_t touched = a.M < a.L ? a.M : a.L;
  // a multiple of 8 for the XCDs; no more than are resident at once
  const int64_t pairs = (tile_bound(a.M, touched + 1, 16) * col_blocks + 7) / 8 * 8;
  const int64_t most = 256 * (KS <= 2 ? 4 : KS == 4 ? 3 : 2);
  expand_kernel<Out, KS><<<dim3(static_cast<unsigned>(pairs < most ? pairs : most)), dim3(256), 0, stream>>>(
      a, col_blocks, wide, splits);
  return hipGetLastError();
}

template <class Out>
hipError_t launch_add(const LoraArgs& a, int wide, hipStream_t stream) {
  const int64_t touched = a.M < a.L ? a.M : a.L;
  const int col_blocks = (a.N + 255) / 256;
  const int64_t small = tile_bound(a.M, touched + 1, 16) * col_blocks;   // and the rows without an adapter
  const int nf = a.R <= 16 ? 1 : a.R <= 32 ? 2 : 4;   // fragments of 16 ranks
  // One launch where no compute unit gets a second workgroup and each one's repeat of the first product
  // is short.  One / two launches, us: 1x4096x4096 rank 8 7.0 / 8.0, 16 8.3 / 8.3, 32 11.7 / 9.4, 64 20.5 / 13.1;
  // 77x1003x2064 rank 32 9.3 / 10.4, 64 13.7 / 14.1; 4x256x1024 rank 64 9.3 / 11.1; 64 adapters' 64 rows of
  // 4096x4096 (1024 workgroups) rank 16 23.3 / 11.2.
  if (a.R <= 64 && small <= 256 && static_cast<int64_t>(16 * nf) * a.K <= 98304) {
    const dim3 grid(static_cast<unsigned>(small)), block(1024);
    if (nf == 1) small_kernel<Out, 1><<<grid, block, 0, stream>>>(a, col_blocks, wide);
    else if (nf == 2) small_kernel<Out, 2><<<grid, block, 0, stream>>>(a, col_blocks, wide);
    else small_kernel<Out, 4><<<grid, block, 0, stream>>>(a, col_blocks, wide);
    return hipGetLastError();
  }
  bool done;
  hipError_t err = launch_lora_tall(a, sizeof(Out) == 4, wide, stream, &done);
  if (err != hipSuccess || done) return err;
  int splits = 1;
  err = nf == 1   ? launch_shrink<1>(a, stream, &splits)
        : nf == 2 ? launch_shrink<2>(a, stream, &splits)
                  : launch_shrink<4>(a, stream, &splits);
  if (err != hipSuccess) return err;
  if (a.R <= 32) return launch_expand<Out, 1>(a, wide, splits, stream);
  if (a.R <= 64) return launch_expand<Out, 2>(a, wide, splits, stream);
  if (a.R <= 128) return launch_expand<Out, 4>(a, wide, splits, stream);
  return launch_expand<Out, 8>(a, wide, splits, stream);
}

}  // namespace

hipError_t launch_lora_add(const LoraArgs& a, bool f32, hipStream_t stream) {
  const int64_t unit = f32 ? 4 : 8;
  const int wide = a.y_stride % unit == 0 && (a.base == nullptr || a.base_stride % unit == 0);
  return f32 ? launch_add<float>(a, wide, stream) : launch_add<uint16_t>(a, wide, stream);
}

}  // namespace moe
