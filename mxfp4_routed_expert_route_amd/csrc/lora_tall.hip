// Adapters over many rows, both products in one launch.
//
// A workgroup of eight wavefronts takes up to 64 rows of one adapter.  x and A go to LDS by loads
// that write it themselves, in whole lines (8 rows x 128 bytes a copy), eight chunks of 64 elements
// of K deep; the wavefronts share a chunk out as 16 rows x 32 elements.  The inner sums become bf16
// parts in LDS, and each wavefront goes over blocks of 64 columns with all the rows: B straight to
// registers and base on its way while the block before is worked on, results through LDS so that
// base is read and y written in whole lines.
//
// The rows of a tile are chosen so that the tiles are just under a multiple of the GPU's 256 CUs: one
// tile more than CUs would take as long as two rounds.
#include <atomic>

#include "block.h"
#include "block_plan.h"
#include "lds_copy.h"
#include "lora_core.h"

namespace moe {
namespace {

extern __shared__ __attribute__((aligned(16))) unsigned char tall_lds[];

template <class Out, int NF_>
struct Tall {
  static constexpr int NF = NF_, KS = (NF + 1) / 2, W = 8, kParts = kPartsOf<Out>;
  static constexpr int MT = sizeof(Out) == 4 ? 3 : 4;      // 16-row fragments (registers)
  static constexpr int kStages = 8, kLines = 64 + 16 * NF, stage = kLines * 128;
  static constexpr int part = 64 * KS * 64, sums_at = kParts * part;   // [part][row][32 KS ranks]
  static constexpr int kPitch = 68, exchange = 16 * kPitch * 4;        // floats of a row; a wavefront's
  static constexpr int later = sums_at + (W * exchange > NF * 4096 ? W * exchange : NF * 4096);
  static constexpr int lds = kStages * stage > later ? kStages * stage : later;
  static_assert(lds <= 160 * 1024, "LDS of a CU");
};

template <class Out, int NF>
__global__ __launch_bounds__(512, 2) void tall_kernel(LoraArgs a, int tile_rows, int wide) {
  using S = Tall<Out, NF>;
  constexpr int KS = S::KS, MT = S::MT, kStages = S::kStages, kParts = S::kParts;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const Tiles<0> tiles(a.offsets, a.L, static_cast<int>(a.M), tile_rows);
  if (static_cast<int>(blockIdx.x) >= tiles.total) return;   // uniform over the workgroup
  const Tile tile = tiles.find(blockIdx.x);
  const bool with = tile.adapter < a.L;   // uniform
  if (!with && a.base == a.y) return;
  auto row_of = [&](int r) {   // -1: none
    const int row = a.rows[tile.begin + (r < tile.rows ? r : 0)];
    return r < tile.rows && static_cast<unsigned>(row) < static_cast<unsigned>(a.M) ? row : -1;
  };

  // ---- inner sums
  if (with) {
    const int K = a.K, chunks = (K + 63) / 64;
    // this wavefront's copies of a chunk: eight of the rows, eight of A's ranks
    const bool copies_x = 8 * wave < tile.rows, copies_a = wave < 2 * NF;
    const int line = 8 * wave + (lane >> 3), piece = (lane & 7) ^ ((line >> 1) & 7);
    const int row = copies_x ? row_of(line) : 0, rank = line < a.R ? line : 0;
    const uint16_t* x = a.x + (row < 0 ? 0 : row) * a.x_stride;
    const uint16_t* w = a.a + (static_cast<int64_t>(tile.adapter) * a.R + rank) * K;
    const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
        (__attribute__((address_space(3))) unsigned char*)tall_lds));
    auto copy = [&](int c) {
      const int at = 64 * c + 8 * piece;
      const int k = at < K ? at : 0;   // past K: any, the operands are zeroed
      const uint32_t to = lds0 + c % kStages * S::stage + 1024 * wave;
      if (copies_x) copy16_global(x + k, to);
      if (copies_a) copy16_global(w + k, to + 64 * 128);
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s)
      if (s < chunks) copy(s);
    floatx4 acc[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[f] = floatx4{0.f, 0.f, 0.f, 0.f};
    const int m = wave & 3, h = wave >> 2;   // rows 16 m .. + 15, elements 32 h .. + 31 of a chunk
    const bool busy = 16 * m < tile.rows;    // uniform per wavefront
    const int place = r16 * 128 + 16 * ((4 * h + g) ^ ((r16 >> 1) & 7));
    const int each = (copies_x ? 1 : 0) + (copies_a ? 1 : 0);
    for (int c = 0; c < chunks; ++c) {
      if (c + kStages - 1 < chunks && each == 2)   // uniform: this chunk's copies are the oldest
        wait_copies<2 * (kStages - 2)>();
      else if (c + kStages - 1 < chunks && each == 1)
        wait_copies<kStages - 2>();
      else
        wait_copies<0>();
      wait_lds();
      barrier();   // all wavefronts' copies of it are there, and the chunk before it has been read
      if (c + kStages - 1 < chunks) copy(c + kStages - 1);
      if (!busy) continue;
      const unsigned char* from = tall_lds + c % kStages * S::stage + place;
      bf16x8 v = *reinterpret_cast<const bf16x8*>(from + m * 2048);
      bf16x8 b[NF];
#pragma unroll
      for (int f = 0; f < NF; ++f) b[f] = *reinterpret_cast<const bf16x8*>(from + 64 * 128 + f * 2048);
      if (64 * c + 64 > K) {   // uniform
        const bool here = 64 * c + 32 * h + 8 * g < K;
        const bf16x8 zero = {0, 0, 0, 0, 0, 0, 0, 0};
        v = here ? v : zero;
#pragma unroll
        for (int f = 0; f < NF; ++f) b[f] = here ? b[f] : zero;
      }
#pragma unroll
      for (int f = 0; f < NF; ++f) acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[f], v, acc[f], 0, 0, 0);
    }
    wait_lds();
    barrier();   // the last chunk has been read: its LDS is free
    floatx4* sums = reinterpret_cast<floatx4*>(tall_lds + S::sums_at) + m * NF * 64 + lane;
    if (h == 1)
#pragma unroll
      for (int f = 0; f < NF; ++f) sums[f * 64] = acc[f];
    wait_lds();
    barrier();
    if (h == 0)
#pragma unroll
      for (int f = 0; f < 2 * KS; ++f) {   // ranks past R and past the fragments are zeros
        floatx4 v = {0.f, 0.f, 0.f, 0.f};
        if (f < NF && 16 * f + 4 * g < a.R) v = acc[f < NF ? f : 0] + sums[f * 64];
        const int r = 16 * m + r16, c = 2 * f + (g >> 1);   // 16-byte piece of the row
        unsigned char* to = tall_lds + r * (KS * 64) + 16 * (KS == 2 ? c ^ ((r >> 1) & 7) : c) + 8 * (g & 1);
        float left[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int q = 0; q < kParts; ++q) {
          float d[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            d[j] = q + 1 < kParts ? __uint_as_float(__float_as_uint(left[j]) & 0xFFFF0000u) : left[j];
            if (q + 1 < kParts) left[j] = fabsf(d[j]) < __builtin_inff() ? left[j] - d[j] : 0.f;
          }
          *reinterpret_cast<uint2*>(to + q * S::part) = make_uint2(pack_bf16x2(d[0], d[1]), pack_bf16x2(d[2], d[3]));
        }
      }
    wait_lds();
    barrier();
  }

  // ---- base + v B^T, 64 columns of all the rows at a time
  constexpr int kPiece = 16 / sizeof(Out), kLanes = 64 / kPiece;   // columns of a lane, lanes of a row
  constexpr int kRows = 64 / kLanes, kGoes = 16 / kRows;           // rows of an access, accesses
  const Out* base = static_cast<const Out*>(a.base);
  Out* y = static_cast<Out*>(a.y);
  const int my_col = kPiece * (lane % kLanes);
  int rows[MT][kGoes];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < kGoes; ++i) rows[m][i] = row_of(16 * m + kRows * i + lane / kLanes);
  const float scaling = with && a.scaling != nullptr ? a.scaling[tile.adapter] : 1.0f;
  const int blocks = (a.N + 63) / 64;
  struct In {
    Cols<Out, kPiece> base[MT][kGoes];
    bf16x8 w[KS][4];
  };
  auto load = [&](In& d, int block) {
    const int n0 = 64 * block, left = a.N - n0 - my_col;
    const bool whole = wide && n0 + 64 <= a.N;   // uniform
    if (with)
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const int n = n0 + 16 * f + r16;
        const uint16_t* from = a.b + (static_cast<int64_t>(tile.adapter) * a.N + (n < a.N ? n : 0)) * a.R;
#pragma unroll
        for (int s = 0; s < KS; ++s) d.w[s][f] = load_bf16x8(from + 32 * s + 8 * g, 32 * s + 8 * g < a.R && n < a.N);
      }
#pragma unroll
    for (int m = 0; m < MT; ++m)
      if (16 * m < tile.rows)   // uniform
#pragma unroll
        for (int i = 0; i < kGoes; ++i) {
          d.base[m][i].zero();
          if (base != nullptr && rows[m][i] >= 0)
            d.base[m][i].load(base + rows[m][i] * a.base_stride + n0 + my_col, left, whole);
        }
  };
  float* exchange = reinterpret_cast<float*>(tall_lds + S::sums_at + wave * S::exchange);
  In in;
  if (wave < blocks) load(in, wave);
  for (int block = wave; block < blocks; block += S::W) {
    In next;
    if (block + S::W < blocks) load(next, block + S::W);
    const int n0 = 64 * block, left = a.N - n0 - my_col;
    const bool whole = wide && n0 + 64 <= a.N;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (16 * m >= tile.rows) break;   // uniform
      if (with) {
        floatx4 acc[4];
#pragma unroll
        for (int f = 0; f < 4; ++f) acc[f] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const int r = 16 * m + r16, c = 4 * s + g;
          const unsigned char* from = tall_lds + r * (KS * 64) + 16 * (KS == 2 ? c ^ ((r >> 1) & 7) : c);
#pragma unroll
          for (int q = 0; q < kParts; ++q) {
            const bf16x8 v = *reinterpret_cast<const bf16x8*>(from + q * S::part);
#pragma unroll
            for (int f = 0; f < 4; ++f)
              acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(in.w[s][f], v, acc[f], 0, 0, 0);
          }
        }
        wave_sync_lds();   // the last ones have been read
#pragma unroll
        for (int f = 0; f < 4; ++f)
          *reinterpret_cast<floatx4*>(exchange + r16 * S::kPitch + 16 * f + 4 * g) = acc[f];
        wave_sync_lds();
#pragma unroll
        for (int i = 0; i < kGoes; ++i)
#pragma unroll
          for (int j = 0; j < kPiece; j += 4) {
            const floatx4 d = *reinterpret_cast<const floatx4*>(
                exchange + (kRows * i + lane / kLanes) * S::kPitch + my_col + j);
            Cols<Out, kPiece>& o = in.base[m][i];
            o.put4(j, fmaf(scaling, d[0], o.get(j)), fmaf(scaling, d[1], o.get(j + 1)),
                   fmaf(scaling, d[2], o.get(j + 2)), fmaf(scaling, d[3], o.get(j + 3)));
          }
      }
#pragma unroll
      for (int i = 0; i < kGoes; ++i)
        if (rows[m][i] >= 0) in.base[m][i].store(y + rows[m][i] * a.y_stride + n0 + my_col, left, whole);
    }
    in = next;
  }
}

template <class Out, int NF>
hipError_t launch(const LoraArgs& a, int64_t tiles, int tile_rows, int wide, hipStream_t stream) {
  using S = Tall<Out, NF>;
  // the kernel's LDS, allowed once on each device
  static std::atomic<uint64_t> allowed{0};
  int dev = 0;
  hipError_t err = hipGetDevice(&dev);
  if (err != hipSuccess) return err;
  const uint64_t bit = uint64_t{1} << (dev & 63);
  if (dev > 63 || !(allowed.load(std::memory_order_relaxed) & bit)) {
    err = hipFuncSetAttribute(reinterpret_cast<const void*>(tall_kernel<Out, NF>),
                              hipFuncAttributeMaxDynamicSharedMemorySize, S::lds);
    if (err != hipSuccess) return err;
    if (dev < 64) allowed.fetch_or(bit, std::memory_order_relaxed);
  }
  tall_kernel<Out, NF><<<dim3(static_cast<unsigned>(tiles)), dim3(512), S::lds, stream>>>(a, tile_rows, wide);
  return hipGetLastError();
}

template <class Out>
hipError_t launch_ranked(const LoraArgs& a, int64_t tiles, int tile_rows, int wide, hipStream_t stream) {
  if (a.R <= 16) return launch<Out, 1>(a, tiles, tile_rows, wide, stream);
  if (a.R <= 32) return launch<Out, 2>(a, tiles, tile_rows, wide, stream);
  return launch<Out, 4>(a, tiles, tile_rows, wide, stream);
}

}  // namespace

hipError_t launch_lora_tall(const LoraArgs& a, bool f32, int wide, int least, hipStream_t stream, bool* done) {
  *done = false;
  constexpr int kCus = 256;
  const int64_t groups = (a.M < a.L ? a.M : a.L) + 1;   // and the rows without an adapter
  const int64_t most = 16 * (f32 ? Tall<float, 4>::MT : Tall<uint16_t, 4>::MT);
  if (a.R > 64) return hipSuccess;
  // the fewest rounds of at most kCus tiles that hold all the rows
  int64_t rounds = (a.M + most * groups + most * kCus - 1) / (most * kCus);
  const int64_t rows = (a.M + rounds * kCus - groups - 1) / (rounds * kCus - groups);
  if (rounds * kCus <= groups || rows < least || rows > most) return hipSuccess;
  const int64_t tiles = (a.M + (rows - 1) * groups) / rows;
  if (tiles >= int64_t{1} << 22) return hipSuccess;   // fewer than 2^32 threads
  *done = true;
  const int r = static_cast<int>(rows);
  return f32 ? launch_ranked<float>(a, tiles, r, wide, stream) : launch_ranked<uint16_t>(a, tiles, r, wide, stream);
}

}  // namespace moe
