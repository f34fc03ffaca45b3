// Adapters over many rows, both products in one launch.
//
// A workgroup of eight wavefronts takes up to 48 rows of one adapter.  x and A go to LDS by loads
// that write it themselves, in whole lines (8 rows x 128 bytes a copy), 128 elements of K a step:
// x, which comes from HBM, eight steps deep, A, which is in L2, three, each copied by wavefronts
// of its own (a wavefront's loads return in order, so one that copied both would wait for the one
// as long as for the other).  The wavefronts share a step out as 16 rows x 64 elements.  The inner
// sums become bf16 parts in LDS, and each wavefront goes over blocks of 64 columns with all the
// rows at once: B straight to registers, it and base on their way while the block before is worked
// on.
//
// The rows of a tile are chosen so that the tiles are just under a multiple of the GPU's 256 CUs: one
// tile more than CUs would take as long as two rounds.
//
// Bound by memory and its requests: 8191 x 4096 x 4096, rank 64, 8 adapters, moves 226 MB by the
// counters (x, base and y once each are 201) in 54 us, 4.2 TB/s, where a copy reaches 5.1; the inner sums
// take about 21 us of that, and with one workgroup a CU the two parts do not overlap.  MFMAs are busy
// 0.15 of the time.  Rank 16 takes 53 us, fp32 base and y (335 MB) 79 at rank 64; without a base, two
// thirds of the bytes, 53.  A second workgroup a CU has neither LDS nor registers: a wavefront holds 202 to
// 256, and of the fp32 form for 64 ranks one spills.  Tried without gain: 16 wavefronts (spills), columns begun
// at another place by each workgroup, non-temporal copies of x.
#include <atomic>
#include <type_traits>

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
  static constexpr int MT = 3, kRows = 16 * MT;                        // 16-row fragments
  static constexpr bool kAhead = sizeof(Out) == 2;                     // base of the next block: registers
  static constexpr int kStepsX = 8, kStepsA = 3;                       // deep
  static constexpr int x_step = kRows * 256, a_step = 16 * NF * 256;   // [half][row][128 bytes]
  static constexpr int a_at = kStepsX * x_step, copies_end = a_at + kStepsA * a_step;
  static constexpr int part = kRows * KS * 64, sums_at = kParts * part;   // [part][row][32 KS ranks]
  static constexpr int kPitch = 68, exchange = 16 * kPitch * 4;        // floats of a row; a wavefront's
  static constexpr int later = sums_at + (W * exchange > MT * NF * 1024 ? W * exchange : MT * NF * 1024);
  static constexpr int lds = copies_end > later ? copies_end : later;   // over half of a CU's: one tile a CU
  static_assert(lds <= 160 * 1024 && lds > 80 * 1024, "LDS of a CU");
};

template <class Out, int NF>
__global__ __launch_bounds__(512, 2) void tall_kernel(LoraArgs a, int tile_rows, int wide) {
  using S = Tall<Out, NF>;
  constexpr int KS = S::KS, kParts = S::kParts;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const Tiles<0> tiles(a.offsets, a.L, static_cast<int>(a.M), tile_rows);
  // consecutive workgroups go to the XCDs in turn: XCD x takes the x-th eighth of the tiles, so that its
  // L2 holds few adapters' weights
  const int per_xcd = (tiles.total + 7) / 8, in_xcd = blockIdx.x / 8;
  const int tile_no = static_cast<int>(blockIdx.x % 8) * per_xcd + in_xcd;
  if (in_xcd >= per_xcd || tile_no >= tiles.total) return;   // uniform over the workgroup
  const Tile tile = tiles.find(tile_no);
  const bool with = tile.adapter < a.L;   // uniform
  if (!with && a.base == a.y) return;

  // ---- inner sums
  if (with) {
    const int K = a.K, steps = (K + 127) / 128;
    // Wavefronts 0 .. 3 copy A, the others x, each two groups of eight ranks or rows, 4 apart.
    const bool is_x = wave >= 4;
    const int group = wave & 3, all = is_x ? (tile.rows + 7) / 8 : 2 * NF;
    const int mine = group + 4 < all ? 2 : group < all ? 1 : 0;   // uniform per wavefront
    const int piece = (lane & 7) ^ (4 * (group & 1) + (lane >> 4));
    const uint16_t* from[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int line = 8 * (group + 4 * i) + (lane >> 3);
      from[i] = a.a + (static_cast<int64_t>(tile.adapter) * a.R + (line < a.R ? line : 0)) * K;
      if (is_x && i < mine) {
        const int row = a.rows[tile.begin + (line < tile.rows ? line : 0)];
        from[i] = a.x + (static_cast<unsigned>(row) < static_cast<unsigned>(a.M) ? row : 0) * a.x_stride;
      }
    }
    const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
        (__attribute__((address_space(3))) unsigned char*)tall_lds));
    auto copy = [&](int step) {
      const uint32_t to = lds0 + 1024 * group +
                          (is_x ? step % S::kStepsX * S::x_step : S::a_at + step % S::kStepsA * S::a_step);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = 128 * step + 64 * h + 8 * piece;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (i < mine)   // past K: any
            copy16_global(from[i] + (at < K ? at : 0), to + 4096 * i + h * (is_x ? S::x_step / 2 : S::a_step / 2));
      }
    };
    const int deep = is_x ? S::kStepsX : S::kStepsA;
    for (int s = 0; s < deep - 1 && s < steps; ++s) copy(s);
    floatx4 acc[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[f] = floatx4{0.f, 0.f, 0.f, 0.f};
    const int m = wave & 3, q = wave >> 2;   // rows 16 m .. + 15, elements 64 q .. + 63 of a step
    const bool busy = 16 * m < tile.rows;    // uniform per wavefront; no rows 48 .. 63
    const int place = r16 * 128 + 16 * (g ^ ((r16 >> 1) & 7));   // piece g; piece g + 4 is at ^ 64
    const unsigned char* x_from = tall_lds + q * (S::x_step / 2) + m * 2048;
    const unsigned char* a_from = tall_lds + S::a_at + q * (S::a_step / 2);
    for (int s = 0; s < steps; ++s) {
      // this step's copies are the oldest
      const int wait = s + deep - 1 < steps ? mine : 0;
      if (wait == 2 && is_x)
        wait_copies<4 * (S::kStepsX - 2)>();
      else if (wait == 1 && is_x)
        wait_copies<2 * (S::kStepsX - 2)>();
      else if (wait == 2)
        wait_copies<4 * (S::kStepsA - 2)>();
      else if (wait == 1)
        wait_copies<2 * (S::kStepsA - 2)>();
      else
        wait_copies<0>();
      wait_lds();
      barrier();   // all wavefronts' copies of it are there, and the step before it has been read
      if (s + deep - 1 < steps) copy(s + deep - 1);
      if (!busy) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = h ? place ^ 64 : place;
        bf16x8 v = *reinterpret_cast<const bf16x8*>(x_from + s % S::kStepsX * S::x_step + at);
        bf16x8 b[NF];
#pragma unroll
        for (int f = 0; f < NF; ++f)
          b[f] = *reinterpret_cast<const bf16x8*>(a_from + s % S::kStepsA * S::a_step + f * 2048 + at);
        if (128 * s + 128 > K) {   // uniform
          const bool here = 128 * s + 64 * q + 32 * h + 8 * g < K;
          const bf16x8 zero = {0, 0, 0, 0, 0, 0, 0, 0};
          v = here ? v : zero;
#pragma unroll
          for (int f = 0; f < NF; ++f) b[f] = here ? b[f] : zero;
        }
#pragma unroll
        for (int f = 0; f < NF; ++f) acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[f], v, acc[f], 0, 0, 0);
      }
    }
    wait_lds();
    barrier();   // the last step has been read: its LDS is free
    floatx4* sums = reinterpret_cast<floatx4*>(tall_lds + S::sums_at) + m * NF * 64 + lane;
    if (q == 1 && busy)
#pragma unroll
      for (int f = 0; f < NF; ++f) sums[f * 64] = acc[f];
    wait_lds();
    barrier();
    if (q == 0 && busy)
#pragma unroll
      for (int f = 0; f < 2 * KS; ++f) {   // ranks past R and past the fragments are zeros
        floatx4 v = {0.f, 0.f, 0.f, 0.f};
        if (f < NF && 16 * f + 4 * g < a.R) {
          v = acc[f < NF ? f : 0] + sums[f * 64];
        }
        const int r = 16 * m + r16, c = 2 * f + (g >> 1);   // 16-byte piece of the row
        unsigned char* to = tall_lds + r * (KS * 64) + 16 * (KS == 2 ? c ^ ((r >> 1) & 7) : c) + 8 * (g & 1);
        float left[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int p = 0; p < kParts; ++p) {
          float d[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            d[j] = p + 1 < kParts ? upper_part<kParts>(left[j]) : left[j];
            if (p + 1 < kParts) left[j] -= d[j];
          }
          *reinterpret_cast<uint2*>(to + p * S::part) = make_uint2(pack_bf16x2(d[0], d[1]), pack_bf16x2(d[2], d[3]));
        }
      }
    wait_lds();
    barrier();
  }

  // ---- base + v B^T, 64 columns of all the rows at a time
  //
  // Without branches around loads and stores: the wait for a block's loads then counts the next
  // block's, which are on their way, as not meant.  (With them it waits for all: 8191 x 4096 x 4096,
  // rank 64, this part alone 47 us.)  A lane whose row is not there does the last row's work as well,
  // and stores the same bits to the same place.
  constexpr int kPiece = 16 / sizeof(Out), kLanes = 64 / kPiece;   // columns of a lane, lanes of a row
  constexpr int kAt = 64 / kLanes, kGoes = 16 / kAt;               // rows of an access, accesses
  // Without a base what is loaded in its place is not used: one row of N * sizeof(Out) <= 2 N R bytes of B, from cache.
  const Out* base = a.base != nullptr ? static_cast<const Out*>(a.base) : reinterpret_cast<const Out*>(a.b);
  const int64_t base_stride = a.base != nullptr ? a.base_stride : 0;
  Out* y = static_cast<Out*>(a.y);
  const int my_row = lane / kLanes, my_col = kPiece * (lane % kLanes);
  float* exchange = reinterpret_cast<float*>(tall_lds + S::sums_at + wave * S::exchange);
  const float scaling = with && a.scaling != nullptr ? a.scaling[tile.adapter] : 1.0f;
  const uint16_t* weights = a.b + static_cast<int64_t>(with ? tile.adapter : 0) * a.N * a.R;
  const bool ragged = a.R < 32 * KS;
  const int blocks = (a.N + 63) / 64, whole = wide ? a.N / 64 : 0;

  auto go = [&](auto fragments) {
    constexpr int MT = decltype(fragments)::value;   // 16-row fragments
    auto there = [&](int r) { return r < tile.rows ? r : tile.rows - 1; };
    int rows[MT][kGoes];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < kGoes; ++i) {
        const int row = a.rows[tile.begin + there(16 * m + kAt * i + my_row)];
        rows[m][i] = static_cast<unsigned>(row) < static_cast<unsigned>(a.M) ? row : 0;
      }
    struct Weights {
      bf16x8 w[KS][4];
    };
    struct Columns {
      Cols<Out, kPiece> c[MT][kGoes];
    };
    // in_full: all 64 columns are there, and rows on 16 bytes
    auto load_weights = [&](auto in_full, Weights& d, int block) {
      constexpr bool kFull = decltype(in_full)::value;
      const int n0 = 64 * block;
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const int n = n0 + 16 * f + r16;
        const uint16_t* from = weights + static_cast<int64_t>(kFull || n < a.N ? n : 0) * a.R;
#pragma unroll
        for (int s = 0; s < KS; ++s) d.w[s][f] = load_bf16x8(from + (32 * s + 8 * g < a.R ? 32 * s + 8 * g : 0), true);
      }
    };
    auto load_base = [&](auto in_full, Columns& d, int block) {
      constexpr bool kFull = decltype(in_full)::value;
      const int n0 = 64 * block, left = a.N - n0 - my_col;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < kGoes; ++i) d.c[m][i].load(base + rows[m][i] * base_stride + n0 + my_col, left, kFull);
    };
    auto work = [&](auto in_full, Weights& b, Columns& d, int block) {
      constexpr bool kFull = decltype(in_full)::value;
      const int n0 = 64 * block, left = a.N - n0 - my_col;
      if (a.base == nullptr)   // uniform, as below
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < kGoes; ++i) d.c[m][i].zero();
      if (with) {
        if (ragged)   // ranks past R: the inner sums are zeros there, an infinity times them would not be
#pragma unroll
          for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int f = 0; f < 4; ++f)
              if (32 * s + 8 * g >= a.R) b.w[s][f] = bf16x8{0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          floatx4 acc[4];
#pragma unroll
          for (int f = 0; f < 4; ++f) acc[f] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            const int r = 16 * m + r16, c = 4 * s + g;   // rows that are not there: any
            const unsigned char* from = tall_lds + r * (KS * 64) + 16 * (KS == 2 ? c ^ ((r >> 1) & 7) : c);
#pragma unroll
            for (int q = 0; q < kParts; ++q) {
              const bf16x8 v = *reinterpret_cast<const bf16x8*>(from + q * S::part);
#pragma unroll
              for (int f = 0; f < 4; ++f)
                acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b.w[s][f], v, acc[f], 0, 0, 0);
            }
          }
          wave_sync_lds();   // the last ones have been read
#pragma unroll
          for (int f = 0; f < 4; ++f)
            *reinterpret_cast<floatx4*>(exchange + r16 * S::kPitch + 16 * f + 4 * g) = acc[f];
          wave_sync_lds();
          if (__builtin_expect(any_nan(acc, 16 * m + r16 < tile.rows), false)) {   // uniform
            const int in_m = tile.rows - 16 * m < 16 ? tile.rows - 16 * m : 16, n = n0 + lane;
#pragma unroll 1
            for (int i = 0; i < in_m; ++i) {
              const int r = 16 * m + i;
              float* at = exchange + i * S::kPitch + lane;
              auto inner = [&](int k) {
                const int c = k >> 3;
                const unsigned char* from = tall_lds + r * (KS * 64) + 16 * (KS == 2 ? c ^ ((r >> 1) & 7) : c) + 2 * (k & 7);
                float s = 0.f;
                for (int q = 0; q < kParts; ++q) s += bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(from + q * S::part));
                return s;
              };
              if (n < a.N && *at != *at) *at = whole_product(inner, weights + static_cast<int64_t>(n) * a.R, a.R);
            }
            wave_sync_lds();
          }
#pragma unroll
          for (int i = 0; i < kGoes; ++i)
#pragma unroll
            for (int j = 0; j < kPiece; j += 4) {
              const int r = there(16 * m + kAt * i + my_row) - 16 * m;   // in fragment m
              const floatx4 v = *reinterpret_cast<const floatx4*>(exchange + r * S::kPitch + my_col + j);
              Cols<Out, kPiece>& o = d.c[m][i];
              o.put4(j, fmaf(scaling, v[0], o.get(j)), fmaf(scaling, v[1], o.get(j + 1)),
                     fmaf(scaling, v[2], o.get(j + 2)), fmaf(scaling, v[3], o.get(j + 3)));
            }
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < kGoes; ++i) d.c[m][i].store(y + rows[m][i] * a.y_stride + n0 + my_col, left, kFull);
    };
    constexpr std::true_type full;
    constexpr std::false_type edge;
    int i = wave;
    Weights w1, w2;   // in turn
    if (i < whole) {
      load_weights(full, w1, i);
      if constexpr (S::kAhead) {
        Columns c1, c2;
        load_base(full, c1, i);
        for (; i + S::W < whole; i += 2 * S::W) {
          load_weights(full, w2, i + S::W);
          load_base(full, c2, i + S::W);
          work(full, w1, c1, i);
          const int after = i + 2 * S::W < whole ? i + 2 * S::W : i;   // past the end: any
          load_weights(full, w1, after);
          load_base(full, c1, after);
          work(full, w2, c2, i + S::W);
        }
        if (i < whole) work(full, w1, c1, i);
      } else {
        for (; i + S::W < whole; i += 2 * S::W) {
          Columns c1, c2;
          load_base(full, c1, i);
          load_weights(full, w2, i + S::W);
          work(full, w1, c1, i);
          load_base(full, c2, i + S::W);
          load_weights(full, w1, i + 2 * S::W < whole ? i + 2 * S::W : i);   // past the end: any
          work(full, w2, c2, i + S::W);
        }
        if (i < whole) {
          Columns c;
          load_base(full, c, i);
          work(full, w1, c, i);
        }
      }
      if (i < whole) i += S::W;
    }
    for (; i < blocks; i += S::W) {
      Columns c;
      load_weights(edge, w1, i);
      load_base(edge, c, i);
      work(edge, w1, c, i);
    }
  };
  if (tile.rows <= 16)
    go(std::integral_constant<int, 1>{});
  else if (tile.rows <= 32)
    go(std::integral_constant<int, 2>{});
  else
    go(std::integral_constant<int, 3>{});
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
  tall_kernel<Out, NF><<<dim3(static_cast<unsigned>((tiles + 7) / 8 * 8)), dim3(512), S::lds, stream>>>(a, tile_rows, wide);
  return hipGetLastError();
}

template <class Out>
hipError_t launch_ranked(const LoraArgs& a, int64_t tiles, int tile_rows, int wide, hipStream_t stream) {
  if (a.R <= 16) return launch<Out, 1>(a, tiles, tile_rows, wide, stream);
  if (a.R <= 32) return launch<Out, 2>(a, tiles, tile_rows, wide, stream);
  return launch<Out, 4>(a, tiles, tile_rows, wide, stream);
}

}  // namespace

hipError_t launch_lora_tall(const LoraArgs& a, bool f32, int wide, hipStream_t stream, bool* done) {
  *done = false;
  constexpr int kCus = 256;
  const int64_t groups = (a.M < a.L ? a.M : a.L) + 1;   // and the rows without an adapter
  const int64_t most = Tall<float, 4>::kRows;
  if (a.R > 64) return hipSuccess;
  // The fewest rounds of at most kCus tiles that hold all the rows: rounds kCus most >= M + most groups, so the
  // rounds have more tiles than groups and the rows come to at most `most`.
  const int64_t rounds = (a.M + most * groups + most * kCus - 1) / (most * kCus);
  const int64_t rows = (a.M + rounds * kCus - groups - 1) / (rounds * kCus - groups);
  // Fewer rows a tile than this read the weights too often for one launch.  One launch / two (us, K = N =
  // 4096, 8 adapters): rank 16, 2048 rows 28.2 / 22.9, 4096 37.1 / 34.0, 5000 40.2 / 41.0, 7000 45.6 / 48.4, 11000
  // 61 / 72; rank 24, 4096 33.8 / 35.8; rank 32, 2048 29.0 / 27.6, 4096 34.5 / 38.5; rank 64, 1500 37.6 / 31.1, 2048
  // 37.8 / 38.6, 3000 39.6 / 43.5.  The rule is not right everywhere: 33 or 34 rows a tile are a third fragment for
  // one or two of them (rank 16, 8191 rows 52.7 / 51.0, 16384 121 / 101), and a rank of 8 gains by two
  // launches up to some 8000 rows (5000 39.9 / 38.3, 9000 54.8 / 57.4).
  const int least = a.R > 32 ? 9 : a.R > 16 ? 17 : 18;
  if (rows < least) return hipSuccess;
  const int64_t tiles = (a.M + (rows - 1) * groups) / rows;
  if (tiles >= (int64_t{1} << 22)) return hipSuccess;   // fewer than 2^32 threads
  *done = true;
  const int r = static_cast<int>(rows);
  return f32 ? launch_ranked<float>(a, tiles, r, wide, stream) : launch_ranked<uint16_t>(a, tiles, r, wide, stream);
}

}  // namespace moe
