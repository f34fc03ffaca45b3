// Block-scaled FP8 product on LDS tiles: TM activation rows x TN weight rows a workgroup.
//
// K goes in steps of one run (128 elements, 128 bytes a row).  A step's weight and
// activation rows and activation scales are copied to LDS by buffer loads that write LDS
// themselves, kStages steps deep, one barrier a step.  The wavefronts share the tile as
// WM x WN; a wavefront's part is MT 16-row activation fragments by NF 16-row weight
// fragments.  Weights are the MFMA's A operand, so a lane of D holds four weight rows
// (output columns) of one activation row, and one multiplier, x_scale * w_scale, serves
// its four values: acc += multiplier * D, with D one run's product from zero.
//
// Which weight row sits in which LDS row is free.  Lane m of fragment f takes the row that
// makes a lane's 4 NF values consecutive output columns (SwiGLU: 2 NF gate columns and the
// same up columns), so results go out in 16-byte stores.
//
// LDS layout.  A row is 128 bytes, eight 16-byte pieces; piece c of row r sits at place
// c ^ ((r >> 1) & 7).  A copy moves 8 rows x 128 contiguous bytes (the read shape that
// streams best), lane l to row l / 8, place l % 8.  An operand read takes pieces g and
// g + 4 of row l % 16 (g = l / 16).  128-bit LDS reads go 16 lanes at a time (0-3, 12-15,
// 20-27; then 4-11, 16-19, 28-31; the same plus 32): over such 16 lanes the places fall on
// 16 different 16-byte columns of the 256-byte bank row.
#include <type_traits>

#include "fp8.h"
#include "fp8_common.h"

namespace moe {
namespace {

extern __shared__ __attribute__((aligned(16))) unsigned char tile_lds[];

__device__ __forceinline__ i32x4 lds_rsrc(const void* base, uint32_t bytes) {
  const uint64_t u = reinterpret_cast<uint64_t>(base);
  return i32x4{__builtin_amdgcn_readfirstlane(static_cast<int>(u)),
               __builtin_amdgcn_readfirstlane(static_cast<int>(u >> 32)),
               __builtin_amdgcn_readfirstlane(static_cast<int>(bytes)), 0x00020000};
}
// 16 (4) bytes a lane from rsrc + voff + soff to LDS address lds + 16 (4) * lane; offsets
// voff past the resource give zeros.  In assembly so that the compiler, which cannot tell
// the stages apart, does not wait for all copies before every LDS read; wait_copies counts
// them.  They write no register.
__device__ __forceinline__ void copy16(i32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
               :: "v"(voff), "s"(rsrc), "s"(soff), "s"(lds) : "memory");
}
__device__ __forceinline__ void copy4(i32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dword %0, %1, %2 offen lds"
               :: "v"(voff), "s"(rsrc), "s"(soff), "s"(lds) : "memory");
}
template <int kLeft>
__device__ __forceinline__ void wait_copies() {
  static_assert(kLeft < 64, "the counter's range");
  // vmcnt in bits 3:0 and 15:14, the other counters at their maximum (no wait)
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((kLeft & 15) | ((kLeft >> 4) << 14) | 0x0F70);
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

typedef __attribute__((address_space(4))) const float const_float;

constexpr int kXcds = 8;

template <int TM_, int TN_, int WM_, int WN_, int ST_>
struct Shape {
  static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_, ST = ST_;
  static constexpr int NW = WM * WN, threads = 64 * NW;
  static constexpr int MT = TM / WM / 16, NF = TN / WN / 16;
  static constexpr int copies_w = TN / 8 / NW;                       // per wavefront and step
  static constexpr int copies_a = TM / 8 >= NW ? TM / 8 / NW : 1;
  static constexpr int copies = copies_w + copies_a + 1;
  static constexpr int w_bytes = TN * 128, a_bytes = TM * 128, s_bytes = NW * 256;
  static constexpr int stage = w_bytes + a_bytes + s_bytes;
  static constexpr int lds = ST * stage;
  static_assert(TN % (8 * NW) == 0 && NW % 2 == 0 && TM <= 64 * NW && lds <= 160 * 1024, "shape");
};

template <class S, int kOut>
__global__ __launch_bounds__(S::threads, S::NW == 8 ? 2 : (2 * S::lds <= 160 * 1024 ? 2 : 1))
void tile_kernel(Fp8Product p, int col_blocks, int64_t n_work) {
  constexpr bool kSwiglu = kOut == kFp8OutSwiglu, kFull = kOut == kFp8OutF32;
  constexpr int MT = S::MT, NF = S::NF, NR = 16 * NF;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int wm = wave / S::WN, wn = wave % S::WN;

  // consecutive workgroups go to the XCDs in turn: XCD x takes row tiles x, x + 8, ...,
  // all column blocks of one from one L2
  const int64_t xcd = blockIdx.x % kXcds, local = blockIdx.x / kXcds;
  const int64_t tile = (local / col_blocks) * kXcds + xcd;
  const int nb_col = static_cast<int>(local % col_blocks);
  int expert = 0, rows;
  int64_t p_begin;
  if (p.tiles != nullptr) {
    if (tile >= *p.n_tiles) return;   // uniform
    const RowTile rt = p.tiles[tile];
    expert = __builtin_amdgcn_readfirstlane(rt.expert);
    p_begin = __builtin_amdgcn_readfirstlane(rt.p_begin);
    rows = __builtin_amdgcn_readfirstlane(rt.p_end) - static_cast<int>(p_begin);
  } else {
    p_begin = tile * S::TM;
    if (p_begin >= p.rows) return;
    rows = p.rows - p_begin < S::TM ? static_cast<int>(p.rows - p_begin) : S::TM;
  }
  const int K = p.K, nk = (K + kFp8Block - 1) / kFp8Block;
  const int half = p.n / 2;
  const int n0 = nb_col * (kSwiglu ? S::TN / 2 : S::TN);   // first output column

  // ---- copies: this lane's place in a copy's 8 rows x 128 bytes, and the piece it fetches
  const int c_row = lane >> 3;                                    // copy j: LDS row 8 j + c_row
  const uint32_t c_piece = 16u * ((lane & 7) ^ (4 * (wave & 1) + (lane >> 4)));   // j % 2 = wave % 2
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) unsigned char*)tile_lds));
  // weights: a resource on the expert's slab (SwiGLU) or on this column block's rows
  const uint8_t* wbase = p.w + (static_cast<int64_t>(expert) * p.n + (kSwiglu ? 0 : n0)) * K;
  const int w_rows = kSwiglu ? p.n : (p.n - n0 < S::TN ? p.n - n0 : S::TN);
  const i32x4 wrs = lds_rsrc(wbase, static_cast<uint32_t>(static_cast<int64_t>(w_rows) * K));
  uint32_t woff[S::copies_w];
#pragma unroll
  for (int t = 0; t < S::copies_w; ++t) {
    const int r = 8 * (wave + S::NW * t) + c_row;   // LDS row: fragment r / 16 % NF of wn = r / NR
    const int m = r & 15, f = (r >> 4) % NF, w = r / NR;
    int n;
    if (kSwiglu) {
      const int i = n0 + w * (NR / 2) + (m >> 2) * (2 * NF) + (f % (NF / 2)) * 4 + (m & 3);
      n = f < NF / 2 ? i : half + i;
    } else {
      n = w * NR + (m >> 2) * (4 * NF) + f * 4 + (m & 3);
    }
    woff[t] = n < w_rows ? static_cast<uint32_t>(n) * static_cast<uint32_t>(K) + c_piece : kRsrcOutOfRange;
  }
  // activations and their scales: dense, a resource on the tile's rows; grouped, on all
  const bool grouped = p.tiles != nullptr;
  const int64_t a_first = grouped ? 0 : p_begin, a_count = grouped ? p.act_rows : rows;
  const i32x4 ars = lds_rsrc(p.act + a_first * K, static_cast<uint32_t>(a_count * K));
  const i32x4 srs = lds_rsrc(p.act_scale + a_first * p.scale_row,
                             static_cast<uint32_t>(4 * (p.scale_k == 1 ? a_count * p.scale_row
                                                                       : nk * p.scale_k)));
  auto act_row = [&](int r) -> int64_t {   // row in the resource, or -1
    if (r >= rows) return -1;
    if (!grouped) return r;
    if (p.gather == nullptr) return p_begin + r;
    const int slot = p.gather[p_begin + r];
    return static_cast<unsigned>(slot) < static_cast<unsigned>(p.rows) ? slot / p.k_top : -1;
  };
  uint32_t aoff[S::copies_a];
#pragma unroll
  for (int t = 0; t < S::copies_a; ++t) {
    const int64_t row = act_row(8 * ((wave + S::NW * t) % (S::TM / 8)) + c_row);
    aoff[t] = row < 0 ? kRsrcOutOfRange : static_cast<uint32_t>(row) * static_cast<uint32_t>(K) + c_piece;
  }
  const int64_t srow = act_row(64 * wave + lane);
  const uint32_t soff = srow < 0 ? kRsrcOutOfRange : static_cast<uint32_t>(srow * p.scale_row * 4);
  auto copy_step = [&](int kb, int slot) {
    const uint32_t at = lds0 + slot * S::stage;
    const uint32_t k0 = static_cast<uint32_t>(kb) * 128u;
    const bool in = static_cast<int>(k0 + c_piece) < K;   // past K (a short last run, or no step): zeros
#pragma unroll
    for (int t = 0; t < S::copies_w; ++t)
      copy16(wrs, in ? woff[t] : kRsrcOutOfRange, k0, at + 1024u * (wave + S::NW * t));
#pragma unroll
    for (int t = 0; t < S::copies_a; ++t)
      copy16(ars, in ? aoff[t] : kRsrcOutOfRange, k0,
             at + S::w_bytes + 1024u * ((wave + S::NW * t) % (S::TM / 8)));
    copy4(srs, kb < nk ? soff : kRsrcOutOfRange, static_cast<uint32_t>(kb) * static_cast<uint32_t>(p.scale_k) * 4u,
          at + S::w_bytes + S::a_bytes + 256u * wave);
  };

  // ---- weight scales: uniform, read through the constant cache
  const int n_blk = (p.n + kFp8Block - 1) / kFp8Block;
  const int col = n0 + wn * (kSwiglu ? NR / 2 : NR);
  auto scale_row = [&](int n) {
    const int b = n / kFp8Block < n_blk ? n / kFp8Block : n_blk - 1;   // past n: any (results unused)
    const int64_t at = (static_cast<int64_t>(expert) * n_blk + __builtin_amdgcn_readfirstlane(b)) * nk;
    return (const_float*)(p.w_scale + at);
  };
  const_float* ws0 = scale_row(col);
  const_float* ws1 = scale_row(kSwiglu ? half + col : col);

  floatx4 acc[MT][NF];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[m][f] = floatx4{0.f, 0.f, 0.f, 0.f};

  const int place = r16 * 128 + 16 * (g ^ ((r16 >> 1) & 7));   // piece g; piece g + 4 is at ^ 64
  const int my_rows = rows - wm * (S::TM / S::WM);              // rows of this wavefront's part
  auto read_frag = [&](const unsigned char* base, int row0) {
    const i32x4 lo = *reinterpret_cast<const i32x4*>(base + row0 * 128 + place);
    const i32x4 hi = *reinterpret_cast<const i32x4*>(base + row0 * 128 + (place ^ 64));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  // one step over the part's first NS activation fragments
  auto step = [&](int kb, int slot, auto frags) {
    constexpr int NS = decltype(frags)::value;
    if constexpr (NS == 0) return;
    const unsigned char* st = tile_lds + slot * S::stage;
    const unsigned char* sa = st + S::w_bytes;
    const float* ss = reinterpret_cast<const float*>(sa + S::a_bytes) + wm * (S::TM / S::WM) + r16;
    const float w0 = ws0[kb], w1 = kSwiglu ? ws1[kb] : w0;
    i32x8 a[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) a[f] = read_frag(st, wn * NR + 16 * f);
    const unsigned char* mine = sa + wm * (S::TM / S::WM) * 128;
    i32x8 b = read_frag(mine, 0);
    float x = ss[0];
#pragma unroll
    for (int m = 0; m < NS; ++m) {
      // the next fragment is read while this one multiplies; the compiler, left alone, reads
      // all of them at once and spills
      i32x8 b_next = b;
      float x_next = x;
      if (m + 1 < NS) {
        b_next = read_frag(mine, 16 * (m + 1));
        x_next = ss[16 * (m + 1)];
      }
      const float s0 = x * w0, s1 = kSwiglu ? x * w1 : s0;
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const floatx4 d = mfma_e4m3<kFull>(a[f], b);
        const float s = f < NF / 2 ? s0 : s1;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][f][i] = fmaf(d[i], s, acc[m][f][i]);
      }
      b = b_next;
      x = x_next;
      if (NS * NF > 16) __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto loop = [&](auto frags) {
#pragma unroll
    for (int s = 0; s < S::ST - 1; ++s) copy_step(s, s);
    int slot = 0, fill = S::ST - 1;
    for (int kb = 0; kb < nk; ++kb) {
      wait_copies<(S::ST - 2) * S::copies>();   // this wavefront's copies of step kb are in LDS
      barrier();                                // everybody's are, and step kb - 1 has been read
      copy_step(kb + S::ST - 1, fill);
      step(kb, slot, frags);
      wait_lds();
      slot = slot + 1 == S::ST ? 0 : slot + 1;
      fill = fill + 1 == S::ST ? 0 : fill + 1;
    }
  };
  // only fragments that hold rows are multiplied: the loop for 0, 1, 2, 4 .. MT of them, chosen
  // per wavefront (uniform; every loop meets the same barriers)
  const int need = (my_rows + 15) / 16;
  if (need <= 0)
    loop(std::integral_constant<int, 0>{});
  else if (need <= 1)
    loop(std::integral_constant<int, 1>{});
  else if (MT <= 2 || need <= 2)
    loop(std::integral_constant<int, MT < 2 ? MT : 2>{});
  else if (MT <= 4 || need <= 4)
    loop(std::integral_constant<int, MT < 4 ? MT : 4>{});
  else
    loop(std::integral_constant<int, MT>{});

  // ---- results: lane has rows wm part + 16 m + r16, 4 NF (SwiGLU 2 NF) consecutive columns
  if constexpr (kSwiglu) {
    // h, quantised by runs of 128 columns: this workgroup's whole column block
    static_assert(S::TN == 256 && NF % 2 == 0, "one run of h per workgroup");
    wait_copies<0>();
    barrier();   // LDS is free (the copies past the last step write zeros)
    uint32_t* red = reinterpret_cast<uint32_t*>(tile_lds);   // [WN][TM] magnitudes
    constexpr int HF = NF / 2;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      uint32_t top = 0;
#pragma unroll
      for (int f = 0; f < HF; ++f)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float h = swiglu_fp8(acc[m][f][i], acc[m][HF + f][i], p.limit, p.clamp != 0);
          acc[m][f][i] = h;
          const uint32_t a = __float_as_uint(h) & 0x7FFFFFFFu;
          top = a > top ? a : top;
        }
#pragma unroll
      for (int d = 16; d < 64; d <<= 1) {
        const uint32_t o = static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), d, 64));
        top = o > top ? o : top;
      }
      if (g == 0) red[wn * S::TM + wm * (S::TM / S::WM) + 16 * m + r16] = top;
    }
    wait_lds();
    barrier();
    uint8_t* hq = static_cast<uint8_t*>(p.out);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int r = wm * (S::TM / S::WM) + 16 * m + r16;
      uint32_t top = 0;
#pragma unroll
      for (int w = 0; w < S::WN; ++w) {
        const uint32_t o = red[w * S::TM + r];
        top = o > top ? o : top;
      }
      const bool finite = top < 0x7F800000u;
      const RunScale q = run_scale(finite ? __uint_as_float(top) : 1.0f);
      uint32_t o[HF];
#pragma unroll
      for (int f = 0; f < HF; ++f) {
        const floatx4 h = acc[m][f];
        o[f] = finite ? pack_e4m3(run_quotient(h[0], q), run_quotient(h[1], q), run_quotient(h[2], q),
                                  run_quotient(h[3], q))
                      : kNanCodes;
      }
      if (r >= rows) continue;
      uint32_t* dst = reinterpret_cast<uint32_t*>(hq + (p_begin + r) * p.ld_out + n0 + wn * (NR / 2) + g * (2 * NF));
      if constexpr (HF == 2) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(o[0], o[1]);
      } else {
#pragma unroll
        for (int f = 0; f < HF; ++f) dst[f] = o[f];
      }
      if (wn == 0 && g == 0)
        p.out_scale[static_cast<int64_t>(n0 / kFp8Block) * p.rows + p_begin + r] =
            finite ? q.scale : __uint_as_float(0x7FC00000u);
    }
  } else {
    const int c0 = n0 + wn * NR + g * (4 * NF);
    const bool wide = p.n % 8 == 0;   // rows start on 16 bytes; columns come in whole eights
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int r = wm * (S::TM / S::WM) + 16 * m + r16;
      if (r >= rows) continue;
      const int64_t at = (p_begin + r) * p.ld_out + c0;
      if constexpr (kOut == kFp8OutF32) {
        float* dst = static_cast<float*>(p.out) + at;
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          if (wide && c0 + 4 * f + 4 <= p.n) {
            *reinterpret_cast<floatx4*>(dst + 4 * f) = acc[m][f];
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (c0 + 4 * f + i < p.n) dst[4 * f + i] = acc[m][f][i];
          }
        }
      } else {
        uint16_t* dst = static_cast<uint16_t*>(p.out) + at;
#pragma unroll
        for (int f = 0; f < NF; f += 2) {
          if (wide && c0 + 4 * f + 8 <= p.n) {
            *reinterpret_cast<uint4*>(dst + 4 * f) =
                make_uint4(pack_bf16x2(acc[m][f][0], acc[m][f][1]), pack_bf16x2(acc[m][f][2], acc[m][f][3]),
                           pack_bf16x2(acc[m][f + 1][0], acc[m][f + 1][1]),
                           pack_bf16x2(acc[m][f + 1][2], acc[m][f + 1][3]));
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (c0 + 4 * f + i < p.n) dst[4 * f + i] = f32_to_bf16_bits(acc[m][f + i / 4][i % 4]);
          }
        }
      }
    }
    wait_copies<0>();   // no copy outlives its workgroup's LDS
  }
}

template <class S, int kOut>
hipError_t launch(const Fp8Product& p, hipStream_t stream) {
  const int cols = kOut == kFp8OutSwiglu ? p.n / 2 : p.n;
  const int per = kOut == kFp8OutSwiglu ? S::TN / 2 : S::TN;
  const int col_blocks = (cols + per - 1) / per;
  const int64_t tiles = p.tiles ? p.tile_bound : (p.rows + S::TM - 1) / S::TM;
  const int64_t work = (tiles + kXcds - 1) / kXcds * kXcds * col_blocks;
  static const hipError_t attr = hipFuncSetAttribute(
      reinterpret_cast<const void*>(tile_kernel<S, kOut>), hipFuncAttributeMaxDynamicSharedMemorySize, S::lds);
  if (attr != hipSuccess) return attr;
  tile_kernel<S, kOut><<<dim3(static_cast<unsigned>(work)), dim3(S::threads), S::lds, stream>>>(p, col_blocks, work);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_tile(int tile_rows, const Fp8Product& p, hipStream_t stream) {
  switch (p.out_kind) {
    case kFp8OutSwiglu:
      if (tile_rows <= 32) return launch<Shape<32, 256, 1, 4, 2>, kFp8OutSwiglu>(p, stream);
      if (tile_rows <= 64) return launch<Shape<64, 256, 1, 4, 2>, kFp8OutSwiglu>(p, stream);
      return launch<Shape<256, 256, 2, 4, 2>, kFp8OutSwiglu>(p, stream);
    case kFp8OutF32:
      return launch<Shape<64, 128, 1, 4, 3>, kFp8OutF32>(p, stream);
    default:
      if (tile_rows <= 32) return launch<Shape<32, 256, 1, 4, 2>, kFp8OutBf16>(p, stream);
      if (tile_rows <= 64) return launch<Shape<64, 256, 1, 4, 2>, kFp8OutBf16>(p, stream);
      return launch<Shape<256, 256, 2, 4, 2>, kFp8OutBf16>(p, stream);
  }
}

}  // namespace moe
