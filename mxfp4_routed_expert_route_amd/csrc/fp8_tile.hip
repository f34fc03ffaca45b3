// Block-scaled FP8 product on LDS tiles: TM activation rows x TN weight rows a workgroup.
//
// K goes in steps of one run (128 elements, 128 bytes a row; KS groups of wavefronts: of KS
// runs, one each, their sums added at the end).  A step's weight and
// activation rows and activation scales are copied to LDS by buffer loads that write LDS
// themselves, ST steps deep, one barrier a step.  A group's wavefronts share the tile as
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
// 16 different 16-byte columns of the 256-byte bank row (no conflicts by the counter).
//
// Measured (rocprofv3).  256 x 256: 8191x4096x4096 125-129 us, 2.2 PFLOP/s, MFMAs busy 0.52 of
// the time; beside them a step's 72 copies take a CU's address unit about 480 ns and the operand
// reads its LDS about 640 of the step's 1950.  Grouped, 12 rows an expert (32 x 256): first product
// 655 us, 6.6 TB/s of weights; 48 rows (96 x 256): 805 us, 5.3 TB/s (MFMAs busy 0.30); each weight is
// read 1.00 times.  One row an expert (16 x 256): 111 us, 6.4 TB/s.
#include <atomic>
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
// 16 bytes a lane from rsrc + voff + soff to LDS address lds + 16 * lane: 8 rows.  The resource's
// range check takes voff alone: rows that are not there have to show in voff, and lanes past the
// resource get zeros.  In assembly so that the compiler, which cannot tell the steps' LDS apart,
// does not wait for all copies before every LDS read; wait_copies counts them.  They write no
// register: the LDS address is an operand in m0, which the compiler sets (the nop is the cycle
// between that and its use).
template <bool kNt>   // kNt: non-temporal
__device__ __forceinline__ void copy16(i32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  if constexpr (kNt)
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen nt lds"
                 :: "v"(voff), "s"(rsrc), "s"(soff), "{m0}"(lds) : "memory");
  else
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
                 :: "v"(voff), "s"(rsrc), "s"(soff), "{m0}"(lds) : "memory");
}
// 4 bytes a lane from rsrc + voff + soff to LDS address lds + 4 * lane.
__device__ __forceinline__ void copy4(i32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_nop 0\n\tbuffer_load_dword %0, %1, %2 offen lds"
               :: "v"(voff), "s"(rsrc), "s"(soff), "{m0}"(lds) : "memory");
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

// Non-temporal: with ordinary stores, the second product of 12,288 rows x 4096 columns (100 MB
// out, 2.1 GB of weights in) takes 436 us, with these 406.
__device__ __forceinline__ void store16(void* p, i32x4 v) {
  __builtin_nontemporal_store(v, static_cast<i32x4*>(p));
}

typedef __attribute__((address_space(4))) const float const_float;
typedef __attribute__((address_space(4))) const int const_int;

constexpr int kXcds = 8;
constexpr int kFewTiles = 64;   // from here on the row tiles spread evenly enough over the XCDs

// Nt: streaming shapes, whose weights are read about once: non-temporal copies of them, the
// column blocks of a tile starting at different runs of K (so that the workgroups of the GPU,
// which step together, do not all read the same columns of the weights, a few kB apart, at a
// time: the 512-token burst's first product 684 -> 660 us), and whole-line stores of h.
// KS: groups of WM x WN wavefronts that take a step's KS runs of K side by side.
template <int TM_, int TN_, int WM_, int WN_, int ST_, bool Nt_, int KS_ = 1>
struct Shape {
  static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_;
  static constexpr int ST = ST_;   // steps in LDS
  static constexpr bool Nt = Nt_;
  static constexpr int KS = KS_;
  static constexpr int NW = WM * WN * KS, threads = 64 * NW;
  static constexpr int MT = TM / WM / 16, NF = TN / WN / 16;
  // 16-byte copies a wavefront issues for a run: activations, then weights.  The rows of
  // activations may not go round evenly: the first `uneven` wavefronts have one more (0: all
  // have copies_a).
  static constexpr int copies_w = TN / 8 / NW, copies_a = (TM / 8 + NW - 1) / NW, uneven = TM / 8 % NW;
  // Scales: one 4-byte copy a step for each 64 rows, by the wavefronts in turn and ahead of the
  // step's other copies.  They are not counted: a wait for the others then also covers them, and
  // one on its way makes a wait end a little later than it has to.  (A 4-byte copy takes a CU's
  // address unit as long as two of the others: one by every wavefront in every step cost the
  // 256 x 256 tile's step 107 of 690 ns of copies.)
  static constexpr int scale_copies = (TM + 63) / 64 == 3 ? 4 : (TM + 63) / 64, turns = NW / scale_copies;
  static constexpr int w_bytes = TN * 128, a_bytes = TM * 128, s_bytes = scale_copies * 256;
  static constexpr int slots = ST * KS, a_at = slots * w_bytes, s_at = a_at + slots * a_bytes;
  static constexpr int red_at = s_at + slots * s_bytes;     // [WN][TM] magnitudes of h's runs
  static constexpr int slots_at = red_at + WN * TM * 4;  // gather entries of the next tile
  static constexpr int h_at = slots_at + s_bytes;        // [TM][128] codes of h
  static constexpr int lds = h_at + (Nt ? TM * 128 : 0);
  static constexpr int per_cu = 160 * 1024 / lds;        // workgroups of a CU
  static_assert(TM % 16 == 0 && TN % (8 * NW) == 0 && NW % scale_copies == 0 && per_cu >= 1, "shape");
  static_assert(ST >= 2 && NW % 2 == 0 && NF % 2 == 0 && (KS == 1 || !Nt), "copies");
};

// Workgroups go through (row tile, column block) pairs; the copies run some steps ahead of the
// products and across pairs, so the next pair's first steps are on their way while this
// one's results are written.
template <class S, int kOut>
__global__ __launch_bounds__(S::threads, S::NW / 4 * S::per_cu)
void tile_kernel(Fp8Product p, int col_blocks) {
  constexpr bool kSwiglu = kOut == kFp8OutSwiglu;
  // which products (mfma_e4m3): the streaming shapes wait for weights, so the gates and ups of
  // h get fp32's there
  constexpr bool kFull = kOut == kFp8OutF32 || (kSwiglu && S::Nt);
  constexpr int MT = S::MT, NF = S::NF, NR = 16 * NF;
  // Steps the copies are ahead.  Streaming shapes fill a step's LDS as soon as its barrier says it
  // has been read; the others a little later, spread over the next step's fragments.
  constexpr int kLate = S::Nt ? 0 : 1, kAhead = S::ST - kLate;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int wm = wave / S::WN % S::WM, wn = wave % S::WN;
  const int ks = wave / (S::WM * S::WN);   // which of a step's runs it takes
  const int K = p.K, nk = (K + kFp8Block - 1) / kFp8Block;
  // steps past nk copy zeros; SwiGLU's next gather entries need some steps to arrive
  constexpr int kLeast = kSwiglu ? 2 * kAhead : kAhead;
  const int all = (nk + S::KS - 1) / S::KS, steps = all < kLeast ? kLeast : all;
  const int half = p.n / 2;
  const int n_blk = (p.n + kFp8Block - 1) / kFp8Block;
  const bool grouped = p.tiles != nullptr;
  const int n_tiles = grouped ? *(const_int*)p.n_tiles : static_cast<int>((p.rows + S::TM - 1) / S::TM);

  // Consecutive workgroups go to the XCDs in turn: XCD x takes row tiles x, x + 8, ..., all
  // column blocks of one from one L2; its workgroups share out the pairs in turn.  With few row
  // tiles it takes column blocks x, x + 8, ... instead where that spreads the pairs more evenly
  // (the FFN of two tokens 70 -> 63 us) or, as evenly, reads fewer bytes: by rows all 8 L2s read all
  // the weights, by columns all the activations (512x4096x2048 13.5 -> 11.2 us).
  const int xcd = blockIdx.x % kXcds;
  const int stride = gridDim.x / kXcds;
  const int most_t = (n_tiles + kXcds - 1) / kXcds * col_blocks;   // the pairs of one XCD
  const int most_c = (col_blocks + kXcds - 1) / kXcds * n_tiles;
  const bool by_cols = n_tiles < kFewTiles && (most_c < most_t || (most_c == most_t && !grouped && p.rows < p.n));
  struct Pair {
    int tile, p_begin, expert, rows, n0;   // n0: first output column
    int first;                             // first run of K it takes
  };
  auto pair_at = [&](int local) {
    Pair w;
    const int per = by_cols ? n_tiles : col_blocks, major = local / per * kXcds + xcd, minor = local % per;
    const int block = by_cols ? major : minor;
    w.tile = by_cols ? (major < col_blocks ? minor : n_tiles) : major;
    w.n0 = block * (kSwiglu ? S::TN / 2 : S::TN);
    w.first = S::Nt ? block * nk / col_blocks : 0;
    w.expert = 0;
    w.rows = 0;
    w.p_begin = 0;
    if (w.tile >= n_tiles) return w;
    if (grouped) {
      const_int* rt = (const_int*)(p.tiles + w.tile);   // expert, p_begin, p_end
      w.expert = rt[0];
      w.p_begin = rt[1];
      w.rows = rt[2] - rt[1];
    } else {
      w.p_begin = w.tile * S::TM;
      const int left = static_cast<int>(p.rows) - w.p_begin;
      w.rows = left < S::TM ? left : S::TM;
    }
    return w;
  };
  int local = blockIdx.x / kXcds;
  Pair cur = pair_at(local);
  if (cur.tile >= n_tiles) return;   // uniform

  // ---- copies: this lane's place in a copy's 8 rows x 128 bytes, and the piece it fetches.
  // A wavefront's copy c goes to LDS rows 8 (wave + NW c) + c_row: all its copies odd or even.
  const int c_row = lane >> 3;
  const uint32_t c_piece = 16u * ((lane & 7) ^ (4 * (wave & 1) + (lane >> 4)));
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) unsigned char*)tile_lds));
  // weight row, from the column block's first, of an LDS row: fragment r / 16 % NF of wn = r / NR
  auto weight_row = [&](int r) {
    const int m = r & 15, f = (r >> 4) % NF, v = r / NR;
    if (!kSwiglu) return v * NR + (f >> 1) * 32 + (m >> 2) * 8 + (f & 1) * 4 + (m & 3);
    const int i = v * (NR / 2) + (m >> 2) * (2 * NF) + (f % (NF / 2)) * 4 + (m & 3);
    return f < NF / 2 ? i : half + i;
  };
  // it is a lane part, weight_row(c_row), plus one that the wavefront shares
  const uint32_t woff = static_cast<uint32_t>(weight_row(c_row)) * static_cast<uint32_t>(K) + c_piece;   // below 2^20
  uint32_t wcopy[S::copies_w];
#pragma unroll
  for (int c = 0; c < S::copies_w; ++c)
    wcopy[c] = static_cast<uint32_t>(weight_row(8 * (wave + S::NW * c))) * static_cast<uint32_t>(K);
  const bool a_short = S::uneven && wave >= S::uneven;   // one copy of activations less
  i32x4 wrs, ars, srs;
  int w_first, a_first;
  uint32_t aoff[S::copies_a], soff;
  const int* next_slots = reinterpret_cast<const int*>(tile_lds + S::slots_at);
  // aims the copies at a pair; its gather entries: read here (first pair) or from LDS
  auto aim = [&](const Pair& w, auto first) {
    // weights: from the column block's first row on, to the expert's last (SwiGLU) or the block's
    const uint8_t* wbase = p.w + (static_cast<int64_t>(w.expert) * p.n + w.n0) * K;
    const int w_rows = kSwiglu ? p.n - w.n0 : (p.n - w.n0 < S::TN ? p.n - w.n0 : S::TN);
    wrs = lds_rsrc(wbase, static_cast<uint32_t>(static_cast<int64_t>(w_rows) * K));
    // activations and their scales: dense, a resource on the tile's rows; grouped, on all
    const int64_t a_row0 = grouped ? 0 : w.p_begin;
    const int64_t a_count = grouped ? p.act_rows : static_cast<int64_t>(w.rows);
    ars = lds_rsrc(p.act + a_row0 * K, static_cast<uint32_t>(a_count * K));
    srs = lds_rsrc(p.act_scale + a_row0 * p.scale_row,
                   static_cast<uint32_t>(4 * ((a_count - 1) * p.scale_row + (nk - 1) * p.scale_k + 1)));
    auto act_row = [&](int r) -> int {   // row in the resource, or -1
      if (r >= w.rows) return -1;
      if (!grouped) return r;
      if (p.gather == nullptr) return w.p_begin + r;
      const int slot = decltype(first)::value ? p.gather[w.p_begin + r] : next_slots[r];
      return static_cast<unsigned>(slot) < static_cast<unsigned>(p.rows) ? slot / p.k_top : -1;
    };
#pragma unroll
    for (int c = 0; c < S::copies_a; ++c) {
      const int row = act_row(8 * (wave + S::NW * c) + c_row);
      aoff[c] = row < 0 ? kRsrcOutOfRange : static_cast<uint32_t>(row) * static_cast<uint32_t>(K) + c_piece;
    }
    const int srow = act_row(64 * (wave % S::scale_copies) + lane);
    soff = srow < 0 ? kRsrcOutOfRange : static_cast<uint32_t>(srow) * static_cast<uint32_t>(p.scale_row) * 4u;
    w_first = a_first = w.first;
  };
  auto run_of = [&](int kb, int first) {   // kb-th run of K; past the last: any
    return kb >= nk ? 0 : S::Nt && kb + first >= nk ? kb + first - nk : kb + first;
  };
  const int short_run = K % kFp8Block ? nk - 1 : -1;   // the run that ends early
  // run kb's scales, if it is this wavefront's turn
  auto copy_s = [&](int kb, int slot) {
    if (static_cast<int>(static_cast<unsigned>(kb) % S::turns) == wave / S::scale_copies)   // uniform
      copy4(srs, soff, static_cast<uint32_t>(run_of(kb, a_first)) * static_cast<uint32_t>(p.scale_k) * 4u,
            lds0 + S::s_at + slot * S::s_bytes + 256 * (wave % S::scale_copies));
  };
  // copy c of run kb's activations.  Past the last run they are not zeros, but the weights are.
  auto copy_a = [&](int c, int kb, int slot) {
    if (c + 1 == S::copies_a && a_short) return;   // uniform
    const int run = run_of(kb, a_first);
    const uint32_t k0 = static_cast<uint32_t>(run) * 128u;
    uint32_t v = aoff[c];
    if (run == short_run) v = static_cast<int>(k0 + c_piece) < K ? v : kRsrcOutOfRange;   // zeros past K
    copy16<false>(ars, v, k0, lds0 + S::a_at + slot * S::a_bytes + 1024 * (wave + S::NW * c));
  };
  // copy c of run kb's weights; zeros past the last run
  auto copy_w = [&](int c, int kb, int slot) {
    const int run = run_of(kb, w_first);
    const uint32_t k0 = static_cast<uint32_t>(run) * 128u;
    // no step: kRsrcOutOfRange and up, with less than 2^20 to add
    uint32_t v = woff + (kb < nk ? wcopy[c] : kRsrcOutOfRange);
    if (run == short_run) v = static_cast<int>(k0 + c_piece) < K ? v : kRsrcOutOfRange;
    copy16<S::Nt>(wrs, v, k0, lds0 + slot * S::w_bytes + 1024 * (wave + S::NW * c));
  };
  constexpr int kRun = 1 + S::copies_a + S::copies_w, kCopies = S::KS * kRun;
  auto copy_part = [&](int part, int step, int slot) {
    const int c = part % kRun, kb = step * S::KS + part / kRun, at = slot * S::KS + part / kRun;
    if (c == 0)
      copy_s(kb, at);
    else if (c <= S::copies_a)
      copy_a(c - 1, kb, at);
    else
      copy_w(c - 1 - S::copies_a, kb, at);
  };
  // waits until only copies on their way for later steps are left, and `more` steps' besides
  auto wait_step = [&](auto more) {
    constexpr int n = S::ST - 2 + decltype(more)::value;
    if (a_short)   // uniform
      wait_copies<n * S::KS * (S::copies_a - 1 + S::copies_w)>();
    else
      wait_copies<n * S::KS * (S::copies_a + S::copies_w)>();
  };
  aim(cur, std::true_type{});
#pragma unroll
  for (int s = 0; s < kAhead; ++s) {
#pragma unroll
    for (int c = 0; c < kCopies; ++c) copy_part(c, s, s);
  }

  const int place = r16 * 128 + 16 * (g ^ ((r16 >> 1) & 7));   // piece g; piece g + 4 is at ^ 64
  auto read_frag = [&](const unsigned char* base, int row0) {
    const i32x4 lo = *reinterpret_cast<const i32x4*>(base + row0 * 128 + place);
    const i32x4 hi = *reinterpret_cast<const i32x4*>(base + row0 * 128 + (place ^ 64));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  const unsigned char* wpart = tile_lds + ks * S::w_bytes;
  const unsigned char* part = tile_lds + S::a_at + ks * S::a_bytes + wm * (S::TM / S::WM) * 128;
  const unsigned char* xpart = tile_lds + S::s_at + ks * S::s_bytes + (wm * (S::TM / S::WM) + r16) * 4;
  int slot = 0, fill = kAhead % S::ST;
  for (;;) {
    local += stride;
    const Pair nxt = pair_at(local);
    const bool more = nxt.tile < n_tiles;
    const int rows = cur.rows, n0 = cur.n0;
    const int64_t p_begin = cur.p_begin;   // 64-bit: output offsets
    const int my_rows = rows - wm * (S::TM / S::WM);   // rows of this wavefront's part

    // weight scales: uniform, read through the constant cache
    const int col = n0 + wn * (kSwiglu ? NR / 2 : NR);
    auto scale_row = [&](int n) {
      const int b = n / kFp8Block < n_blk ? n / kFp8Block : n_blk - 1;   // past n: any (results unused)
      return (const_float*)(p.w_scale + (static_cast<int64_t>(cur.expert) * n_blk + b) * nk);
    };
    const_float* ws0 = scale_row(col);
    const_float* ws1 = scale_row(kSwiglu ? half + col : col);

    floatx4 acc[MT][NF];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int f = 0; f < NF; ++f) acc[m][f] = floatx4{0.f, 0.f, 0.f, 0.f};

    // The K loop over the part's first NS activation fragments.  Within a step, fragment m's
    // MFMAs are issued before fragment m - 1's multiply-adds, which then do not wait for their
    // MFMAs, and fragment m + 1 is read meanwhile.  The step's barrier stands before its last
    // fragment, when its LDS has been read: behind it the next step's weight fragments replace
    // this one's as the last MFMAs take them, and the slot is filled again during the next
    // step, a few copies a fragment (all at once, the wavefronts would stand at the full copy
    // queue instead of multiplying).
    constexpr bool kPast = !kSwiglu && (S::KS > 1 || kAhead > 1);
    constexpr bool kStops = MT * NF <= 24;   // (the largest tile has no registers left for branches)
    auto loop = [&](auto frags) {
      constexpr int NS = decltype(frags)::value;
      wait_step(std::integral_constant<int, kLate ? 0 : 1>{});
      barrier();
      if (kSwiglu && more && wave < S::scale_copies) {
        // the next tile's gather entries: in LDS before they are needed, as the waits of this pair's
        // later steps cover them
        const int r = 64 * wave + lane;
        const i32x4 grs = lds_rsrc(p.gather, static_cast<uint32_t>(p.rows) * 4u);
        copy4(grs, r < nxt.rows ? static_cast<uint32_t>(nxt.p_begin + r) * 4u : kRsrcOutOfRange, 0,
              lds0 + S::slots_at + 256 * wave);
      }
      i32x8 a[NF], b{};
      const int first = S::KS == 1 ? cur.first : ks < nk ? ks : 0;
      float x = 0.f, w0 = ws0[first], w1 = ws1[first];
      if constexpr (NS > 0) {
#pragma unroll
        for (int f = 0; f < NF; ++f) a[f] = read_frag(wpart + slot * S::KS * S::w_bytes, wn * NR + 16 * f);
        b = read_frag(part + slot * S::KS * S::a_bytes, 0);
        x = *reinterpret_cast<const float*>(xpart + slot * S::KS * S::s_bytes);
      }
      // the copies of this pair's steps, then of the next pair's first ones
      int kb = 0, ahead = kAhead;
      bool copying = true;
#pragma unroll 1
      for (int lap = 0; lap < 2; ++lap) {
        const int end = lap == 0 ? steps - kAhead : steps;
        if (lap == 1) {
          copying = more || !kStops;
          ahead = more ? kAhead - steps : 1 << 20;   // no step: zeros
          if (more) aim(nxt, std::false_type{});
        }
#pragma unroll 1
        for (; kb < end; ++kb) {
          const int next = slot + 1 == S::ST ? 0 : slot + 1;
          int kn = (kb + 1) * S::KS + ks;   // its next run
          kn = kn < nk ? kn + cur.first : 0;
          if (S::Nt && kn >= nk) kn -= nk;
          const float w0n = ws0[kn], w1n = kSwiglu ? ws1[kn] : w0n;
          floatx4 d[NF];
          float s0 = 0.f, s1 = 0.f;
#pragma unroll
          for (int m = 0; m < (NS > 0 ? NS : 1); ++m) {
            const bool last = m + 1 >= NS;
            // Where the copies go: streaming shapes, at once behind the barrier; the 256 x 256 tile,
            // some ahead of each of the first half's fragments (its copies are one step ahead only:
            // behind the MFMAs, 8191 x 4096 x 4096 takes 136 instead of 127 us); the others, behind the first
            // fragment's MFMAs (a CU takes in one such copy every 16 cycles, and the wavefronts
            // stand meanwhile), unless the step has no other fragment before its wait.
            constexpr bool kAfter = kLate && NS >= 2 && MT * NF <= 16;
            constexpr int kOver = NS >= 4 ? NS / 2 : 1, kEach = (kCopies + kOver - 1) / kOver;
            if (kLate && !kAfter && (!kStops || copying)) {   // uniform
#pragma unroll
              for (int c = 0; c < kCopies; ++c)
                if (c / kEach == m) copy_part(c, kb + ahead, fill);
            }
            i32x8 b_next = b;
            float x_next = x;
            if (!last) {
              b_next = read_frag(part + slot * S::KS * S::a_bytes, 16 * (m + 1));
              x_next = *reinterpret_cast<const float*>(xpart + slot * S::KS * S::s_bytes + 64 * (m + 1));
            } else {
              wait_lds();
              // this wavefront's copies of the next step; none behind them: all
              if (!kStops || copying)
                wait_step(std::integral_constant<int, 0>{});
              else
                wait_copies<0>();
              barrier();                                     // everybody's; and this step has been read
              if (!kLate && (!kStops || copying)) {
#pragma unroll
                for (int c = 0; c < kCopies; ++c) copy_part(c, kb + ahead, fill);
              }
            }
            if constexpr (NS > 0) {
              if (m > 0) {   // keeps the multiply-adds of fragment m - 1 in this part of the code
#pragma unroll
                for (int f = 0; f < NF; ++f) asm volatile("" : "+v"(d[f]));
              }
              floatx4 dn[NF];
              // past the last run the weights are zeros, the scales any (grouped: none infinite)
              const bool run = !kPast || kb * S::KS + ks < nk;
              const float t0 = run ? x * w0 : 0.f, t1 = kSwiglu ? (run ? x * w1 : 0.f) : t0;
#pragma unroll
              for (int f = 0; f < NF; ++f) {
                dn[f] = mfma_e4m3<kFull>(a[f], b);
                if (last) a[f] = read_frag(wpart + next * S::KS * S::w_bytes, wn * NR + 16 * f);
                if (m > 0) {
                  const float s = f < NF / 2 ? s0 : s1;
#pragma unroll
                  for (int i = 0; i < 4; ++i) acc[m - 1][f][i] = fmaf(d[f][i], s, acc[m - 1][f][i]);
                }
              }
              if (last) {
                b_next = read_frag(part + next * S::KS * S::a_bytes, 0);
                x_next = *reinterpret_cast<const float*>(xpart + next * S::KS * S::s_bytes);
              }
              if (kAfter && m == 0 && (!kStops || copying)) {
                __builtin_amdgcn_sched_barrier(0);   // the MFMAs first
#pragma unroll
                for (int c = 0; c < kCopies; ++c) copy_part(c, kb + ahead, fill);
              }
#pragma unroll
              for (int f = 0; f < NF; ++f) d[f] = dn[f];
              s0 = t0;
              s1 = t1;
              b = b_next;
              x = x_next;
              if (NS * NF > 16) {
#pragma unroll
                for (int f = 0; f < NF; ++f) {
                  __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // one MFMA,
                  __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // one LDS read,
                  __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);   // multiply-adds
                }
                __builtin_amdgcn_sched_barrier(0);
              }
            }
          }
          if constexpr (NS > 0) {
#pragma unroll
            for (int f = 0; f < NF; ++f)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                acc[NS - 1][f][i] = fmaf(d[f][i], f < NF / 2 ? s0 : s1, acc[NS - 1][f][i]);
          }
          w0 = w0n;
          w1 = w1n;
          slot = next;
          fill = fill + 1 == S::ST ? 0 : fill + 1;
        }
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

    // the groups' sums, added in the groups' order: each group finishes every KS-th pair of
    // weight fragments
    auto mine = [&](int m, int f) { return S::KS == 1 || (m * (NF / 2) + f / 2) % S::KS == ks; };
    if constexpr (S::KS > 1) {
      static_assert(S::NW * MT * NF * 1024 <= S::s_at, "in the steps' LDS");
      floatx4* sums = reinterpret_cast<floatx4*>(tile_lds) + wave % (S::WM * S::WN) * (MT * NF * 64) + lane;
      constexpr int kGroup = S::WM * S::WN * MT * NF * 64;
      wait_copies<0>();
      wait_lds();
      barrier();   // no copy and no read of the steps' LDS is left: this was the only pair
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int f = 0; f < NF; ++f) sums[ks * kGroup + (m * NF + f) * 64] = acc[m][f];
      wait_lds();
      barrier();
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int f = 0; f < NF; ++f)
          if (mine(m, f)) {
            floatx4 s = sums[(m * NF + f) * 64];
#pragma unroll
            for (int o = 1; o < S::KS; ++o) s += sums[o * kGroup + (m * NF + f) * 64];
            acc[m][f] = s;
          }
    }

    // ---- results: lane has rows wm part + 16 m + r16, 4 NF (SwiGLU 2 NF) consecutive columns
    if constexpr (kSwiglu) {
      // h, quantised by runs of 128 columns: this workgroup's whole column block
      static_assert(S::TN == 256 && NF % 2 == 0, "one run of h per workgroup");
      uint32_t* red = reinterpret_cast<uint32_t*>(tile_lds + S::red_at);   // [WN][TM] magnitudes
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
        // streaming shapes gather a row's 128 bytes in LDS and store whole lines; the others write
        // their 4 HF bytes
        const int c = wn * (NR / 2) + g * (2 * NF);
        uint32_t* dst = reinterpret_cast<uint32_t*>(
            S::Nt ? tile_lds + S::h_at + r * 128 + c
                  : static_cast<unsigned char*>(hq) + (p_begin + r) * p.ld_out + n0 + c);
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
      if constexpr (S::Nt) {
        wait_lds();
        barrier();
        for (int i = threadIdx.x; i < rows * 8; i += S::threads)
          store16(hq + (p_begin + i / 8) * p.ld_out + n0 + 16 * (i % 8),
                  *reinterpret_cast<const i32x4*>(tile_lds + S::h_at + 16 * i));
      }
    } else {
      // eight columns from 8 g on of every 32
      const int c0 = n0 + wn * NR + 8 * g;
      const bool wide = p.n % 8 == 0;   // rows start on 16 bytes; columns come in whole eights
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int r = wm * (S::TM / S::WM) + 16 * m + r16;
        if (r >= rows) continue;
        const int64_t at = (p_begin + r) * p.ld_out;
#pragma unroll
        for (int f = 0; f < NF; f += 2) {
          if (!mine(m, f)) continue;
          const int c = c0 + 16 * f;
          if (wide && c < p.n) {
            if constexpr (kOut == kFp8OutF32) {
              store16(static_cast<float*>(p.out) + at + c, __builtin_bit_cast(i32x4, acc[m][f]));
              store16(static_cast<float*>(p.out) + at + c + 4, __builtin_bit_cast(i32x4, acc[m][f + 1]));
            } else {
              store16(static_cast<uint16_t*>(p.out) + at + c,
                      i32x4{static_cast<int>(pack_bf16x2(acc[m][f][0], acc[m][f][1])),
                            static_cast<int>(pack_bf16x2(acc[m][f][2], acc[m][f][3])),
                            static_cast<int>(pack_bf16x2(acc[m][f + 1][0], acc[m][f + 1][1])),
                            static_cast<int>(pack_bf16x2(acc[m][f + 1][2], acc[m][f + 1][3]))});
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (c + i >= p.n) break;
              const float v = acc[m][f + i / 4][i % 4];
              if constexpr (kOut == kFp8OutF32)
                static_cast<float*>(p.out)[at + c + i] = v;
              else
                static_cast<uint16_t*>(p.out)[at + c + i] = f32_to_bf16_bits(v);
            }
          }
        }
      }
    }
    if (!more) break;
    cur = nxt;
  }
  wait_copies<0>();   // no copy outlives its workgroup's LDS
}

template <class S, int kOut>
hipError_t launch(const Fp8Product& p, hipStream_t stream) {
  const int cols = kOut == kFp8OutSwiglu ? p.n / 2 : p.n;
  const int per = kOut == kFp8OutSwiglu ? S::TN / 2 : S::TN;
  const int col_blocks = (cols + per - 1) / per;
  const int64_t tiles = p.tiles ? p.tile_bound : (p.rows + S::TM - 1) / S::TM;
  // either way of giving pairs to XCDs; with KS > 1 (outputs of few tiles) a workgroup takes one
  const int64_t by_tiles = (tiles + kXcds - 1) / kXcds * col_blocks, by_cols = (col_blocks + kXcds - 1) / kXcds * tiles;
  const int64_t pairs = kXcds * (by_tiles > by_cols ? by_tiles : by_cols);
  const int64_t most = static_cast<int64_t>(kFp8Cus) * S::per_cu;
  // the kernel's LDS, allowed once on each device
  static std::atomic<uint64_t> allowed{0};
  int dev = 0;
  hipError_t err = hipGetDevice(&dev);
  if (err != hipSuccess) return err;
  const uint64_t bit = uint64_t{1} << (dev & 63);
  if (dev > 63 || !(allowed.load(std::memory_order_relaxed) & bit)) {
    err = hipFuncSetAttribute(reinterpret_cast<const void*>(tile_kernel<S, kOut>),
                              hipFuncAttributeMaxDynamicSharedMemorySize, S::lds);
    if (err != hipSuccess) return err;
    if (dev < 64) allowed.fetch_or(bit, std::memory_order_relaxed);
  }
  tile_kernel<S, kOut><<<dim3(static_cast<unsigned>(pairs < most || S::KS > 1 ? pairs : most)), dim3(S::threads), S::lds,
                         stream>>>(p, col_blocks);
  return hipGetLastError();
}

// fp8_tile_rows has the rule for the rows.  Up to 96 rows the weights are the traffic; at 32 rows
// two workgroups fit a CU and cover each other's barriers and stores.
template <int kOut>
hipError_t launch_grouped(int tile_rows, const Fp8Product& p, hipStream_t stream) {
  if (tile_rows == 16) return launch<Shape<16, 256, 1, 8, 4, true>, kOut>(p, stream);
  if (tile_rows == 32) return launch<Shape<32, 256, 1, 4, 2, true>, kOut>(p, stream);
  if (tile_rows == 96) return launch<Shape<96, 256, 2, 4, 3, true>, kOut>(p, stream);
  return launch<Shape<256, 256, 2, 4, 2, false>, kOut>(p, stream);
}

// The smallest tile of which the output has at most one per CU (fp8_rows.hip has the smallest).
// Small tiles are bound by what a step costs beside its products, so K is shared out as well.
// Measured (us in a graph; the 32 x 64 tile with K in 4 / the rows kernel's / the 64 x 128 tile):
// 128x4096x4096 10.7 / 15.9 / 16.7, 128x4096x2048 8.1 / 9.7 / 10.7; the 32 x 32 tile with K in 4 /
// the rows kernel's: 256x1024x4096 8.6 / 11.8, 64x4096x4096 10.1 / 12.0; the 64 x 64 tile with K
// in 2 / the 64 x 128 tile: 256x4096x4096 13.2 / 16.8, 256x4096x1024 7.2 / 7.6.  The 64 x 128
// tile gains nothing from K in 2 (512 rows: K = 4096 18.0 / 18.5, 2048 11.7 / 11.4, 1024 8.6 / 7.8).
// Two wavefronts a SIMD, one reading while the other multiplies, beat one: 64 x 64 15.6 -> 13.2
// (256x4096x4096), 64 x 128 and a fourth step 18.5 -> 17.5 (512x4096x4096); 128 x 128 as 4 x 2
// wavefronts instead of 2 x 4 26.9 -> 24.8 (1024x4096x4096).
// fp32 results, whose products are bf16 MFMAs on converted operands, take the same tiles but the
// largest (registers); 4096x4096x4096: 130 us with 128 x 256, 172 with 64 x 128.
// Up to 32 rows of more than 65536 columns are a stream of weights, as the grouped FFN's are, and
// take its tile; the 256 x 256 tile (fp32: 128 x 256) / it: 1x70000x4096 114 / 55 (fp32 104 / 55),
// 32x70000x4096 120 / 62, 32x131072x1024 38.5 / 25.7, 1x131072x4096 140 / 87 (6.2 TB/s).
template <int kOut>
hipError_t launch_dense(const Fp8Product& p, hipStream_t stream) {
  auto fits = [&](int tm, int tn) {
    return (p.rows + tm - 1) / tm * ((p.n + tn - 1) / tn) <= kFp8Cus;
  };
  if (fits(32, 32)) return launch<Shape<32, 32, 1, 1, 4, false, 4>, kOut>(p, stream);
  if (fits(32, 64)) return launch<Shape<32, 64, 1, 2, 3, false, 4>, kOut>(p, stream);
  if (fits(64, 64)) return launch<Shape<64, 64, 2, 2, 4, false, 2>, kOut>(p, stream);
  if (fits(64, 128)) return launch<Shape<64, 128, 2, 4, 4, false>, kOut>(p, stream);
  if (fits(128, 128)) return launch<Shape<128, 128, 4, 2, 4, false>, kOut>(p, stream);
  if (fits(128, 256)) return launch<Shape<128, 256, 2, 4, 3, false>, kOut>(p, stream);
  if (p.rows <= 32) return launch<Shape<32, 256, 1, 4, 2, true>, kOut>(p, stream);
  if constexpr (kOut == kFp8OutF32) return launch<Shape<128, 256, 2, 4, 3, false>, kOut>(p, stream);
  if constexpr (kOut == kFp8OutBf16) return launch<Shape<256, 256, 2, 4, 2, false>, kOut>(p, stream);
}

}  // namespace

hipError_t launch_fp8_grouped(int tile_rows, const Fp8Product& p, hipStream_t stream) {
  return p.out_kind == kFp8OutSwiglu ? launch_grouped<kFp8OutSwiglu>(tile_rows, p, stream)
                                     : launch_grouped<kFp8OutBf16>(tile_rows, p, stream);
}

hipError_t launch_fp8_dense(const Fp8Product& p, hipStream_t stream) {
  return p.out_kind == kFp8OutF32 ? launch_dense<kFp8OutF32>(p, stream) : launch_dense<kFp8OutBf16>(p, stream);
}

}  // namespace moe
