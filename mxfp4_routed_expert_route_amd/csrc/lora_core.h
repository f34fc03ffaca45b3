// Shared pieces of the adapters' kernels: tiles of rows, results' columns, inner sums' parts.
#pragma once
#include "block_common.h"

namespace moe {

// Orders a wavefront's LDS accesses where its lanes read what others wrote.
__device__ __forceinline__ void wave_sync_lds() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

struct Tile {
  int adapter;       // L: rows without an adapter
  int begin, rows;   // positions in the grouped order
};

__device__ __forceinline__ int lane_value(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

// Inclusive sums over the wavefront's lanes: row shifts, then broadcasts of rows' last lanes.
__device__ __forceinline__ int lanes_upto(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
  return v;
}

// The batch's tiles, of kRows (0: `size`) rows of one adapter (its last one may have fewer), in the grouped
// order; behind them those of the rows without an adapter.  A wavefront looks at all adapters at
// once, a lane at `per` neighbouring ones, and keeps what it has read.
template <int kRows>
struct Tiles {
  const int32_t* offsets;
  int L, M, size, per;
  int from, rows;   // the lane's adapter, if per is 1
  int n, upto;      // tiles of the lane's adapters, and of all up to them
  int adapters_end, total;

  __device__ __forceinline__ int tile_size() const { return kRows ? kRows : size; }
  __device__ __forceinline__ int tiles_of(int r) const {
    const unsigned each = tile_size();
    return r > 0 ? static_cast<int>((r + each - 1) / each) : 0;
  }
  __device__ __forceinline__ int clamp(int v) const { return v < 0 ? 0 : v > M ? M : v; }

  __device__ __forceinline__ Tiles(const int32_t* offsets_, int L_, int M_, int size_ = kRows)
      : offsets(offsets_), L(L_), M(M_), size(size_), per((L_ + 63) / 64), from(0), rows(0), n(0) {
    const int lane = threadIdx.x & 63;
    adapters_end = clamp(offsets[L]);
    for (int i = 0; i < per; ++i) {   // uniform
      const int a = lane * per + i;
      if (a < L) {
        from = clamp(offsets[a]);
        rows = clamp(offsets[a + 1]) - from;
        n += tiles_of(rows);
      }
    }
    upto = lanes_upto(n);
    adapters_end = __builtin_amdgcn_readfirstlane(adapters_end);
    total = lane_value(upto, 63) + tiles_of(M - adapters_end);
  }
  // Tile t < total.
  __device__ __forceinline__ Tile find(int t) const {
    const uint64_t behind = __builtin_amdgcn_ballot_w64(upto > t);
    if (behind == 0ull) {
      const int begin = adapters_end + (t - lane_value(upto, 63)) * tile_size();
      return cut(L, begin, M - begin);
    }
    const int owner = static_cast<int>(__builtin_ctzll(behind));
    int left = t - (lane_value(upto, owner) - lane_value(n, owner));
    if (per == 1)
      return cut(owner, lane_value(from, owner) + left * tile_size(), lane_value(rows, owner) - left * tile_size());
    // the owner's adapters, one a lane
    const int lane = threadIdx.x & 63, a = owner * per + lane;
    int f = 0, r = 0;
    if (lane < per && a < L) {
      f = clamp(offsets[a]);
      r = clamp(offsets[a + 1]) - f;
    }
    const int own = tiles_of(r), sums = lanes_upto(own);
    const int at = static_cast<int>(__builtin_ctzll(__builtin_amdgcn_ballot_w64(sums > left) | (1ull << 63)));
    left -= lane_value(sums, at) - lane_value(own, at);
    return cut(owner * per + at, lane_value(f, at) + left * tile_size(), lane_value(r, at) - left * tile_size());
  }
  __device__ __forceinline__ Tile cut(int adapter, int begin, int left) const {
    return Tile{adapter, begin, left < tile_size() ? left : tile_size()};
  }
};

__device__ __forceinline__ bf16x8 load_bf16x8(const uint16_t* p, bool here) {
  uint4 d = make_uint4(0u, 0u, 0u, 0u);
  if (here) d = *reinterpret_cast<const uint4*>(p);
  return __builtin_bit_cast(bf16x8, d);
}

__device__ __forceinline__ void load_f32x8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// The first of kParts bf16 parts of v; what it leaves, v less that, is split further.  Three parts are the upper bits
// of what is left each time, the last one rounded: together all 24 bits, for fp32 results.  Of two,
// the first is rounded as well, so that what it leaves is half as much and they hold all but 2^-17 of v, far
// under a bf16 result's step (cut off instead, they lack up to 2^-16).  Sums under 2^-110 hold
// fewer bits: lower parts are subnormal there.  Of an infinity or NaN the last part is one, the others finite.
template <int kParts>
__device__ __forceinline__ float upper_part(float v) {
  constexpr float kMost = kParts > 2 ? 0x1.fffffep+127f : 0x1.fep+127f;   // what does not become an infinity
  v = __builtin_amdgcn_fmed3f(v, -kMost, kMost);
  return kParts > 2 ? __uint_as_float(__float_as_uint(v) & 0xFFFF0000u) : bf16_bits_to_f32(f32_to_bf16_bits(v));
}
template <int kParts>
__device__ __forceinline__ void split(const float (&v)[8], bf16x8 (&part)[kParts]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float left = v[j];
#pragma unroll
    for (int i = 0; i < kParts - 1; ++i) {
      const float h = upper_part<kParts>(left);
      part[i][j] = static_cast<__bf16>(h);
      left -= h;
    }
    part[kParts - 1][j] = static_cast<__bf16>(left);
  }
}
// Infinite weights: the first part of an inner sum makes of one what the sum does, but a lower part may be
// 0, and 0 times an infinity is NaN.  So results that are NaN are made again from whole inner sums, one by
// one: few results, or ones that stay NaN.  `here`: the lane's results are any row's.
template <int n>
__device__ __forceinline__ bool any_nan(const floatx4 (&v)[n], bool here) {   // over the wavefront
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < n; ++i) s += (v[i][0] + v[i][1]) + (v[i][2] + v[i][3]);
  return __builtin_amdgcn_ballot_w64(here && s != s) != 0ull;
}
// sum_r v(r) b[r], up to the first NaN: one in an inner sum, of a row that holds one, costs a term.
template <class Inner>
__device__ __forceinline__ float whole_product(Inner v, const uint16_t* b, int R) {
  float s = 0.f;
#pragma unroll 1
  for (int r = 0; r < R && s == s; ++r) s = fmaf(v(r), bf16_bits_to_f32(b[r]), s);
  return s;
}
template <class Out>
constexpr int kPartsOf = sizeof(Out) == 4 ? 3 : 2;

typedef uint32_t Words __attribute__((ext_vector_type(4)));

// kCols neighbouring columns of a row (4 or a multiple of 8), `left` of them within the matrix;
// whole: all of them, on 16 bytes (4 bf16: on 8).
template <class Out, int kCols>
struct Cols {
  static constexpr int kWords = kCols * sizeof(Out) / 4;
  uint32_t w[kWords];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void load(const Out* p, int left, bool whole) {
    if (whole) {
      if constexpr (kWords == 2) {
        const uint2 d = *reinterpret_cast<const uint2*>(p);
        w[0] = d.x; w[1] = d.y;
      } else {
#pragma unroll
        for (int i = 0; i < kWords; i += 4) {
          const Words d = __builtin_nontemporal_load(reinterpret_cast<const Words*>(p + i * 4 / sizeof(Out)));
          w[i] = d[0]; w[i + 1] = d[1]; w[i + 2] = d[2]; w[i + 3] = d[3];
        }
      }
    } else {
      zero();
#pragma unroll
      for (int j = 0; j < kCols; ++j)
        if (j < left) {
          if constexpr (sizeof(Out) == 4)
            w[j] = __float_as_uint(p[j]);
          else
            w[j / 2] |= static_cast<uint32_t>(p[j]) << (16 * (j & 1));
        }
    }
  }
  __device__ __forceinline__ float get(int j) const {
    if constexpr (sizeof(Out) == 4)
      return __uint_as_float(w[j]);
    else
      return j & 1 ? __uint_as_float(w[j / 2] & 0xFFFF0000u) : bf16_bits_to_f32(w[j / 2] & 0xFFFFu);
  }
  // Four results from column j on.
  __device__ __forceinline__ void put4(int j, float a, float b, float c, float d) {
    if constexpr (sizeof(Out) == 4) {
      w[j] = __float_as_uint(a); w[j + 1] = __float_as_uint(b);
      w[j + 2] = __float_as_uint(c); w[j + 3] = __float_as_uint(d);
    } else {
      w[j / 2] = pack_bf16x2(a, b);
      w[j / 2 + 1] = pack_bf16x2(c, d);
    }
  }
  __device__ __forceinline__ void store(Out* p, int left, bool whole) const {
    if (whole) {
      if constexpr (kWords == 2) {
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
      } else {
#pragma unroll
        for (int i = 0; i < kWords; i += 4)
          __builtin_nontemporal_store(Words{w[i], w[i + 1], w[i + 2], w[i + 3]},
                                      reinterpret_cast<Words*>(p + i * 4 / sizeof(Out)));
      }
    } else {
#pragma unroll
      for (int j = 0; j < kCols; ++j)
        if (j < left) {
          if constexpr (sizeof(Out) == 4)
            p[j] = __uint_as_float(w[j]);
          else
            p[j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
        }
    }
  }
};

}  // namespace moe
