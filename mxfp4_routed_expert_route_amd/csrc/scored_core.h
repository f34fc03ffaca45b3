// Scored top-k routing of one token by one wavefront.
//
// score s_e = softmax(l)_e or sigmoid(l_e); key = s_e + bias_e; optionally only the
// experts of the best groups; the k largest keys, ties to the lower index.
//
// Layout.  The 64 lanes are cut into G2 = (groups rounded up to a power of two) runs of
// L = 64 / G2 lanes.  Group g's experts g*per .. g*per + per-1 (per = E / groups) sit in
// lanes gL .. gL + L-1, expert g*per + sub + L*i in slot i of lane gL + sub, so a group's
// largest keys come from exchanges within its L lanes and need no LDS.  groups = 1 is the
// plain layout: expert lane + 64 i.
//
// Order.  The keys are ordered as 64-bit arithmetic orders them, at fp32's price: a first
// pass computes them in fp32 and looks at every comparison that the answer rests on (each
// chosen key against the next one; with groups, those taken against those left).  If one of
// them is closer than the fp32 keys can be off, the token is done again with fp64 keys.  With
// E = 256, k = 6, normal logits and a bias of sigma 0.1 that is one token in 40,000 (softmax)
// or 1,600 (sigmoid); such a token's wavefront then takes about 2 us longer.  Without a bias
// the scores' order is the logits', which are compared as they are; only sums of two scores
// (group_top 2) are then rounded.
//   Error of an fp32 key, u = 2^-24: sigmoid = 1 / (1 + e^-l): e^-l within 3u, the sum u, the
//   reciprocal 2u: at most 6u of a score <= 1.  Softmax: the argument l - m is rounded
//   (u |l - m|), the exponential adds 3u; the sum, taken in fp64, is off by at most
//   sum_e p_e (u d_e + 3u) <= u (3 + ln E) (d_e = m - l_e, and sum p d <= ln E); its reciprocal
//   and the product 3u; so p is off by at most p u (d + 3) + 10 p u + 3 p u <= 16.4 u pmax, as
//   p d <= 0.37 pmax.  Adding the bias rounds by u |key|.  Two keys: 35 u max(smax, |key|)
//   in all; kKeyTol is 40 u.  A group's key is one or two of these: off by at most 33 u smax and
//   u times the sum of its terms' magnitudes, and as much again for rounding their sum, which
//   may be far smaller than they are (biases of opposite sign).  With a kGroupTol of 36 u for
//   smax and a kTermTol of 4 u for the magnitudes there is room for rounding the bound itself.
//   Each group has its own error, so all that are taken are compared with all that are left.
//
// Selection.  Up to 8 keys a lane are sorted there first (largest first, equal ones by slot),
// and each of the k rounds then takes the wave-wide maximum of the lanes' first keys and moves
// the winner's list up; with more, each round looks through all of a lane's keys.  With 8 the
// compiler keeps the swaps' masks in more scalar registers than there are (556 spilled, on the
// ordinary path too): 8191 x 512 takes 43 us, 8191 x 1024, unsorted, 26.
#pragma once
#include "routing_core.h"

namespace moe {

struct ScoreArgs {
  int score;         // 0 softmax, 1 sigmoid
  const float* bias; // nullptr: none
  int groups, per;   // groups, experts per group
  int topk_groups, group_top, renormalize;
  float scale;
  int lane_bits;     // log2 L
};

constexpr float kKeyTol = 40 * 0x1p-24f, kGroupTol = 36 * 0x1p-24f, kTermTol = 4 * 0x1p-24f;

// Order-preserving bits; 0: no expert here or already taken, 1: excluded expert.
__device__ __forceinline__ uint32_t key_bits(float f) { return order_bits(f); }
__device__ __forceinline__ uint64_t key_bits(double f) {
  uint64_t u = __builtin_bit_cast(uint64_t, f);
  if ((u << 1) == 0ull) u = 0ull;
  return (u >> 63) ? ~u : (u | (1ull << 63));
}
__device__ __forceinline__ float key_value(uint32_t k) { return order_bits_to_f32(k); }
__device__ __forceinline__ double key_value(uint64_t k) {
  return __builtin_bit_cast(double, (k >> 63) ? (k & ~(1ull << 63)) : ~k);
}

// Lane exchanges on the vector ALU (DPP); lanes a control does not reach read 0.
template <int kCtrl, int kRowMask = 0xF>
__device__ __forceinline__ uint32_t dpp0(uint32_t v) {
  return static_cast<uint32_t>(
      __builtin_amdgcn_update_dpp(0, static_cast<int>(v), kCtrl, kRowMask, 0xF, false));
}
template <int kCtrl, int kRowMask = 0xF>
__device__ __forceinline__ uint64_t dpp0(uint64_t v) {
  return (static_cast<uint64_t>(dpp0<kCtrl, kRowMask>(static_cast<uint32_t>(v >> 32))) << 32) |
         dpp0<kCtrl, kRowMask>(static_cast<uint32_t>(v));
}
template <int kCtrl, int kRowMask = 0xF>
__device__ __forceinline__ double dpp0(double v) {
  return __builtin_bit_cast(double, dpp0<kCtrl, kRowMask>(__builtin_bit_cast(uint64_t, v)));
}
__device__ __forceinline__ uint32_t max_of(uint32_t a, uint32_t b) { return a > b ? a : b; }
// Maximum over the wavefront, wave-uniform: row shifts, then broadcasts of rows' last lanes
// (0 is below every key, so the lanes that a step does not reach keep theirs).
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max_of(v, dpp0<0x111>(v));
  v = max_of(v, dpp0<0x112>(v));
  v = max_of(v, dpp0<0x114>(v));
  v = max_of(v, dpp0<0x118>(v));
  v = max_of(v, dpp0<0x142, 0xA>(v));
  v = max_of(v, dpp0<0x143, 0xC>(v));
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
  const uint32_t hi = static_cast<uint32_t>(v >> 32);
  const uint32_t top = wave_max(hi);
  const uint32_t low = wave_max(hi == top ? static_cast<uint32_t>(v) : 0u);
  return (static_cast<uint64_t>(top) << 32) | low;
}
__device__ __forceinline__ uint32_t read_lane(uint32_t v, int l) {
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), l));
}
__device__ __forceinline__ uint64_t read_lane(uint64_t v, int l) {
  return (static_cast<uint64_t>(read_lane(static_cast<uint32_t>(v >> 32), l)) << 32) |
         read_lane(static_cast<uint32_t>(v), l);
}
__device__ __forceinline__ float read_lane(float v, int l) {
  return __uint_as_float(read_lane(__float_as_uint(v), l));
}
__device__ __forceinline__ double read_lane(double v, int l) {
  return __builtin_bit_cast(double, read_lane(__builtin_bit_cast(uint64_t, v), l));
}
// A value of the other half of the lane's group of 2 d lanes, whose halves each hold one value
// in all their lanes: a swap of neighbours, of pairs, mirrored half rows and rows, then any lane.
template <class Key>
__device__ __forceinline__ Key other_half(Key v, int d) {
  switch (d) {   // uniform
    case 1: return dpp0<0xB1>(v);
    case 2: return dpp0<0x4E>(v);
    case 4: return dpp0<0x141>(v);
    case 8: return dpp0<0x140>(v);
  }
  if constexpr (sizeof(Key) == 4)
    return static_cast<Key>(__shfl_xor(static_cast<int>(v), d, 64));
  else
    return (static_cast<Key>(__shfl_xor(static_cast<int>(v >> 32), d, 64)) << 32) |
           static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), d, 64));
}
__device__ __forceinline__ double wave_sum(double v) {
  v += dpp0<0x111>(v);
  v += dpp0<0x112>(v);
  v += dpp0<0x114>(v);
  v += dpp0<0x118>(v);
  v += dpp0<0x142, 0xA>(v);
  v += dpp0<0x143, 0xC>(v);
  return read_lane(v, 63);
}

// e^x: 2^(x log2 e) by the hardware's exponential, whose argument is rounded, times what the
// rounding left out; off by at most 3u.  Below -110 it is 0 (fp32's smallest is e^-103.3).
__device__ __forceinline__ float exp_of(float x) {
  constexpr float kLog2E = 0x1.715476p+0f, kLog2ELow = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;
  x = x > -110.f ? x : -110.f;
  x = x < 110.f ? x : 110.f;
  const float hi = x * kLog2E;
  const float lo = fmaf(x, kLog2ELow, fmaf(x, kLog2E, -hi));
  return __builtin_amdgcn_exp2f(hi) * fmaf(lo, kLn2, 1.0f);
}
__device__ __forceinline__ double exp_of(double x) { return exp(x); }
__device__ __forceinline__ float inverse(float x) { return __builtin_amdgcn_rcpf(x); }   // 1 ulp
__device__ __forceinline__ double inverse(double x) { return 1.0 / x; }

__device__ __forceinline__ bool excluded(float l) { return !(l > -__builtin_inff()); }

// exp(l - m) with l = m giving 1 (also at +inf) and an excluded expert 0.
template <class F>
__device__ __forceinline__ F exp_below(float l, float m) {
  const F d = l == m ? F(0) : static_cast<F>(l) - static_cast<F>(m);
  const F e = exp_of(d);
  return excluded(l) ? F(0) : e;
}
template <class F>
__device__ __forceinline__ F sigmoid_of(float l) {
  const F s = inverse(F(1) + exp_of(-static_cast<F>(l)));
  return excluded(l) ? F(0) : s;
}

// What the scores of a token rest on: its largest logit and the softmax sum.
struct TokenStats {
  float m;
  double sum;
};

// One selection with keys of type Key (uint32_t: fp32 keys, uint64_t: fp64 keys).  Lane
// j < k returns slot j's expert.  Returns false if fp32 keys cannot decide
// (wave-uniform); fp64 keys always decide.
template <int EPL, class Key>
__device__ __forceinline__ bool select_experts(const float (&l)[EPL], const float (&b)[EPL],
                                               const float (&ex)[EPL],
                                               const ScoreArgs& a, const TokenStats& st, int k,
                                               int lane, int n_mine, int& my_id) {
  using F = decltype(key_value(Key{}));
  constexpr bool kCheck = sizeof(Key) == 4;
  const int L = 1 << a.lane_bits, sub = lane & (L - 1), g = lane >> a.lane_bits;
  const bool has_bias = a.bias != nullptr;
  // softmax: fp32 multiplies by the reciprocal, fp64 divides, as the definition does
  const F sum = static_cast<F>(st.sum), inv = F(1) / sum;
  auto softmax_of = [&](F e) -> F {
    return !(st.sum > 0.0) ? F(0) : kCheck ? e * inv : e / sum;
  };
  auto score = [&](float x) -> F {
    return a.score ? sigmoid_of<F>(x) : softmax_of(exp_below<F>(x, st.m));
  };
  Key key[EPL];
  if (has_bias) {   // uniform, like the score
    F v[EPL];
    if (a.score) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) v[i] = sigmoid_of<F>(l[i]);
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        if constexpr (kCheck)
          v[i] = softmax_of(ex[i]);
        else
          v[i] = softmax_of(exp_below<F>(l[i], st.m));
      }
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const F s = v[i] + static_cast<F>(b[i]);
      key[i] = s == s ? key_bits(s) : Key(1);   // a NaN bias excludes its expert
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = static_cast<Key>(key_bits(l[i]));
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) key[i] = i >= n_mine ? Key(0) : excluded(l[i]) ? Key(1) : key[i];
  // largest score, the unit of a key's error
  const float smax = a.score ? 1.0f : static_cast<float>(inv);

  // expert of each key; sorted by key for the small counts
  constexpr bool kSorted = EPL <= 8;
  int at[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) at[i] = g * a.per + sub + L * i;
  if constexpr (kSorted) {
#pragma unroll
    for (int pass = 0; pass < EPL; ++pass)   // neighbours in turn: equal keys keep their order
#pragma unroll
      for (int i = pass & 1; i + 1 < EPL; i += 2) {
        const bool swap = key[i + 1] > key[i];
        const Key hi = swap ? key[i + 1] : key[i], lo = swap ? key[i] : key[i + 1];
        const int ahi = swap ? at[i + 1] : at[i], alo = swap ? at[i] : at[i + 1];
        key[i] = hi;
        key[i + 1] = lo;
        at[i] = ahi;
        at[i + 1] = alo;
      }
  }

  if (a.groups > 1) {
    Key k1 = key[0], k2 = 0;   // the group's two largest keys
    if constexpr (kSorted) {
      if constexpr (EPL > 1) k2 = key[1];
    } else {
      k1 = 0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        if (key[i] > k1) {
          k2 = k1;
          k1 = key[i];
        } else if (key[i] > k2) {
          k2 = key[i];
        }
      }
    }
    for (int d = 1; d < L; d <<= 1) {
      const Key o1 = other_half(k1, d), o2 = other_half(k2, d);
      const Key hi = o1 > k1 ? o1 : k1, lo = o1 > k1 ? k1 : o1;
      const Key s = o2 > k2 ? o2 : k2;
      k1 = hi;
      k2 = lo > s ? lo : s;
    }
    Key gk = k1;
    const bool summed = a.group_top == 2, rounded = has_bias || summed;   // else logits, as they are
    const bool counted = k1 > 1;
    F v = 0, size = 0;   // the group's key, and its terms' magnitudes
    if (rounded && counted) {
      const bool two = summed && k2 > 1;
      if (has_bias) {
        const F v1 = key_value(k1), v2 = two ? key_value(k2) : F(0);
        v = v1 + v2;
        size = fabs(v1) + fabs(v2);
      } else {
        v = score(key_value(static_cast<uint32_t>(k1)));
        if (two) v += score(key_value(static_cast<uint32_t>(k2)));
        size = v;
      }
      gk = key_bits(v);
    }
    int rank = 0;
    for (int o = 0; o < a.groups; ++o) {
      const Key ok = read_lane(gk, o * L);
      rank += (ok > gk || (ok == gk && o < g)) ? 1 : 0;
    }
    const bool live = g < a.groups, kept = live && rank < a.topk_groups;
    if (kCheck && rounded && a.topk_groups < a.groups) {
      // every group taken, at its least, against every group left, at its most (groups of excluded
      // experts only are left last in any arithmetic: not counted)
      const F err = F(kGroupTol) * static_cast<F>(smax) + F(kTermTol) * size;
      const Key least = static_cast<Key>(~wave_max(static_cast<Key>(kept && counted ? ~key_bits(v - err) : 0)));
      const Key most = wave_max(static_cast<Key>(live && !kept && counted ? key_bits(v + err) : 0));
      if (most != 0 && least <= most) return false;
      if (__builtin_amdgcn_ballot_w64(counted && !(err < __builtin_inff()))) return false;   // past fp32's range
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (!kept) key[i] = 0;
  }

  my_id = 0;
  Key my_key = 0;
  const int rounds = kCheck && has_bias ? k + 1 : k;   // one more: the first key left
  for (int j = 0; j < rounds; ++j) {
    Key mine = key[0];
    int e = at[0];
    if constexpr (!kSorted) {
#pragma unroll
      for (int i = 1; i < EPL; ++i) {   // the lowest expert of the largest
        e = key[i] > mine ? at[i] : e;
        mine = key[i] > mine ? key[i] : mine;
      }
    }
    const Key best = wave_max(mine);   // wave-uniform; 0: nothing left past the k-th
    my_key = lane == j ? best : my_key;
    if (j == k) break;
    // of the lanes that hold it, the one with the lowest expert
    uint64_t holders = __builtin_amdgcn_ballot_w64(mine == best);
    if (holders & (holders - 1)) {   // several lanes (wave-uniform)
      const uint32_t low = ~wave_max(mine == best ? ~static_cast<uint32_t>(e) : 0u);
      holders = __builtin_amdgcn_ballot_w64(mine == best && e == static_cast<int>(low));
    }
    const int win = static_cast<int>(__builtin_ctzll(holders));
    const bool won = lane == win;
    const int e_best = __builtin_amdgcn_readlane(e, win);
    my_id = lane == j ? e_best : my_id;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      if constexpr (kSorted) {
        key[i] = won ? (i + 1 < EPL ? key[i + 1 < EPL ? i + 1 : i] : Key(0)) : key[i];
        if (i + 1 < EPL) at[i] = won ? at[i + 1 < EPL ? i + 1 : i] : at[i];
      } else {
        key[i] = won && at[i] == e ? Key(0) : key[i];
      }
    }
  }
  if (kCheck && has_bias) {
    // lane j: its key against the next one's (excluded experts' keys give NaN: decided)
    const Key below = dpp0<0x101>(my_key);   // lane j + 1 (k + 1 lanes of a row of 16)
    const F cur = key_value(my_key), next = key_value(below);
    const F unit = fmax(static_cast<F>(smax), fmax(fabs(cur), fabs(next)));
    const bool close = lane < k && below != 0 && cur - next <= F(kKeyTol) * unit;
    if (__builtin_amdgcn_ballot_w64(close)) return false;
  }
  return true;
}

__device__ __forceinline__ float logit_f32(float v) { return v; }
__device__ __forceinline__ float logit_f32(uint16_t v) { return bf16_bits_to_f32(v); }

template <int EPL, class Logit>
__device__ __forceinline__ void route_scored_token(const Logit* __restrict__ row, int k, int lane,
                                                   const ScoreArgs& a, int& my_id,
                                                   float& my_weight) {
  const int L = 1 << a.lane_bits, sub = lane & (L - 1), g = lane >> a.lane_bits;
  const int n_mine = g < a.groups ? (a.per - sub + L - 1) >> a.lane_bits : 0;   // <= 0: none
  float l[EPL], b[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = i < n_mine ? g * a.per + sub + L * i : 0;   // a load for every lane, no branch
    l[i] = logit_f32(row[e]);
    b[i] = a.bias != nullptr ? a.bias[e] : 0.f;   // uniform
    if (i >= n_mine) l[i] = -__builtin_inff();
  }
  TokenStats st{0.f, 1.0};
  float ex[EPL] = {};   // softmax: exp(l - m)
  if (a.score == 0) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const uint32_t o = excluded(l[i]) ? 0u : order_bits(l[i]);
      top = o > top ? o : top;
    }
    top = wave_max(top);
    st.m = top ? order_bits_to_f32(top) : 0.f;
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      ex[i] = exp_below<float>(l[i], st.m);
      s += static_cast<double>(ex[i]);
    }
    st.sum = wave_sum(s);
  }
  if (!select_experts<EPL, uint32_t>(l, b, ex, a, st, k, lane, n_mine, my_id)) {   // uniform
    TokenStats fine = st;
    if (a.score == 0) {
      double s = 0.0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) s += exp_below<double>(l[i], st.m);
      fine.sum = wave_sum(s);
    }
    select_experts<EPL, uint64_t>(l, b, ex, a, fine, k, lane, n_mine, my_id);
  }
  // weights of the chosen; fp64 argument and sum, one fp32 quotient
  const bool mine = lane < k;
  const float lg = mine ? logit_f32(row[my_id]) : -__builtin_inff();   // in a cache by now
  float m = st.m;
  if (a.score == 0 && a.renormalize) {   // relative to the largest chosen logit: no underflow
    const uint32_t top = wave_max(excluded(lg) ? 0u : order_bits(lg));
    m = top ? order_bits_to_f32(top) : 0.f;
  }
  double s;
  if (a.score) {   // uniform
    s = static_cast<double>(sigmoid_of<float>(lg));
    // far below 0 the scores of the chosen may leave fp32's range: fp64
    if (__builtin_amdgcn_ballot_w64(!excluded(lg) && lg < -60.f)) s = sigmoid_of<double>(lg);
  } else {
    // e^(lg - m) with the difference's rounding put back by one term of the series
    const double d = lg == m ? 0.0 : static_cast<double>(lg) - static_cast<double>(m);
    const float hi = static_cast<float>(d);
    const double back = hi > -110.f ? d - static_cast<double>(hi) : 0.0;
    s = excluded(lg) ? 0.0 : static_cast<double>(exp_of(hi)) * (1.0 + back);
  }
  double div = 1.0;
  if (a.renormalize) {
    div = 0.0;
    for (int j = 0; j < k; ++j) div += read_lane(s, j);
  } else if (a.score == 0) {
    div = st.sum;
  }
  // scores of a small sum may be denormal in fp32, or 0: divided in fp64 (sigmoid only: the
  // other sums are 1 or more).  From 2^-20 on what fp32 loses of a score is below 2^-130 of the sum.
  const float q = div < 0x1p-20 ? static_cast<float>(s / div)   // uniform
                                : static_cast<float>(s) / static_cast<float>(div);
  my_weight = div > 0.0 ? a.scale * q : 0.f;
}

}  // namespace moe
