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
// chosen key against the next one; with groups, the last group taken against the first
// left).  If one of them is closer than the two fp32 keys can be off, the token is done
// again with fp64 keys.  With E = 256 normal logits and a bias of sigma 0.1 that is about
// one token in a hundred.  Without a bias the scores' order is the logits', which are
// compared as they are; only sums of two scores (group_top 2) are then rounded.
//   Error of an fp32 key, u = 2^-24: sigmoid = 1 / (1 + e^-l): e^-l within 2u, the sum and
//   the quotient u each: at most 4u of a score <= 1.  Softmax: the argument l - m is rounded
//   (u |l - m|), the exponential adds 2u; the sum, taken in fp64, is off by at most
//   sum_e p_e (u d_e + 2u) <= u (2 + ln E) (d_e = m - l_e, and sum p d <= ln E); conversion
//   and quotient 2u; so p is off by at most p u (d + 2) + 9 p u + 2 p u <= 14 u pmax, as
//   p d <= 0.37 pmax.  Adding the bias rounds by u |key|.  Two keys: 30 u max(smax, |key|)
//   in all; kKeyTol is 32 u, for sums of two keys twice that.
#pragma once
#include "routing_core.h"

namespace moe {

struct ScoreArgs {
  int score;         // 0 softmax, 1 sigmoid
  const float* bias; // nullptr: none
  int groups, per;   // groups, experts per group
  int topk_groups, group_top, renormalize;
  float scale;
  int lanes;         // L
};

constexpr float kKeyTol = 0x1p-19f;

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

__device__ __forceinline__ uint32_t wave_max(uint32_t v) { return wave_max_u32(v); }
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
  const uint32_t hi = static_cast<uint32_t>(v >> 32);
  const uint32_t top = wave_max_u32(hi);
  const uint32_t low = wave_max_u32(hi == top ? static_cast<uint32_t>(v) : 0u);
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
__device__ __forceinline__ uint32_t shfl_xor_key(uint32_t v, int d) {
  return static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), d, 64));
}
__device__ __forceinline__ uint64_t shfl_xor_key(uint64_t v, int d) {
  return (static_cast<uint64_t>(shfl_xor_key(static_cast<uint32_t>(v >> 32), d)) << 32) |
         shfl_xor_key(static_cast<uint32_t>(v), d);
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

__device__ __forceinline__ float exp_of(float x) { return expf(x); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }

__device__ __forceinline__ bool excluded(float l) { return !(l > -__builtin_inff()); }

// exp(l - m) with l = m giving 1 (also at +inf) and an excluded expert 0.
template <class F>
__device__ __forceinline__ F exp_below(float l, float m) {
  if (excluded(l)) return F(0);
  return l == m ? F(1) : exp_of(static_cast<F>(l) - static_cast<F>(m));
}
template <class F>
__device__ __forceinline__ F sigmoid_of(float l) {
  return excluded(l) ? F(0) : F(1) / (F(1) + exp_of(-static_cast<F>(l)));
}

// What the scores of a token rest on: its largest logit and the softmax sum.
struct TokenStats {
  float m;
  double sum;
};

// One selection with keys of type Key (uint32_t: fp32 keys, uint64_t: fp64 keys).  Lane
// j < k returns slot j's expert and logit.  Returns false if fp32 keys cannot decide
// (wave-uniform); fp64 keys always decide.
template <int EPL, class Key>
__device__ __forceinline__ bool select_experts(const float (&l)[EPL], const float (&b)[EPL],
                                               const ScoreArgs& a, const TokenStats& st, int k,
                                               int lane, int n_mine, int& my_id, float& my_logit) {
  using F = decltype(key_value(Key{}));
  constexpr bool kCheck = sizeof(Key) == 4;
  const int L = a.lanes, sub = lane % L, g = lane / L;
  const bool has_bias = a.bias != nullptr;
  const F inv = F(1) / static_cast<F>(st.sum);   // softmax; unused for an empty row
  auto score = [&](float x) -> F {
    if (a.score) return sigmoid_of<F>(x);
    return st.sum > 0.0 ? exp_below<F>(x, st.m) / static_cast<F>(st.sum) : F(0);
  };
  Key key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    if (i >= n_mine) {
      key[i] = 0;
    } else if (excluded(l[i])) {
      key[i] = 1;
    } else if (has_bias) {
      const F v = score(l[i]) + static_cast<F>(b[i]);
      key[i] = v == v ? key_bits(v) : Key(1);   // a NaN bias excludes its expert
    } else {
      key[i] = static_cast<Key>(key_bits(l[i]));
    }
  }
  // largest score, the unit of a key's error
  const float smax = a.score ? 1.0f : static_cast<float>(inv);

  if (a.groups > 1) {
    Key k1 = 0, k2 = 0;   // the group's two largest keys
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      if (key[i] > k1) {
        k2 = k1;
        k1 = key[i];
      } else if (key[i] > k2) {
        k2 = key[i];
      }
    }
    for (int d = 1; d < L; d <<= 1) {
      const Key o1 = shfl_xor_key(k1, d), o2 = shfl_xor_key(k2, d);
      const Key hi = o1 > k1 ? o1 : k1, lo = o1 > k1 ? k1 : o1;
      const Key s = o2 > k2 ? o2 : k2;
      k1 = hi;
      k2 = lo > s ? lo : s;
    }
    Key gk = k1;
    const bool summed = a.group_top == 2;
    if (summed && k1 > 1) {
      F v;
      if (has_bias) {
        v = key_value(k1);
        if (k2 > 1) v += key_value(k2);
      } else {
        v = score(key_value(static_cast<uint32_t>(k1)));
        if (k2 > 1) v += score(key_value(static_cast<uint32_t>(k2)));
      }
      gk = key_bits(v);
    }
    int rank = 0;
    for (int o = 0; o < a.groups; ++o) {
      const Key ok = read_lane(gk, o * L);
      rank += (ok > gk || (ok == gk && o < g)) ? 1 : 0;
    }
    const bool live = g < a.groups, kept = live && rank < a.topk_groups;
    if (kCheck && (has_bias || summed) && a.topk_groups < a.groups) {
      // the last group taken against the first left (excluded groups give NaN: decided)
      const F last = key_value(static_cast<Key>(~wave_max(static_cast<Key>(kept ? ~gk : 0))));
      const F next = key_value(wave_max(static_cast<Key>(live && !kept ? gk : 0)));
      const F unit = fmax(static_cast<F>(smax), fmax(fabs(last), fabs(next)));
      if (last - next <= F(2) * F(kKeyTol) * unit) return false;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (!kept) key[i] = 0;
  }

  my_id = 0;
  my_logit = 0.f;
  F prev = F(0);
  const int rounds = kCheck && has_bias ? k + 1 : k;   // one more: the first key left
  for (int j = 0; j < rounds; ++j) {
    Key mine = key[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) mine = key[i] > mine ? key[i] : mine;
    const Key best = wave_max(mine);   // wave-uniform
    if (best == 0) break;              // nothing left past the k-th
    if (kCheck && has_bias) {
      const F cur = key_value(best);
      if (j > 0 && prev - cur <= F(kKeyTol) * fmax(static_cast<F>(smax), fmax(fabs(prev), fabs(cur))))
        return false;
      prev = cur;
      if (j == k) break;
    }
    // lowest expert holding it: lowest slot within a lane, lowest expert over the lanes
    int at = -1;
    float lg = 0.f;
#pragma unroll
    for (int i = EPL - 1; i >= 0; --i)
      if (key[i] == best) {
        at = i;
        lg = l[i];
      }
    uint64_t holders = __builtin_amdgcn_ballot_w64(at >= 0);
    const int e = g * a.per + sub + L * at;
    if (holders & (holders - 1)) {   // several lanes (wave-uniform)
      const uint32_t low = ~wave_max_u32(at >= 0 ? ~static_cast<uint32_t>(e) : 0u);
      holders = __builtin_amdgcn_ballot_w64(at >= 0 && e == static_cast<int>(low));
    }
    const int win = static_cast<int>(__builtin_ctzll(holders));
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane == win && i == at) key[i] = 0;
    const int e_best = __builtin_amdgcn_readlane(e, win);
    const float l_best = read_lane(lg, win);
    if (lane == j) {
      my_id = e_best;
      my_logit = l_best;
    }
  }
  return true;
}

__device__ __forceinline__ float logit_f32(float v) { return v; }
__device__ __forceinline__ float logit_f32(uint16_t v) { return bf16_bits_to_f32(v); }

template <int EPL, class Logit>
__device__ __forceinline__ void route_scored_token(const Logit* __restrict__ row, int k, int lane,
                                                   const ScoreArgs& a, int& my_id,
                                                   float& my_weight) {
  const int L = a.lanes, sub = lane % L, g = lane / L;
  const int n_mine = g < a.groups && sub < a.per ? (a.per - sub + L - 1) / L : 0;
  float l[EPL], b[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = g * a.per + sub + L * i;
    l[i] = i < n_mine ? logit_f32(row[e]) : -__builtin_inff();
    b[i] = i < n_mine && a.bias != nullptr ? a.bias[e] : 0.f;
  }
  TokenStats st{0.f, 1.0};
  if (a.score == 0) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const uint32_t o = excluded(l[i]) ? 0u : order_bits(l[i]);
      top = o > top ? o : top;
    }
    top = wave_max_u32(top);
    st.m = top ? order_bits_to_f32(top) : 0.f;
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) s += static_cast<double>(exp_below<float>(l[i], st.m));
    st.sum = wave_sum(s);
  }
  float lg;
  if (!select_experts<EPL, uint32_t>(l, b, a, st, k, lane, n_mine, my_id, lg)) {   // uniform
    TokenStats fine = st;
    if (a.score == 0) {
      double s = 0.0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) s += exp_below<double>(l[i], st.m);
      fine.sum = wave_sum(s);
    }
    select_experts<EPL, uint64_t>(l, b, a, fine, k, lane, n_mine, my_id, lg);
  }
  // weights of the chosen: fp32 exponentials, the argument's rounding put back by one
  // term of the series; fp64 sum and quotient
  const bool mine = lane < k;
  float m = st.m;
  if (a.score == 0 && a.renormalize) {   // relative to the largest chosen logit: no underflow
    const uint32_t top = wave_max_u32(mine && !excluded(lg) ? order_bits(lg) : 0u);
    m = top ? order_bits_to_f32(top) : 0.f;
  }
  double s = 0.0;
  if (mine && !excluded(lg)) {
    if (a.score) {
      // below -60 the sum of the chosen scores may leave fp32's range: fp64
      s = lg < -60.f ? sigmoid_of<double>(lg) : static_cast<double>(sigmoid_of<float>(lg));
    } else if (lg == m) {
      s = 1.0;
    } else {
      const double d = static_cast<double>(lg) - static_cast<double>(m);
      const float hi = static_cast<float>(d);
      if (hi > -104.f)   // below, the exponential is under fp32's range
        s = static_cast<double>(expf(hi)) * (1.0 + (d - static_cast<double>(hi)));
    }
  }
  double div = 1.0;
  if (a.renormalize) {
    div = 0.0;
    for (int j = 0; j < k; ++j) div += __shfl(s, j, 64);
  } else if (a.score == 0) {
    div = st.sum;
  }
  my_weight = div > 0.0 ? static_cast<float>(static_cast<double>(a.scale) * s / div) : 0.f;
}

}  // namespace moe
