// The loss that balances the router's load, and its gradient, over packed sequences.
//
// With c the counts of a token's sequence, everything that a token adds is d = sum_i p_i c_i: the
// loss is E / (k n^2) times the sum of d over the sequence, and the gradient is that factor times
// p_e (c_e - d).  So the counts come first, and one pass over the logits then gives the loss and
// the gradient: no sum per expert is kept.  A workgroup counts a short sequence itself, from all its
// ids; long ones are counted by a launch in front.
//   c is taken less its mean's integer part: p sums to 1, so c_e - d does not change, and an even
//   load, whose gradient is a small difference of large numbers, keeps its digits.
//
// Layout: LPT lanes (16, 32 or 64, by E) take a token, four neighbouring experts a lane and step, so
// that a wavefront's reductions over lanes serve several tokens.
//
// Bound by memory, and by the launches around it: 65536 x 256 with the gradient reads and writes 136
// MB, 26.6 us at a copy's rate; counting takes 5, the main launch 33 to 36, the loss 4.  Fewer and longer
// sequences cost more, since each workgroup adds up its sequence's counting chunks itself: k = 8, with the
// gradient (loss alone), in 16 sequences 39 us (26), in 4 52 (37), in one 100 (86).
#include "block.h"
#include "block_common.h"
#include "block_plan.h"
#include "scored_core.h"

// The kernel's forms give the same bits: no product and sum are one operation but where it says so.
#pragma clang fp contract(off)

namespace moe {
namespace {

// The sequences' offsets.  Up to 63 of them a wavefront holds in its lanes; of more it looks at 64 at a
// time.
struct Sequences {
  const int32_t* offsets;   // nullptr: one of all tokens
  int n;
  int64_t T;
  int mine;                 // offsets[lane], if n < 64

  __device__ __forceinline__ Sequences(const int32_t* offsets_, int n_, int64_t T_)
      : offsets(offsets_), n(n_), T(T_), mine(0) {
    const int lane = threadIdx.x & 63;
    if (offsets != nullptr && n < 64) mine = offsets[lane < n ? lane : n];
  }
  __device__ __forceinline__ int64_t at(int s) const {   // s uniform
    return n < 64 ? __builtin_amdgcn_readlane(mine, s) : __builtin_amdgcn_readfirstlane(offsets[s]);
  }
  // How many of offsets[1 .. n] are at most t: the sequence of token t, n behind the last.
  __device__ __forceinline__ int of(int64_t t) const {
    const int lane = threadIdx.x & 63;
    if (n < 64) return __popcll(__builtin_amdgcn_ballot_w64(lane >= 1 && lane <= n && mine <= t));
    int lo = 0, hi = n;
    while (lo < hi) {
      const int step = (hi - lo + 63) / 64;
      const int64_t i = lo + static_cast<int64_t>(lane + 1) * step;
      const bool below = i <= hi && offsets[i] <= t;
      lo += __popcll(__builtin_amdgcn_ballot_w64(below)) * step;
      const int64_t end = static_cast<int64_t>(lo) + step - 1;
      hi = end < hi ? static_cast<int>(end) : hi;
    }
    return __builtin_amdgcn_readfirstlane(lo);
  }
};

// The tokens from t on that belong together: sequence s (n_seqs: padding) up to `end` <= t1, and where
// the sequence begins and its length.  Offsets that break the rules still give t < end <= t1 and
// 0 <= begin <= t, begin + n <= T.
struct Segment {
  int s;
  int64_t end, begin, n;
};
__device__ __forceinline__ Segment segment_at(const Sequences& q, int64_t t, int64_t t1) {
  if (q.offsets == nullptr) return Segment{0, t1, 0, q.T};
  const int s = q.of(t);
  if (s >= q.n) return Segment{q.n, t1, 0, 1};
  const int64_t begin = q.at(s) > 0 ? q.at(s) : 0;
  int64_t end = q.at(s + 1);
  if (t < begin) return Segment{q.n, begin < t1 ? begin : t1, 0, 1};   // in front of the first
  if (end <= t) end = t + 1;
  if (end > q.T) end = q.T;
  return Segment{s, end < t1 ? end : t1, begin, end - begin};
}

__global__ __launch_bounds__(256) void zero_kernel(int32_t* p, int64_t n) {
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) p[i] = 0;
}

// Counts the experts of pairs i0 .. i1 - 1 in `bins` in LDS, by the whole workgroup; they are there
// after the caller's next barrier.  Eight ids a thread are on their way at once.
__device__ __forceinline__ void count_pairs(const int32_t* ids, int64_t i0, int64_t i1, int E, int* bins) {
  const int n = blockDim.x;
  int e[8];
  auto load = [&](int64_t i) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int64_t at = i + static_cast<int64_t>(u) * n;
      const int id = ids[at < i1 ? at : i1 - 1];
      e[u] = at < i1 ? id : -1;
    }
  };
  load(i0 + threadIdx.x);
  for (int b = threadIdx.x; b < E; b += n) bins[b] = 0;
  __syncthreads();
  for (int64_t i = i0 + threadIdx.x; i < i1; i += 8 * n) {
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (static_cast<unsigned>(e[u]) < static_cast<unsigned>(E)) atomicAdd(&bins[e[u]], 1);
    if (i + 8 * n < i1) load(i + 8 * n);
  }
}

// The long sequences' counts within a chunk of tokens.
__global__ __launch_bounds__(1024) void count_kernel(BalanceArgs a, int chunk) {
  __shared__ int bins[kMaxE];
  const Sequences q(a.offsets, a.n_seqs, a.T);
  int64_t t = static_cast<int64_t>(blockIdx.x) * chunk;
  const int64_t t1 = t + chunk < a.T ? t + chunk : a.T;
  while (t < t1) {   // uniform over the workgroup
    const Segment g = segment_at(q, t, t1);
    if (g.s < a.n_seqs && g.n * a.k > kShortPairs) {
      count_pairs(a.ids, t * a.k, g.end * a.k, a.E, bins);
      __syncthreads();
      int32_t* to = a.partial + (blockIdx.x + g.begin / kLongTokens) * a.E;
      for (int e = threadIdx.x; e < a.E; e += 1024) to[e] = bins[e];
      __syncthreads();
    }
    t = g.end;
  }
}

__device__ __forceinline__ float logit_of(float l) { return l; }
__device__ __forceinline__ float logit_of(uint16_t l) { return bf16_bits_to_f32(l); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = f32_to_bf16_bits(v); }

// Four elements from `e` on of a row of E; past E: `other`.  wide: all four are there, on 16 bytes (8).
template <class Logit>
__device__ __forceinline__ void load4(const Logit* row, int e, int E, bool wide, float other, float (&v)[4]) {
  if (wide) {
    if constexpr (sizeof(Logit) == 4) {
      const float4 d = *reinterpret_cast<const float4*>(row + e);
      v[0] = d.x; v[1] = d.y; v[2] = d.z; v[3] = d.w;
    } else {
      const uint2 d = *reinterpret_cast<const uint2*>(row + e);
      v[0] = bf16_bits_to_f32(d.x & 0xFFFFu); v[1] = __uint_as_float(d.x & 0xFFFF0000u);
      v[2] = bf16_bits_to_f32(d.y & 0xFFFFu); v[3] = __uint_as_float(d.y & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = e + j < E ? logit_of(row[e + j]) : other;
  }
}
template <class Logit>
__device__ __forceinline__ void store4(Logit* row, int e, int E, bool wide, const float (&v)[4]) {
  if (wide) {
    if constexpr (sizeof(Logit) == 4)
      *reinterpret_cast<float4*>(row + e) = make_float4(v[0], v[1], v[2], v[3]);
    else
      *reinterpret_cast<uint2*>(row + e) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (e + j < E) put(row + e + j, v[j]);
  }
}

// exp_of for -110 <= x <= 0.
__device__ __forceinline__ float exp_not_above(float x) {
  constexpr float kLog2E = 0x1.715476p+0f, kLog2ELow = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;
  const float hi = x * kLog2E;
  const float lo = fmaf(x, kLog2ELow, fmaf(x, kLog2E, -hi));
  return __builtin_amdgcn_exp2f(hi) * fmaf(lo, kLn2, 1.0f);
}

// Sigmoid scores under e^-40 are divided as softmax scores: sigmoid(l) = e^l (1 - e^l + ...).
constexpr float kSigmoidLow = -40.f;

// What a launch does: anything, by its arguments; or, for rows of whole aligned fours, one thing alone,
// without a branch around a load or store: the wait for a token's loads then leaves the stores of
// the token before on their way (with branches it waits for those too: 65536 x 256, softmax, 50 us
// for loss and gradient).  A lane behind the last expert does the last four's work as well, kept
// out of the sums, and stores the same bits to the same place.
enum Mode : int { kAny, kLossOnly, kGradient, kGradientAdd };

template <class Logit, int LPT, int I, bool kSigmoid, int kMode>
__global__ __launch_bounds__(256) void balance_kernel(BalanceArgs a, int chunk, int count_chunk) {
  constexpr int G = 64 / LPT, kAtOnce = 4 * G;   // tokens per wavefront, per workgroup
  __shared__ double part[kAtOnce];
  __shared__ int live[kAtOnce];
  __shared__ int bins[kMaxE];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int sub = lane & (LPT - 1), group = wave * G + lane / LPT;
  const int E = a.E;
  constexpr bool kWide = kMode != kAny;
  const bool gradient = kMode == kAny ? a.dlogits != nullptr : kMode != kLossOnly;
  const bool adds = kMode == kAny ? a.add != nullptr : kMode == kGradientAdd;
  const Logit* logits = static_cast<const Logit*>(a.logits);
  const Logit* add = static_cast<const Logit*>(a.add);
  Logit* out = static_cast<Logit*>(a.dlogits);
  int at[I];   // the lane's first experts
  bool here[I];
#pragma unroll
  for (int i = 0; i < I; ++i) {
    at[i] = 4 * (sub + LPT * i);
    here[i] = at[i] < E;
    if (kWide && !here[i]) at[i] = E - 4;
  }
  const Sequences q(a.offsets, a.n_seqs, a.T);
  int64_t t = static_cast<int64_t>(blockIdx.x) * chunk;
  const int64_t t1 = t + chunk < a.T ? t + chunk : a.T;
  while (t < t1) {   // uniform over the workgroup
    const Segment g = segment_at(q, t, t1);
    if (g.s >= a.n_seqs) {   // padding
      if (gradient)
        for (int64_t r = t + group; r < g.end; r += kAtOnce)
#pragma unroll
          for (int i = 0; i < I; ++i) {
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            if (adds) load4(add + r * E, at[i], E, kWide, 0.f, v);
            store4(out + r * E, at[i], E, kWide, v);
          }
      t = g.end;
      continue;
    }
    float l[I][4], v[I][4];
    auto load = [&](int64_t r) {   // past the end: the last token again
      const int64_t row = r < g.end ? r : g.end - 1;
#pragma unroll
      for (int i = 0; i < I; ++i) {
        load4(logits + row * E, at[i], E, kWide, -__builtin_inff(), l[i]);
        if (adds) load4(add + row * E, at[i], E, kWide, 0.f, v[i]);
      }
    };
    load(t + group);   // on their way while the counts are made
    const int64_t mean = g.n * a.k / E;
    float c[I][4];
    const int32_t* counts = a.counts + static_cast<int64_t>(g.s) * E;
    if (a.ids != nullptr) {
      if (g.n * a.k <= kShortPairs) {
        count_pairs(a.ids, g.begin * a.k, (g.begin + g.n) * a.k, E, bins);
      } else {
        const int64_t first = g.begin / count_chunk, last = (g.begin + g.n - 1) / count_chunk;
        for (int e = threadIdx.x; e < E; e += 256) {
          int n = 0;
          for (int64_t j = first; j <= last; ++j) n += a.partial[(j + g.begin / kLongTokens) * E + e];
          bins[e] = n;
        }
      }
      __syncthreads();
      if (t == g.begin)
        for (int e = threadIdx.x; e < E; e += 256) a.counts[static_cast<int64_t>(g.s) * E + e] = bins[e];
      counts = bins;
    }
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = at[i] + j;
        c[i][j] = e < E ? static_cast<float>(counts[e] - mean) : 0.f;
      }
    float factor = 0.f;
    if (gradient)
      factor = static_cast<float>(static_cast<double>(a.dloss[g.s]) * E /
                                  (static_cast<double>(a.k) * g.n * g.n));
    double total = 0.0;
    int tokens = 0;
    for (int64_t r = t + group; r < g.end; r += kAtOnce) {
      float m = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < I; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) m = fmaxf(m, l[i][j]);   // a NaN is left out
      m = run_max<LPT>(m);
      const bool sigmoid = kSigmoid && m > kSigmoidLow, infinite = m == __builtin_inff();
      float p[I][4], slope[I][4], sum = 0.f, dot = 0.f;
#pragma unroll
      for (int i = 0; i < I; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (sigmoid) {
            // 1 / (1 + e^-l), and 1 minus that as e^-l times it; below -87 0, and for -inf and NaN
            const float y = l[i][j] >= -87.f ? exp_of(-l[i][j]) : 0x1p+126f, s = inverse(1.0f + y);
            p[i][j] = l[i][j] >= -87.f ? s : 0.f;
            slope[i][j] = y < 0x1p+126f ? y * s : 1.0f;
          } else {
            // below -110, and for -inf and NaN, 0: the maximum with a number drops a NaN
            const float d = fmaxf(l[i][j] - m, -110.f);
            p[i][j] = exp_not_above(infinite && l[i][j] == m ? 0.f : d);
            slope[i][j] = 1.0f;
          }
          const float s = kWide && !here[i] ? 0.f : p[i][j];
          sum += s;
          dot = fmaf(s, c[i][j], dot);
        }
      sum = run_sum<LPT>(sum);
      dot = run_sum<LPT>(dot);
      const float inv = sum > 0.f ? inverse(sum) : 0.f;
      const float d = dot * inv;
      total += d;
      tokens += sum > 0.f;
      if (gradient) {   // uniform
        const float by = factor * inv;
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float y = by * p[i][j] * (c[i][j] - d);
            if (kSigmoid) y *= slope[i][j];
            p[i][j] = adds ? y + v[i][j] : y;
          }
      }
      load(r + kAtOnce);   // the next token's on their way
      if (gradient)
#pragma unroll
        for (int i = 0; i < I; ++i) store4(out + r * E, at[i], E, kWide, p[i]);
    }
    if (a.slots != nullptr) {
      if (sub == 0) part[group] = total, live[group] = tokens;
      __syncthreads();
      if (threadIdx.x == 0) {
        double sum = 0.0;
        int n = 0;
        for (int i = 0; i < kAtOnce; ++i) sum += part[i], n += live[i];
        a.slots[blockIdx.x + static_cast<int64_t>(g.s)] = sum + static_cast<double>(mean) * n;
      }
    }
    if (a.ids != nullptr) __syncthreads();   // the bins and sums are free
    t = g.end;
  }
}

// loss[s]: a wavefront adds the sums that the chunks left for its sequence; an empty one's counts.
__global__ __launch_bounds__(256) void loss_kernel(BalanceArgs a, int chunk) {
  const int lane = threadIdx.x & 63;
  const int64_t s = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (s >= a.n_seqs) return;   // uniform per wavefront
  int64_t begin = 0, end = a.T;
  if (a.offsets != nullptr) {
    begin = a.offsets[s] > 0 ? a.offsets[s] : 0;
    end = a.offsets[s + 1] < a.T ? a.offsets[s + 1] : a.T;
  }
  double v = 0.0;
  if (begin < end)
    for (int64_t c = begin / chunk + lane; c <= (end - 1) / chunk; c += 64) v += a.slots[c + s];
  v = wave_sum(v);
  const double n = static_cast<double>(end - begin);
  if (begin >= end)
    for (int e = lane; e < a.E; e += 64) a.counts[s * a.E + e] = 0;
  if (lane == 0) a.loss[s] = begin < end ? static_cast<float>(v * a.E / (n * n * a.k)) : 0.f;
}

template <class Logit, int LPT, int I>
hipError_t launch(const BalanceArgs& a, int mode, int chunk, int count_chunk, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>((a.T + chunk - 1) / chunk)), block(256);
#define MOE_BALANCE(MODE)                                                                          \
  a.sigmoid ? balance_kernel<Logit, LPT, I, true, MODE><<<grid, block, 0, stream>>>(a, chunk, count_chunk) \
            : balance_kernel<Logit, LPT, I, false, MODE><<<grid, block, 0, stream>>>(a, chunk, count_chunk)
  switch (mode) {
    case kLossOnly: MOE_BALANCE(kLossOnly); break;
    case kGradient: MOE_BALANCE(kGradient); break;
    case kGradientAdd: MOE_BALANCE(kGradientAdd); break;
    default: MOE_BALANCE(kAny);
  }
#undef MOE_BALANCE
  return hipGetLastError();
}

template <class Logit>
hipError_t launch_typed(const BalanceArgs& a, int chunk, int count_chunk, hipStream_t stream) {
  auto fits = [&](const void* p) { return reinterpret_cast<uintptr_t>(p) % (4 * sizeof(Logit)) == 0; };
  const bool wide = a.E % 4 == 0 && fits(a.logits) && fits(a.add) && fits(a.dlogits);
  const int mode = !wide ? kAny : a.dlogits == nullptr ? kLossOnly : a.add == nullptr ? kGradient : kGradientAdd;
  if (a.E <= 64) return launch<Logit, 16, 1>(a, mode, chunk, count_chunk, stream);
  // two tokens a wavefront / four / one: 65536 x 256, loss and gradient 46.8 us / 50.8 / 48.0, gradient
  // added 42.4 / 47.9 / 41.6
  if (a.E <= 128) return launch<Logit, 32, 1>(a, mode, chunk, count_chunk, stream);
  if (a.E <= 256) return launch<Logit, 32, 2>(a, mode, chunk, count_chunk, stream);
  if (a.E <= 512) return launch<Logit, 32, 4>(a, mode, chunk, count_chunk, stream);
  return launch<Logit, 64, 4>(a, mode, chunk, count_chunk, stream);
}

// Tokens per workgroup: T stays below 2^31, so with 256 a launch has fewer than 2^32 threads.
int chunk_of(int64_t T) {
  int chunk = kBalanceMinChunk;
  // up to 2048 workgroups: 65536 x 256 46.8 us; 1024 48.4, 4096 52.3
  while (chunk < 256 && T > static_cast<int64_t>(chunk) * 2048) chunk *= 2;
  return chunk;
}
// Of the counting launch: a long sequence's counts are the sum of at most 128 chunks' or so.
int count_chunk_of(int64_t T) {
  int chunk = kCountChunk;
  while (T > static_cast<int64_t>(chunk) * 128) chunk *= 2;
  return chunk;
}

}  // namespace

hipError_t launch_balance(const BalanceArgs& a, bool bf16, hipStream_t stream) {
  if (a.T == 0) {   // every sequence is empty
    const int64_t n = static_cast<int64_t>(a.n_seqs) * a.E, groups = (n + 255) / 256;
    zero_kernel<<<dim3(static_cast<unsigned>(groups < 4096 ? groups : 4096)), dim3(256), 0, stream>>>(a.counts, n);
    zero_kernel<<<dim3(static_cast<unsigned>((a.n_seqs + 255) / 256)), dim3(256), 0, stream>>>(
        reinterpret_cast<int32_t*>(a.loss), a.n_seqs);
    return hipGetLastError();
  }
  const int chunk = chunk_of(a.T), count_chunk = count_chunk_of(a.T);
  if (a.ids != nullptr && a.T * a.k > kShortPairs) {
    count_kernel<<<dim3(static_cast<unsigned>((a.T + count_chunk - 1) / count_chunk)), dim3(1024), 0, stream>>>(
        a, count_chunk);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  const hipError_t err = bf16 ? launch_typed<uint16_t>(a, chunk, count_chunk, stream)
                              : launch_typed<float>(a, chunk, count_chunk, stream);
  if (err != hipSuccess || a.loss == nullptr) return err;
  loss_kernel<<<dim3(static_cast<unsigned>((a.n_seqs + 3) / 4)), dim3(256), 0, stream>>>(a, chunk);
  return hipGetLastError();
}

}  // namespace moe
