// The loss that balances the router's load, and its gradient, over packed sequences.
//
// With c the counts of a token's sequence, everything that a token adds is d = sum_i p_i c_i: the
// loss is E / (k n^2) times the sum of d over the sequence, and the gradient is that factor times
// p_e (c_e - d).  So the counts come first (integers, whose order of addition does not matter), and
// one pass over the logits then gives the loss and the gradient: no sum per expert is kept.
//   c is taken less its mean's integer part: p sums to 1, so c_e - d does not change, and an even
//   load, whose gradient is a small difference of large numbers, keeps its digits.
//
// Layout: LPT lanes (16, 32 or 64, by E) take a token, four neighbouring experts a lane and step.
#include "block.h"
#include "block_common.h"
#include "block_plan.h"
#include "scored_core.h"

namespace moe {
namespace {

constexpr int kCountTokens = 1024;   // tokens per workgroup of the counting kernel

// How many of offsets[1 .. n] are at most t: the sequence of token t, n behind the last.  All lanes of
// a wavefront look at 64 of them at a time.
__device__ __forceinline__ int sequence_of(const int32_t* offsets, int n, int64_t t) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = n;
  while (lo < hi) {
    const int step = (hi - lo + 63) / 64;
    const int64_t i = lo + static_cast<int64_t>(lane + 1) * step;
    const bool below = i <= hi && offsets[i] <= t;
    const int c = __popcll(__builtin_amdgcn_ballot_w64(below));
    lo += c * step;
    const int64_t end = static_cast<int64_t>(lo) + step - 1;
    hi = end < hi ? static_cast<int>(end) : hi;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// The tokens from t on that belong together: sequence s (n_seqs: padding) up to `end` <= t1, and the
// sequence's length.  Offsets that break the rules still give t < end <= t1.
struct Segment {
  int s;
  int64_t end, n;
};
__device__ __forceinline__ Segment segment_at(const int32_t* offsets, int n_seqs, int64_t T, int64_t t,
                                              int64_t t1) {
  if (offsets == nullptr) return Segment{0, t1, T};
  const int s = sequence_of(offsets, n_seqs, t);
  if (s >= n_seqs) return Segment{n_seqs, t1, 1};
  const int64_t begin = offsets[s], end = offsets[s + 1];
  if (t < begin) return Segment{n_seqs, begin < t1 ? begin : t1, 1};   // in front of the first
  return Segment{s, end < t1 ? (end > t ? end : t + 1) : t1, end - begin > 0 ? end - begin : 1};
}

__global__ __launch_bounds__(256) void zero_kernel(int32_t* p, int64_t n) {
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) p[i] = 0;
}

// Counts: a histogram in LDS for each sequence of the workgroup's tokens, added to the whole.
__global__ __launch_bounds__(256) void count_kernel(const int32_t* __restrict__ ids, int64_t T, int E, int k,
                                                    const int32_t* __restrict__ offsets, int n_seqs,
                                                    int32_t* __restrict__ counts) {
  __shared__ int bins[kMaxE];
  int64_t t = static_cast<int64_t>(blockIdx.x) * kCountTokens;
  const int64_t t1 = t + kCountTokens < T ? t + kCountTokens : T;
  while (t < t1) {   // uniform over the workgroup
    const Segment g = segment_at(offsets, n_seqs, T, t, t1);
    if (g.s < n_seqs) {
      for (int e = threadIdx.x; e < E; e += 256) bins[e] = 0;
      __syncthreads();
      for (int64_t i = t * k + threadIdx.x; i < g.end * k; i += 256) {
        const int e = ids[i];
        if (static_cast<unsigned>(e) < static_cast<unsigned>(E)) atomicAdd(&bins[e], 1);
      }
      __syncthreads();
      for (int e = threadIdx.x; e < E; e += 256)
        if (bins[e]) atomicAdd(&counts[static_cast<int64_t>(g.s) * E + e], bins[e]);
      __syncthreads();
    }
    t = g.end;
  }
}

__device__ __forceinline__ float logit_of(float l) { return l; }
__device__ __forceinline__ float logit_of(uint16_t l) { return bf16_bits_to_f32(l); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = f32_to_bf16_bits(v); }

// Four elements from `e` on of a row of E; past E: `other`.
template <class Logit>
__device__ __forceinline__ void load4(const Logit* row, int e, int E, bool wide, float other, float (&v)[4]) {
  if (wide) {   // uniform: E is a multiple of 4 and rows are aligned to four elements
    if (e < E) {
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
      for (int j = 0; j < 4; ++j) v[j] = other;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = e + j < E ? logit_of(row[e + j]) : other;
  }
}
template <class Logit>
__device__ __forceinline__ void store4(Logit* row, int e, int E, bool wide, const float (&v)[4]) {
  if (wide) {
    if (e >= E) return;
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

// Sigmoid scores under e^-40 are divided as softmax scores: sigmoid(l) = e^l (1 - e^l + ...).
constexpr float kSigmoidLow = -40.f;

template <class Logit, int LPT, int I>
__global__ __launch_bounds__(256) void balance_kernel(BalanceArgs a, int chunk, int wide) {
  constexpr int G = 64 / LPT;   // tokens per wavefront
  __shared__ double part[4 * G];
  __shared__ int live[4 * G];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int sub = lane & (LPT - 1), group = wave * G + lane / LPT;
  const int E = a.E;
  const Logit* logits = static_cast<const Logit*>(a.logits);
  const Logit* add = static_cast<const Logit*>(a.add);
  Logit* out = static_cast<Logit*>(a.dlogits);
  int64_t t = static_cast<int64_t>(blockIdx.x) * chunk;
  const int64_t t1 = t + chunk < a.T ? t + chunk : a.T;
  while (t < t1) {   // uniform over the workgroup
    const Segment g = segment_at(a.offsets, a.n_seqs, a.T, t, t1);
    const bool padding = g.s >= a.n_seqs;
    if (padding) {
      if (out != nullptr)
        for (int64_t r = t + group; r < g.end; r += 4 * G)
#pragma unroll
          for (int i = 0; i < I; ++i) {
            const int e = 4 * (sub + LPT * i);
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            if (add != nullptr) load4(add + r * E, e, E, wide, 0.f, v);
            store4(out + r * E, e, E, wide, v);
          }
      t = g.end;
      continue;
    }
    const int64_t mean = g.n * a.k / E;
    float c[I][4];
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = 4 * (sub + LPT * i) + j;
        c[i][j] = e < E ? static_cast<float>(a.counts[static_cast<int64_t>(g.s) * E + e] - mean) : 0.f;
      }
    float factor = 0.f;
    if (out != nullptr)
      factor = static_cast<float>(static_cast<double>(a.dloss[g.s]) * E /
                                  (static_cast<double>(a.k) * g.n * g.n));
    double total = 0.0;
    int tokens = 0;
    for (int64_t r = t + group; r < g.end; r += 4 * G) {
      float l[I][4], p[I][4];
      float m = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < I; ++i) {
        load4(logits + r * E, 4 * (sub + LPT * i), E, wide, -__builtin_inff(), l[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) m = fmaxf(m, l[i][j]);   // a NaN is left out
      }
      m = run_max<LPT>(m);
      const bool sigmoid = a.sigmoid && m > kSigmoidLow;
      float sum = 0.f, dot = 0.f;
#pragma unroll
      for (int i = 0; i < I; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          p[i][j] = sigmoid ? sigmoid_of<float>(l[i][j]) : exp_below<float>(l[i][j], m);
          sum += p[i][j];
          dot = fmaf(p[i][j], c[i][j], dot);
        }
      sum = run_sum<LPT>(sum);
      dot = run_sum<LPT>(dot);
      const float inv = sum > 0.f ? 1.0f / sum : 0.f;
      const float d = dot * inv;
      total += d;
      tokens += sum > 0.f;
      if (out != nullptr) {   // uniform
        const float by = factor * inv;
#pragma unroll
        for (int i = 0; i < I; ++i) {
          const int e = 4 * (sub + LPT * i);
          float v[4] = {0.f, 0.f, 0.f, 0.f};
          if (add != nullptr) load4(add + r * E, e, E, wide, 0.f, v);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float x = by * p[i][j] * (c[i][j] - d);
            if (a.sigmoid) x *= inverse(1.0f + exp_of(l[i][j]));   // 1 - sigmoid
            v[j] += x;
          }
          store4(out + r * E, e, E, wide, v);
        }
      }
    }
    if (a.slots != nullptr) {
      if (sub == 0) part[group] = total, live[group] = tokens;
      __syncthreads();
      if (threadIdx.x == 0) {
        double v = 0.0;
        int n = 0;
        for (int i = 0; i < 4 * G; ++i) v += part[i], n += live[i];
        a.slots[blockIdx.x + static_cast<int64_t>(g.s)] = v + static_cast<double>(mean) * n;
      }
      __syncthreads();
    }
    t = g.end;
  }
}

// loss[s]: a wavefront adds the sums that the chunks left for its sequence.
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
  if (lane == 0) a.loss[s] = begin < end ? static_cast<float>(v * a.E / (n * n * a.k)) : 0.f;
}

template <class Logit, int LPT, int I>
hipError_t launch(const BalanceArgs& a, int chunk, int wide, hipStream_t stream) {
  balance_kernel<Logit, LPT, I>
      <<<dim3(static_cast<unsigned>((a.T + chunk - 1) / chunk)), dim3(256), 0, stream>>>(a, chunk, wide);
  return hipGetLastError();
}

template <class Logit>
hipError_t launch_typed(const BalanceArgs& a, int chunk, hipStream_t stream) {
  auto fits = [&](const void* p) { return reinterpret_cast<uintptr_t>(p) % (4 * sizeof(Logit)) == 0; };
  const int wide = a.E % 4 == 0 && fits(a.logits) && fits(a.add) && fits(a.dlogits);
  if (a.E <= 64) return launch<Logit, 16, 1>(a, chunk, wide, stream);
  if (a.E <= 128) return launch<Logit, 32, 1>(a, chunk, wide, stream);
  if (a.E <= 256) return launch<Logit, 64, 1>(a, chunk, wide, stream);
  if (a.E <= 512) return launch<Logit, 64, 2>(a, chunk, wide, stream);
  return launch<Logit, 64, 4>(a, chunk, wide, stream);
}

// Tokens per workgroup: T stays below 2^31, so with 256 a launch has fewer than 2^32 threads.
int chunk_of(int64_t T) {
  int chunk = kBalanceMinChunk;
  while (chunk < 256 && T > static_cast<int64_t>(chunk) * 1024) chunk *= 2;
  return chunk;
}

}  // namespace

hipError_t launch_balance(const BalanceArgs& a, bool bf16, hipStream_t stream) {
  const int chunk = chunk_of(a.T);
  if (a.ids != nullptr || a.T == 0) {
    const int64_t n = static_cast<int64_t>(a.n_seqs) * a.E;
    const int64_t groups = (n + 255) / 256;
    zero_kernel<<<dim3(static_cast<unsigned>(groups < 4096 ? groups : 4096)), dim3(256), 0, stream>>>(a.counts, n);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    if (a.T > 0) {
      count_kernel<<<dim3(static_cast<unsigned>((a.T + kCountTokens - 1) / kCountTokens)), dim3(256), 0, stream>>>(
          a.ids, a.T, a.E, a.k, a.offsets, a.n_seqs, a.counts);
      err = hipGetLastError();
      if (err != hipSuccess) return err;
    }
  }
  if (a.T > 0) {
    const hipError_t err = bf16 ? launch_typed<uint16_t>(a, chunk, stream) : launch_typed<float>(a, chunk, stream);
    if (err != hipSuccess) return err;
  }
  if (a.loss == nullptr) return hipSuccess;
  BalanceArgs l = a;
  if (a.T == 0) l.offsets = nullptr;   // every sequence is empty
  loss_kernel<<<dim3(static_cast<unsigned>((a.n_seqs + 3) / 4)), dim3(256), 0, stream>>>(l, chunk);
  return hipGetLastError();
}

}  // namespace moe
