// Scored routing (softmax or sigmoid scores, balance bias, expert groups): one wavefront
// per token (route_scored_token in scored_core.h).  As for plain top-k, a few tokens are
// routed and grouped by expert in one launch of one workgroup (one_launch has the rule);
// above, the routing kernel also writes the bit matrix and the expert-offsets kernels follow.
//
// Bound by the vector ALU: about 610 instructions a token (E = 256, softmax and bias), of which
// the k + 1 rounds are a quarter.  8191 tokens take 11.6 us by the kernel trace (10.9 to 12.0 in a
// row of calls); their 8.8 MB would need 1.7.  Sigmoid scores in 8 groups take 14.0.  The one-launch
// form is one workgroup's chain of dependent steps: 8 tokens of 256 experts routed and grouped, in
// those groups, in 7.4 us.
#include "group_core.h"
#include "launch.h"
#include "scored_core.h"

namespace moe {
namespace {

template <int EPL, class Logit>
__global__ __launch_bounds__(256) void route_scored_kernel(
    const Logit* __restrict__ logits, int64_t T, int E, int k, ScoreArgs a,
    int32_t* __restrict__ ids, float* __restrict__ weights, uint32_t* __restrict__ bm) {
  const int lane = threadIdx.x & 63;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (t >= T) return;   // uniform per wavefront
  int id;
  float w;
  route_scored_token<EPL>(logits + t * E, k, lane, a, id, w);
  if (lane < k) {
    ids[t * k + lane] = id;
    weights[t * k + lane] = w;
  }
  if (bm != nullptr) {   // uniform: the token's bit-matrix row, lane w writing word w
    const int words = (E + 31) / 32;
    uint32_t word = 0;
    for (int j = 0; j < k; ++j) {
      const int e = __shfl(id, j, 64);
      if ((e >> 5) == lane) word |= 1u << (e & 31);
    }
    if (lane < words) bm[t * words + lane] = word;
  }
}

template <int EPL, class Logit>
__global__ __launch_bounds__(1024) void scored_front_kernel(
    const Logit* __restrict__ logits, int T, int E, int k, ScoreArgs a, int words,
    int32_t* __restrict__ ids, float* __restrict__ weights, uint32_t* __restrict__ bm,
    int32_t* __restrict__ counts, int32_t* __restrict__ offsets, int32_t* __restrict__ gather,
    int32_t* __restrict__ scatter) {
  __shared__ FrontLds lds;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n_waves = blockDim.x >> 6;
  for (int t = wave; t < T; t += n_waves) {
    int id;
    float w;
    route_scored_token<EPL>(logits + static_cast<int64_t>(t) * E, k, lane, a, id, w);
    if (lane < k) {
      ids[t * k + lane] = id;
      weights[t * k + lane] = w;
      lds.ids[t * k + lane] = id;
    }
  }
  group_small<EPL>(lds, T, E, k, words, bm, counts, offsets, gather, scatter, 1, 0, nullptr,
                   nullptr);
}

ScoreArgs score_args(const ScoredRouting& r, int E) {
  int bits = 6;   // log2 of 64 / (groups rounded up to a power of two)
  for (int g2 = 1; g2 < r.groups; g2 *= 2) --bits;
  return ScoreArgs{r.score,     r.bias,        r.groups, E / r.groups, r.topk_groups,
                   r.group_top, r.renormalize, r.scale,  bits};
}

// At most 32: per / L < 2 E / 64.
int experts_per_lane(const ScoreArgs& a) { return (a.per + (1 << a.lane_bits) - 1) >> a.lane_bits; }
// One launch for a few tokens: its 16 wavefronts take them in turn, while the routing and
// offsets kernels spread them over the GPU.  Measured (us in a graph, softmax and bias, k = 6),
// one launch / those kernels: 256 experts 8 tokens 6.6 / 11.3, 16 8.4 / 11.2, 24 10.0 / 11.2, 25
// 11.5 / 11.3, 64 23 / 11.5; 64 experts 24 7.7 / 8.6, 32 9.3 / 8.6.  With 8 experts a lane the
// one-launch form spills (128 registers a lane with 16 wavefronts; 164 bytes of scratch): 512
// experts 1 token 14.9 / 20.2, 8 19.9 / 21.6, 12 25.0 / 21.5, 64 94 / 22.
bool one_launch(int64_t T, int epl) { return epl <= 4 ? T <= 24 : epl <= 8 && T <= 8; }
static_assert(kFrontMaxTokens >= 24, "the workgroup's LDS");

template <class Logit>
hipError_t launch_route(const Logit* logits, int64_t T, int E, int k, const ScoreArgs& a,
                        int32_t* ids, float* weights, uint32_t* bm, hipStream_t stream) {
  const int epl = experts_per_lane(a);
  const int words = (E + 31) / 32;
  // a launch has fewer than 2^32 threads: 2^22 tokens at a time
  for (int64_t at = 0; at < T; at += 1 << 22) {
    const int64_t n = T - at < (1 << 22) ? T - at : 1 << 22;
    const dim3 grid(static_cast<unsigned>((n + 3) / 4)), block(256);
#define MOE_ROUTE(EPL)                                                                         \
  route_scored_kernel<EPL><<<grid, block, 0, stream>>>(logits + at * E, n, E, k, a, ids + at * k, \
                                                       weights + at * k, bm ? bm + at * words : bm)
    if (epl <= 1)
      MOE_ROUTE(1);
    else if (epl <= 2)
      MOE_ROUTE(2);
    else if (epl <= 4)
      MOE_ROUTE(4);
    else if (epl <= 8)
      MOE_ROUTE(8);
    else if (epl <= 16)
      MOE_ROUTE(16);
    else
      MOE_ROUTE(32);
#undef MOE_ROUTE
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

template <class Logit>
hipError_t launch_front(const Logit* logits, int T, int E, int k, const ScoreArgs& a, int32_t* ids,
                        float* weights, uint32_t* bm, int32_t* counts, int32_t* offsets,
                        int32_t* gather, int32_t* scatter, hipStream_t stream) {
  const int epl = experts_per_lane(a);
  const int words = (E + 31) / 32;
#define MOE_FRONT(EPL)                                                                        \
  scored_front_kernel<EPL><<<1, 1024, 0, stream>>>(logits, T, E, k, a, words, ids, weights, bm, \
                                                   counts, offsets, gather, scatter)
  if (epl <= 1)
    MOE_FRONT(1);
  else if (epl <= 2)
    MOE_FRONT(2);
  else if (epl <= 4)
    MOE_FRONT(4);
  else
    MOE_FRONT(8);
#undef MOE_FRONT
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route_scored(const void* logits, bool bf16, int64_t T, int E, int k,
                               const ScoredRouting& r, int32_t* ids, float* weights, uint32_t* bm,
                               hipStream_t stream) {
  const ScoreArgs a = score_args(r, E);
  return bf16 ? launch_route(static_cast<const uint16_t*>(logits), T, E, k, a, ids, weights, bm, stream)
              : launch_route(static_cast<const float*>(logits), T, E, k, a, ids, weights, bm, stream);
}

hipError_t launch_route_scored_and_group(const void* logits, bool bf16, int64_t T, int E, int k,
                                         const ScoredRouting& r, int32_t* ids, float* weights,
                                         uint32_t* bm, int32_t* counts, int32_t* offsets,
                                         int32_t* gather, int32_t* scatter, void* ws,
                                         hipStream_t stream) {
  const ScoreArgs a = score_args(r, E);
  if (!one_launch(T, experts_per_lane(a))) {
    const hipError_t err = launch_route_scored(logits, bf16, T, E, k, r, ids, weights, bm, stream);
    if (err != hipSuccess) return err;
    return launch_offsets(bm, ids, T, E, k, counts, offsets, gather, scatter, ws, stream);
  }
  const int t = static_cast<int>(T);
  return bf16 ? launch_front(static_cast<const uint16_t*>(logits), t, E, k, a, ids, weights, bm,
                             counts, offsets, gather, scatter, stream)
              : launch_front(static_cast<const float*>(logits), t, E, k, a, ids, weights, bm,
                             counts, offsets, gather, scatter, stream);
}

}  // namespace moe
