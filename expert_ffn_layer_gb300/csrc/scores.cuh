// What the router's losses and its backward pass need of one token's logits, held by
// a warp: lane l has experts 2 l, 2 l + 1, 64 + 2 l, .. (at most 256), so that two
// neighbours' 16-bit values go out in one store.
#pragma once
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

constexpr int kPerLane = 8;  // experts of a lane
__device__ __forceinline__ int expert_of(int lane, int j) { return 64 * (j >> 1) + 2 * lane + (j & 1); }
__device__ __forceinline__ int lane_of(int e) { return (e & 63) >> 1; }
__device__ __forceinline__ int slot_of(int e) { return 2 * (e >> 6) + (e & 1); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// The sequence of token t, or -1 where the token counts nowhere (a negative
// number, or one past the last sequence, which is flagged).
__device__ __forceinline__ int token_seq(const int32_t *seq_id, int n_seq, int t, unsigned *err) {
  if (seq_id == nullptr) return 0;
  const int b = __ldg(seq_id + t);
  if (b >= n_seq) {
    atomicOr(err, MOE_DEVERR_INDEX);
    return -1;
  }
  return b < 0 ? -1 : b;
}
__device__ __forceinline__ int checked_expert(int e, int E, unsigned *err) {
  if (e < 0 || e >= E) {
    atomicOr(err, MOE_DEVERR_INDEX);
    return e < 0 ? 0 : E - 1;
  }
  return e;
}

// Sequences with tokens, and all counted tokens, by the whole CTA (`sh` is shared).
__device__ __forceinline__ int2 sequence_totals(const int32_t *tokens, int n_seq, int *sh) {
  if (n_seq == 1) {
    const int n = __ldcg(tokens);
    return make_int2(n > 0, n);
  }
  if (threadIdx.x < 2) sh[threadIdx.x] = 0;
  __syncthreads();
  int full = 0, total = 0;
  for (int b = threadIdx.x; b < n_seq; b += blockDim.x) {
    const int n = __ldcg(tokens + b);
    full += n > 0;
    total += n;
  }
  full = __reduce_add_sync(0xffffffffu, full);
  total = __reduce_add_sync(0xffffffffu, total);
  if ((threadIdx.x & 31) == 0 && full) {
    atomicAdd(&sh[0], full);
    atomicAdd(&sh[1], total);
  }
  __syncthreads();
  return make_int2(sh[0], sh[1]);
}

struct TokenScores {
  float p[kPerLane];     // softmax of the logits (0 past the last expert)
  float s[kPerLane];     // sigmoid mode: sigmoid of the logits
  float miss[kPerLane];  // sigmoid mode: 1 - s, from the other end
  float total;           // sigmoid mode: the sum of s over all experts
  float lse;             // log of the sum of the logits' exponentials
};
__device__ __forceinline__ void load_logits(const float *lg, int E, int lane, float (&v)[kPerLane]) {
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) v[j] = expert_of(lane, j) < E ? __ldg(lg + expert_of(lane, j)) : -INFINITY;
}
template <bool SIGMOID>
__device__ __forceinline__ TokenScores token_scores(const float (&v)[kPerLane], int E, int lane) {
  TokenScores r;
  {
    float mx = v[0];
#pragma unroll
    for (int j = 1; j < kPerLane; ++j) mx = fmaxf(mx, v[j]);
    mx = warp_max(mx);
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      r.p[j] = expert_of(lane, j) < E ? expf(v[j] - mx) : 0.0f;
      sum += r.p[j];
    }
    sum = warp_sum(sum);
    const float inv = 1.0f / sum;
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) r.p[j] *= inv;
    r.lse = mx + logf(sum);
  }
  r.total = 0.0f;
  if (SIGMOID) {
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      // both ends from one exponential, which cannot overflow, and one reciprocal of a
      // value in [1, 2]; past the last expert v = -infinity, so s = 0
      const float t = expf(-fabsf(v[j])), big = __fdividef(1.0f, 1.0f + t), small = t * big;
      r.s[j] = v[j] >= 0.0f ? big : small;
      r.miss[j] = v[j] >= 0.0f ? small : big;
      if (v[j] != v[j]) r.s[j] = r.miss[j] = v[j];
      r.total += r.s[j];
    }
    r.total = warp_sum(r.total);
  }
  return r;
}

}  // namespace moe
