// Scoring and top-k selection of one token by one warp, shared by the router's
// top-k kernel and the one-kernel layer for few tokens.
#pragma once
#include <math_constants.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

__device__ __forceinline__ bool better(float k1, int e1, float k2, int e2) {
  return k1 > k2 || (k1 == k2 && e1 < e2);
}

// Routing rule of a call (moe_dims' fields of the same names).
struct TopkRule {
  const float *bias;  // [E] or nullptr
  int E, top_k, score_mode;
  float route_scale, renorm_eps;
};

// From the token's logits lg[0..E): lane j < top_k gets the j-th expert in
// descending key order (equal keys: the lower index) and its combine weight.
__device__ __forceinline__ void warp_select_topk(const TopkRule &p, const float *lg, int lane, int &expert,
                                                 float &weight) {
  const int E = p.E, k = p.top_k;
  const int nj = (E + 31) >> 5;
  float v[8], key[8], sc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = (j < nj && lane + 32 * j < E) ? lg[lane + 32 * j] : 0.0f;
  if (p.score_mode == MOE_SCORE_SIGMOID_BIAS) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = lane + 32 * j;
      const float s = 1.0f / (1.0f + expf(-v[j]));
      const float kk = s + ((p.bias != nullptr && j < nj && e < E) ? p.bias[e] : 0.0f);
      sc[j] = s;
      key[j] = (kk == kk) ? kk : -INFINITY;
    }
  } else {
    float mx = -INFINITY;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < nj && lane + 32 * j < E) mx = fmaxf(mx, v[j]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    float ex[8], sum = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      ex[j] = (j < nj && lane + 32 * j < E) ? expf(v[j] - mx) : 0.0f;
      sum += ex[j];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sc[j] = ex[j] / sum;
      key[j] = (sc[j] == sc[j]) ? sc[j] : -INFINITY;
    }
  }
  uint32_t taken = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (!(j < nj && lane + 32 * j < E)) taken |= 1u << j;
  int my_e = 0;
  float my_s = 0.0f;
  for (int rnd = 0; rnd < k; ++rnd) {
    float bk = -INFINITY, bs = 0.0f;
    int be = 0x7fffffff;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = lane + 32 * j;
      if (!((taken >> j) & 1u) && better(key[j], e, bk, be)) {
        bk = key[j];
        be = e;
        bs = sc[j];
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float ok2 = __shfl_xor_sync(0xffffffffu, bk, o);
      const int oe = __shfl_xor_sync(0xffffffffu, be, o);
      const float os = __shfl_xor_sync(0xffffffffu, bs, o);
      if (better(ok2, oe, bk, be)) {
        bk = ok2;
        be = oe;
        bs = os;
      }
    }
    if (be < E && (be & 31) == lane) taken |= 1u << (be >> 5);
    if (lane == rnd) {
      my_e = be < E ? be : 0;
      my_s = bs;
    }
  }
  float tot = lane < k ? my_s : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
  if (lane < k) {
    expert = my_e;
    weight = p.score_mode == MOE_SCORE_SIGMOID_BIAS ? my_s / tot * p.route_scale : my_s / fmaxf(tot, p.renorm_eps);
  }
}

}  // namespace moe
