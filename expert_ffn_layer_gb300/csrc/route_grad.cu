// The routing's backward pass (include/moe.h, moe_route_backward): gradients of the
// combine weights and of the router's losses with respect to the logits, and from
// those with respect to the hidden state and the router weight.
//
// One token's logits l, scores s, gradient g_j of its combine weights, u_j = s_j / sum
// over the selected s:
//   sigmoid   dl_ej += R u_j (g_j - sum_i g_i u_i) (1 - s_j)
//   softmax   dl_ej += u_j (g_j - sum_i g_i u_i); where the clamp acts (w = p / eps)
//             dl_e  += p_e (a_e - sum_j a_j p_j), a_j = g_j / eps at the selected e
//   balance   dl_e  += G0 q_e (F_e - sum F q) (times 1 - s_e in sigmoid mode),
//             F_e = E c_be / (k n_b^2 B)
//   z         dl_e  += G1 2 lse / n softmax_e
#include "internal.h"
#include "ptx.cuh"
#include "scores.cuh"

namespace moe {

namespace {
constexpr int kThreads = 256;
}

// A warp per token.  1 - s is taken as the sigmoid of the negated logit, which keeps
// its digits where s is near one.
template <bool SIGMOID>
__global__ void __launch_bounds__(kThreads) grad_logits_kernel(const RouteGradParams p) {
  __shared__ int nb[2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = p.E, k = p.top_k;
  pdl_launch_dependents();
  pdl_wait();
  float full = 1.0f, total = 1.0f, g0 = 0.0f, g1 = 0.0f;
  if (p.grad_losses != nullptr) {
    if (threadIdx.x < 2) nb[threadIdx.x] = 0;
    __syncthreads();
    int f = 0, n = 0;
    for (int b = threadIdx.x; b < p.n_seq; b += kThreads) {
      const int m = __ldg(p.tokens + b);
      f += m > 0;
      n += m;
    }
    f = __reduce_add_sync(0xffffffffu, f);
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) {
      atomicAdd(&nb[0], f);
      atomicAdd(&nb[1], n);
    }
    __syncthreads();
    full = (float)max(nb[0], 1);
    total = (float)max(nb[1], 1);
    g0 = __ldg(p.grad_losses);
    g1 = __ldg(p.grad_losses + 1);
  }
  for (unsigned t = blockIdx.x * (kThreads / 32) + warp; t < (unsigned)p.T; t += gridDim.x * (kThreads / 32)) {
    const int b = token_seq(p.seq_id, p.n_seq, t, p.err);
    float d[kPerLane];
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) d[j] = 0.0f;
    if (b >= 0) {
      const TokenScores r = token_scores<SIGMOID, true>(p.logits + (size_t)t * E, E, lane);
      if (p.grad_losses != nullptr) {
        const int32_t *c = p.counts + (size_t)b * E;
        const float n = (float)max(__ldg(p.tokens + b), 1);
        const float load = (float)E / (float)k / (n * n) / full, inv = SIGMOID ? 1.0f / r.total : 1.0f;
        float F[kPerLane], dot = 0.0f;
#pragma unroll
        for (int j = 0; j < kPerLane; ++j) {
          F[j] = lane + 32 * j < E ? (float)__ldg(c + lane + 32 * j) * load : 0.0f;
          dot = fmaf(F[j], (SIGMOID ? r.s[j] : r.p[j]) * inv, dot);
        }
        dot = warp_sum(dot);
        const float gz = g1 * 2.0f * r.lse / total;
#pragma unroll
        for (int j = 0; j < kPerLane; ++j) {
          const float q = (SIGMOID ? r.s[j] : r.p[j]) * inv;
          d[j] = g0 * q * (F[j] - dot) * (SIGMOID ? r.miss[j] : 1.0f) + gz * r.p[j];
        }
      }
      if (p.grad_w != nullptr) {
        // lane i < k holds slot i
        int e = 0;
        float g = 0.0f;
        if (lane < k) {
          e = checked_expert(__ldg(p.topk_idx + (size_t)t * k + lane), E, p.err);
          g = __ldg(p.grad_w + (size_t)t * k + lane);
        }
        float score = 0.0f, rest = 0.0f;  // of the slot's expert, from the lane that has it
#pragma unroll
        for (int j = 0; j < kPerLane; ++j) {
          const float a = __shfl_sync(0xffffffffu, SIGMOID ? r.s[j] : r.p[j], e & 31);
          if (e >> 5 == j) score = a;
          if (SIGMOID) {
            const float m = __shfl_sync(0xffffffffu, r.miss[j], e & 31);
            if (e >> 5 == j) rest = m;
          }
        }
        if (lane >= k) score = 0.0f;
        const float sel = warp_sum(score);
        float v;  // the slot's contribution to its expert's logit
        float spread = 0.0f;
        if (!SIGMOID && !(sel >= p.renorm_eps)) {  // the clamp acts: w = p / eps
          const float a = g / p.renorm_eps;
          spread = warp_sum(a * score);
          v = a * score;
        } else {
          const float u = score / sel, mean = warp_sum(g * u);
          v = u * (g - mean) * (SIGMOID ? p.route_scale * rest : 1.0f);
        }
        for (int i = 0; i < k; ++i) {
          const int ei = __shfl_sync(0xffffffffu, e, i);
          const float vi = __shfl_sync(0xffffffffu, v, i);
          if ((ei & 31) == lane) {
#pragma unroll
            for (int j = 0; j < kPerLane; ++j)
              if (ei >> 5 == j) d[j] += vi;
          }
        }
        if (spread != 0.0f) {
#pragma unroll
          for (int j = 0; j < kPerLane; ++j) d[j] = fmaf(-spread, r.p[j], d[j]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kPerLane; ++j)
      if (lane + 32 * j < E) p.dl[(size_t)t * E + lane + 32 * j] = d[j];
  }
}

// grad_hidden[t, h] = sum_e dl[t, e] W[e, h]: 16 tokens x 256 columns a CTA.
__global__ void __launch_bounds__(kThreads) grad_hidden_kernel(const RouteGradParams p) {
  __shared__ float dl[16][256];
  pdl_launch_dependents();
  pdl_wait();
  const int t0 = blockIdx.y * 16, h = blockIdx.x * kThreads + threadIdx.x;
  for (int i = threadIdx.x; i < 16 * p.E; i += kThreads) {
    const int t = i / p.E, e = i - t * p.E;
    dl[t][e] = t0 + t < p.T ? __ldcg(p.dl + (size_t)(t0 + t) * p.E + e) : 0.0f;
  }
  __syncthreads();
  if (h >= p.H) return;
  float a[16] = {};
  for (int e = 0; e < p.E; ++e) {
    const float w = __ldg(p.router_w + (size_t)e * p.H + h);
#pragma unroll
    for (int t = 0; t < 16; ++t) a[t] = fmaf(dl[t][e], w, a[t]);
  }
#pragma unroll
  for (int t = 0; t < 16; ++t)
    if (t0 + t < p.T) p.grad_hidden[(size_t)(t0 + t) * p.H + h] = __float2bfloat16_rn(a[t]);
}

// grad_router_w[e, h] = sum_t dl[t, e] x[t, h] over counted tokens: 16 experts x 256
// columns a CTA, sums of 64 tokens added up in fp32.
__global__ void __launch_bounds__(kThreads) grad_router_w_kernel(const RouteGradParams p) {
  __shared__ float dl[64][16];
  __shared__ int live[64];
  pdl_launch_dependents();
  pdl_wait();
  const int e0 = blockIdx.y * 16, h = blockIdx.x * kThreads + threadIdx.x;
  float sum[16] = {};
  for (int t0 = 0; t0 < p.T; t0 += 64) {
    __syncthreads();
    for (int i = threadIdx.x; i < 64 * 16; i += kThreads) {
      const int t = i >> 4, e = e0 + (i & 15);
      dl[t][i & 15] = t0 + t < p.T && e < p.E ? __ldcg(p.dl + (size_t)(t0 + t) * p.E + e) : 0.0f;
    }
    if (threadIdx.x < 64)
      live[threadIdx.x] = t0 + threadIdx.x < p.T && token_seq(p.seq_id, p.n_seq, t0 + threadIdx.x, p.err) >= 0;
    __syncthreads();
    if (h >= p.H) continue;
    float a[16] = {};
    for (int t = 0; t < 64; ++t) {
      if (!live[t]) continue;
      const float x = __bfloat162float(p.hidden[(size_t)(t0 + t) * p.H + h]);
#pragma unroll
      for (int e = 0; e < 16; ++e) a[e] = fmaf(dl[t][e], x, a[e]);
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) sum[e] += a[e];
  }
  if (h >= p.H) return;
#pragma unroll
  for (int e = 0; e < 16; ++e)
    if (e0 + e < p.E) p.grad_router_w[(size_t)(e0 + e) * p.H + h] = sum[e];
}

cudaError_t launch_route_grad(const RouteGradParams &p, int num_sms, cudaStream_t stream) {
  void *args[] = {(void *)&p};
  int blocks = (p.T + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 8 * num_sms) blocks = 8 * num_sms;
  cudaError_t e = launch_ex(p.sigmoid ? (const void *)grad_logits_kernel<true> : (const void *)grad_logits_kernel<false>,
                            dim3(blocks), dim3(kThreads), 0, stream, true, 1, args);
  const unsigned hb = (p.H + kThreads - 1) / kThreads;
  if (e == cudaSuccess && p.grad_hidden != nullptr)
    e = launch_ex((const void *)grad_hidden_kernel, dim3(hb, (p.T + 15) / 16), dim3(kThreads), 0, stream, true, 1, args);
  if (e == cudaSuccess && p.grad_router_w != nullptr)
    e = launch_ex((const void *)grad_router_w_kernel, dim3(hb, (p.E + 15) / 16), dim3(kThreads), 0, stream, false, 1, args);
  return e;
}

}  // namespace moe
