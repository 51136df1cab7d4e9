// Per-expert counts of each sequence's choices, the balance loss and the z loss of
// the router's logits (include/moe.h, moe_balance_loss).
//
//   balance = sum over counted tokens t of sequence b, experts e of F_be q_te,
//             F_be = E c_be / (k n_b) / (n_b B),  q_te the normalised score
//   z       = mean over counted tokens of lse_t^2
//
// Written this way round (the counts first) the loss needs no sum per expert over
// a sequence's tokens: each token contributes one number.  Kernels: the
// counts (in one, or zero and count), and the logits' pass, whose CTAs leave one pair of sums each; the last
// CTA adds them in a fixed order, so that results do not depend on timing (the counts
// are sums of integers).  Latency-bound: T = 4096, E = 192 (3.3 MB) 4.5 us for the
// counts and 9 for the pass.
#include "internal.h"
#include "ptx.cuh"
#include "scores.cuh"

namespace moe {

namespace {
constexpr int kThreads = 256;
constexpr int kClusterCtas = 8, kClusterThreads = 1024;
constexpr int kClusterCounters = 11000;   // 44 KB of shared memory
constexpr int kClusterSlots = 8 * kClusterCtas * kClusterThreads;  // 8 choices a thread
}

__global__ void __launch_bounds__(kThreads) balance_zero_kernel(int32_t *counts, int32_t *tokens, long long nc, int n_seq) {
  pdl_wait();
  pdl_launch_dependents();
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < nc + n_seq; i += (long long)gridDim.x * kThreads) {
    if (i < nc) counts[i] = 0;
    else tokens[i - nc] = 0;
  }
}

// A CTA's tokens are mostly of one sequence: the choices of its first token's
// sequence are counted in shared memory and added at the end, the others' at once.
__global__ void __launch_bounds__(kThreads) balance_count_kernel(const BalanceParams p, int per_cta) {
  __shared__ int hist[256];
  __shared__ int here;
  pdl_launch_dependents();
  const int t0 = blockIdx.x * per_cta, t1 = min(p.T, t0 + per_cta);
  if (threadIdx.x == 0) here = 0;
  for (int e = threadIdx.x; e < p.E; e += kThreads) hist[e] = 0;
  pdl_wait();
  const int home = p.seq_id == nullptr ? 0 : __ldg(p.seq_id + t0);
  __syncthreads();
  for (unsigned i = (unsigned)t0 * p.top_k + threadIdx.x; i < (unsigned)t1 * p.top_k; i += kThreads) {
    const int t = (int)(i / p.top_k);
    const int b = token_seq(p.seq_id, p.n_seq, t, p.err);
    if (b < 0) continue;
    const int e = checked_expert(__ldg(p.topk_idx + i), p.E, p.err);
    const bool first = i == (unsigned)t * p.top_k;
    if (b == home) {
      atomicAdd(&hist[e], 1);
      if (first) atomicAdd(&here, 1);
    } else {
      atomicAdd(p.counts + (size_t)b * p.E + e, 1);
      if (first) atomicAdd(p.tokens + b, 1);
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kThreads)
    if (hist[e]) atomicAdd(p.counts + (size_t)home * p.E + e, hist[e]);
  if (threadIdx.x == 0 && here) atomicAdd(p.tokens + home, here);
}

// Zero and count in one launch where the counters of all sequences fit in shared
// memory and there is no more to count than a few CTAs do quickly: a cluster, each
// CTA counting a part of the choices; then each adds up a part of the counters over
// the cluster's shared memory.
__global__ void __launch_bounds__(kClusterThreads) balance_cluster_kernel(const BalanceParams p) {
  extern __shared__ int hist[];  // [n_seq][E] choices, [n_seq] tokens
  pdl_wait();
  pdl_launch_dependents();
  const int n = p.n_seq * p.E + p.n_seq, parts = gridDim.x, rank = blockIdx.x;
  for (int i = threadIdx.x; i < n; i += kClusterThreads) hist[i] = 0;
  __syncthreads();
  const int S = p.T * p.top_k;
  for (int i = rank * kClusterThreads + threadIdx.x; i < S; i += parts * kClusterThreads) {
    const int t = i / p.top_k;
    const int b = token_seq(p.seq_id, p.n_seq, t, p.err);
    if (b < 0) continue;
    atomicAdd(&hist[b * p.E + checked_expert(__ldg(p.topk_idx + i), p.E, p.err)], 1);
    if (i == t * p.top_k) atomicAdd(&hist[p.n_seq * p.E + b], 1);
  }
  cluster_sync();
  for (int i = rank * kClusterThreads + threadIdx.x; i < n; i += parts * kClusterThreads) {
    int v[kClusterCtas];
#pragma unroll
    for (int r = 0; r < kClusterCtas; ++r) {
      v[r] = 0;
      if (r < parts)
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v[r]) : "r"(map_cluster(smem_u32(hist + i), (uint32_t)r)) : "memory");
    }
    int sum = 0;
#pragma unroll
    for (int r = 0; r < kClusterCtas; ++r) sum += v[r];
    if (i < p.n_seq * p.E) p.counts[i] = sum;
    else p.tokens[i - p.n_seq * p.E] = sum;
  }
  cluster_sync();  // nobody leaves while its counters are being read
}

template <bool SIGMOID>
__global__ void __launch_bounds__(kThreads) balance_loss_kernel(const BalanceParams p) {
  __shared__ double sums[2][kThreads / 32];
  __shared__ int nb[2];
  __shared__ bool last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_launch_dependents();
  pdl_wait();
  // a warp's few tokens are added in fp32 with the rounding carried along (Kahan)
  float balance = 0.0f, z = 0.0f, balance_c = 0.0f, z_c = 0.0f;
  auto add = [](float &sum, float &c, float x) {
    const float y = __fsub_rn(x, c), t = __fadd_rn(sum, y);
    c = __fsub_rn(__fsub_rn(t, sum), y);
    sum = t;
  };
  const unsigned step = gridDim.x * (kThreads / 32);
  unsigned t = blockIdx.x * (kThreads / 32) + warp;
  float v[kPerLane];
  int seq = -1;
  if (t < (unsigned)p.T) {
    seq = token_seq(p.seq_id, p.n_seq, t, p.err);
    load_logits(p.logits + (size_t)t * p.E, p.E, lane, v);
  }
  while (t < (unsigned)p.T) {
    const int here = seq;
    int c[kPerLane];
    float n = 1.0f, now[kPerLane];
    if (here >= 0) {
      // through L1: every token reads the same few lines, which L2 would serve one by one
      // (the logits' pass 29 against 17 us at 16384 tokens)
      const int32_t *of = p.counts + (size_t)here * p.E;
#pragma unroll
      for (int j = 0; j < kPerLane; ++j) c[j] = expert_of(lane, j) < p.E ? __ldg(of + expert_of(lane, j)) : 0;
      n = (float)__ldg(p.tokens + here);
    }
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) now[j] = v[j];
    t += step;
    if (t < (unsigned)p.T) {  // the next token's, while this one is worked on
      seq = token_seq(p.seq_id, p.n_seq, t, p.err);
      load_logits(p.logits + (size_t)t * p.E, p.E, lane, v);
    }
    if (here < 0) continue;
    const TokenScores r = token_scores<SIGMOID>(now, p.E, lane);
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) dot = fmaf((float)c[j], SIGMOID ? r.s[j] : r.p[j], dot);
    dot = warp_sum(dot);
    add(balance, balance_c, dot / ((SIGMOID ? r.total : 1.0f) * n) / n);
    add(z, z_c, r.lse * r.lse);
  }
  if (lane == 0) {
    sums[0][warp] = (double)balance - balance_c;
    sums[1][warp] = (double)z - z_c;
  }
  __syncthreads();
  if (warp == 0) {
    double v = 0.0;
    if (lane < 2) {
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) v += sums[lane][w];
      p.part[2 * blockIdx.x + lane] = v;
      __threadfence();
    }
    __syncwarp();
    if (lane == 0) last = atomicAdd(p.done, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  // every CTA's pair at once, then added in a fixed order
  double a = 0.0, b = 0.0;
  for (int i = threadIdx.x; i < (int)gridDim.x; i += kThreads) {
    a += __ldcg(p.part + 2 * i);
    b += __ldcg(p.part + 2 * i + 1);
  }
  const int2 nt = sequence_totals(p.tokens, p.n_seq, nb);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if (lane == 0) {
    sums[0][warp] = a;
    sums[1][warp] = b;
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    double v = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) v += sums[threadIdx.x][w];
    p.losses[threadIdx.x] = threadIdx.x == 0 ? (float)v * ((float)p.E / (float)p.top_k) / (float)max(nt.x, 1)
                                             : (float)v / (float)max(nt.y, 1);
    if (threadIdx.x == 0) *p.done = 0;
  }
}

cudaError_t launch_balance(const BalanceParams &p, int num_sms, cudaStream_t stream) {
  const long long counters = (long long)p.n_seq * p.E + p.n_seq, slots = (long long)p.T * p.top_k;
  const bool one = counters <= kClusterCounters && slots <= kClusterSlots;
  if (one) {
    int parts = 1;
    while (parts < kClusterCtas && parts * kClusterThreads < slots) parts *= 2;
    void *args[] = {(void *)&p};
    const cudaError_t e = launch_ex((const void *)balance_cluster_kernel, dim3(parts), dim3(kClusterThreads),
                                    (size_t)counters * 4, stream, true, parts, args);
    if (e != cudaSuccess) return e;
  } else {
    const long long nc = (long long)p.n_seq * p.E, n = nc + p.n_seq;
    long long blocks = (n + 4 * kThreads - 1) / (4 * kThreads);
    if (blocks > num_sms) blocks = num_sms;
    int32_t *counts = p.counts, *tokens = p.tokens;
    int n_seq = p.n_seq;
    long long nc_ = nc;
    void *args[] = {(void *)&counts, (void *)&tokens, (void *)&nc_, (void *)&n_seq};
    const cudaError_t e = launch_ex((const void *)balance_zero_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, stream,
                                    true, 1, args);
    if (e != cudaSuccess) return e;
  }
  if (p.T == 0) return p.losses ? cudaMemsetAsync(p.losses, 0, 2 * sizeof(float), stream) : cudaSuccess;
  if (!one) {
    int per = 32;  // tokens of a CTA
    while ((p.T + per - 1) / per > 4 * num_sms) per *= 2;
    void *args[] = {(void *)&p, (void *)&per};
    const cudaError_t e = launch_ex((const void *)balance_count_kernel, dim3((p.T + per - 1) / per), dim3(kThreads), 0,
                                    stream, true, 1, args);
    if (e != cudaSuccess) return e;
  }
  if (p.losses == nullptr) return cudaSuccess;
  int blocks = (p.T + kThreads / 32 - 1) / (kThreads / 32);
  // a few tokens a warp and one wave: each CTA's end costs about as much as two tokens
  if (blocks > 3 * num_sms) blocks = 3 * num_sms;
  if (blocks > kBalanceMaxCtas) blocks = kBalanceMaxCtas;
  void *args[] = {(void *)&p};
  return launch_ex(p.sigmoid ? (const void *)balance_loss_kernel<true> : (const void *)balance_loss_kernel<false>,
                   dim3(blocks), dim3(kThreads), 0, stream, true, 1, args);
}

}  // namespace moe
