// Step a9: top-k weighted combine back to token order plus the shared branch.
//   out[t] = sum_j w[t, j] * y_sorted[inv[t*k + j]] + y_shared[t]
// "Hy3 Preview inference optimisation case", section 3 (top-k weighted
// aggregation done at the end of the chain); HunyuanImage 3.0 post, Routed
// Experts (outputs viewed as [T, k, H], multiplied by the weights, summed over
// k) and Shared MLP (the shared output is added).
//
// HBM-bound streaming: one thread per 8 hidden values (16-byte vectors), fp32
// accumulation in j order, one bf16 rounding at the end.
#include "internal.h"
#include "ptx.cuh"

namespace moe {

namespace {
constexpr int kThreads = 256;
constexpr int kMaxK = 16;  // top_k limit of the ABI

__device__ __forceinline__ void acc8(float (&a)[8], const uint4 &v, float w) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[2 * i] = fmaf(w, __uint_as_float(u[i] << 16), a[2 * i]);
    a[2 * i + 1] = fmaf(w, __uint_as_float(u[i] & 0xffff0000u), a[2 * i + 1]);
  }
}
}  // namespace

// BATCHED: every slot's loads in flight at once (latency-bound small batches;
// the register cost of top-16 halves residency, which large, bandwidth-bound
// batches need more), else one slot at a time; K8: top-8 exactly, its eight
// rows (and the shared one) in flight together with half that register cost.
// All add in slot order.
template <bool BATCHED, bool K8 = false>
__global__ void __launch_bounds__(kThreads) combine_kernel(const CombineParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int hv = p.H >> 3;
  const long long total = (long long)p.T * hv;
  for (long long idx = (long long)blockIdx.x * kThreads + threadIdx.x; idx < total;
       idx += (long long)gridDim.x * kThreads) {
    const int t = (int)(idx / hv);
    const int c = (int)(idx - (long long)t * hv);
    float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if constexpr (K8) {
      uint4 v[8];
      float wt[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int pos = min(max(__ldg(p.inv + (size_t)t * 8 + j), 0), p.S - 1);
        wt[j] = __ldg(p.topk_w + (size_t)t * 8 + j);
        v[j] = __ldcs(reinterpret_cast<const uint4 *>(p.y_sorted + (size_t)pos * p.H) + c);
      }
      uint4 z = make_uint4(0u, 0u, 0u, 0u);
      if (p.y_shared != nullptr) z = __ldcs(reinterpret_cast<const uint4 *>(p.y_shared + (size_t)t * p.H) + c);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc8(a, v[j], wt[j]);
      if (p.y_shared != nullptr) acc8(a, z, 1.0f);
    } else if constexpr (!BATCHED) {
      for (int j = 0; j < p.top_k; ++j) {
        const int pos = min(max(__ldg(p.inv + (size_t)t * p.top_k + j), 0), p.S - 1);
        const float w = __ldg(p.topk_w + (size_t)t * p.top_k + j);
        acc8(a, __ldcs(reinterpret_cast<const uint4 *>(p.y_sorted + (size_t)pos * p.H) + c), w);
      }
      if (p.y_shared != nullptr)
        acc8(a, __ldcs(reinterpret_cast<const uint4 *>(p.y_shared + (size_t)t * p.H) + c), 1.0f);
    } else {
      // every slot's index and weight, then every row piece, in flight at once
      // (top_k <= 16); accumulated in slot order
      int pos[kMaxK];
      float wt[kMaxK];
#pragma unroll
      for (int j = 0; j < kMaxK; ++j) {
        if (j < p.top_k) {
          pos[j] = min(max(__ldg(p.inv + (size_t)t * p.top_k + j), 0), p.S - 1);
          wt[j] = __ldg(p.topk_w + (size_t)t * p.top_k + j);
        }
      }
      uint4 v[kMaxK];
#pragma unroll
      for (int j = 0; j < kMaxK; ++j)
        if (j < p.top_k) v[j] = __ldcs(reinterpret_cast<const uint4 *>(p.y_sorted + (size_t)pos[j] * p.H) + c);
      uint4 z = make_uint4(0u, 0u, 0u, 0u);
      if (p.y_shared != nullptr) z = __ldcs(reinterpret_cast<const uint4 *>(p.y_shared + (size_t)t * p.H) + c);
#pragma unroll
      for (int j = 0; j < kMaxK; ++j)
        if (j < p.top_k) acc8(a, v[j], wt[j]);
      if (p.y_shared != nullptr) acc8(a, z, 1.0f);
    }
    uint4 o;
    uint32_t *ou = reinterpret_cast<uint32_t *>(&o);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(a[2 * i], a[2 * i + 1]);
      ou[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    reinterpret_cast<uint4 *>(p.out + (size_t)t * p.H)[c] = o;
  }
}

// Gradients of the combine.  A CTA per token, or (WARP: rows of at most 2048 values,
// which leave much of a CTA idle) a warp: its row of grad_out against the rows of
// its slots, 8 values a thread step; the sums over H are added in a fixed order.  HBM-bound: K slots' loads in flight together (8 for top-8 and fewer:
// Hy3 T = 4096, 571 MB, 98 us, 5.8 TB/s, against 121 one slot at a time), then their
// stores.
template <int K, bool WARP>
__global__ void __launch_bounds__(kThreads, K <= 8 ? 3 : 1) combine_grad_kernel(const CombineGradParams p) {
  __shared__ float sums[kThreads / 32][K];
  pdl_wait();
  pdl_launch_dependents();
  const int hv = p.H >> 3, k = p.top_k;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kTokens = WARP ? kThreads / 32 : 1, kPerToken = WARP ? 32 : kThreads;
  for (unsigned t = blockIdx.x * kTokens + (WARP ? warp : 0); t < (unsigned)p.T; t += gridDim.x * kTokens) {
    int pos[K];
    float wt[K], acc[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      acc[j] = 0.0f;
      wt[j] = 0.0f;
      pos[j] = 0;
      if (j < k) {
        pos[j] = min(max(__ldg(p.inv + (size_t)t * k + j), 0), p.S - 1);
        if (p.grad_y != nullptr) wt[j] = __ldg(p.topk_w + (size_t)t * k + j);
      }
    }
    for (int c = WARP ? lane : (int)threadIdx.x; c < hv; c += kPerToken) {
      float g[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      const uint4 go = __ldg(reinterpret_cast<const uint4 *>(p.grad_out + (size_t)t * p.H) + c);
      if (p.grad_w != nullptr) {
        uint4 v[K];
#pragma unroll
        for (int j = 0; j < K; ++j)
          if (j < k) v[j] = __ldcs(reinterpret_cast<const uint4 *>(p.y_sorted + (size_t)pos[j] * p.H) + c);
        acc8(g, go, 1.0f);
#pragma unroll
        for (int j = 0; j < K; ++j)
          if (j < k) {
            const uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              acc[j] = fmaf(g[2 * i], __uint_as_float(u[i] << 16), acc[j]);
              acc[j] = fmaf(g[2 * i + 1], __uint_as_float(u[i] & 0xffff0000u), acc[j]);
            }
          }
      } else {
        acc8(g, go, 1.0f);
      }
      if (p.grad_y != nullptr) {
#pragma unroll
        for (int j = 0; j < K; ++j)
          if (j < k) {
            uint4 o;
            uint32_t *ou = reinterpret_cast<uint32_t *>(&o);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(wt[j] * g[2 * i], wt[j] * g[2 * i + 1]);
              ou[i] = *reinterpret_cast<const uint32_t *>(&b);
            }
            __stcs(reinterpret_cast<uint4 *>(p.grad_y + (size_t)pos[j] * p.H) + c, o);
          }
      }
    }
    if (p.grad_w == nullptr) continue;
#pragma unroll
    for (int j = 0; j < K; ++j) {
      if (j >= k) break;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
      if (lane == 0) {
        if (WARP) p.grad_w[(size_t)t * k + j] = acc[j];
        else sums[warp][j] = acc[j];
      }
    }
    if (WARP) continue;
    __syncthreads();
    if (threadIdx.x < (unsigned)k) {
      float s = 0.0f;
      for (int w = 0; w < kThreads / 32; ++w) s += sums[w][threadIdx.x];
      p.grad_w[(size_t)t * k + threadIdx.x] = s;
    }
    __syncthreads();
  }
}

cudaError_t launch_combine_grad(const CombineGradParams &p, cudaStream_t stream) {
  static thread_local int nsm = 0, dev_cached = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev != dev_cached) {
    cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
    dev_cached = dev;
  }
  const int cap = (nsm > 0 ? nsm : 1) * 8;
  void *args[] = {(void *)&p};
  // H = 2048: 16384 tokens, top-8, 183 us with a warp a token, 213 with a CTA; H = 4096,
  // 4096 tokens, top-8, 114 and 98.  Fewer tokens than CTAs: a CTA each, all at once.
  const bool warp = p.H <= 2048 && p.T > cap;
  const void *fn = p.top_k <= 2   ? warp ? (const void *)combine_grad_kernel<2, true> : (const void *)combine_grad_kernel<2, false>
                   : p.top_k <= 8 ? warp ? (const void *)combine_grad_kernel<8, true> : (const void *)combine_grad_kernel<8, false>
                   : warp         ? (const void *)combine_grad_kernel<kMaxK, true>
                                  : (const void *)combine_grad_kernel<kMaxK, false>;
  const int blocks = warp ? (p.T + kThreads / 32 - 1) / (kThreads / 32) : p.T;
  return launch_ex(fn, dim3(blocks < cap ? blocks : cap), dim3(kThreads), 0, stream, true, 1, args);
}

cudaError_t launch_combine(const CombineParams &p, cudaStream_t stream, bool pdl) {
  static thread_local int nsm = 0, dev_cached = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev != dev_cached) {
    cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
    dev_cached = dev;
  }
  const long long total = (long long)p.T * (p.H >> 3);
  long long blocks = (total + kThreads - 1) / kThreads;
  const long long cap = (long long)nsm * 8;
  if (blocks > cap) blocks = cap;
  if (blocks < 1) blocks = 1;
  void *args[] = {(void *)&p};
  const bool batched = total <= (long long)nsm * kThreads;  // one wave of threads
  const void *fn = batched ? (const void *)combine_kernel<true>
                   : p.top_k == 8 ? (const void *)combine_kernel<false, true>
                                  : (const void *)combine_kernel<false>;
  return launch_ex(fn, dim3((unsigned)blocks), dim3(kThreads), 0, stream, pdl, 1, args);
}

}  // namespace moe
