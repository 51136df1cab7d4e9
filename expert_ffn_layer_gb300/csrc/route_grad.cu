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

// A value as three bf16 pieces whose sum it is: its first 8 bits, the next rounded to
// nearest even, the rest (at most 8 bits).  Below 2^-110 or so the rest runs out of
// bf16's range.  Infinities and NaN are in the first piece alone.
struct Pieces {
  uint32_t hi, mid, lo;  // bf16 bits
};
__device__ __forceinline__ Pieces pieces_of(float v) {
  Pieces r;
  const uint32_t u = __float_as_uint(v);
  if ((u & 0x7F800000u) == 0x7F800000u) {
    r.hi = (u & 0x7FFFFFu) ? 0x7FC0u : u >> 16;
    r.mid = r.lo = 0;
    return r;
  }
  r.hi = u >> 16;
  const float rest = v - __uint_as_float(r.hi << 16);
  const __nv_bfloat16 m = __float2bfloat16_rn(rest);
  r.mid = __bfloat16_as_ushort(m);
  r.lo = __bfloat16_as_ushort(__float2bfloat16_rn(rest - __bfloat162float(m)));
  return r;
}
}  // namespace

// What the losses' gradient needs of the whole batch.
struct BatchTerms {
  float load, gz, g0;  // E / (k B), 2 G1 / n, G0
};
__device__ __forceinline__ BatchTerms batch_terms(const RouteGradParams &p, int *sh) {
  BatchTerms r = {0.0f, 0.0f, 0.0f};
  if (p.grad_losses == nullptr) return r;
  r.g0 = __ldg(p.grad_losses);
  const float g1 = __ldg(p.grad_losses + 1);
  const int2 nt = sequence_totals(p.tokens, p.n_seq, sh);
  r.load = (float)p.E / (float)p.top_k / (float)max(nt.x, 1);
  r.gz = g1 * 2.0f / (float)max(nt.y, 1);
  return r;
}

// The gradient of token t's logits, by a warp.  1 - s is taken as the sigmoid of the
// negated logit, which keeps its digits where s is near one.
template <bool SIGMOID>
__device__ __forceinline__ void token_grad(const RouteGradParams &p, const BatchTerms &bt, int t, int lane,
                                           float (&d)[kPerLane]) {
  const int E = p.E, k = p.top_k;
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) d[j] = 0.0f;
  // everything that is read goes out first; a padded token's is not used
  const int b = token_seq(p.seq_id, p.n_seq, t, p.err);
  float v[kPerLane];
  load_logits(p.logits + (size_t)t * E, E, lane, v);
  int e = 0;
  float g = 0.0f;  // lane i < k holds slot i
  if (p.grad_w != nullptr && lane < k) {
    e = __ldg(p.topk_idx + (size_t)t * k + lane);
    g = __ldg(p.grad_w + (size_t)t * k + lane);
  }
  if (b < 0) return;
  int c[kPerLane];
  float n = 1.0f;
  if (p.grad_losses != nullptr) {
    const int32_t *of = p.counts + (size_t)b * E;
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) c[j] = expert_of(lane, j) < E ? __ldg(of + expert_of(lane, j)) : 0;
    n = (float)max(__ldg(p.tokens + b), 1);
  }
  const TokenScores r = token_scores<SIGMOID>(v, E, lane);
  if (p.grad_losses != nullptr) {
    const float load = bt.load / n / n, inv = SIGMOID ? 1.0f / r.total : 1.0f;
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) dot = fmaf((float)c[j] * load, (SIGMOID ? r.s[j] : r.p[j]) * inv, dot);
    dot = warp_sum(dot);
    const float gz = bt.gz * r.lse;
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      const float q = (SIGMOID ? r.s[j] : r.p[j]) * inv;
      d[j] = bt.g0 * q * ((float)c[j] * load - dot) * (SIGMOID ? r.miss[j] : 1.0f) + gz * r.p[j];
    }
  }
  if (p.grad_w != nullptr) {
    if (lane < k) e = checked_expert(e, E, p.err);
    float score = 0.0f, rest = 0.0f;  // of the slot's expert, from the lane that has it
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      const float a = __shfl_sync(0xffffffffu, SIGMOID ? r.s[j] : r.p[j], lane_of(e));
      if (slot_of(e) == j) score = a;
      if (SIGMOID) {
        const float m = __shfl_sync(0xffffffffu, r.miss[j], lane_of(e));
        if (slot_of(e) == j) rest = m;
      }
    }
    if (lane >= k) score = 0.0f;
    const float sel = warp_sum(score);
    float w;  // the slot's contribution to its expert's logit
    float spread = 0.0f;
    if (!SIGMOID && !(sel >= p.renorm_eps)) {  // the clamp acts: the weight is p / eps
      w = g / p.renorm_eps * score;
      spread = warp_sum(w);
    } else {
      const float u = score / sel, mean = warp_sum(g * u);
      w = u * (g - mean) * (SIGMOID ? p.route_scale * rest : 1.0f);
    }
    for (int i = 0; i < k; ++i) {
      const int ei = __shfl_sync(0xffffffffu, e, i);
      const float wi = __shfl_sync(0xffffffffu, w, i);
#pragma unroll
      for (int j = 0; j < kPerLane; ++j)
        if (ei == expert_of(lane, j)) d[j] += wi;
    }
    if (spread != 0.0f) {
#pragma unroll
      for (int j = 0; j < kPerLane; ++j) d[j] = fmaf(-spread, r.p[j], d[j]);
    }
  }
}

// A warp per token: bound by the latency of its loads and shuffles (E = 192: 5 us at
// T = 4096, 21 at 16384, 25 MB).  The CTAs past logit_blocks split the router weight into the
// pieces that grad_hidden takes.
template <bool SIGMOID>
__global__ void __launch_bounds__(kThreads) grad_logits_kernel(const __grid_constant__ RouteGradParams p) {
  __shared__ int sh[2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = p.E;
  pdl_wait();
  pdl_launch_dependents();
  if ((int)blockIdx.x >= p.logit_blocks) {
    const long long n8 = (long long)E * p.H / 8;
    for (long long i = (long long)(blockIdx.x - p.logit_blocks) * kThreads + threadIdx.x; i < n8;
         i += (long long)(gridDim.x - p.logit_blocks) * kThreads) {
      const float4 a = __ldg(reinterpret_cast<const float4 *>(p.router_w) + 2 * i);
      const float4 b = __ldg(reinterpret_cast<const float4 *>(p.router_w) + 2 * i + 1);
      const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      uint32_t hi[4], mid[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const Pieces x = pieces_of(v[2 * j]), y = pieces_of(v[2 * j + 1]);
        hi[j] = x.hi | y.hi << 16;
        mid[j] = x.mid | y.mid << 16;
      }
      reinterpret_cast<uint4 *>(p.w_pieces)[i] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      reinterpret_cast<uint4 *>(p.w_pieces)[n8 + i] = make_uint4(mid[0], mid[1], mid[2], mid[3]);
    }
    return;
  }
  const BatchTerms bt = batch_terms(p, sh);
  for (unsigned t = blockIdx.x * (kThreads / 32) + warp; t < (unsigned)p.T; t += p.logit_blocks * (kThreads / 32)) {
    float d[kPerLane];
    token_grad<SIGMOID>(p, bt, (int)t, lane, d);
    if (p.dl != nullptr) {
#pragma unroll
      for (int j = 0; j < kPerLane; ++j)
        if (expert_of(lane, j) < E) p.dl[(size_t)t * E + expert_of(lane, j)] = d[j];
    }
    if (p.pieces != nullptr) {
      const size_t plane = (size_t)p.T * p.Epad;
      uint16_t *row = p.pieces + (size_t)t * p.Epad + 2 * lane;
#pragma unroll
      for (int j = 0; j < kPerLane; j += 2)
        if (32 * j < p.Epad) {  // zeros past the last expert
          const Pieces x = pieces_of(d[j]), y = pieces_of(d[j + 1]);
          uint32_t *at = reinterpret_cast<uint32_t *>(row + 32 * j);
          at[0] = x.hi | y.hi << 16;
          at[plane / 2] = x.mid | y.mid << 16;
          at[plane] = x.lo | y.lo << 16;
        }
    }
  }
}

// The whole pass for few tokens in one kernel: every CTA forms all the logits'
// gradients itself (a warp two tokens) and takes 32 columns of both products in
// fp32.  The products are a read and a write of the router weight's size (Hy3's
// router, T = 8: 6.4 MB, 12 us as against 22 in three kernels, most of it the launch
// and the chain of loads).
template <bool SIGMOID>
__global__ void __launch_bounds__(kThreads) grad_few_kernel(const __grid_constant__ RouteGradParams p) {
  __shared__ int sh[2];
  __shared__ float dl[kFewTokens][256];
  __shared__ float part[kThreads / 32][kFewTokens][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = p.E, T = p.T, h = blockIdx.x * 32 + lane;
  constexpr int kWarps = kThreads / 32;
  pdl_wait();
  pdl_launch_dependents();
  const BatchTerms bt = batch_terms(p, sh);
  for (int t = warp; t < T; t += kWarps) {
    float d[kPerLane];
    token_grad<SIGMOID>(p, bt, t, lane, d);
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      dl[t][expert_of(lane, j)] = d[j];
      if (p.dl != nullptr && blockIdx.x == 0 && expert_of(lane, j) < E) p.dl[(size_t)t * E + expert_of(lane, j)] = d[j];
    }
  }
  __syncthreads();
  // this lane's column: warp w takes experts w, w + 8, .. of both products
  if (p.grad_router_w != nullptr) {
    float x[kFewTokens];
#pragma unroll
    for (int t = 0; t < kFewTokens; ++t) {
      x[t] = 0.0f;
      if (t < T && token_seq(p.seq_id, p.n_seq, t, p.err) >= 0) x[t] = __bfloat162float(p.hidden[(size_t)t * p.H + h]);
    }
    for (int e = warp; e < E; e += kWarps) {
      float a = 0.0f;
#pragma unroll
      for (int t = 0; t < kFewTokens; ++t)
        if (t < T) a = fmaf(dl[t][e], x[t], a);
      p.grad_router_w[(size_t)e * p.H + h] = a;
    }
  }
  if (p.grad_hidden == nullptr) return;
  float a[kFewTokens];
#pragma unroll
  for (int t = 0; t < kFewTokens; ++t) a[t] = 0.0f;
#pragma unroll 4
  for (int e = warp; e < E; e += kWarps) {
    const float w = __ldg(p.router_w + (size_t)e * p.H + h);
#pragma unroll
    for (int t = 0; t < kFewTokens; ++t)
      if (t < T) a[t] = fmaf(dl[t][e], w, a[t]);
  }
#pragma unroll
  for (int t = 0; t < kFewTokens; ++t) part[warp][t][lane] = a[t];
  __syncthreads();
  for (int t = warp; t < T; t += kWarps) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += part[w][t][lane];
    p.grad_hidden[(size_t)t * p.H + h] = __float2bfloat16_rn(s);
  }
}

// ------------------------------------------------------------- the products
// grad_hidden = dl W and grad_router_w = dl^T x on the tensor cores.  An fp32 factor
// goes in as bf16 pieces that add up to it: a first piece cut off after 8 bits, the
// next rounded, the third what is left (exact).  grad_router_w takes all three pieces
// of dl (x is bf16: its products are exact, rounding is that of the fp32 sums);
// grad_hidden, rounded to bf16 in the end, two pieces of dl and of W and three of
// their four products (relative error of a product 2^-15 at most).
//
// grad_hidden: a CTA keeps the pieces of W's 128 columns (at most 128 KB) as the M
// operand and walks over 256 tokens at a time as the N one (128 tokens as M and 128
// columns as N read shared memory faster than it answers: 79 us against 65 at 16384
// tokens), their pieces of dl in a ring of 64-expert steps.
// grad_router_w: a CTA has 128 columns of x and a part of the tokens, in steps of
// 64; both operands lie with their row dimension inner (MN-major).  The tensor cores'
// fp32 sums are cut off, not rounded, at each step, which over thousands of tokens
// would shrink the result (by 2.4e-6 of itself over 1024): two accumulators take 128
// tokens in turn, and the epilogue warps add them up in registers.  The parts of one
// tile are a cluster, which adds its fp32 tiles over shared memory in rank order.
// Hy3's router (H = 4096, E = 192) at T = 4096: 22 and 29 us, of which the MMAs of three
// products take 9.7 each; at 16384 70 and 80 us, MMAs 39.
constexpr int kSmemMax = 232448;  // 227 KB opt-in per block
constexpr int kBox = 64 * 128;    // 64 rows of 128 bytes
constexpr int kProdThreads = 320;  // warp 0 TMA, 1 MMA, 2-9 epilogue (TMEM lane quarters 2,3,0,1, twice)
constexpr int kStep = 64;          // tokens of a step of grad_router_w
constexpr int kWBox = kStep * 128;  // its boxes: 64 rows of 128 bytes
constexpr int kChunk = 2;          // steps before the accumulator changes
constexpr int kMaxSplit = 8;

// Shared-memory matrix descriptor of an operand with its row dimension (M or N)
// inner, 128-byte swizzle: atoms of 64 rows x 8 of K, 1024 bytes from one group of 8
// of K to the next, `atom` bytes from one 64 rows to the next.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr, uint32_t atom) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(atom >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
constexpr uint32_t kTransA = 1u << 15, kTransB = 1u << 16;  // instruction descriptor: the operand is MN-major

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *m, uint32_t bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          dst),
      "l"(m), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// Barriers, TMEM slot and abort flag of either product, behind its operands.
struct ProdShared {
  uint64_t full[8], empty[8], ready[8], afull[2], aempty[2], bfull;
  uint32_t tmem;
  int abort;
};

__global__ void __launch_bounds__(kProdThreads, 1) grad_hidden_kernel(const __grid_constant__ RouteGradParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const int eb = p.Epad >> 6, nst = p.hidden_stages;
  const int w_piece = eb * 2 * kBox;  // one piece of W: eb steps of two 64-column boxes
  uint8_t *ring = smem + 2 * w_piece;
  constexpr int kStage = 4 * kBox;  // one piece of dl: 256 tokens x 64 experts
  ProdShared *sh = (ProdShared *)(ring + nst * kStage);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h0 = blockIdx.x * 128, tiles = (p.T + 255) >> 8;
  volatile int *abort_flag = &sh->abort;
  unsigned *err = p.err;
  if (threadIdx.x == 0) {
    for (int s = 0; s < nst; ++s) {
      mbar_init(smem_u32(&sh->full[s]), 1);
      mbar_init(smem_u32(&sh->empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&sh->afull[a]), 1);
      mbar_init(smem_u32(&sh->aempty[a]), 8);
    }
    mbar_init(smem_u32(&sh->bfull), 1);
    sh->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sh->tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem;
  pdl_wait();  // the pieces come from the kernel before
  pdl_launch_dependents();
  bool ok = true;
  if (warp == 0) {
    if (lane == 0) {
      const uint32_t bb = smem_u32(&sh->bfull);
      mbar_arrive_expect_tx(bb, (uint32_t)(2 * w_piece));
      for (int pc = 0; pc < 2; ++pc)
        for (int e = 0; e < eb; ++e)
          for (int x = 0; x < 2; ++x)
            tma_load_3d(smem_u32(smem + pc * w_piece + (2 * e + x) * kBox), &p.map_w, bb, h0 + 64 * x, 64 * e, pc);
      int i = 0;
      for (int t = blockIdx.y; t < tiles && ok; t += gridDim.y) {
        const bool both = p.T - 256 * t > 128;  // boxes of 128 tokens
        for (int j = 0; j < 2 * eb; ++j, ++i) {  // step j: 64 experts j / 2, piece j % 2
          const int s = i % nst;
          ok = mbar_wait(smem_u32(&sh->empty[s]), ((uint32_t)(i / nst) & 1u) ^ 1u, err, abort_flag);
          if (!ok) break;
          const uint32_t fb = smem_u32(&sh->full[s]), st = smem_u32(ring + s * kStage);
          mbar_arrive_expect_tx(fb, both ? kStage : kStage / 2);
          tma_load_3d(st, &p.map_dl_k, fb, 32 * (j & ~1), 256 * t, j & 1);
          if (both) tma_load_3d(st + 2 * kBox, &p.map_dl_k, fb, 32 * (j & ~1), 256 * t + 128, j & 1);
        }
      }
      if (!ok) {  // leave no copy in flight
        mbar_wait(bb, 0, err, nullptr);
        for (int j = i - nst < 0 ? 0 : i - nst; j < i; ++j)
          mbar_wait(smem_u32(&sh->full[j % nst]), (uint32_t)(j / nst) & 1u, err, nullptr);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      ok = mbar_wait(smem_u32(&sh->bfull), 0, err, abort_flag);
      int i = 0, na = 0;
      for (int t = blockIdx.y; t < tiles && ok; t += gridDim.y, ++na) {
        const int acc = na & 1, n = min(256, (p.T - 256 * t + 15) & ~15);
        ok = mbar_wait(smem_u32(&sh->aempty[acc]), ((uint32_t)(na >> 1) & 1u) ^ 1u, err, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint32_t dst = tmem + 256u * acc, idesc = idesc_bf16(128, n) | kTransA;
        for (int j = 0; j < 2 * eb; ++j, ++i) {
          const int s = i % nst;
          ok = mbar_wait(smem_u32(&sh->full[s]), (uint32_t)(i / nst) & 1u, err, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint32_t wb = smem_u32(smem + (j & ~1) * kBox);
          const uint64_t bd = sdesc_sw128(smem_u32(ring + s * kStage));
          const uint64_t a0 = sdesc_mn(wb, kBox), a1 = sdesc_mn(wb + w_piece, kBox);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {  // 16 experts: 16 rows of W, 32 bytes along dl's rows
            umma_bf16(dst, a0 + 128 * kk, bd + 2 * kk, idesc, (j > 0 || kk > 0) ? 1u : 0u);
            if (!(j & 1)) umma_bf16(dst, a1 + 128 * kk, bd + 2 * kk, idesc, 1u);
          }
          umma_commit(smem_u32(&sh->empty[s]));
        }
        if (!ok) break;
        umma_commit(smem_u32(&sh->afull[acc]));
      }
    }
  } else {
    // TMEM lane: a column of W; its columns: tokens, 128 of the lane quarter's 256 to
    // each of its two warps.  Four lanes swap four tokens' values, so that each
    // stores four neighbouring columns of one token.
    const int q = warp & 3, half = (warp - 2) >> 2;
    const int h = h0 + 32 * q + (lane & ~3), sub = lane & 3;
    int na = 0;
    for (int t = blockIdx.y; t < tiles && ok; t += gridDim.y, ++na) {
      const int acc = na & 1, t0 = 256 * t + 128 * half;
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&sh->afull[acc]), (uint32_t)(na >> 1) & 1u, err, abort_flag));
      if (!ok) break;
      tc_fence_after();
      const uint32_t base = tmem + 256u * acc + 128u * half + ((uint32_t)(32 * q) << 16);
#pragma unroll 1
      for (int c = 0; c < 128 && t0 + c < p.T; c += 32) {
        float v[32];
        tmem_ld32(base + (uint32_t)c, v);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          uint32_t w[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {  // lanes l and l ^ 1: tokens j + 2 u and the next
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[j + 2 * u], v[j + 2 * u + 1]);
            const uint32_t mine = *reinterpret_cast<const uint32_t *>(&b), other = __shfl_xor_sync(0xffffffffu, mine, 1);
            w[u] = lane & 1 ? __byte_perm(other, mine, 0x7632) : __byte_perm(mine, other, 0x5410);
          }
          const uint32_t got = __shfl_xor_sync(0xffffffffu, lane & 2 ? w[0] : w[1], 2);
          const uint2 o = lane & 2 ? make_uint2(got, w[1]) : make_uint2(w[0], got);
          const int tok = t0 + c + j + sub;
          if (tok < p.T && h < p.H) *reinterpret_cast<uint2 *>(p.grad_hidden + (size_t)tok * p.H + h) = o;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh->aempty[acc]));
    }
  }
  tc_fence_before();
  __syncwarp();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

__global__ void __launch_bounds__(kProdThreads, 1) grad_router_w_kernel(const __grid_constant__ RouteGradParams p,
                                                                     int waited) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const int eb = p.Epad >> 6, nst = p.w_stages;
  const int stage = (2 + 3 * eb) * kWBox;  // 128 columns of x and three pieces of dl
  ProdShared *sh = (ProdShared *)(smem + p.w_smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = gridDim.x, rank = blockIdx.x, h0 = blockIdx.y * 128;
  const int blocks = (p.T + kStep - 1) / kStep;
  const int k0 = (int)((long long)blocks * rank / split), k1 = (int)((long long)blocks * (rank + 1) / split);
  volatile int *abort_flag = &sh->abort;
  unsigned *err = p.err;
  uint32_t tmem_cols = 32;
  while (tmem_cols < 2u * p.Epad) tmem_cols <<= 1;
  if (threadIdx.x == 0) {
    for (int s = 0; s < nst; ++s) {
      mbar_init(smem_u32(&sh->full[s]), 1);
      mbar_init(smem_u32(&sh->empty[s]), 1);
      mbar_init(smem_u32(&sh->ready[s]), 4);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&sh->afull[a]), 1);
      mbar_init(smem_u32(&sh->aempty[a]), 8);
    }
    sh->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sh->tmem), tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem;
  // Behind grad_hidden_kernel, whose CTAs let this kernel start once each of them has
  // waited for the pieces, they are there already; its own end is waited for below.
  if (!waited) pdl_wait();
  pdl_launch_dependents();
  // whether any of this part's tokens is padding
  bool masked = false;
  if (p.seq_id != nullptr) {
    int any = 0;
    for (int t = kStep * k0 + threadIdx.x; t < min(p.T, kStep * k1); t += kProdThreads)
      any |= token_seq(p.seq_id, p.n_seq, t, err) < 0;
    masked = __syncthreads_or(any);
  }
  bool ok = true;
  if (warp == 0) {
    if (lane == 0) {
      int i = 0;
      for (int b = k0; b < k1; ++b, ++i) {
        const int s = i % nst;
        ok = mbar_wait(smem_u32(&sh->empty[s]), ((uint32_t)(i / nst) & 1u) ^ 1u, err, abort_flag);
        if (!ok) break;
        const uint32_t fb = smem_u32(&sh->full[s]), st = smem_u32(smem + s * stage);
        mbar_arrive_expect_tx(fb, (uint32_t)stage);
        tma_load_2d(st, &p.map_x, fb, h0, kStep * b);
        tma_load_2d(st + kWBox, &p.map_x, fb, h0 + 64, kStep * b);
        for (int pc = 0; pc < 3; ++pc)
          for (int e = 0; e < eb; ++e)
            tma_load_3d(st + (2 + pc * eb + e) * kWBox, &p.map_dl_mn, fb, 64 * e, kStep * b, pc);
      }
      if (!ok)
        for (int j = i - nst < 0 ? 0 : i - nst; j < i; ++j)
          mbar_wait(smem_u32(&sh->full[j % nst]), (uint32_t)(j / nst) & 1u, err, nullptr);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16(128, p.Epad) | kTransA | kTransB;
      for (int i = 0; i < k1 - k0; ++i) {
        const int s = i % nst, chunk = i / kChunk, acc = chunk & 1;
        if (i % kChunk == 0) {
          ok = mbar_wait(smem_u32(&sh->aempty[acc]), ((uint32_t)(chunk >> 1) & 1u) ^ 1u, err, abort_flag);
          if (!ok) break;
          tc_fence_after();
        }
        ok = mbar_wait(smem_u32(masked ? &sh->ready[s] : &sh->full[s]), (uint32_t)(i / nst) & 1u, err, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint32_t st = smem_u32(smem + s * stage);
        const uint64_t a = sdesc_mn(st, kWBox);
#pragma unroll
        for (int pc = 2; pc >= 0; --pc) {  // the small pieces first
          const uint64_t bd = sdesc_mn(st + (2 + pc * eb) * kWBox, kWBox);
#pragma unroll
          for (int kk = 0; kk < kStep / 16; ++kk)
            umma_bf16(tmem + (uint32_t)(acc * p.Epad), a + 128 * kk, bd + 128 * kk, idesc,
                      (i % kChunk || pc < 2 || kk > 0) ? 1u : 0u);
        }
        umma_commit(smem_u32(&sh->empty[s]));
        if (i % kChunk == kChunk - 1 || i == k1 - k0 - 1) umma_commit(smem_u32(&sh->afull[acc]));
      }
    }
  } else {
    // TMEM lane: a column of x; its columns: the experts, 16-column groups of the lane
    // quarter in turn to its two warps, whose sums stay in registers
    const int q = warp & 3, half = (warp - 2) >> 2, h = h0 + 32 * q + lane;
    float sum[8][16];
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
      for (int j = 0; j < 16; ++j) sum[c][j] = 0.0f;
    // padded tokens' rows of x are overwritten with zeros before they are multiplied
    // (their rows of dl are zero, which NaN times would not be): the first four warps
    const bool mask = masked && half == 0;
    const int tid = threadIdx.x - 64, row = tid & (kStep - 1), box = (tid / kStep) & 1;
    const int steps = k1 - k0, chunks = (steps + kChunk - 1) / kChunk;
    int cleared = 0;
    for (int n = 0; n < chunks && ok; ++n) {
      if (mask) {
        // up to the end of the chunk after this one, as far as the ring reaches: the
        // products of chunk n + 1 need not wait for the sums of chunk n
        const int until = min(steps, min(kChunk * (n + 2), kChunk * (n + 1) + nst - 1));
        for (; cleared < until; ++cleared) {
          const int s = cleared % nst, t = kStep * (k0 + cleared) + row;
          const bool off = t < p.T && token_seq(p.seq_id, p.n_seq, t, err) < 0;
          ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&sh->full[s]), (uint32_t)(cleared / nst) & 1u, err, abort_flag));
          if (!ok) break;
          if (off) {
            const uint32_t at = smem_u32(smem + s * stage + box * kWBox + row * 128);
#pragma unroll
            for (int c = 0; c < 8; ++c) st_shared_v4(at + 16 * c, make_uint4(0u, 0u, 0u, 0u));
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh->ready[s]));
        }
        if (!ok) break;
      }
      const int acc = n & 1;
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&sh->afull[acc]), (uint32_t)(n >> 1) & 1u, err, abort_flag));
      if (!ok) break;
      tc_fence_after();
      const uint32_t base = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(acc * p.Epad + 16 * half);
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (32 * c + 16 * half < p.E) {
          float v[16];
          tmem_ld16(base + (uint32_t)(32 * c), v);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) sum[c][j] += v[j];
        }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh->aempty[acc]));
    }
    if (ok) {
      float *tile = reinterpret_cast<float *>(smem);  // [E][128]: every copy and product is done
#pragma unroll
      for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int e = 32 * c + 16 * half + j;
          if (e < p.E) {
            if (split > 1) tile[e * 128 + 32 * q + lane] = sum[c][j];
            else if (h < p.H) p.grad_router_w[(size_t)e * p.H + h] = sum[c][j];
          }
        }
    }
  }
  tc_fence_before();
  __syncwarp();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, tmem_cols);
  }
  if (split > 1) {
    cluster_sync();
    // rank r adds up experts r, r + split, ..: a warp a row of 128 columns
    const int col = 4 * lane;
#pragma unroll 2
    for (int e = rank + split * warp; e < p.E; e += split * (kProdThreads / 32)) {
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      float4 v[kMaxSplit];
#pragma unroll
      for (int r = 0; r < kMaxSplit; ++r)
        if (r < split) {
          const uint32_t at = map_cluster(smem_u32(smem) + (uint32_t)(e * 128 + col) * 4, (uint32_t)r);
          asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                       : "=f"(v[r].x), "=f"(v[r].y), "=f"(v[r].z), "=f"(v[r].w)
                       : "r"(at)
                       : "memory");
        }
#pragma unroll
      for (int r = 0; r < kMaxSplit; ++r)
        if (r < split) a = make_float4(a.x + v[r].x, a.y + v[r].y, a.z + v[r].z, a.w + v[r].w);
      if (h0 + col < p.H) *reinterpret_cast<float4 *>(p.grad_router_w + (size_t)e * p.H + h0 + col) = a;
    }
    cluster_sync();  // nobody leaves while its tile is being read
  }
  if (waited) pdl_wait();  // the next kernel waits for this one alone
}

cudaError_t launch_route_grad(RouteGradParams p, int num_sms, cudaStream_t stream) {
  static thread_local unsigned long long attr_h = 0, attr_w = 0;
  const int eb = p.Epad >> 6, tail = (int)sizeof(ProdShared) + 1024;
  if (p.T <= kFewTokens && p.pieces != nullptr) {
    void *args[] = {(void *)&p};
    return launch_ex(p.sigmoid ? (const void *)grad_few_kernel<true> : (const void *)grad_few_kernel<false>,
                     dim3(p.H / 32), dim3(kThreads), 0, stream, true, 1, args);
  }
  int blocks = (p.T + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 8 * num_sms) blocks = 8 * num_sms;
  p.logit_blocks = blocks;
  if (p.grad_hidden != nullptr) {
    const long long n = ((long long)p.E * p.H / 8 + kThreads - 1) / kThreads;
    blocks += (int)(n < 2 * num_sms ? n : 2 * num_sms);
  }
  {
    void *args[] = {(void *)&p};
    const cudaError_t e = launch_ex(p.sigmoid ? (const void *)grad_logits_kernel<true> : (const void *)grad_logits_kernel<false>,
                                    dim3(blocks), dim3(kThreads), 0, stream, true, 1, args);
    if (e != cudaSuccess) return e;
  }
  const int hb = (p.H + 127) >> 7;
  if (p.grad_hidden != nullptr) {
    const cudaError_t e0 = set_smem_attr_once((const void *)grad_hidden_kernel, kSmemMax, attr_h);
    if (e0 != cudaSuccess) return e0;
    const int tiles = (p.T + 255) >> 8;
    int rows = num_sms / hb;  // CTAs that share the token tiles: one wave
    if (rows < 1) rows = 1;
    if (rows > tiles) rows = tiles;
    p.hidden_stages = (kSmemMax - tail - 4 * eb * kBox) / (4 * kBox);
    if (p.hidden_stages > 4) p.hidden_stages = 4;
    const size_t smem = (size_t)(4 * eb + 4 * p.hidden_stages) * kBox + tail;
    void *args[] = {(void *)&p};
    const cudaError_t e = launch_ex((const void *)grad_hidden_kernel, dim3(hb, rows), dim3(kProdThreads), smem, stream, true,
                                    1, args);
    if (e != cudaSuccess) return e;
  }
  if (p.grad_router_w != nullptr) {
    const cudaError_t e0 = set_smem_attr_once((const void *)grad_router_w_kernel, kSmemMax, attr_w);
    if (e0 != cudaSuccess) return e0;
    const int steps = (p.T + kStep - 1) / kStep, stage = (2 + 3 * eb) * kWBox;
    // parts of the tokens, a cluster, of at least four steps each (512 tokens at H = 4096:
    // two parts 24 us in all, four 29)
    int split = 1;
    while (2 * split <= kMaxSplit && 8 * split <= steps && hb * 2 * split <= num_sms) split *= 2;
    p.w_stages = (kSmemMax - tail) / stage;
    if (p.w_stages > 8) p.w_stages = 8;
    p.w_smem = p.w_stages * stage;
    if (p.w_smem < p.E * 512) p.w_smem = (p.E * 512 + 127) & ~127;  // the tile that the cluster adds up
    int waited = p.grad_hidden != nullptr;
    void *args[] = {(void *)&p, (void *)&waited};
    return launch_ex((const void *)grad_router_w_kernel, dim3(split, hb), dim3(kProdThreads), (size_t)p.w_smem + tail, stream,
                     true, split, args);
  }
  return cudaSuccess;
}

}  // namespace moe
