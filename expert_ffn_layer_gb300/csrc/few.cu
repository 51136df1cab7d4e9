// The MoE FFN layer for few tokens (at most 32) in one kernel: router, top-k,
// the experts' gate/up, SiLU(gate) * up and down products, the shared expert and
// the weighted combine; and, with a routing given, the expert FFN alone.
//
//   logits[t, e] = x[t] . Wr[e]                      (fp32, [hy3] Model facts)
//   a[p, i]  = SiLU(x[t] . Wg[e, i]) * (x[t] . Wu[e, i])   p = (e, t), e in top-k of t
//   y[p, h]  = a[p] . Wd[e, h]
//   out[t]   = sum_j w[t, j] y[p(t, j)] + shared FFN(x[t])
//
// What bounds it: the active experts' weights, each read once.  A token or two per
// expert is no work for the tensor cores -- the products are matrix-vector -- so
// every choice serves the weight stream.  mma.sync (m16n8k16) is used rather than
// tcgen05 because its A operand comes straight from registers: weights go from
// memory to the lane that multiplies them, with no shared tile, no barrier and no
// conversion pass between (MXFP4 codes become fp16 in registers), and its rate is
// an order of magnitude above what the stream can feed at 8 tokens.
//
// Work.  One CTA of 16 warps per SM, all resident (cooperative launch).  A unit is
// 16 RG gate rows and the same up rows (gate/up), or 32 RG rows of w_down (down), of
// one expert; warp w takes row group w / KS and K slice w % KS (RG KS = 16), and the
// KS partial products are added in a fixed order through shared memory.  Units go
// to CTAs round robin; KS is chosen so that the last round is as short as it can be.
// Nothing is added by atomics: results do not depend on timing.
//
// Weights travel through a ring of NST steps per warp (64 bytes of each of 32 rows)
// by cp.async.  Each lane copies exactly the 16-byte pieces it will read itself, so
// the ring needs no barrier; it keeps filling across units, and before the wait
// between the two products it already holds the first steps of the second.
//
// Two grid-wide waits order the phases (logits -> selection, activations -> down).
// They are bounded like every wait here: a CTA that gives up sets
// MOE_DEVERR_TIMEOUT and the kernel winds down.
#include "internal.h"
#include "mxfp4.cuh"
#include "ptx.cuh"
#include "silu.cuh"
#include "topk.cuh"

namespace moe {

namespace {

constexpr int kFewWarps = 16, kFewThreads = kFewWarps * 32;
constexpr int kStepBytes = 64;               // bytes of one row in a step
constexpr int kStageW = 32 * kStepBytes;     // 32 rows: two 16-row operand tiles
constexpr int kMaxPos = kFewMaxT * 16 + kFewMaxT;  // routed positions and shared rows
constexpr int kMaxSegs = 256 + kFewMaxT * 16 / 8;

template <int WT>
struct Fmt {  // weights: 0 bf16, 1 MXFP4
  static constexpr int kStep = WT ? 128 : 32;   // K values of a step
  static constexpr int kGroups = kStep / 32;    // groups of 32 K values (two matrix instructions each)
  static constexpr int kStage = kStageW + (WT ? 128 : 0);  // with the 32 rows' four scale bytes
};

template <int NT>
struct FewLayout {
  static constexpr int kNst = 4;
  static constexpr int kRedBufs = NT <= 2 ? 2 : 1;  // double-buffered where it fits
  static constexpr int kRedFloats = kFewWarps * 2 * NT * 128;
};

// Tables every CTA builds for itself from the routing.
struct FewTables {
  // active segments in expert order (the shared expert is not in the list): an
  // expert's positions, in pieces of at most 8 NT -- a given routing may name an
  // expert more than once for a token
  int seg_e[kMaxSegs];
  int seg_row0[kMaxSegs + 1];  // first position of each
  int tok[kMaxPos];   // token of each routed position
  int pos[kFewMaxT * 16];      // position of slot t * k + j
  float w[kFewMaxT * 16];      // combine weight of each slot
  int idx[kFewMaxT * 16];
  unsigned mask[256];          // tokens of each expert
  int base[256];               // first position of each expert
  int nact, nsh;               // active routed segments; 1 with a shared expert
  int last, abort_flag;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// D += A B on a 16 x 8 tile, K = 16.
template <bool HALF>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  if constexpr (HALF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The power of two that brings a largest magnitude (its fp32 bits) into
// [2^14, 2^15), and its reciprocal: a row so scaled keeps every bf16 value's eight
// bits in fp16 down to 2^-28 of the row's maximum, and what is cut below that is
// under 2^-39 of it.
__device__ __forceinline__ float fp16_scale(uint32_t top) {
  const uint32_t ex = min(max(top >> 23, 15u), 254u);
  return __uint_as_float((268u - ex) << 23);
}
__device__ __forceinline__ float fp16_unscale(uint32_t top) {
  const uint32_t ex = min(max(top >> 23, 15u), 254u);
  return __uint_as_float((ex - 14u) << 23);
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ void grid_arrive(unsigned *counter) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(counter, 1u);
  }
}
// Waits until every CTA has arrived; false (in every thread) when the wait ran out.
__device__ __forceinline__ bool grid_wait(const FewParams &p, unsigned *counter, FewTables &tb) {
  if (threadIdx.x == 0) {
    const unsigned long long t0 = globaltimer();
    unsigned v;
    for (unsigned it = 1;; ++it) {
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(counter) : "memory");
      if (v >= gridDim.x) break;
      if ((it & 63u) == 0u && globaltimer() - t0 > kWaitLimitNs) {
        atomicOr(p.err, MOE_DEVERR_TIMEOUT);
        tb.abort_flag = 1;
        break;
      }
    }
  }
  __syncthreads();
  return tb.abort_flag == 0;
}

// Units of one phase and how the warps share one.
struct Plan {
  int ks, rg_shift;   // K slices, log2 of the row groups
  int unit_rows;      // rows (pairs of rows for gate/up) of a unit
  int rows_r, rows_s; // rows of a routed / the shared expert
  int rb_r, rb_s;     // units of each
  int steps_r, steps_s;
  int units;
};

// KS by the shortest makespan: rounds of units over the CTAs, each as long as its
// warps' steps (about 1400 cycles of the SM's share of the memory rate, 16 warps
// together) and the exchange of partial products (about 300).
template <bool DOWN>
__device__ Plan make_plan(const FewTables &tb, int rows_r, int rows_s, int steps_r, int steps_s) {
  Plan best = {};
  int best_cost = 0x7fffffff;
  for (int sh = 0; sh <= 4; ++sh) {  // RG = 2^sh
    Plan q;
    q.rg_shift = sh;
    q.ks = kFewWarps >> sh;
    q.unit_rows = (DOWN ? 32 : 16) << sh;
    q.rows_r = rows_r;
    q.rows_s = rows_s;
    q.steps_r = steps_r;
    q.steps_s = steps_s;
    q.rb_r = (rows_r + q.unit_rows - 1) / q.unit_rows;
    q.rb_s = tb.nsh ? (rows_s + q.unit_rows - 1) / q.unit_rows : 0;
    q.units = q.rb_s + tb.nact * q.rb_r;
    const int rounds = (q.units + gridDim.x - 1) / gridDim.x;
    const int cost = rounds * (((max(steps_r, tb.nsh ? steps_s : 0) + q.ks - 1) / q.ks) * 1400 + 300);
    if (cost < best_cost) {
      best_cost = cost;
      best = q;
    }
  }
  return best;
}

struct Unit {
  int seg;   // index in the active list, -1 the shared expert
  int e;     // expert (0 for the shared one)
  int rb, row0, ntok;
  int s0, n; // this warp's first step and its number of steps
};

__device__ __forceinline__ Unit decode_unit(const FewParams &p, const FewTables &tb, const Plan &q, int u, int warp,
                                            int warp_rows) {
  Unit t;
  int steps, rows;
  if (u < q.rb_s) {
    t.seg = -1;
    t.e = 0;
    t.rb = u;
    t.row0 = p.S;
    t.ntok = p.T;
    steps = q.steps_s;
    rows = q.rows_s;
  } else {
    const int v = u - q.rb_s;
    t.seg = v / q.rb_r;
    t.rb = v - t.seg * q.rb_r;
    t.e = tb.seg_e[t.seg];
    t.row0 = tb.seg_row0[t.seg];
    t.ntok = tb.seg_row0[t.seg + 1] - t.row0;
    steps = q.steps_r;
    rows = q.rows_r;
  }
  const int ks = warp & (q.ks - 1), rg = warp / q.ks;
  t.s0 = steps * ks / q.ks;
  t.n = steps * (ks + 1) / q.ks - t.s0;
  if (t.rb * q.unit_rows + rg * warp_rows >= rows) t.n = 0;  // past the expert's last rows
  return t;
}

// One phase over this CTA's units.  DOWN: the products with w_down, else gate/up.
template <int WT, int NT, bool DOWN>
__device__ void run_phase(const FewParams &p, FewTables &tb, uint8_t *ring, float *red, unsigned *wait_for, bool &ok) {
  constexpr int NST = FewLayout<NT>::kNst, G = Fmt<WT>::kGroups, STAGE = Fmt<WT>::kStage;
  constexpr int kRows = DOWN ? 32 : 16;  // rows a warp's unit advances by
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int K_r = DOWN ? p.I : p.H, K_s = DOWN ? p.Is : p.H;
  const Plan q = make_plan<DOWN>(tb, DOWN ? p.H : p.I, DOWN ? p.H : p.Is, K_r / Fmt<WT>::kStep, K_s / Fmt<WT>::kStep);
  const int rg = warp / q.ks;
  const uint32_t my_ring = smem_u32(ring) + warp * NST * STAGE;

  // ---- the weight stream: position (unit, step) of the next step to copy
  int fu = blockIdx.x, fs = 0, fn = 0, fslot = 0;
  const uint8_t *f0 = nullptr, *f1 = nullptr, *fsc = nullptr;
  size_t f8 = 0;  // bytes from a row to the one eight below
  auto f_unit = [&]() {  // settle on the next unit in which this warp has steps
    while (fu < q.units) {
      const Unit t = decode_unit(p, tb, q, fu, warp, kRows);
      if (t.n > 0) {
        const bool sh = t.seg < 0;
        const int K = sh ? K_s : K_r;
        const size_t rowb = WT ? (size_t)K / 2 : (size_t)K * 2;
        const size_t row = (size_t)t.e * (DOWN ? p.H : p.I) + t.rb * q.unit_rows + rg * kRows;
        const uint8_t *m0 = DOWN ? (sh ? p.s_down : p.down) : (sh ? p.s_gate : p.gate);
        const uint8_t *m1 = DOWN ? m0 + 16 * rowb : (sh ? p.s_up : p.up);
        f0 = m0 + (row + g) * rowb + t.s0 * kStepBytes + t4 * 16;
        f1 = m1 + (row + g) * rowb + t.s0 * kStepBytes + t4 * 16;
        f8 = 8 * rowb;
        if constexpr (WT) {
          const size_t sb = (size_t)K / 32;
          const uint8_t *c0 = DOWN ? (sh ? p.s_down_scale : p.down_scale) : (sh ? p.s_gate_scale : p.gate_scale);
          const uint8_t *c1 = DOWN ? c0 + 16 * sb : (sh ? p.s_up_scale : p.up_scale);
          fsc = (lane < 16 ? c0 : c1) + (row + (lane & 15)) * sb + t.s0 * 4;
        }
        fs = 0;
        fn = t.n;
        return;
      }
      fu += gridDim.x;
    }
  };
  f_unit();
  auto fill = [&]() {  // copy one step and commit it (an empty group past the end)
    if (fu < q.units) {
      const uint32_t d = my_ring + fslot * STAGE + g * kStepBytes + t4 * 16;
      cp_async16(d, f0);
      cp_async16(d + 8 * kStepBytes, f0 + f8);
      cp_async16(d + 16 * kStepBytes, f1);
      cp_async16(d + 24 * kStepBytes, f1 + f8);
      f0 += kStepBytes;
      f1 += kStepBytes;
      if constexpr (WT) {
        cp_async4(my_ring + fslot * STAGE + kStageW + lane * 4, fsc);
        fsc += 4;
      }
      if (++fs == fn) {
        fu += gridDim.x;
        f_unit();
      }
    }
    cp_async_commit();
    fslot = fslot + 1 == NST ? 0 : fslot + 1;
  };
  for (int i = 0; i < NST - 1; ++i) fill();

  if (wait_for != nullptr && !grid_wait(p, wait_for, tb)) {
    ok = false;
    cp_async_wait<0>();
    return;
  }

  // ---- the token operand of one step: this lane's 8 values of each group of 32, for column n
  constexpr int NB = DOWN ? 2 * G : G;
  auto load_b = [&](uint4 (&b)[NB], const Unit &t, int s, int n) {
    if (n >= t.ntok) {
#pragma unroll
      for (int i = 0; i < NB; ++i) b[i] = make_uint4(0u, 0u, 0u, 0u);
      return;
    }
    const int k0 = (t.s0 + s) * Fmt<WT>::kStep + t4 * 8;
    if constexpr (DOWN) {
      const float *row = t.seg < 0 ? p.act_s + (size_t)n * p.Is : p.act + (size_t)(t.row0 + n) * p.I;
      const uint4 *src = reinterpret_cast<const uint4 *>(row + k0);
#pragma unroll
      for (int i = 0; i < G; ++i) {
        b[2 * i] = src[8 * i];
        b[2 * i + 1] = src[8 * i + 1];
      }
    } else {
      const int tk = t.seg < 0 ? n : tb.tok[t.row0 + n];
      const uint4 *src = reinterpret_cast<const uint4 *>(p.x + (size_t)tk * p.H + k0);
#pragma unroll
      for (int i = 0; i < G; ++i) b[i] = src[4 * i];
    }
  };

  int slot = 0, buf = 0;
  for (int u = blockIdx.x; u < q.units; u += gridDim.x) {
    const Unit t = decode_unit(p, tb, q, u, warp, kRows);
    const int nts = (t.ntok + 7) >> 3;
    float acc[2][NT][4];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[a][n][i] = 0.0f;
    float bscale[NT];  // MXFP4 down: the activation row's power of two
    if constexpr (WT && DOWN) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
        bscale[n] = n * 8 + g < t.ntok ? fp16_scale(__ldcg(p.amax + t.row0 + n * 8 + g)) : 0.0f;
    }
    for (int s = 0; s < t.n; ++s) {
      cp_async_wait<NST - 2>();
      __syncwarp();
      fill();  // into the slot read in the previous step
      const uint32_t st = my_ring + slot * STAGE;
      slot = slot + 1 == NST ? 0 : slot + 1;
      const uint32_t wa = st + g * kStepBytes + t4 * 16;
      uint4 v[4];  // tile 0 rows g, g + 8; tile 1 rows g, g + 8
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = lds128(wa + i * 8 * kStepBytes);
      uint32_t sc[4];
      if constexpr (WT) {
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[i] = lds32(st + kStageW + (i * 8 + g) * 4);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (n < nts) {
          uint4 b[NB];
          load_b(b, t, s, n * 8 + g);
#pragma unroll
          for (int gr = 0; gr < G; ++gr) {
            uint32_t bh[4], bl[4];
            if constexpr (DOWN) {
              const uint4 x0 = b[2 * gr], x1 = b[2 * gr + 1];
              const uint32_t xu[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float fa = __uint_as_float(xu[2 * i]), fb = __uint_as_float(xu[2 * i + 1]);
                if constexpr (WT) {
                  bh[i] = pack_f16(fa * bscale[n], fb * bscale[n]);
                } else {
                  // the fp32 activation as the sum of two bf16 values (16 of its 24 bits)
                  bh[i] = pack_bf16(fa, fb);
                  bl[i] = pack_bf16(fa - __uint_as_float(bh[i] << 16), fb - __uint_as_float(bh[i] & 0xFFFF0000u));
                }
              }
            } else {
              bh[0] = b[gr].x, bh[1] = b[gr].y, bh[2] = b[gr].z, bh[3] = b[gr].w;
            }
#pragma unroll
            for (int a = 0; a < 2; ++a) {
              if constexpr (WT) {
                const uint4 &r0 = v[2 * a], &r8 = v[2 * a + 1];
                uint32_t h0[4], h8[4];
                e2m1x8_to_f16(gr == 0 ? r0.x : gr == 1 ? r0.y : gr == 2 ? r0.z : r0.w, h0);
                e2m1x8_to_f16(gr == 0 ? r8.x : gr == 1 ? r8.y : gr == 2 ? r8.z : r8.w, h8);
                float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                mma16<true>(part, h0[0], h8[0], h0[1], h8[1], bh[0], bh[1]);
                mma16<true>(part, h0[2], h8[2], h0[3], h8[3], bh[2], bh[3]);
                const float s0 = __uint_as_float((gr < 3 ? sc[2 * a] << (23 - 8 * gr) : sc[2 * a] >> 1) & 0x7F800000u);
                const float s8 =
                    __uint_as_float((gr < 3 ? sc[2 * a + 1] << (23 - 8 * gr) : sc[2 * a + 1] >> 1) & 0x7F800000u);
                acc[a][n][0] = fmaf(s0, part[0], acc[a][n][0]);
                acc[a][n][1] = fmaf(s0, part[1], acc[a][n][1]);
                acc[a][n][2] = fmaf(s8, part[2], acc[a][n][2]);
                acc[a][n][3] = fmaf(s8, part[3], acc[a][n][3]);
              } else {
                const uint4 &r0 = v[2 * a], &r8 = v[2 * a + 1];
                mma16<false>(acc[a][n], r0.x, r8.x, r0.y, r8.y, bh[0], bh[1]);
                mma16<false>(acc[a][n], r0.z, r8.z, r0.w, r8.w, bh[2], bh[3]);
                if constexpr (DOWN) {
                  mma16<false>(acc[a][n], r0.x, r8.x, r0.y, r8.y, bl[0], bl[1]);
                  mma16<false>(acc[a][n], r0.z, r8.z, r0.w, r8.w, bl[2], bl[3]);
                }
              }
            }
          }
        }
      }
    }

    // ---- the warps' partial products, then the sums in slice order
    float *rd = red + buf * FewLayout<NT>::kRedFloats;
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (n < nts)
          *reinterpret_cast<float4 *>(rd + ((warp * 2 + a) * NT + n) * 128 + lane * 4) =
              make_float4(acc[a][n][0], acc[a][n][1], acc[a][n][2], acc[a][n][3]);
    __syncthreads();
    const int rgs = 1 << q.rg_shift;
    const bool sh = t.seg < 0;
    if constexpr (!DOWN) {
      const int rows = sh ? q.rows_s : q.rows_r;
      for (int o = threadIdx.x; o < (rgs * nts) << 7; o += kFewThreads) {
        const int e = o & 127, nr = o >> 7, n = nr % nts, r = nr / nts;
        const int c = e & 3, ln = e >> 2;
        const int col = n * 8 + 2 * (ln & 3) + (c & 1), row = t.rb * q.unit_rows + r * 16 + (ln >> 2) + 8 * (c >> 1);
        float a = 0.0f;
        if (col < t.ntok && row < rows) {
          float gs = 0.0f, us = 0.0f;
          const float *src = rd + (r * q.ks * 2 * NT + n) * 128 + e;
          for (int k = 0; k < q.ks; ++k, src += 2 * NT * 128) {
            gs += src[0];
            us += src[NT * 128];
          }
          if constexpr (WT) {
            const float un = __ldcg(p.x_unscale + (sh ? col : tb.tok[t.row0 + col]));
            gs *= un;
            us *= un;
          }
          a = silu_mul(gs, us);
          (sh ? p.act_s + (size_t)col * p.Is : p.act + (size_t)(t.row0 + col) * p.I)[row] = a;
        }
        if constexpr (WT) {  // the largest magnitude of each activation row: its four lanes' rows first
          uint32_t m = __float_as_uint(a) & 0x7FFFFFFFu;
          m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
          m = max(m, __shfl_xor_sync(0xffffffffu, m, 16));
          if ((lane & 18) == 0 && col < t.ntok) atomicMax(p.amax + t.row0 + col, m);
        }
      }
    } else {
      for (int o = threadIdx.x; o < (2 * rgs * nts) << 7; o += kFewThreads) {
        const int e = o & 127, nr = o >> 7, n = nr % nts, ra = nr / nts, r = ra >> 1, a = ra & 1;
        const int c = e & 3, ln = e >> 2;
        const int col = n * 8 + 2 * (ln & 3) + (c & 1);
        const int row = t.rb * q.unit_rows + r * 32 + a * 16 + (ln >> 2) + 8 * (c >> 1);
        if (col < t.ntok && row < p.H) {
          float y = 0.0f;
          const float *src = rd + ((r * q.ks * 2 + a) * NT + n) * 128 + e;
          for (int k = 0; k < q.ks; ++k, src += 2 * NT * 128) y += *src;
          if constexpr (WT) y *= fp16_unscale(__ldcg(p.amax + t.row0 + col));
          if (p.y != nullptr) p.y[(size_t)(t.row0 + col) * p.H + row] = y;
          else if (sh) p.y_shared[(size_t)col * p.H + row] = __float2bfloat16_rn(y);
          else p.y_sorted[(size_t)(t.row0 + col) * p.H + row] = __float2bfloat16_rn(y);
        }
      }
      if (p.y != nullptr) {
        // the last segment to finish a block of rows combines it, in slot order
        __syncthreads();
        if (threadIdx.x == 0) {
          __threadfence();
          tb.last = atomicAdd(p.done + t.rb, 1u) == (unsigned)(tb.nact + tb.nsh - 1);
          __threadfence();
        }
        __syncthreads();
        if (tb.last) {
          const int w0 = t.rb * q.unit_rows, w1 = min(p.H, w0 + q.unit_rows), nw = (w1 - w0) >> 2;
          for (int o = threadIdx.x; o < p.T * nw; o += kFewThreads) {
            const int tk = o / nw, h = w0 + 4 * (o - tk * nw);
            float4 s4 = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int j = 0; j < p.top_k; ++j) {
              const float w = tb.w[tk * p.top_k + j];
              const float4 y = __ldcg(
                  reinterpret_cast<const float4 *>(p.y + (size_t)tb.pos[tk * p.top_k + j] * p.H + h));
              s4 = make_float4(fmaf(w, y.x, s4.x), fmaf(w, y.y, s4.y), fmaf(w, y.z, s4.z), fmaf(w, y.w, s4.w));
            }
            if (tb.nsh) {
              const float4 y = __ldcg(reinterpret_cast<const float4 *>(p.y + (size_t)(p.S + tk) * p.H + h));
              s4 = make_float4(s4.x + y.x, s4.y + y.y, s4.z + y.z, s4.w + y.w);
            }
            *reinterpret_cast<uint2 *>(p.out + (size_t)tk * p.H + h) =
                make_uint2(pack_bf16(s4.x, s4.y), pack_bf16(s4.z, s4.w));
          }
        }
      }
    }
    if (FewLayout<NT>::kRedBufs == 1) __syncthreads();
    else buf ^= 1;
  }
  cp_async_wait<0>();
}

// ---- router logits of this CTA's experts, two at a time: each thread the same
// pieces of H for both experts and eight tokens, a tree over the lanes, then the
// warps' sums in order.
__device__ void router_rows(const FewParams &p, float *red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h4 = p.H >> 2;
  for (int e0 = blockIdx.x; e0 < p.E; e0 += 2 * gridDim.x) {
    const int e1 = e0 + gridDim.x;
    const bool two = e1 < p.E;
    const float4 *w0 = reinterpret_cast<const float4 *>(p.router_w + (size_t)e0 * p.H);
    const float4 *w1 = reinterpret_cast<const float4 *>(p.router_w + (size_t)(two ? e1 : e0) * p.H);
    for (int t0 = 0; t0 < p.T; t0 += 8) {
      float acc[2][8];
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[0][i] = acc[1][i] = 0.0f;
      for (int i = threadIdx.x; i < h4; i += kFewThreads) {
        const float4 a = __ldg(w0 + i), b = __ldg(w1 + i);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (t0 + j < p.T) {
            const uint2 x = __ldg(reinterpret_cast<const uint2 *>(p.hidden + (size_t)(t0 + j) * p.H) + i);
            const float x0 = __uint_as_float(x.x << 16), x1 = __uint_as_float(x.x & 0xFFFF0000u);
            const float x2 = __uint_as_float(x.y << 16), x3 = __uint_as_float(x.y & 0xFFFF0000u);
            acc[0][j] = fmaf(a.w, x3, fmaf(a.z, x2, fmaf(a.y, x1, fmaf(a.x, x0, acc[0][j]))));
            acc[1][j] = fmaf(b.w, x3, fmaf(b.z, x2, fmaf(b.y, x1, fmaf(b.x, x0, acc[1][j]))));
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          acc[0][j] += __shfl_xor_sync(0xffffffffu, acc[0][j], o);
          acc[1][j] += __shfl_xor_sync(0xffffffffu, acc[1][j], o);
        }
        if (lane == 0) {
          red[(warp * 2 + 0) * 8 + j] = acc[0][j];
          red[(warp * 2 + 1) * 8 + j] = acc[1][j];
        }
      }
      __syncthreads();
      if (threadIdx.x < 16) {
        const int r = threadIdx.x >> 3, j = threadIdx.x & 7;
        if (t0 + j < p.T && (r == 0 || two)) {
          float s = 0.0f;
          for (int w = 0; w < kFewWarps; ++w) s += red[(w * 2 + r) * 8 + j];
          p.logits[(size_t)(t0 + j) * p.E + (r ? e1 : e0)] = s;
        }
      }
      __syncthreads();
    }
  }
}

// MXFP4: token t's hidden row as fp16, scaled by the power of two of its largest
// magnitude (exact for bf16 values within 2^-28 of it).
__device__ void convert_token(const FewParams &p, int t, unsigned *top_smem) {
  const uint4 *src = reinterpret_cast<const uint4 *>(p.hidden + (size_t)t * p.H);
  const int n8 = p.H >> 3;
  uint32_t m = 0;
  for (int i = threadIdx.x; i < n8; i += kFewThreads) {
    const uint4 v = __ldg(src + i);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max(m, max(u[j] & 0x7FFFu, (u[j] >> 16) & 0x7FFFu));
  }
  if (threadIdx.x == 0) *top_smem = 0u;
  __syncthreads();
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) atomicMax(top_smem, m);
  __syncthreads();
  const uint32_t top = *top_smem << 16;
  const float s = fp16_scale(top);
  if (threadIdx.x == 0) p.x_unscale[t] = fp16_unscale(top);
  uint4 *dst = reinterpret_cast<uint4 *>(p.x16 + (size_t)t * p.H);
  for (int i = threadIdx.x; i < n8; i += kFewThreads) {
    const uint4 v = __ldg(src + i);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = pack_f16(__uint_as_float(u[j] << 16) * s, __uint_as_float(u[j] & 0xFFFF0000u) * s);
    dst[i] = make_uint4(o[0], o[1], o[2], o[3]);
  }
  __syncthreads();
}

// Selection and tables from the logits.
__device__ void tables_from_logits(const FewParams &p, FewTables &tb, float *lg_smem) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = p.top_k;
  for (int e = threadIdx.x; e < 256; e += kFewThreads) tb.mask[e] = 0u;
  __syncthreads();
  const TopkRule rule = {p.bias, p.E, k, p.score_mode, p.route_scale, p.renorm_eps};
  float *lg = lg_smem + warp * 256;
  for (int t = warp; t < p.T; t += kFewWarps) {
    for (int e = lane; e < p.E; e += 32) lg[e] = __ldcg(p.logits + (size_t)t * p.E + e);
    __syncwarp();
    int e = 0;
    float w = 0.0f;
    warp_select_topk(rule, lg, lane, e, w);
    if (lane < k) {
      tb.idx[t * k + lane] = e;
      tb.w[t * k + lane] = w;
      atomicOr(&tb.mask[e], 1u << t);
    }
    __syncwarp();
  }
  __syncthreads();
  if (warp == 0) {
    int rows = 0, act = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane, cnt = e < p.E ? __popc(tb.mask[e]) : 0;
      int incl = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const unsigned live = __ballot_sync(0xffffffffu, cnt > 0);
      if (cnt > 0) {
        const int a = act + __popc(live & ((1u << lane) - 1u));
        tb.seg_e[a] = e;
        tb.seg_row0[a] = tb.base[e] = rows + incl - cnt;
      }
      rows += __shfl_sync(0xffffffffu, incl, 31);
      act += __popc(live);
    }
    if (lane == 0) {
      tb.seg_row0[act] = rows;
      tb.nact = act;
    }
  }
  __syncthreads();
  for (int s = threadIdx.x; s < p.S; s += kFewThreads) {
    const int t = s / k, e = tb.idx[s];
    const int pos = tb.base[e] + __popc(tb.mask[e] & ((1u << t) - 1u));
    tb.pos[s] = pos;
    tb.tok[pos] = t;
  }
  __syncthreads();
}

// Tables from a given permutation.  Offsets that are not a partition of the slots
// leave no routed work; slots out of range read token 0; both are recorded.
__device__ void tables_from_perm(const FewParams &p, FewTables &tb, int cap) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    bool good = __ldg(p.offsets) == 0 && __ldg(p.offsets + p.E) == p.S;
    for (int e = lane; e < p.E; e += 32) good = good && __ldg(p.offsets + e) <= __ldg(p.offsets + e + 1);
    good = __all_sync(0xffffffffu, good);
    int act = 0;
    if (good) {
      for (int e0 = 0; e0 < p.E; e0 += 32) {
        const int e = e0 + lane;
        const int lo = e < p.E ? __ldg(p.offsets + e) : 0, hi = e < p.E ? __ldg(p.offsets + e + 1) : 0;
        const int pieces = (hi - lo + cap - 1) / cap;
        int incl = pieces;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        for (int i = 0, a = act + incl - pieces; i < pieces; ++i, ++a) {
          tb.seg_e[a] = e;
          tb.seg_row0[a] = lo + i * cap;
        }
        act += __shfl_sync(0xffffffffu, incl, 31);
      }
    } else if (blockIdx.x == 0 && lane == 0) {
      atomicOr(p.err, MOE_DEVERR_OFFSETS);
    }
    if (lane == 0) {
      tb.seg_row0[act] = p.S;
      tb.nact = act;
    }
  }
  for (int i = threadIdx.x; i < p.S; i += kFewThreads) {
    const int slot = __ldg(p.perm + i);
    int t = slot / p.top_k;
    if (slot < 0 || t >= p.T) {
      t = 0;
      if (blockIdx.x == 0) atomicOr(p.err, MOE_DEVERR_INDEX);
    }
    tb.tok[i] = t;
  }
  __syncthreads();
}

template <int WT, int NT>
struct FewSmem {
  static constexpr int kRing = kFewWarps * FewLayout<NT>::kNst * Fmt<WT>::kStage;
  static constexpr int kRed = FewLayout<NT>::kRedBufs * FewLayout<NT>::kRedFloats * 4;
  static constexpr int kTables = (int)sizeof(FewTables);
  static constexpr int kBytes = kRing + kRed + kTables;
  static_assert(kBytes <= 232448, "shared memory budget");
  static_assert(kRed >= kFewWarps * 256 * 4, "the logits' staging shares the reduction buffer");
};

}  // namespace

template <int WT, int NT>
__global__ void __launch_bounds__(kFewThreads, 1) few_kernel(const __grid_constant__ FewParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  using L = FewSmem<WT, NT>;
  uint8_t *ring = smem;
  float *red = reinterpret_cast<float *>(smem + L::kRing);
  FewTables &tb = *reinterpret_cast<FewTables *>(smem + L::kRing + L::kRed);
  unsigned *bar0 = p.sync + kSyncFew, *bar1 = p.sync + kSyncFew + 1, *exits = p.sync + kSyncFew + 2;
  if (threadIdx.x == 0) {
    tb.abort_flag = 0;
    tb.nsh = p.has_shared ? 1 : 0;
  }
  // counters and maxima of this call
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < p.S + p.T; i += kFewThreads) p.amax[i] = 0u;
    for (int i = threadIdx.x; i < (p.H + 31) / 32; i += kFewThreads) p.done[i] = 0u;
  }
  if (WT)
    for (int t = gridDim.x - 1 - blockIdx.x; t < p.T; t += gridDim.x) convert_token(p, t, reinterpret_cast<unsigned *>(red));
  __syncthreads();
  if (p.router_w != nullptr) router_rows(p, red);
  grid_arrive(bar0);
  bool ok = grid_wait(p, bar0, tb);
  if (ok) {
    if (p.router_w != nullptr) tables_from_logits(p, tb, red);
    else tables_from_perm(p, tb, 8 * NT);
    run_phase<WT, NT, false>(p, tb, ring, red, nullptr, ok);
    __syncthreads();
  }
  grid_arrive(bar1);  // also after a wait that ran out: the others need not wait for theirs to do so
  if (ok) run_phase<WT, NT, true>(p, tb, ring, red, bar1, ok);
  __syncthreads();
  // the last CTA out zeroes the counters
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(exits, 1u) == gridDim.x - 1) {
      volatile unsigned *s = p.sync + kSyncFew;
      s[0] = s[1] = 0;
      __threadfence();
      s[2] = 0;
    }
  }
}

namespace {
template <int WT, int NT>
cudaError_t launch_few_one(const FewParams &p, int num_ctas, cudaStream_t stream) {
  using L = FewSmem<WT, NT>;
  static thread_local unsigned long long attr_ctx = 0;
  const cudaError_t e = set_smem_attr_once((const void *)few_kernel<WT, NT>, L::kBytes, attr_ctx);
  if (e != cudaSuccess) return e;
  void *args[] = {(void *)&p};
  return launch_coop((const void *)few_kernel<WT, NT>, dim3(num_ctas), dim3(kFewThreads), L::kBytes, stream, args);
}
template <int WT>
cudaError_t launch_few_wt(const FewParams &p, int num_ctas, cudaStream_t stream) {
  if (p.T <= 8) return launch_few_one<WT, 1>(p, num_ctas, stream);
  if (p.T <= 16) return launch_few_one<WT, 2>(p, num_ctas, stream);
  return launch_few_one<WT, 4>(p, num_ctas, stream);
}
}  // namespace

cudaError_t launch_few(const FewParams &p, bool mxfp4, int num_ctas, cudaStream_t stream) {
  return mxfp4 ? launch_few_wt<1>(p, num_ctas, stream) : launch_few_wt<0>(p, num_ctas, stream);
}

}  // namespace moe
