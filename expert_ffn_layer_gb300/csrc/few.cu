// The MoE FFN layer for few tokens in one kernel: router, top-k, the experts'
// gate/up, SiLU(gate) * up and down products, the shared expert and the weighted
// combine; and, with a routing given, the expert FFN alone.
//
//   logits[t, e] = x[t] . Wr[e]                            (fp32)
//   a[p, i]  = SiLU(x[t] . Wg[e, i]) * (x[t] . Wu[e, i])   p = (e, t), e in the top-k of t
//   y[p, h]  = a[p] . Wd[e, h]
//   out[t]   = sum_j w[t, j] y[p(t, j)] + shared FFN(x[t])
//
// "hy3 -- tencent/Hy3 GGUF Converter and Inference Engine", Model facts (router, MoE
// routing); HunyuanImage 3.0 post (easy_topk, Routed Experts, Shared MLP).  Weights
// are bf16, or MXFP4 (mxfp4.cuh).
//
// What bounds it: the active experts' weights, each read once.  A token or two per
// expert is no work for the tensor cores -- the products are matrix-vector -- so
// every choice serves the weight stream.  mma.sync (m16n8k16) is used rather than
// tcgen05 because its A operand comes from registers: MXFP4 codes become fp16 there,
// two by an instruction, with no pass through shared memory between.  Its pipe is
// under a quarter busy.  With MXFP4 no unit is: at T = 8 half the issue slots, 45 % of
// the ALU pipe, 55 % of the memory.  Four warps a scheduler wait out the latencies of
// steps (32 rows x 128 codes) of about 280 instructions, of which 64 expand codes and
// 64 to 100 apply the blocks' scales.
//
// Measured (GB300, Hy3 shape, time of a call and share of the measured copy bandwidth
// that the active weights come in at): bf16 T = 1 64 us (0.78), T = 8 336 us (56 active
// experts, 0.94), T = 32 818 us (0.95); MXFP4 layer T = 1 39 us (0.36), T = 8 124 us
// (0.68); MXFP4 expert FFN T = 8 114 us (0.71).  Percentages further down compare two
// versions of this file in turn on one box, also Hy3 shape.
//
// Work.  One CTA of 16 warps per SM, all resident (cooperative launch).  Units of 32
// rows go to teams of warps that split K (Plan below); the partial products are added
// in a fixed order through shared memory, and experts' outputs in slot order by a last
// phase.  Nothing is added by atomics: results do not depend on timing.
//
// Weights travel through a ring of steps per warp by cp.async.  No other warp reads a
// ring, so it needs no barrier; it keeps filling across units, and before the wait
// between the two products it already holds the first steps of the second.  (Bringing
// more of the second's weights into L2 during that wait: no gain at T = 8.)
//
// Three grid-wide waits order the phases (logits -> selection, activations -> down,
// outputs -> combine).  They are bounded like every wait here: a CTA that gives up sets
// MOE_DEVERR_TIMEOUT and the kernel winds down.
#include <climits>

#include "internal.h"
#include "mxfp4.cuh"
#include "ptx.cuh"
#include "silu.cuh"

namespace moe {

namespace {

constexpr int kFewWarps = 16, kFewThreads = kFewWarps * 32;
constexpr int kStageW = 2048;  // weight bytes of a ring slot
constexpr int kMaxSegs = 256 + kFewFfnMaxS / 8;
static_assert(kFewMaxT * 16 <= kFewFfnMaxS && kFewFfnMaxS + kFewFfnMaxT <= 4096, "positions in 12 bits");

template <int WT>
struct Fmt {  // weights: 0 bf16, 1 MXFP4
  // K values of a step, and its ring slots: both 16-row tiles' 64 bytes a row in one slot
  // (MXFP4), or a slot for each tile's 128 bytes a row (bf16: whole lines, as the memory
  // likes them: 4 % less time than half lines at T = 8, 2 % at T = 32)
  static constexpr int kStep = WT ? 128 : 64;
  static constexpr int kSlots = WT ? 1 : 2;
  static constexpr int kGroups = kStep / 32;    // groups of 32 K values (two matrix instructions each)
  static constexpr int kStage = kStageW + (WT ? 128 : 0);  // with the 32 rows' four scale bytes
  // Steps of a warp's ring.  MXFP4: three, which leaves 32 KB more of L1 to the token
  // operand (expert FFN T = 8 3 % faster than with four); bf16 is better off with the
  // fourth (T = 1 4 % faster).
  static constexpr int kNst = WT ? 3 : 4;
};

constexpr int kRedCol = 20;     // floats from one column of a partial 16 x 8 tile to the next (16 rows: no bank conflicts)
constexpr int kRedTile = 8 * kRedCol;
constexpr int kRedFloats = kFewWarps * 2 * kRedTile;  // one of two buffers

// Tables every CTA builds for itself from the routing.
struct FewTables {
  // segments: the active experts in order, each in pieces of at most 8 positions
  // (the columns of a product).  An expert of more re-reads its weights, by then in
  // L2.
  uint16_t seg_e[kMaxSegs];
  uint16_t seg_row0[kMaxSegs];  // first position of each
  uint16_t seg_n[kMaxSegs];     // positions of each
  uint16_t tok[kFewFfnMaxS];    // token of each routed position
  int pos[kFewMaxT * 16];      // position of slot t * k + j
  float w[kFewMaxT * 16];      // combine weight of each slot
  int idx[kFewMaxT * 16];
  unsigned mask[256];          // tokens of each expert
  float bias[256];             // of the keys
  int base[256];               // first position of each expert
  int scan[8];                 // build_segments' warp totals
  int nact, nsh;               // routed segments; the shared expert's pieces of 8 tokens
  int abort_flag;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy) : "memory");
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
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D = A B in fp16 operands, K = 16.
__device__ __forceinline__ void mma16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
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

// Scale byte i of a word as a power of two, 2^(byte - 127) (0 counts as zero, 255 is infinite).
__device__ __forceinline__ float scale_of(uint32_t w, int i) {
  return __uint_as_float((i < 3 ? w << (23 - 8 * i) : w >> 1) & 0x7F800000u);
}
__device__ __forceinline__ uint32_t word_of(const uint4 &v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
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

// How the warps share the units of one phase.  A unit is 32 rows of one segment
// (32 pairs of rows for gate/up); a team of warps takes one: KS slices of K, and for
// gate/up two warps a slice (16 gate and 16 up rows each).  The CTA's teams go their
// own ways, each with its own units and its own barrier.
//
// The units are dealt out in two parts: as many whole rounds over all teams as there
// are, with KS slices, and the rest, which would leave teams idle in a last round, with
// at least as many slices (larger teams, shorter units).
struct Plan {
  int rows_r, rows_s;    // rows of a routed / the shared expert, multiples of 32
  int steps_r, steps_s;
  int units, units_a;    // all, and those of the first part
  int ks_shift[2];       // log2 of the parts' K slices
};

// KS of both parts by the shortest makespan: a round lasts its warps' steps (C cycles
// each, the 16 warps of an SM together) and the exchange of partial products (C_unit).
// One lane tries one pair.
template <int WT, bool DOWN>
__device__ Plan make_plan(const FewTables &tb, int rows_r, int rows_s, int steps_r, int steps_s, int lane) {
  constexpr int kChoices = DOWN ? 5 : 4, kStepCycles = WT ? 2000 : 2800, kUnitCycles = WT ? 2000 : 600;
  Plan q;
  q.rows_r = rows_r;
  q.rows_s = rows_s;
  q.steps_r = steps_r;
  q.steps_s = steps_s;
  q.units = (tb.nsh * rows_s + tb.nact * rows_r) >> 5;
  const int a = lane / kChoices, b = lane % kChoices, steps = max(steps_r, tb.nsh ? steps_s : 0);
  unsigned cost = 0x7fffffffu;
  // bf16, bound by the memory: at least as many slices as leave a warp three steps, up to
  // eight -- fewer and longer ones spread the reads (T = 8: four down slices 1.5 % slower
  // than eight; two 9 % slower, when steps were half as wide).
  // MXFP4, whose steps take longer than their bytes, gains from few.
  const bool near = WT || a >= 3 || steps >> (a + 1) < 3;
  if (a < kChoices && b >= a && near) {
    auto round = [&](int sh) { return ((steps + (1 << sh) - 1) >> sh) * kStepCycles + kUnitCycles; };
    auto teams = [&](int sh) { return (int)gridDim.x * (kFewWarps >> (DOWN ? sh : sh + 1)); };
    const int ra = q.units / teams(a), rest = q.units - ra * teams(a);
    cost = (unsigned)(ra * round(a) + (rest + teams(b) - 1) / teams(b) * round(b));
  }
  const unsigned best = __reduce_min_sync(0xffffffffu, cost);
  const int win = __ffs(__ballot_sync(0xffffffffu, cost == best)) - 1;
  q.ks_shift[0] = win / kChoices;
  q.ks_shift[1] = win % kChoices;
  const int ta = gridDim.x * (kFewWarps >> (DOWN ? q.ks_shift[0] : q.ks_shift[0] + 1));
  q.units_a = q.units / ta * ta;
  return q;
}

// A warp's place in one part: its team, K slice and units.
struct Part {
  int ks_shift, tw_shift;  // log2 of K slices and of a team's warps
  int team, teams, mine;   // the team's number, how many there are, units of this one
  int off;                 // the warp's first row in a unit
  int s0[2], n[2];         // its first step and number of steps: routed, shared
};
template <bool DOWN>
__device__ __forceinline__ Part make_part(const Plan &q, int i, int warp) {
  Part r;
  r.ks_shift = i ? q.ks_shift[1] : q.ks_shift[0];
  r.tw_shift = DOWN ? r.ks_shift : r.ks_shift + 1;
  const int ks = warp & ((1 << r.ks_shift) - 1), units = i ? q.units - q.units_a : q.units_a;
  r.off = DOWN ? 0 : (warp >> r.ks_shift & 1) * 16;
  r.teams = gridDim.x * (kFewWarps >> r.tw_shift);
  // neighbouring units to neighbouring CTAs (to the teams of one CTA: 10 % slower)
  r.team = (warp >> r.tw_shift) * gridDim.x + blockIdx.x;
  r.mine = units > r.team ? (units - 1 - r.team) / r.teams + 1 : 0;
  r.s0[0] = q.steps_r * ks >> r.ks_shift;
  r.s0[1] = q.steps_s * ks >> r.ks_shift;
  r.n[0] = (q.steps_r * (ks + 1) >> r.ks_shift) - r.s0[0];
  r.n[1] = (q.steps_s * (ks + 1) >> r.ks_shift) - r.s0[1];
  return r;
}

// One of a team's units, for one of its warps.
struct Unit {
  int w_row;           // this warp's first row of the stacked weight matrix
  int sh, row0, ntok;  // of the shared expert; first position; number of positions (0: past the last unit)
  int row;             // the unit's first row in its expert
  int s0, n;           // this warp's first step and its number of steps
};

// A warp's units in order, decoded 32 at a time, one by each lane, and read by
// shuffles -- which also tells the compiler that they are the warp's, not the lane's.
// Packed: positions (4 bits), first position (12), first row / 32 (10), shared (1),
// and the steps: first (10), number (11).
struct UnitList {
  int base, w_row, word, steps;

  template <bool DOWN>
  __device__ __forceinline__ void decode(const FewTables &tb, const Plan &q, int S, int T, int warp, int first, int lane) {
    base = first;
    const Part a = make_part<DOWN>(q, 0, warp), b = make_part<DOWN>(q, 1, warp);
    const int i = first + lane, rb_s = q.rows_s >> 5, rb_r = q.rows_r >> 5, n_sh = tb.nsh * rb_s;
    const bool in_a = i < a.mine;
    const int u = in_a ? a.team + i * a.teams : i - a.mine < b.mine ? q.units_a + b.team + (i - a.mine) * b.teams : q.units;
    const int off = in_a ? a.off : b.off;
    word = w_row = steps = 0;
    if (u < q.units) {
      const bool sh = u < n_sh;
      if (sh) {
        const int seg = u / rb_s, rb = u - seg * rb_s;
        w_row = rb * 32 + off;
        word = min(8, T - 8 * seg) | (S + 8 * seg) << 4 | rb << 16 | 1 << 26;
      } else {
        const int v = u - n_sh, seg = v / rb_r, rb = v - seg * rb_r;
        w_row = tb.seg_e[seg] * q.rows_r + rb * 32 + off;
        word = tb.seg_n[seg] | tb.seg_row0[seg] << 4 | rb << 16;
      }
      const int s0 = sh ? (in_a ? a.s0[1] : b.s0[1]) : in_a ? a.s0[0] : b.s0[0];
      steps = s0 | (sh ? (in_a ? a.n[1] : b.n[1]) : in_a ? a.n[0] : b.n[0]) << 10;
    }
  }
  // unit i, 0 <= i - base < 32
  __device__ __forceinline__ Unit get(int i) const {
    Unit t;
    const int x = __shfl_sync(0xffffffffu, word, i - base), st = __shfl_sync(0xffffffffu, steps, i - base);
    t.w_row = __shfl_sync(0xffffffffu, w_row, i - base);
    t.ntok = x & 15;
    t.row0 = x >> 4 & 4095;
    t.row = (x >> 16 & 1023) << 5;
    t.sh = x >> 26;
    t.s0 = st & 1023;
    t.n = st >> 10;
    return t;
  }
};

// One phase over this CTA's units.  DOWN: the products with w_down, else gate/up.
template <int WT, bool DOWN>
__device__ void run_phase(const FewParams &p, FewTables &tb, uint8_t *ring, float *red, unsigned *wait_for, bool &ok) {
  constexpr int G = Fmt<WT>::kGroups, STAGE = Fmt<WT>::kStage, kNst = Fmt<WT>::kNst, kSlots = Fmt<WT>::kSlots;
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int K_r = DOWN ? p.I : p.H, K_s = DOWN ? p.Is : p.H;
  const Plan q = make_plan<WT, DOWN>(tb, DOWN ? p.H : p.I, DOWN ? p.H : p.Is, K_r / Fmt<WT>::kStep,
                                     K_s / Fmt<WT>::kStep, lane);
  const int mine_a = make_part<DOWN>(q, 0, warp).mine, mine = mine_a + make_part<DOWN>(q, 1, warp).mine;
  UnitList list{};  // of the products
  list.decode<DOWN>(tb, q, p.S, p.T, warp, 0, lane);
  UnitList flist = list;  // of the weight stream ahead of them
  const uint32_t my_ring = smem_u32(ring) + warp * kNst * STAGE;
  // With at most 8 tokens every weight is read once: evict-first, so that the stream
  // leaves the rest in L2 -- the code above all, whose lines every launch would fetch
  // from memory again (T = 1: 4 us less with either weights).
  const uint64_t pol = p.T <= 8 ? policy_evict_first() : policy_evict_normal();

  // ---- the weight stream: the unit and step to copy next
  int fi = 0, fs = 0, fn = 0, fslot = 0;
  const uint8_t *f0 = nullptr, *f1 = nullptr, *fsc = nullptr;
  uint32_t f_rows = 0;  // bytes from a lane's row to its next
  auto fill = [&]() {  // copy one step and commit it (an empty group past the end)
    if (fs == fn) {    // on to the next unit in which this warp has steps
      fs = fn = 0;
      while (fi < mine && fn == 0) {
        if (fi - flist.base == 32) flist.decode<DOWN>(tb, q, p.S, p.T, warp, fi, lane);
        const Unit f = flist.get(fi++);
        fn = f.n;
        if (fn > 0) {
          const int K = f.sh ? K_s : K_r;
          const uint32_t rowb = WT ? K / 2 : K * 2;
          const uint8_t *m0 = DOWN ? (f.sh ? p.s_down : p.down) : (f.sh ? p.s_gate : p.gate);
          const uint8_t *m1 = DOWN ? m0 + 16 * rowb : (f.sh ? p.s_up : p.up);
          // MXFP4: lane (g, t) copies the 16 bytes of rows g, g + 8 of both tiles that it will
          // itself read; bf16: eight lanes copy a line, four rows at a time
          const size_t at = WT ? (size_t)(f.w_row + g) * rowb + f.s0 * 64 + t4 * 16
                               : (size_t)(f.w_row + (lane >> 3)) * rowb + f.s0 * 128 + (lane & 7) * 16;
          f0 = m0 + at;
          f1 = m1 + at;
          f_rows = (WT ? 8 : 4) * rowb;
          fn *= kSlots;
          if constexpr (WT) {
            const uint32_t sb = K / 32;
            const uint8_t *c0 = DOWN ? (f.sh ? p.s_down_scale : p.down_scale) : (f.sh ? p.s_gate_scale : p.gate_scale);
            const uint8_t *c1 = DOWN ? c0 + 16 * sb : (f.sh ? p.s_up_scale : p.up_scale);
            fsc = (lane < 16 ? c0 : c1) + (size_t)(f.w_row + (lane & 15)) * sb + f.s0 * 4;
          }
        }
      }
    }
    if (fs < fn) {
      const uint32_t d = my_ring + fslot * STAGE;
      if constexpr (WT) {
        const uint32_t dw = d + g * 64 + t4 * 16;
        cp_async16(dw, f0, pol);
        cp_async16(dw + 512, f0 + f_rows, pol);
        cp_async16(dw + 1024, f1, pol);
        cp_async16(dw + 1536, f1 + f_rows, pol);
        f0 += 64;
        f1 += 64;
        cp_async4(d + kStageW + lane * 4, fsc);
        fsc += 4;
      } else {
        // odd rows' halves change places, so that the reads below meet all banks
        const uint32_t dw = d + (lane >> 3) * 128 + ((lane & 7) ^ (lane >> 1 & 4)) * 16;
        const uint8_t *src = fs & 1 ? f1 : f0;
#pragma unroll
        for (int i = 0; i < 4; ++i) cp_async16(dw + i * 512, src + i * f_rows, pol);
        if (fs & 1) {
          f0 += 128;
          f1 += 128;
        }
      }
      ++fs;
    }
    cp_async_commit();
    fslot = fslot + 1 == kNst ? 0 : fslot + 1;
  };
#pragma unroll 1
  for (int i = 0; i < kNst - 1; ++i) fill();

  if (wait_for != nullptr && !grid_wait(p, wait_for, tb)) {
    ok = false;
    cp_async_wait<0>();
    return;
  }

  // ---- the token operand: this lane's 8 values of each group of 32, for column g
  // (columns past the segment's repeat its last: their sums are not read), a step
  // ahead of their use.  MXFP4: each register is loaded anew as soon as the step has
  // used it; bf16, whose steps are shorter: a second set of registers.
  constexpr int kB = (DOWN && !WT) ? 2 * G : G;
  uint4 bv[kB];
  uint32_t ex[2] = {0u, 0u};            // MXFP4 down: the groups' exponents for columns 2 t, 2 t + 1
  const uint4 *bp = nullptr;            // the next values to load
  const uint32_t *xp[2] = {nullptr, nullptr};
  auto point = [&](const Unit &u) {  // bp and xp at a unit's first step
    const int col = min(g, u.ntok - 1);
    const int k0 = u.s0 * Fmt<WT>::kStep + t4 * 8;
    if constexpr (DOWN) {
      // first value of position row0, and values from a position to the next
      const size_t at = u.sh ? (size_t)p.S * p.I + (size_t)(u.row0 - p.S) * p.Is : (size_t)u.row0 * p.I;
      const int ld = u.sh ? p.Is : p.I;
      if constexpr (WT) {
        bp = reinterpret_cast<const uint4 *>(p.act16 + at + (size_t)col * ld + k0);
#pragma unroll
        for (int c = 0; c < 2; ++c)
          xp[c] = reinterpret_cast<const uint32_t *>(p.act_exp + (at + (size_t)min(2 * t4 + c, u.ntok - 1) * ld) / 32) + u.s0;
      } else {
        bp = reinterpret_cast<const uint4 *>(p.act + at + (size_t)col * ld + k0);
      }
    } else {
      const int tk = u.sh ? u.row0 - p.S + col : tb.tok[u.row0 + col];
      bp = reinterpret_cast<const uint4 *>(p.x + (size_t)tk * p.H + k0);
    }
  };
  auto load_b = [&](int i) {
    if constexpr (DOWN && !WT) {
      bv[2 * i] = bp[8 * i];
      bv[2 * i + 1] = bp[8 * i + 1];
    } else {
      bv[i] = bp[4 * i];
    }
  };
  constexpr int kBStep = (DOWN && !WT) ? 8 * G : 4 * G;  // 16-byte pieces from a step to the next
  auto first_b = [&](const Unit &u) {
    point(u);
#pragma unroll
    for (int i = 0; i < G; ++i) load_b(i);
    if constexpr (DOWN && WT) ex[0] = *xp[0], ex[1] = *xp[1];
  };

  int slot = 0, buf = 0;
  auto next_slot = [&]() {  // the next slot of the ring, once its copies are there
    cp_async_wait<kNst - 2>();
    __syncwarp();
    fill();  // into the slot read before it
    const uint32_t st = my_ring + slot * STAGE;
    slot = slot + 1 == kNst ? 0 : slot + 1;
    return st;
  };
  Unit nxt = list.get(0);
  if (nxt.n > 0) first_b(nxt);
#pragma unroll 1
  for (int ui = 0; ui < mine; ++ui) {
    const Unit t = nxt;
    if (ui + 1 - list.base == 32) list.decode<DOWN>(tb, q, p.S, p.T, warp, ui + 1, lane);
    nxt = list.get(ui + 1);
    float acc[2][4];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[a][i] = 0.0f;
    if (t.n == 0 && nxt.n > 0) first_b(nxt);
#pragma unroll 1
    for (int s = 0; s < t.n; ++s) {
      // where the registers' next values come from (after the last step: anywhere valid)
      if (s + 1 < t.n) {
        bp += kBStep;
        if constexpr (DOWN && WT) ++xp[0], ++xp[1];
      } else if (nxt.n > 0) {
        point(nxt);
      }
      if constexpr (WT) {
        const uint32_t st = next_slot();
        uint4 v[4];  // tile 0 rows g, g + 8; tile 1 rows g, g + 8
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = lds128(st + g * 64 + t4 * 16 + i * 512);
        uint32_t sc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[i] = lds32(st + kStageW + (i * 8 + g) * 4);
        const uint32_t e0 = ex[0], e1 = ex[1];
        if constexpr (DOWN) ex[0] = *xp[0], ex[1] = *xp[1];
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
          float part[2][4];
#pragma unroll
          for (int a = 0; a < 2; ++a) {
            uint32_t h0[4], h8[4];
            e2m1x8_to_f16(word_of(v[2 * a], gr), h0);
            e2m1x8_to_f16(word_of(v[2 * a + 1], gr), h8);
            mma16_first(part[a], h0[0], h8[0], h0[1], h8[1], bv[gr].x, bv[gr].y);
            mma16<true>(part[a], h0[2], h8[2], h0[3], h8[3], bv[gr].z, bv[gr].w);
          }
          load_b(gr);
#pragma unroll
          for (int a = 0; a < 2; ++a) {
            const float s0 = scale_of(sc[2 * a], gr), s8 = scale_of(sc[2 * a + 1], gr);
            if constexpr (DOWN) {
              const float x0 = scale_of(e0, gr), x1 = scale_of(e1, gr);
              acc[a][0] = fmaf(s0 * x0, part[a][0], acc[a][0]);
              acc[a][1] = fmaf(s0 * x1, part[a][1], acc[a][1]);
              acc[a][2] = fmaf(s8 * x0, part[a][2], acc[a][2]);
              acc[a][3] = fmaf(s8 * x1, part[a][3], acc[a][3]);
            } else {
              acc[a][0] = fmaf(s0, part[a][0], acc[a][0]);
              acc[a][1] = fmaf(s0, part[a][1], acc[a][1]);
              acc[a][2] = fmaf(s8, part[a][2], acc[a][2]);
              acc[a][3] = fmaf(s8, part[a][3], acc[a][3]);
            }
          }
        }
      } else {
        uint32_t bh[2][4], bl[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if constexpr (DOWN) {  // the fp32 activation as the sum of two bf16 values (16 of its 24 bits)
            const uint4 x0 = bv[kB > 2 ? 2 * h : 0], x1 = bv[kB > 2 ? 2 * h + 1 : 0];
            const uint32_t xu[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float fa = __uint_as_float(xu[2 * i]), fb = __uint_as_float(xu[2 * i + 1]);
              bh[h][i] = pack_bf16(fa, fb);
              bl[h][i] = pack_bf16(fa - __uint_as_float(bh[h][i] << 16), fb - __uint_as_float(bh[h][i] & 0xFFFF0000u));
            }
          } else {
            bh[h][0] = bv[h].x, bh[h][1] = bv[h].y, bh[h][2] = bv[h].z, bh[h][3] = bv[h].w;
          }
          load_b(h);
        }
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          const uint32_t st = next_slot() + g * 128;
          uint4 v[2][2];  // both halves of 32 values, rows g, g + 8
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t at = st + (((t4 | h << 2) ^ (g << 2 & 4)) << 4);
            v[h][0] = lds128(at);
            v[h][1] = lds128(at + 1024);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 &r0 = v[h][0], &r8 = v[h][1];
            mma16<false>(acc[a], r0.x, r8.x, r0.y, r8.y, bh[h][0], bh[h][1]);
            mma16<false>(acc[a], r0.z, r8.z, r0.w, r8.w, bh[h][2], bh[h][3]);
            if constexpr (DOWN) {
              mma16<false>(acc[a], r0.x, r8.x, r0.y, r8.y, bl[h][0], bl[h][1]);
              mma16<false>(acc[a], r0.z, r8.z, r0.w, r8.w, bl[h][2], bl[h][3]);
            }
          }
        }
      }
    }

    // ---- the team's partial products, then the sums in slice order: a warp takes the
    // unit's 32 rows of one column, a lane each.  Two buffers: the next unit's products
    // are written while these are added, and the barrier before their sums orders both.
    // (A team of the second part is made of whole teams of the first, so its first
    // barrier also orders what those still read; it has other barriers, as the first
    // part's may still be in use.)
    const int ksh = ui >= mine_a ? q.ks_shift[1] : q.ks_shift[0], tsh = DOWN ? ksh : ksh + 1;
    const int tsh_a = DOWN ? q.ks_shift[0] : q.ks_shift[0] + 1;
    const int tw = 1 << tsh, wi = warp & (tw - 1), n_ks = 1 << ksh;
    float *rd = red + buf * kRedFloats + (warp - wi) * 2 * kRedTile;
    buf ^= 1;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      float *d = rd + (wi * 2 + a) * kRedTile + 2 * t4 * kRedCol + g;
      d[0] = acc[a][0];
      d[kRedCol] = acc[a][1];
      d[8] = acc[a][2];
      d[kRedCol + 8] = acc[a][3];
    }
    if (tw == 1) __syncwarp();
    else named_bar_sync(1 + (warp >> tsh) + (tsh_a > 0 && tsh > tsh_a ? 8 : 0), 32 * tw);
    const int row = t.row + lane;
    for (int col = wi; col < t.ntok; col += tw) {
      if constexpr (!DOWN) {
        // row group lane / 16 is its KS warps' gate and up tiles
        const float *src = rd + ((lane >> 4) << ksh) * 2 * kRedTile + col * kRedCol + (lane & 15);
        float gs = 0.0f, us = 0.0f;
        for (int k = 0; k < n_ks; ++k, src += 2 * kRedTile) {
          gs += src[0];
          us += src[kRedTile];
        }
        const size_t at =
            (t.sh ? (size_t)p.S * p.I + (size_t)(t.row0 - p.S + col) * p.Is : (size_t)(t.row0 + col) * p.I) + row;
        if constexpr (WT) {
          const float un = __ldcg(p.x_unscale + (t.sh ? t.row0 - p.S + col : tb.tok[t.row0 + col]));
          const float a = silu_mul(gs * un, us * un);
          const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(a) & 0x7FFFFFFFu);
          p.act16[at] = __half_as_ushort(__float2half_rn(a * fp16_scale(top)));
          if (lane == 0) p.act_exp[at / 32] = (uint8_t)(__float_as_uint(fp16_unscale(top)) >> 23);
        } else {
          p.act[at] = silu_mul(gs, us);
        }
      } else {
        const float *src = rd + (lane >> 4) * kRedTile + col * kRedCol + (lane & 15);
        float y = 0.0f;
        for (int k = 0; k < n_ks; ++k, src += 2 * kRedTile) y += *src;
        if (p.y != nullptr) p.y[(size_t)(t.row0 + col) * p.H + row] = y;
        else if (t.sh) p.y_shared[(size_t)(t.row0 - p.S + col) * p.H + row] = __float2bfloat16_rn(y);
        else p.y_sorted[(size_t)(t.row0 + col) * p.H + row] = __float2bfloat16_rn(y);
      }
    }
  }
  cp_async_wait<0>();
}

// out[t] = sum_j w[t, j] y[pos(t, j)] + y_shared[t], in slot order, rounded once.
// A warp takes 128 values of a token; warps are dealt out over the CTAs.
__device__ void combine_rows(const FewParams &p, const FewTables &tb) {
  const int lane = threadIdx.x & 31, h4 = p.H >> 2;
  for (int o = (blockIdx.x + (int)gridDim.x * (threadIdx.x >> 5)) * 32 + lane; o < p.T * h4; o += gridDim.x * kFewThreads) {
    const int tk = o / h4, h = 4 * (o - tk * h4);
    float4 s4 = make_float4(0.0f, 0.0f, 0.0f, 0.0f), z = s4;
    if (tb.nsh) z = __ldcg(reinterpret_cast<const float4 *>(p.y + (size_t)(p.S + tk) * p.H + h));
    for (int j0 = 0; j0 < p.top_k; j0 += 8) {  // eight rows in flight
      float4 y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j0 + j < p.top_k)
          y[j] = __ldcg(reinterpret_cast<const float4 *>(p.y + (size_t)tb.pos[tk * p.top_k + j0 + j] * p.H + h));
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j0 + j < p.top_k) {
          const float w = tb.w[tk * p.top_k + j0 + j];
          s4 = make_float4(fmaf(w, y[j].x, s4.x), fmaf(w, y[j].y, s4.y), fmaf(w, y[j].z, s4.z), fmaf(w, y[j].w, s4.w));
        }
    }
    if (tb.nsh) s4 = make_float4(s4.x + z.x, s4.y + z.y, s4.z + z.z, s4.w + z.w);
    *reinterpret_cast<uint2 *>(p.out + (size_t)tk * p.H + h) = make_uint2(pack_bf16(s4.x, s4.y), pack_bf16(s4.z, s4.w));
  }
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

// Segments and first positions from the experts' counts, one thread per expert
// (threads 0..255; cnt is 0 past E).  Positions are counted on in expert order.
__device__ __forceinline__ void build_segments(FewTables &tb, int cnt) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // positions in the low half, pieces of 8 in the high half of one scanned word
  const int mine = cnt | (((cnt + 7) >> 3) << 16);
  int incl = mine;
  if (threadIdx.x < 256) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) tb.scan[warp] = incl;
  }
  __syncthreads();
  if (threadIdx.x < 256) {
    int before = incl - mine;
#pragma unroll
    for (int w = 0; w < 8; ++w) before += w < warp ? tb.scan[w] : 0;
    const int row0 = before & 0xFFFF, a = before >> 16;
    tb.base[threadIdx.x] = row0;
    for (int i = 0; 8 * i < cnt; ++i) {
      tb.seg_e[a + i] = threadIdx.x;
      tb.seg_row0[a + i] = row0 + 8 * i;
      tb.seg_n[a + i] = min(8, cnt - 8 * i);
    }
    if (threadIdx.x == 255) tb.nact = (before + mine) >> 16;
  }
}

// An fp32 value as an integer of the same order.
__device__ __forceinline__ int ordered(float f) {
  const int b = __float_as_int(f);
  return b ^ ((b >> 31) & 0x7FFFFFFF);
}

// Selection of token t by a warp, with the rule and results of the router's top-k
// kernel: each round the largest key by one integer reduction over the lanes, the
// lower of equal experts by another.  Every CTA runs it once a call, so what it costs
// is fetching its code: rolled loops over scores and keys in shared memory (2 KB a
// warp) rather than unrolled ones in registers (T = 1 with a cold L2: 7 to 8 us less).
__device__ __forceinline__ void select_token(const FewParams &p, FewTables &tb, int t, float *sc, int lane) {
  const int E = p.E, k = p.top_k;
  int *key = reinterpret_cast<int *>(sc + 256);
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = lane + 32 * j < E ? __ldcg(p.logits + (size_t)t * E + lane + 32 * j) : -INFINITY;
#pragma unroll
  for (int j = 0; j < 8; ++j) sc[lane + 32 * j] = v[j];  // a lane reads only what it wrote
  const bool sigmoid = p.score_mode == MOE_SCORE_SIGMOID_BIAS;
  float mx = 0.0f, sum = 1.0f;
  if (!sigmoid) {
    mx = -INFINITY;
#pragma unroll 1
    for (int e = lane; e < E; e += 32) mx = fmaxf(mx, sc[e]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    sum = 0.0f;
#pragma unroll 1
    for (int e = lane; e < E; e += 32) sum += expf(sc[e] - mx);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
#pragma unroll 1
  for (int e = lane; e < E; e += 32) {
    const float x = expf(sigmoid ? -sc[e] : sc[e] - mx);
    const float s = (sigmoid ? 1.0f : x) / (sigmoid ? 1.0f + x : sum);
    const float kk = s + tb.bias[e] + 0.0f;  // -0 as 0
    sc[e] = s;
    key[e] = kk == kk ? ordered(kk) : ordered(-INFINITY);
  }
  int my_e = 0;
#pragma unroll 1
  for (int r = 0; r < k; ++r) {
    int bk = INT_MIN, be = 0x7fffffff;
    int x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = lane + 32 * j < E ? key[lane + 32 * j] : INT_MIN;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (x[j] > bk) {
        bk = x[j];
        be = lane + 32 * j;
      }
    const int top = __reduce_max_sync(0xffffffffu, bk);
    const int e = __reduce_min_sync(0xffffffffu, bk == top ? be : 0x7fffffff);
    if (lane == r) my_e = e;
    if (be == e) key[e] = INT_MIN;  // taken
  }
  __syncwarp();
  const float s = lane < k ? sc[my_e] : 0.0f;
  float tot = s;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
  if (lane < k) {
    tb.idx[t * k + lane] = my_e;
    tb.w[t * k + lane] = sigmoid ? s / tot * p.route_scale : s / fmaxf(tot, p.renorm_eps);
    atomicOr(&tb.mask[my_e], 1u << t);
  }
}

// Selection and tables from the logits (tb.mask is zero).
__device__ void tables_from_logits(const FewParams &p, FewTables &tb, float *scratch) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = p.top_k;
#pragma unroll 1
  for (int t = warp; t < p.T; t += kFewWarps) select_token(p, tb, t, scratch + warp * 512, lane);
  __syncthreads();
  build_segments(tb, threadIdx.x < 256 ? __popc(tb.mask[threadIdx.x]) : 0);
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
__device__ void tables_from_perm(const FewParams &p, FewTables &tb) {
  const int e = threadIdx.x;
  const int lo = e <= p.E ? __ldg(p.offsets + e) : p.S, hi = e < p.E ? __ldg(p.offsets + e + 1) : lo;
  const bool good = __syncthreads_and(hi >= lo && (e != 0 || lo == 0) && (e != p.E || lo == p.S));
  if (!good && e == 0 && blockIdx.x == 0) atomicOr(p.err, MOE_DEVERR_OFFSETS);
  build_segments(tb, good && e < 256 ? hi - lo : 0);
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

// The shared expert's weights into L2 while the routing is found: none of them
// depends on it, and the memory is idle then.
template <int WT>
__device__ void prefetch_shared(const FewParams &p) {
  constexpr unsigned kPiece = 8192;
  const size_t n = (size_t)p.Is * p.H * (WT ? 1 : 4) / 2;  // bytes of one matrix, a multiple of 16
  const uint8_t *m[3] = {p.s_gate, p.s_up, p.s_down};
#pragma unroll
  for (int i = 0; i < 3; ++i)
    for (size_t at = ((size_t)blockIdx.x * 32 + (threadIdx.x & 31)) * kPiece; at < n; at += (size_t)gridDim.x * 32 * kPiece)
      prefetch_l2_bulk(m[i] + at, (uint32_t)min((size_t)kPiece, n - at));
}

template <int WT>
struct FewSmem {
  static constexpr int kRing = kFewWarps * Fmt<WT>::kNst * Fmt<WT>::kStage;
  static constexpr int kRed = 2 * kRedFloats * 4;
  static_assert(kRed >= kFewWarps * 2048, "the selection's scores and keys share the reduction buffer");
  static constexpr int kBytes = kRing + kRed + (int)sizeof(FewTables);
  static_assert(kBytes <= 232448, "shared memory budget");
};

}  // namespace

template <int WT>
__global__ void __launch_bounds__(kFewThreads, 1) few_kernel(const __grid_constant__ FewParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  using L = FewSmem<WT>;
  uint8_t *ring = smem;
  float *red = reinterpret_cast<float *>(smem + L::kRing);
  FewTables &tb = *reinterpret_cast<FewTables *>(smem + L::kRing + L::kRed);
  unsigned *bar = p.sync + kSyncFew, *exits = bar + 3;
  const bool route = p.router_w != nullptr;
  if (threadIdx.x == 0) {
    tb.abort_flag = 0;
    tb.nsh = p.has_shared ? (p.T + 7) >> 3 : 0;
  }
  if (threadIdx.x < 256) tb.mask[threadIdx.x] = 0u;
  if (threadIdx.x < 256) tb.bias[threadIdx.x] = p.bias != nullptr && (int)threadIdx.x < p.E ? __ldg(p.bias + threadIdx.x) : 0.0f;
  if (WT)
    for (int t = gridDim.x - 1 - blockIdx.x; t < p.T; t += gridDim.x) convert_token(p, t, reinterpret_cast<unsigned *>(red));
  __syncthreads();
  if (route) router_rows(p, red);
  if (route || WT) grid_arrive(bar);
  if (p.has_shared && threadIdx.x < 32) prefetch_shared<WT>(p);
  if (!route) tables_from_perm(p, tb);
  bool ok = true;
  if (route || WT) ok = grid_wait(p, bar, tb);
  if (ok) {
    if (route) tables_from_logits(p, tb, red);
    run_phase<WT, false>(p, tb, ring, red, nullptr, ok);
  }
  grid_arrive(bar + 1);  // also after a wait that ran out: the others need not wait for theirs to do so
  if (ok) run_phase<WT, true>(p, tb, ring, red, bar + 1, ok);
  if (route) {
    grid_arrive(bar + 2);
    if (ok && grid_wait(p, bar + 2, tb)) combine_rows(p, tb);
  }
  __syncthreads();
  // the last CTA out zeroes the counters
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(exits, 1u) == gridDim.x - 1) {
      volatile unsigned *s = bar;
      s[0] = s[1] = s[2] = 0;
      __threadfence();
      s[3] = 0;
    }
  }
}

namespace {
template <int WT>
cudaError_t launch_few_wt(const FewParams &p, int num_ctas, cudaStream_t stream) {
  using L = FewSmem<WT>;
  static thread_local unsigned long long attr_ctx = 0;
  const cudaError_t e = set_smem_attr_once((const void *)few_kernel<WT>, L::kBytes, attr_ctx);
  if (e != cudaSuccess) return e;
  void *args[] = {(void *)&p};
  return launch_coop((const void *)few_kernel<WT>, dim3(num_ctas), dim3(kFewThreads), L::kBytes, stream, args);
}
}  // namespace

cudaError_t launch_few(const FewParams &p, bool mxfp4, int num_ctas, cudaStream_t stream) {
  return mxfp4 ? launch_few_wt<1>(p, num_ctas, stream) : launch_few_wt<0>(p, num_ctas, stream);
}

}  // namespace moe
