// 8-bit integer experts: the row quantiser that makes their weights, the way back
// to bf16, and the quantiser of the hidden state that the expert kernel reads.
// The rule is in int8.cuh.
#include <type_traits>

#include "int8.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace moe {

namespace {
constexpr int kThreads = 256;  // eight rows (one per warp) per CTA step

// Largest magnitudes of the even and of the odd of eight bf16 values, as 16-bit
// integers, which order as the values do with NaN above infinity.
__device__ __forceinline__ uint32_t top_bits(const uint4 &v, uint32_t m) {
  m = __vimax3_u16x2(m, v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu);
  return __vimax3_u16x2(m, v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu);
}
// The largest of a warp's, as an fp32 value.
__device__ __forceinline__ float warp_top(uint32_t m) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16)) << 16);
}
}  // namespace

// One warp per row, 8 values (16 bytes) per lane and piece.  V > 0: rows of at most
// 256 V values, read once and kept in registers (the row maximum is wanted first);
// V = 0: longer rows, read twice, the second time from L1 or L2.  Bound by HBM: 64
// stacked matrices of 1536 x 4096 (805 MB in, 403 out) take 196 us, 0.91 of the copy
// bandwidth; reading each row twice, 250.
// F16: the codes as fp16 values, the form in which the expert kernel multiplies them,
// else bytes.
template <bool F16, int V>
__global__ void __launch_bounds__(kThreads) int8_rows_kernel(const __nv_bfloat16 *__restrict__ src,
                                                             void *__restrict__ codes, float *__restrict__ scales,
                                                             long long rows, int cols) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int n8 = cols >> 3;
  auto put = [&](long long at, const uint4 &v, const Int8Row &q) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = int8_round(__uint_as_float(u[j] << 16), q);
      f[2 * j + 1] = int8_round(__uint_as_float(u[j] & 0xFFFF0000u), q);
    }
    if (F16)
      reinterpret_cast<uint4 *>(codes)[at] = make_uint4(int8_f16x2(f[0], f[1]), int8_f16x2(f[2], f[3]),
                                                        int8_f16x2(f[4], f[5]), int8_f16x2(f[6], f[7]));
    else
      reinterpret_cast<uint2 *>(codes)[at] =
          make_uint2(int8_pack4(f[0], f[1], f[2], f[3]), int8_pack4(f[4], f[5], f[6], f[7]));
  };
  for (long long r = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); r < rows;
       r += (long long)gridDim.x * (kThreads / 32)) {
    const uint4 *row = reinterpret_cast<const uint4 *>(src + r * cols);
    uint32_t m = 0;
    uint4 v[V > 0 ? V : 1];
    if constexpr (V > 0) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (lane + 32 * i < n8) v[i] = __ldcs(row + lane + 32 * i);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (lane + 32 * i < n8) m = top_bits(v[i], m);
    } else {
      for (int i = lane; i < n8; i += 32) m = top_bits(row[i], m);
    }
    const Int8Row q = int8_row(warp_top(m));
    if (lane == 0) scales[r] = q.scale;
    if constexpr (V > 0) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (lane + 32 * i < n8) put(r * n8 + lane + 32 * i, v[i], q);
    } else {
      for (int i = lane; i < n8; i += 32) put(r * n8 + i, row[i], q);
    }
  }
}

// A CTA per row of the hidden state, for batches that leave most of the device idle
// with a warp a row.
__global__ void __launch_bounds__(kThreads) int8_row_cta_kernel(const __nv_bfloat16 *__restrict__ src,
                                                                uint4 *__restrict__ codes, float *__restrict__ scales,
                                                                int cols) {
  constexpr int V = 16384 / 8 / kThreads;  // pieces of a thread, the widest row
  __shared__ uint32_t top[kThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  const int n8 = cols >> 3;
  const size_t r = blockIdx.x;
  const uint4 *row = reinterpret_cast<const uint4 *>(src + r * cols);
  uint4 v[V];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if ((int)threadIdx.x + kThreads * i < n8) v[i] = row[threadIdx.x + kThreads * i];
#pragma unroll
  for (int i = 0; i < V; ++i)
    if ((int)threadIdx.x + kThreads * i < n8) m = top_bits(v[i], m);
  m = __float_as_uint(warp_top(m));
  if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) m = max(m, top[w]);
  const Int8Row q = int8_row(__uint_as_float(m));
  if (threadIdx.x == 0) scales[r] = q.scale;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if ((int)threadIdx.x + kThreads * i < n8) {
      const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = int8_f16x2(int8_round(__uint_as_float(u[j] << 16), q), int8_round(__uint_as_float(u[j] & 0xFFFF0000u), q));
      codes[r * n8 + threadIdx.x + kThreads * i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// A warp per row: code * scale in fp32, rounded once to bf16.  16 codes (W = 4 words)
// per lane step where the rows' width allows, else 8; four steps' loads in flight.
template <int W>
__global__ void __launch_bounds__(kThreads) int8_values_kernel(const int8_t *__restrict__ codes,
                                                               const float *__restrict__ scales,
                                                               __nv_bfloat16 *__restrict__ dst, long long rows,
                                                               int cols) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int n = cols / (4 * W);
  using Vec = typename std::conditional<W == 4, uint4, uint2>::type;
  for (long long r = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); r < rows;
       r += (long long)gridDim.x * (kThreads / 32)) {
    const float s = __ldg(scales + r);
    const Vec *row = reinterpret_cast<const Vec *>(codes) + r * n;
    uint4 *out = reinterpret_cast<uint4 *>(dst) + r * n * (W / 2);
    for (int i0 = 0; i0 < n; i0 += 128) {
      Vec v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i0 + 32 * u + lane < n) v[u] = __ldcs(row + i0 + 32 * u + lane);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i0 + 32 * u + lane < n) {
          const uint32_t *w = reinterpret_cast<const uint32_t *>(&v[u]);
#pragma unroll
          for (int h = 0; h < W / 2; ++h) {
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              // code + 128 as the low byte of 2^23 + code + 128
              const uint32_t x = w[2 * h + j / 2] ^ 0x80808080u;
              const float a = __uint_as_float(__byte_perm(x, 0x4B000000u, j & 1 ? 0x7442 : 0x7440)) - 8388736.0f;
              const float b = __uint_as_float(__byte_perm(x, 0x4B000000u, j & 1 ? 0x7443 : 0x7441)) - 8388736.0f;
              const __nv_bfloat162 p = __floats2bfloat162_rn(a * s, b * s);
              o[j] = *reinterpret_cast<const uint32_t *>(&p);
            }
            __stcs(out + (size_t)(i0 + 32 * u + lane) * (W / 2) + h, make_uint4(o[0], o[1], o[2], o[3]));
          }
        }
    }
  }
}

namespace {
int sms() {
  static thread_local int dev_cached = -1, n = 1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev != dev_cached) {
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    dev_cached = dev;
  }
  return n;
}
unsigned row_blocks(long long rows) {
  const long long blocks = (rows + kThreads / 32 - 1) / (kThreads / 32), cap = (long long)sms() * 8;
  return (unsigned)(blocks < cap ? blocks : cap);
}
template <bool F16>
const void *rows_kernel(int cols) {
  if (cols <= 512) return (const void *)int8_rows_kernel<F16, 2>;
  if (cols <= 1536) return (const void *)int8_rows_kernel<F16, 6>;
  if (cols <= 4096) return (const void *)int8_rows_kernel<F16, 16>;
  return (const void *)int8_rows_kernel<F16, 0>;
}
}  // namespace

cudaError_t launch_quantize_int8(const __nv_bfloat16 *src, void *codes, bool f16, float *scales, long long rows,
                                 int cols, cudaStream_t stream) {
  if (f16 && cols <= 16384 && rows <= 2 * sms()) {
    uint4 *out = static_cast<uint4 *>(codes);
    void *args[] = {(void *)&src, (void *)&out, (void *)&scales, (void *)&cols};
    return launch_ex((const void *)int8_row_cta_kernel, dim3((unsigned)rows), dim3(kThreads), 0, stream, true, 1, args);
  }
  void *args[] = {(void *)&src, (void *)&codes, (void *)&scales, (void *)&rows, (void *)&cols};
  return launch_ex(f16 ? rows_kernel<true>(cols) : rows_kernel<false>(cols), dim3(row_blocks(rows)), dim3(kThreads), 0,
                   stream, true, 1, args);
}

cudaError_t launch_dequantize_int8(const int8_t *codes, const float *scales, __nv_bfloat16 *dst, long long rows,
                                   int cols, cudaStream_t stream) {
  void *args[] = {(void *)&codes, (void *)&scales, (void *)&dst, (void *)&rows, (void *)&cols};
  return launch_ex(cols % 16 ? (const void *)int8_values_kernel<2> : (const void *)int8_values_kernel<4>,
                   dim3(row_blocks(rows)), dim3(kThreads), 0, stream, true, 1, args);
}

}  // namespace moe
