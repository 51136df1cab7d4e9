// 8-bit integer experts: the row quantiser that makes their weights, the way back
// to bf16, and the quantiser of the hidden state that the expert kernel reads.
// The rule is in int8.cuh.
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

// Codes of eight values, at piece `at`.  F16: as fp16 values, the form in which the
// expert kernel multiplies them, else bytes.
template <bool F16>
__device__ __forceinline__ void put8(void *codes, long long at, const uint4 &v, const Int8Row &q) {
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
}

// A warp per row of at most 2048 values, which are read once and kept in registers
// (the row's maximum is wanted first), or of any width, read twice (V = 0).
template <bool F16, int V>
__global__ void __launch_bounds__(kThreads) int8_rows_kernel(const __nv_bfloat16 *__restrict__ src,
                                                             void *__restrict__ codes, float *__restrict__ scales,
                                                             long long rows, int cols) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int n8 = cols >> 3;
  for (long long r = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); r < rows;
       r += (long long)gridDim.x * (kThreads / 32)) {
    const uint4 *row = reinterpret_cast<const uint4 *>(src + r * cols);
    uint32_t m = 0;
    uint4 v[V > 0 ? V : 1];
    if constexpr (V > 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = lane + 32 * i < n8 ? __ldcs(row + lane + 32 * i) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int i = 0; i < V; ++i) m = top_bits(v[i], m);
    } else {
      for (int i = lane; i < n8; i += 32) m = top_bits(row[i], m);
    }
    const Int8Row q = int8_row(warp_top(m));
    if (lane == 0) scales[r] = q.scale;
    if constexpr (V > 0) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (lane + 32 * i < n8) put8<F16>(codes, r * n8 + lane + 32 * i, v[i], q);
    } else {
      for (int i = lane; i < n8; i += 32) put8<F16>(codes, r * n8 + i, row[i], q);
    }
  }
}

// Wider rows, up to 1024 V values: a CTA of four warps per row, again read once.
// Bound by HBM: 98304 rows of 4096 values (805 MB in, 403 out) take 187 us, 6.5 TB/s,
// against 250 with a warp a row that reads it twice.
constexpr int kWideThreads = 128;
template <bool F16, int V>
__global__ void __launch_bounds__(kWideThreads) int8_wide_rows_kernel(const __nv_bfloat16 *__restrict__ src,
                                                                      void *__restrict__ codes,
                                                                      float *__restrict__ scales, long long rows,
                                                                      int cols) {
  __shared__ float top[2][kWideThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  const int n8 = cols >> 3, tid = threadIdx.x;
  int par = 0;
  for (long long r = blockIdx.x; r < rows; r += gridDim.x, par ^= 1) {
    const uint4 *row = reinterpret_cast<const uint4 *>(src + r * cols);
    uint4 v[V];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
      v[i] = tid + kWideThreads * i < n8 ? __ldcs(row + tid + kWideThreads * i) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < V; ++i) m = top_bits(v[i], m);
    const float mine = warp_top(m);
    if ((tid & 31) == 0) top[par][tid >> 5] = mine;
    __syncthreads();  // one a row: the next row's maxima go to the other place
    uint32_t t = 0;
#pragma unroll
    for (int w = 0; w < kWideThreads / 32; ++w) t = max(t, __float_as_uint(top[par][w]));  // NaN above all
    const Int8Row q = int8_row(__uint_as_float(t));
    if (tid == 0) scales[r] = q.scale;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (tid + kWideThreads * i < n8) put8<F16>(codes, r * n8 + tid + kWideThreads * i, v[i], q);
  }
}

// A warp per row: code * scale in fp32, rounded to bf16.  Eight codes a lane and step,
// so that a lane's values are one whole 16-byte store (sixteen, stored as two halves
// of every other sector: 264 against 197 us for 403 M values); eight steps' loads in
// flight.
__global__ void __launch_bounds__(kThreads) int8_values_kernel(const int8_t *__restrict__ codes,
                                                               const float *__restrict__ scales,
                                                               __nv_bfloat16 *__restrict__ dst, long long rows,
                                                               int cols) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kSteps = 8;
  const int lane = threadIdx.x & 31;
  const int n8 = cols >> 3;
  for (long long r = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); r < rows;
       r += (long long)gridDim.x * (kThreads / 32)) {
    const float s = __ldg(scales + r);
    const uint2 *row = reinterpret_cast<const uint2 *>(codes) + r * n8;
    uint4 *out = reinterpret_cast<uint4 *>(dst) + r * n8;
    for (int i0 = lane; i0 < n8; i0 += 32 * kSteps) {
      uint2 v[kSteps];
#pragma unroll
      for (int u = 0; u < kSteps; ++u)
        if (i0 + 32 * u < n8) v[u] = __ldcs(row + i0 + 32 * u);
#pragma unroll
      for (int u = 0; u < kSteps; ++u)
        if (i0 + 32 * u < n8) {
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // code + 128 as the low byte of 2^23 + code + 128
            const uint32_t x = (j < 2 ? v[u].x : v[u].y) ^ 0x80808080u;
            const float a = __uint_as_float(__byte_perm(x, 0x4B000000u, j & 1 ? 0x7442 : 0x7440)) - 8388736.0f;
            const float b = __uint_as_float(__byte_perm(x, 0x4B000000u, j & 1 ? 0x7443 : 0x7441)) - 8388736.0f;
            const __nv_bfloat162 p = __floats2bfloat162_rn(a * s, b * s);
            o[j] = *reinterpret_cast<const uint32_t *>(&p);
          }
          __stcs(out + i0 + 32 * u, make_uint4(o[0], o[1], o[2], o[3]));
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
cudaError_t launch_rows(const __nv_bfloat16 *src, void *codes, float *scales, long long rows, int cols, cudaStream_t stream) {
  void *args[] = {(void *)&src, (void *)&codes, (void *)&scales, (void *)&rows, (void *)&cols};
  if (cols > 2048 && cols <= 16384) {
    const long long cap = 16LL * sms();
    return launch_ex(cols <= 4096 ? (const void *)int8_wide_rows_kernel<F16, 4> : (const void *)int8_wide_rows_kernel<F16, 16>,
                     dim3((unsigned)(rows < cap ? rows : cap)), dim3(kWideThreads), 0, stream, true, 1, args);
  }
  return launch_ex(cols <= 1024   ? (const void *)int8_rows_kernel<F16, 4>
                   : cols <= 2048 ? (const void *)int8_rows_kernel<F16, 8>
                                  : (const void *)int8_rows_kernel<false, 0>,  // no hidden state is this wide
                   dim3(row_blocks(rows)), dim3(kThreads), 0, stream, true, 1, args);
}
}  // namespace

cudaError_t launch_quantize_int8(const __nv_bfloat16 *src, void *codes, bool f16, float *scales, long long rows,
                                 int cols, cudaStream_t stream) {
  return f16 ? launch_rows<true>(src, codes, scales, rows, cols, stream)
             : launch_rows<false>(src, codes, scales, rows, cols, stream);
}

cudaError_t launch_dequantize_int8(const int8_t *codes, const float *scales, __nv_bfloat16 *dst, long long rows,
                                   int cols, cudaStream_t stream) {
  void *args[] = {(void *)&codes, (void *)&scales, (void *)&dst, (void *)&rows, (void *)&cols};
  return launch_ex((const void *)int8_values_kernel, dim3(row_blocks(rows)), dim3(kThreads), 0, stream, true, 1, args);
}

}  // namespace moe
