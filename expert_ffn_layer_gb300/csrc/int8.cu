// 8-bit integer experts: the row quantiser that makes their weights, the way back
// to bf16, and the quantiser of the hidden state that the expert kernel reads.
// The rule is in int8.cuh.
#include "int8.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace moe {

namespace {
constexpr int kThreads = 256;  // eight rows (one per warp) per CTA step

// Largest magnitude of eight bf16 values as integer bits, which order as the
// values do with NaN above infinity.
__device__ __forceinline__ uint32_t top_bits(const uint4 &v, uint32_t m) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) m = max(m, max(u[j] << 16 & 0x7FFFFFFFu, u[j] & 0x7FFF0000u));
  return m;
}
}  // namespace

// One warp per row: the row maximum first, then the codes, 8 values per lane
// step (the second reading is from L1 or L2).  F16: the codes as fp16 values, the
// form in which the expert kernel multiplies them, else bytes.
template <bool F16>
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
    for (int i = lane; i < n8; i += 32) m = top_bits(row[i], m);
    m = __reduce_max_sync(0xffffffffu, m);
    const Int8Row q = int8_row(__uint_as_float(m));
    if (lane == 0) scales[r] = q.scale;
    for (int i = lane; i < n8; i += 32) {
      const uint4 v = row[i];
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
      float f[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[2 * j] = int8_round(__uint_as_float(u[j] << 16), q);
        f[2 * j + 1] = int8_round(__uint_as_float(u[j] & 0xFFFF0000u), q);
      }
      if (F16)
        reinterpret_cast<uint4 *>(codes)[r * n8 + i] = make_uint4(int8_f16x2(f[0], f[1]), int8_f16x2(f[2], f[3]),
                                                                  int8_f16x2(f[4], f[5]), int8_f16x2(f[6], f[7]));
      else
        reinterpret_cast<uint2 *>(codes)[r * n8 + i] =
            make_uint2(int8_pack4(f[0], f[1], f[2], f[3]), int8_pack4(f[4], f[5], f[6], f[7]));
    }
  }
}

// Eight values per thread step: code * scale in fp32, rounded once to bf16.
__global__ void __launch_bounds__(kThreads) int8_values_kernel(const int8_t *__restrict__ codes,
                                                               const float *__restrict__ scales,
                                                               __nv_bfloat16 *__restrict__ dst, long long rows,
                                                               int cols) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int n8 = cols >> 3;
  for (long long r = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); r < rows;
       r += (long long)gridDim.x * (kThreads / 32)) {
    const float s = scales[r];
    for (int i = lane; i < n8; i += 32) {
      const uint2 w = reinterpret_cast<const uint2 *>(codes)[r * n8 + i];
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t pair = (j < 2 ? w.x : w.y) >> (16 * (j & 1));
        const __nv_bfloat162 b = __floats2bfloat162_rn((float)(int8_t)(pair & 0xFF) * s, (float)(int8_t)(pair >> 8 & 0xFF) * s);
        o[j] = *reinterpret_cast<const uint32_t *>(&b);
      }
      reinterpret_cast<uint4 *>(dst)[r * n8 + i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

namespace {
unsigned row_blocks(long long rows) {
  int dev = 0, nsm = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
  const long long blocks = (rows + kThreads / 32 - 1) / (kThreads / 32), cap = (long long)(nsm > 0 ? nsm : 1) * 8;
  return (unsigned)(blocks < cap ? blocks : cap);
}
}  // namespace

cudaError_t launch_quantize_int8(const __nv_bfloat16 *src, void *codes, bool f16, float *scales, long long rows,
                                 int cols, cudaStream_t stream) {
  void *args[] = {(void *)&src, (void *)&codes, (void *)&scales, (void *)&rows, (void *)&cols};
  return launch_ex(f16 ? (const void *)int8_rows_kernel<true> : (const void *)int8_rows_kernel<false>,
                   dim3(row_blocks(rows)), dim3(kThreads), 0, stream, true, 1, args);
}

cudaError_t launch_dequantize_int8(const int8_t *codes, const float *scales, __nv_bfloat16 *dst, long long rows,
                                   int cols, cudaStream_t stream) {
  void *args[] = {(void *)&codes, (void *)&scales, (void *)&dst, (void *)&rows, (void *)&cols};
  return launch_ex((const void *)int8_values_kernel, dim3(row_blocks(rows)), dim3(kThreads), 0, stream, true, 1, args);
}

}  // namespace moe
