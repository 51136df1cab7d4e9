// MXFP4 expert weights: rows of bf16 to packed E2M1 codes and scale bytes, and back.
//
// The Ascend deployment article (section 8.2) runs the routed experts with MXFP4
// weights and fixes no further detail.  Here: the OCP Microscaling format, blocks
// of 32 along a row, scale 2^(floor(log2 max|block|) - 2) (at least 2^-127), codes
// nearest-even of value / scale with magnitudes past 6 saturated.  Both directions
// are exact but for that one rounding: a scale is a power of two.
//
// Both kernels stream: 2 bytes read and 17/32 written a value, or the reverse, and
// nothing is read twice, so the memory bounds them.  Over 403 M values 171 us there
// (6.0 TB/s) and 148 us back (6.9); both over 6.3 M values 6.7 us in a graph (a call of
// each from Python takes 11.5).
#include "internal.h"
#include "mxfp4.cuh"
#include "ptx.cuh"

namespace moe {

namespace {
constexpr int kMxThreads = 256;
constexpr int kMxLoads = 4;  // 8-value pieces of a thread, all in flight before the first is used
constexpr long long kMxTile = (long long)kMxThreads * kMxLoads;  // a warp takes 128 neighbouring pieces of it
}  // namespace

// One lane per 8 values: four lanes share a block's maximum, sixteen lanes a
// 64-byte piece.  The maximum is taken on the magnitudes' bit patterns, which
// order finite values by size and put infinities and NaN above them all.
__global__ void __launch_bounds__(kMxThreads) quantize_mxfp4_kernel(const __nv_bfloat16 *__restrict__ src,
                                                                    uint8_t *__restrict__ codes,
                                                                    uint8_t *__restrict__ scales, long long n8) {
  pdl_wait();
  pdl_launch_dependents();
  const int l = threadIdx.x & 15, q = l >> 2, t = l & 3;
  const unsigned group = 0xFu << (threadIdx.x & 28u);  // a block's lanes: n8 is a multiple of 16, so all are in range or none
  for (long long i0 = blockIdx.x * kMxTile + (threadIdx.x >> 5) * 128 + (threadIdx.x & 31); i0 < n8; i0 += gridDim.x * kMxTile) {
    uint4 v[kMxLoads];
#pragma unroll
    for (int u = 0; u < kMxLoads; ++u) {
      const long long i = i0 + u * 32;
      if (i < n8) v[u] = __ldcs(reinterpret_cast<const uint4 *>(src) + i);
    }
#pragma unroll
    for (int u = 0; u < kMxLoads; ++u) {
      const long long i = i0 + u * 32;
      if (i >= n8) break;
      const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) top = max(top, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
      top = max(top, __shfl_xor_sync(group, top, 1));
      top = max(top, __shfl_xor_sync(group, top, 2));
      const uint32_t ex = top >> 7;  // biased exponent of the largest magnitude
      const uint32_t e = ex == 255u ? 255u : ex > 2u ? ex - 2u : 0u;
      const float inv = __uint_as_float((254u - min(e, 253u)) << 23);  // 2^(127 - e)
      float f[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16) * inv;
        f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u) * inv;
      }
      reinterpret_cast<uint32_t *>(codes)[(i & ~15ll) + 4 * t + q] = f32x8_to_e2m1(f);
      if (t == 0) scales[i >> 2] = (uint8_t)e;
    }
  }
}

__global__ void __launch_bounds__(kMxThreads) dequantize_mxfp4_kernel(const uint8_t *__restrict__ codes,
                                                                      const uint8_t *__restrict__ scales,
                                                                      __nv_bfloat16 *__restrict__ dst, long long n8) {
  pdl_wait();
  pdl_launch_dependents();
  const int l = threadIdx.x & 15, q = l >> 2, t = l & 3;
  for (long long i0 = blockIdx.x * kMxTile + (threadIdx.x >> 5) * 128 + (threadIdx.x & 31); i0 < n8; i0 += gridDim.x * kMxTile) {
    uint32_t w[kMxLoads], e[kMxLoads];
#pragma unroll
    for (int u = 0; u < kMxLoads; ++u) {
      const long long i = i0 + u * 32;
      if (i < n8) {
        w[u] = __ldcs(reinterpret_cast<const uint32_t *>(codes) + (i & ~15ll) + 4 * t + q);
        e[u] = __ldcs(scales + (i >> 2));
      }
    }
#pragma unroll
    for (int u = 0; u < kMxLoads; ++u) {
      const long long i = i0 + u * 32;
      if (i >= n8) break;
      const float s = e8m0_value(e[u]);
      uint32_t h[4], o[4];
      e2m1x8_to_f16(w[u], h);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[j]));
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s, f.y * s);
        o[j] = *reinterpret_cast<const uint32_t *>(&b);
      }
      __stcs(reinterpret_cast<uint4 *>(dst) + i, make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
}

namespace {
// A CTA for each tile (a grid of eight CTAs an SM that strides over the tiles: 355 us
// for both ways over 403 M values against 319).
unsigned stream_blocks(long long n8) {
  const long long blocks = (n8 + kMxTile - 1) / kMxTile, cap = 0x7fffffff;
  return (unsigned)(blocks < cap ? blocks : cap);
}
}  // namespace

cudaError_t launch_quantize_mxfp4(const __nv_bfloat16 *src, uint8_t *codes, uint8_t *scales, long long n,
                                  cudaStream_t stream) {
  long long n8 = n / 8;
  void *args[] = {(void *)&src, (void *)&codes, (void *)&scales, (void *)&n8};
  return launch_ex((const void *)quantize_mxfp4_kernel, dim3(stream_blocks(n8)), dim3(kMxThreads), 0, stream, true, 1,
                   args);
}

cudaError_t launch_dequantize_mxfp4(const uint8_t *codes, const uint8_t *scales, __nv_bfloat16 *dst, long long n,
                                    cudaStream_t stream) {
  long long n8 = n / 8;
  void *args[] = {(void *)&codes, (void *)&scales, (void *)&dst, (void *)&n8};
  return launch_ex((const void *)dequantize_mxfp4_kernel, dim3(stream_blocks(n8)), dim3(kMxThreads), 0, stream, true,
                   1, args);
}

}  // namespace moe
