// 8-bit integer rows (int8.cu, and the int8 expert kernel's activations): scale
// = m / 127 in fp32 with m the row's largest magnitude (1 for a row of zeros),
// code = 127 x / m to the nearest integer, ties to even, with no rounding before
// that one.
#pragma once
#include <cuda_fp16.h>
#include <stdint.h>

namespace moe {

// What a row's values are multiplied by.  `pre` lifts rows of tiny values (bf16
// reaches down to 2^-133) so that 127 / m stays finite.
struct Int8Row {
  float scale, pre, mul;
};
// m: the largest magnitude, of bf16 values.  Infinities (and NaN, where m carries
// it) make the scale NaN, so that whatever reads the row is NaN.
__device__ __forceinline__ Int8Row int8_row(float m) {
  Int8Row r;
  r.scale = m > 0.0f ? __fdiv_rn(m, 127.0f) : 1.0f;
  if (!(m <= 3.4e38f)) r.scale = __int_as_float(0x7FC00000);
  r.pre = m < 5.421010862427522e-20f ? 1.8446744073709552e19f : 1.0f;  // 2^-64, 2^64
  r.mul = m > 0.0f ? __fdiv_rn(127.0f, m * r.pre) : 0.0f;
  return r;
}

// 127 x / m, rounded to the nearest integer with ties to even, plus 1.5 * 2^23:
// the sum's low byte is the code.  x and m are bf16: x / m = 2^k a / b with 8-bit
// integers a and b, so 127 x / m is either exactly half way between integers or at
// least v / (127 * 255) away from that, v being its magnitude: more than 2^-16 for
// v >= 1/2.  The fused product (off by at most 127 * 2^-24 < 2^-17) is rounded to a
// multiple of 2^-15 (by adding 384, where fp32's spacing is that), which restores
// the half-way values and crosses none, and then to an integer (384 comes off in the
// same addition).
__device__ __forceinline__ float int8_round(float x, const Int8Row &r) {
  return __fadd_rn(__fmaf_rn(x * r.pre, r.mul, 384.0f), 12582528.0f);
}
// Four codes from four int8_round() results, the first in the low byte.
__device__ __forceinline__ uint32_t int8_pack4(float a, float b, float c, float d) {
  const uint32_t lo = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}
// Two codes as fp16 (exact) from two int8_round() results.
__device__ __forceinline__ uint32_t int8_f16x2(float a, float b) {
  const __half2 h = __floats2half2_rn(a - 12582912.0f, b - 12582912.0f);
  return *reinterpret_cast<const uint32_t *>(&h);
}
// Four codes (bytes of w) to four fp16 values, exactly: code + 128 as the low byte
// of 1024 + code + 128 (fp16's spacing there is 1), less 1152.
__device__ __forceinline__ uint2 int8x4_to_f16(uint32_t w) {
  const uint32_t u = w ^ 0x80808080u;
  const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
  const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), off);
  const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&b), off);
  return make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
}

}  // namespace moe
