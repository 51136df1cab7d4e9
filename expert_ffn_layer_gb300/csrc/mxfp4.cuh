// MXFP4 building blocks (OCP Microscaling): E2M1 elements, one power-of-two
// scale byte e (standing for 2^(e - 127)) per block of 32 values along a row.
//
// Packed rows.  A row of K values (K a multiple of 128) is K / 128 pieces of 64
// bytes, and 32-bit word 4 t + q of a piece (t, q in 0..3) holds the codes of the
// piece's values 32 q + 8 t .. + 7, the first in the lowest four bits: the plain
// order (word 4 q + t) with its 4 x 4 matrix of words transposed.  One 16-byte
// load of lane t then brings, for each of four blocks, the eight values whose
// products the lanes t = 0..3 of a matrix instruction add up -- so that a matrix
// instruction never mixes two blocks and the block's scale can multiply its
// accumulator.
#pragma once
#include <cuda_fp16.h>
#include <stdint.h>

namespace moe {

// Eight E2M1 codes to four fp16 pairs, the lower code in the lower half (every
// E2M1 value is an fp16 value).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n.reg .b8 b0, b1, b2, b3;\nmov.b32 {b0, b1, b2, b3}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\ncvt.rn.f16x2.e2m1x2 %1, b1;\n"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\ncvt.rn.f16x2.e2m1x2 %3, b3;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Eight fp32 values to E2M1 codes (nearest, ties to the even code, magnitudes
// past 6 saturated), the first in the lowest four bits.
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float (&f)[8]) {
  uint32_t w;
  asm("{\n.reg .b8 b0, b1, b2, b3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\ncvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\ncvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      "mov.b32 %0, {b0, b1, b2, b3};\n}"
      : "=r"(w)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return w;
}

// The value of a scale byte: 2^(e - 127); 255 is the format's NaN.
__device__ __forceinline__ float e8m0_value(uint32_t e) {
  return __uint_as_float(e == 0u ? 0x00400000u : e == 255u ? 0x7FFFFFFFu : e << 23);
}

}  // namespace moe
