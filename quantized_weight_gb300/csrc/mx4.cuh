// mx4.cuh -- the microscaled 4-bit format (include/qmm.h): e2m1 codes, blocks of 32 with a power of two each, and
// where a block's scale stands.
//
// Scales are kept in tiles of 128 rows by 4 blocks (512 bytes), the shape in which tcgen05.cp hands them to the tensor
// core: byte 16 * (row % 32) + 4 * (row / 32) + block of a tile.  The tiles of 128 rows follow one another along K.
#pragma once
#include <cstdint>
#include <cuda_fp16.h>

#include "mx4_layout.h"

namespace qmm {

// Offset of the four scales of a row in K tile `kt` of a matrix with `k_tiles` of them a row.
__device__ __forceinline__ int64_t mx4_scale_word(int64_t row, int64_t kt, int64_t k_tiles) {
  return ((row >> 7) * k_tiles + kt) * kMxTileBytes + (row & 31) * 16 + ((row >> 5) & 3) * 4;
}

// 2 ** (scale - 127); 255 is NaN.
__device__ __forceinline__ float mx4_scale(uint32_t scale) {
  return __uint_as_float(scale == 255 ? 0x7FC00000u : scale == 0 ? 0x00400000u : scale << 23);
}

// The two values of a byte of codes, the low nibble's first.
__device__ __forceinline__ float2 mx4_pair(uint32_t byte) {
  uint32_t h;
  asm("{\n\t.reg .b8 b;\n\tcvt.u8.u32 b, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(h) : "r"(byte));
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// Eight values to a word of codes, the first in the lowest nibble: nearest, halves to the even code, at most 6.
__device__ __forceinline__ uint32_t mx4_encode(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// The largest of three, NaN if one is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

}  // namespace qmm
