// Block-scaled e4m3: the arithmetic of the format.
//
// Over the values x of one block (1 x 128 of a row, or 128 x 128):
//   a = max(max |x|, 7 * 2^-58), scale = a / 448, inv = 448 / a,
//   code = e4m3(x * inv),
// each operation rounded to fp32.  The product with inv instead of a division by
// scale costs one multiplication a value and differs from it by at most 2^-23
// relative, far inside the half step (2^-4) of an e4m3 value.
#pragma once

#include "dcn_common.cuh"

namespace dcn {

constexpr float kE4m3Max = 448.f;
constexpr float kE4m3Floor = 0x1.cp-56f;  // 7 * 2^-58: scale >= 2^-64, inv <= 2^64
constexpr int kFp8Block = 128;

// max that passes a NaN on.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

struct BlockScale {
  float scale, inv;
};

__device__ __forceinline__ BlockScale block_scale(float amax) {
  BlockScale s;
  const float a = max_nan(amax, kE4m3Floor);
  if (a <= 3.402823466e38f) {
    s.scale = __fdiv_rn(a, kE4m3Max);
    s.inv = __fdiv_rn(kE4m3Max, a);
  } else {  // a NaN or an infinity in the block
    s.scale = s.inv = __int_as_float(0x7FC00000);
  }
  return s;
}

// Two codes in the low 16 bits, lo in the low byte (nearest, ties to even; NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

}  // namespace dcn
