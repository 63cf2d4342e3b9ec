// The 8-bit block format shared by the kernels that write or read it:
// e4m3 values with one fp32 scale per block, value = q * scale.
//   rows    - one scale per 128 consecutive columns of a row;
//   weights - one scale per 128 x 128 block of a matrix.
// A block with largest magnitude m has scale max(m, 2^-100) / 448 (448 is the
// largest e4m3 value) and q = e4m3(v / scale), nearest even.  The floor keeps
// the reciprocal finite; a block of zeros is stored as zeros.  A NaN stays a
// NaN; a block that holds an infinity has an infinite scale, and every value
// of it reads back as NaN.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

constexpr int kQuantBlock = 128;
constexpr float kFp8Max = 448.f;
constexpr float kQuantFloor = 7.888609052210118e-31f;   // 2^-100

// The scale of a block from its largest magnitude.
__device__ __forceinline__ float fp8_scale(float amax) { return fmaxf(amax, kQuantFloor) / kFp8Max; }

// Two values to packed e4m3 (the first in the low byte), nearest even,
// saturating at +-448.
__device__ __forceinline__ uint16_t fp8_pack2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d) {
  return static_cast<uint32_t>(fp8_pack2(a, b)) | static_cast<uint32_t>(fp8_pack2(c, d)) << 16;
}

}  // namespace moe
