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

// v / scale for the values v of one block, from multiples u of them: u * 448 /
// max|u| is the same quotient with fewer roundings.  For bf16 values, and for
// products of two, u * 448 is exact in fp32, so that a quotient which is a tie
// of the rounding to e4m3 is one here too: the product with the reciprocal is
// corrected by its exact remainder (Markstein's final step, 1990), two FMAs;
// IEEE divisions made the norm of 16384 x 2048 values 52 -> 59 us.
__device__ __forceinline__ bool fp8_direct(float largest_u) {   // far from fp32's ends
  return largest_u > 1e-30f && largest_u < 1e30f;
}
__device__ __forceinline__ float fp8_quotient(float u, float largest_u, float reciprocal) {
  const float a = u * kFp8Max;
  const float q = a * reciprocal;
  return fmaf(fmaf(-q, largest_u, a), reciprocal, q);
}

// The same for values of any size: v times `by` over `top` is v / scale, as the
// quotient by the largest magnitude where that is far from fp32's ends, else by
// the scale itself.  (An infinite scale gives NaN for every value.)
struct Fp8Divisor {
  float by, top, reciprocal;
  __device__ __forceinline__ Fp8Divisor(float amax, float scale) {
    const bool direct = fp8_direct(amax);
    by = direct ? kFp8Max : 1.f;
    top = direct ? amax : scale;
    reciprocal = 1.f / top;
  }
  __device__ __forceinline__ float operator()(float v) const {
    const float a = v * by;
    const float q = a * reciprocal;
    return fmaf(fmaf(-q, top, a), reciprocal, q);
  }
};

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
