// Division by a scale whose reciprocal is at hand.  Host and device: a host test
// compares it with the division.
#pragma once

#include <hip/hip_runtime.h>

namespace awq {

// v / s rounded to nearest even, from y = RN(1 / s), for v of at most 4 significant bits (an e4m3 or e2m1 element
// times a power of two) and v, s, y and the quotient in the normal range, or v a zero: q = RN(v y), then
// q + RN(v - s q) y rounded.  For a zero the sum would lose its sign, so the result takes q's.
__host__ __device__ __forceinline__ float mx_quotient(float v, float s, float y) {
  const float q = v * y;
  return __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-s, q, v), y, q), q);
}

}  // namespace awq
