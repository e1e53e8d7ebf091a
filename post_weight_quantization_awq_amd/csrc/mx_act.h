// Activation functions of the microscaled operators.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace awq {

// g / (1 + e^-g) to a few units of the last place, in 8 operations besides the
// exponential and the reciprocal: e^-g = 2^t (1 + r ln 2) with t = RN(-g log2 e)
// and r the rest of the product.  For g >= -87 only: below, the reciprocal of
// 1 + e^-g leaves the normal range.  Gates past 128 (t would overflow for the
// largest bf16 ones) count as 128 in the exponential, which is 0 there.
constexpr float kLog2eHi = 1.44269502162933349609375f, kLog2eLo = 1.92596298909109e-8f, kLn2 = 0.693147182464599609375f;
template <int DT>
__device__ __forceinline__ float silu(float g) {
  const float x = DT == 0 ? -g : __builtin_fmaxf(-g, -128.0f);
  const float t = x * kLog2eHi;
  const float r = __builtin_fmaf(x, kLog2eLo, __builtin_fmaf(x, kLog2eHi, -t));
  const float d = __builtin_fmaf(__builtin_amdgcn_exp2f(t), __builtin_fmaf(r, kLn2, 1.0f), 1.0f);
  return g * __builtin_amdgcn_rcpf(d);
}

constexpr uint32_t kFarGate = 0xC2AE0000u;  // the pattern of -87; those of lesser values are larger
// g e^g up, which is g / (1 + e^-g) up to 2^-125 of it for g < -87.  e^g is taken as four equal factors, multiplied
// up so that nothing on the way passes the range, and what vanishes on the way vanishes in the result.
__device__ __forceinline__ float far_silu_mul(float g, float up) {
  const float x = __builtin_fmaxf(g, -1024.0f);
  const float t = x * kLog2eHi;
  const float r = __builtin_fmaf(x, kLog2eLo, __builtin_fmaf(x, kLog2eHi, -t));
  const float q = __builtin_amdgcn_exp2f(0.25f * t);
  return g * q * up * q * q * (q * __builtin_fmaf(r, kLn2, 1.0f));
}

// 2^64 e^z for z <= 0 to a few units of the last place, also where e^z itself leaves the normal range
__device__ __forceinline__ float exp_up(float z) {
  z = __builtin_fmaxf(z, -1024.0f);
  const float t = z * kLog2eHi;
  const float r = __builtin_fmaf(z, kLog2eLo, __builtin_fmaf(z, kLog2eHi, -t));
  const float q = __builtin_amdgcn_exp2f(0.5f * t) * 0x1p32f;
  return q * q * __builtin_fmaf(r, kLn2, 1.0f);
}

// v / (1 + e^-s) for any s; for s < 0 as v e^s / (1 + e^s), multiplied up by 2^64 on the way
__device__ __forceinline__ float sigmoid_mul(float v, float s) {
  const float e = exp_up(-__builtin_fabsf(s));
  const float d = __builtin_amdgcn_rcpf(__builtin_fmaf(e, 0x1p-64f, 1.0f));
  return s < 0.0f ? v * e * d * 0x1p-64f : v * d;
}

// v (1 + erf(v / sqrt 2)) / 2 = v (1 - erfc(x) / 2) or, for v < 0, v erfc(x) / 2 with x = |v| / sqrt 2 and
//   erfc(x) = t e^(p(t) - x^2), t = 1 / (1 + x / 2),
// p the polynomial of degree 9 that meets ln(erfc(x) / t) + x^2 at the Chebyshev points of 0 <= x <= 10.5 within
// 2^-22 in fp32 arithmetic (fitted for this kernel); erfc(10.5) is below fp32's range.
__device__ __forceinline__ float gelu(float v) {
  const float x = __builtin_fabsf(v) * 0.70710678118654752f;
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.5f, x, 1.0f));
  float p = 0.1487911492586136f;
  p = __builtin_fmaf(p, t, -0.70184725522995f);
  p = __builtin_fmaf(p, t, 1.2061694860458374f);
  p = __builtin_fmaf(p, t, -0.7619841694831848f);
  p = __builtin_fmaf(p, t, -0.0259946808218956f);
  p = __builtin_fmaf(p, t, -0.027512092143297195f);
  p = __builtin_fmaf(p, t, 0.04436234384775162f);
  p = __builtin_fmaf(p, t, 0.38460636138916016f);
  p = __builtin_fmaf(p, t, 0.9988684058189392f);
  p = __builtin_fmaf(p, t, -1.2654595375061035f);
  const float e = 0.5f * t * exp_up(__builtin_fmaf(-0.5f * v, v, p));  // 2^63 erfc(x)
  return v < 0.0f ? v * e * 0x1p-64f : v * __builtin_fmaf(e, -0x1p-64f, 1.0f);
}

constexpr int kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4;
// relu keeps NaN; gelu_tanh = v (1 + tanh u) / 2 = v / (1 + e^-2u), u = sqrt(2 / pi) (v + 0.044715 v^3)
template <int N>
__device__ __forceinline__ void activate(float (&v)[N], int act) {
  if (act == kActNone) return;
  if (act == kActRelu) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = v[j] < 0.0f ? 0.0f : v[j];
  } else if (act == kActSilu) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = sigmoid_mul(v[j], v[j]);
  } else if (act == kActGeluTanh) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float c = v[j] * v[j] * 0.0713548162726f;  // 2 sqrt(2 / pi) 0.044715
      v[j] = sigmoid_mul(v[j], v[j] * (c + 1.59576912160573f));
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = gelu(v[j]);
  }
}

}  // namespace awq
