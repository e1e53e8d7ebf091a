// Activation functions of the microscaled operators.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

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

constexpr int kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4;
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kFar = -87.0f;  // e^-s passes fp32's range not far below

// v 2^w for w far below 0, as four equal factors of 2^w: what vanishes on the way vanishes in the result
__device__ __forceinline__ float far_exp2_mul(float v, float w) {
  const float q = __builtin_amdgcn_exp2f(0.25f * __builtin_fmaxf(w, -1024.0f));
  return v * q * q * q * q;
}

__device__ __forceinline__ float gelu_poly(float t) {
  float p = -0.2732841968536377f;
  p = __builtin_fmaf(p, t, 1.0939927101135254f);
  p = __builtin_fmaf(p, t, -1.4604928493499756f);
  p = __builtin_fmaf(p, t, 0.519133985042572f);
  p = __builtin_fmaf(p, t, -0.06438025832176208f);
  p = __builtin_fmaf(p, t, 0.5703367590904236f);
  p = __builtin_fmaf(p, t, 1.4403741359710693f);
  p = __builtin_fmaf(p, t, -2.825681447982788f);
  return p;
}

// 8 values at once, with as few operations a value as their accuracy allows (they are not hidden behind the matrix
// products: 21 us of 8192 x 4096 values at 26 operations).  Exponents below kFar are rare and take a branch.
//   relu   keeps NaN
//   silu   v / (1 + e^-v): the rounding of v log2 e is 2^-17.5 of the value at most
//   gelu_tanh   v (1 + tanh u) / 2 = v / (1 + e^-2u), u = sqrt(2 / pi) (v + 0.044715 v^3); 2 u log2 e within 5 roundings
//   gelu   v (1 + erf(v / sqrt 2)) / 2 = v (1 - E) or, for v < 0, v E, where with x = |v| / sqrt 2
//     E = erfc(x) / 2 = t 2^(p(t) - x^2 log2 e), t = 1 / (1 + x / 2),
//   the form that Press et al., Numerical Recipes, give erfc, with p the polynomial of degree 7 that meets log2(erfc(x) /
//   t) + x^2 log2 e - 1 at the Chebyshev points of 0 <= x <= 10.5 within 2^-19.6 in fp32 arithmetic (fitted for this
//   kernel); erfc(10.5) is below fp32's range.
// -inf: NaN by the formulas but for relu.  What the tails' 2^-15 to 2^-17 cost a result of 8 bits does not show: 4096 x
// 12288 x 4096 with 4-bit operands has 8e-7 of its codes off with gelu_tanh, 4e-7 without, as fp32 operations do.
template <int N>
__device__ __forceinline__ void activate(float (&v)[N], int act) {
  if (act == kActNone) return;
  if (act == kActRelu) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = v[j] < 0.0f ? 0.0f : v[j];
    return;
  }
  float least = 0.0f, in[N];
#pragma unroll
  for (int j = 0; j < N; ++j) in[j] = v[j], least = __builtin_fminf(least, v[j]);
  if (act == kActGelu) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(__builtin_fabsf(v[j]), 0.5f * 0.70710678118654752f, 1.0f));
      const float p = gelu_poly(t);
      const float e = t * __builtin_amdgcn_exp2f(__builtin_fmaf(-0.5f * kLog2e * v[j], v[j], p));
      v[j] *= v[j] < 0.0f ? e : 1.0f - e;
    }
    if (__builtin_expect(least < -12.5f, false)) {  // E leaves the normal range at -13
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (in[j] < -12.5f) {
          const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(in[j], -0.5f * 0.70710678118654752f, 1.0f));
          const float p = gelu_poly(t);
          v[j] = far_exp2_mul(in[j] * t, __builtin_fmaf(-0.5f * kLog2e * in[j], in[j], p));
        }
    }
    return;
  }
  // silu, gelu_tanh: s = v or 2 u
  constexpr float c1 = 1.59576912160573078f, c3 = 0.0713548162726009f;
  auto sigmoid = [&](auto tanh_t) {
    constexpr bool tanh = decltype(tanh_t)::value;
    constexpr float far = tanh ? -9.9f : kFar;  // 2 u = -87 at -10.0
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float s = -kLog2e * v[j];
      if (tanh) s *= __builtin_fmaf(v[j] * v[j], c3, c1);
      v[j] *= __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(s));
    }
    if (__builtin_expect(least < far, false)) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        float s = kLog2e * in[j];
        if (tanh) s *= __builtin_fmaf(in[j] * in[j], c3, c1);
        if (in[j] < far) v[j] = far_exp2_mul(in[j], s);
      }
    }
  };
  if (act == kActGeluTanh) sigmoid(std::true_type{});
  else sigmoid(std::false_type{});
}

}  // namespace awq
