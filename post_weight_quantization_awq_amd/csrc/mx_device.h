// Device-side helpers of the microscaled (MX) formats (gfx950, wave64).
//
// A row is cut into blocks of 32 values that share one power of two 2^e, stored
// as the byte e + 127 (e8m0).  The elements are e4m3 (8 bits, largest 448) or
// e2m1 (4 bits, largest 6; two to a byte, the even column in the low half).
//   e = floor(log2 max|v|) - emax, emax = 8 (e4m3) or 2 (e2m1), at least -127;
//   element = v / 2^e rounded to nearest even and saturated.
// The maximum of a block then lands in [2^emax, 2^(emax + 1)): the elements
// above the format's largest value saturate.  A block that holds a NaN or an
// infinity gets the scale byte 255 (NaN) and zero elements, so that everything
// computed from it is NaN.
#pragma once

#include "awq_device.h"
#include "mx_format.h"

namespace awq {

typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2v __attribute__((ext_vector_type(2)));

// 16-bit input types: 0 fp16, 1 bf16 (AWQ_F16, AWQ_BF16)
template <int DT>
__device__ __forceinline__ float x2f(uint32_t h) {
  if constexpr (DT == 0) return h2f((uint16_t)h);
  else return bf2f((uint16_t)h);
}
template <int DT>
__device__ __forceinline__ uint32_t f2x(float f) {
  if constexpr (DT == 0) return f2h_bits(f);
  else return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)f);  // nearest even, NaN stays NaN
}
template <int DT>
__device__ __forceinline__ void unpack8(const uint4 u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = x2f<DT>(w[j] & 0xFFFFu);
    f[2 * j + 1] = x2f<DT>(w[j] >> 16);
  }
}
template <int DT>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = f2x<DT>(f[2 * j]) | (f2x<DT>(f[2 * j + 1]) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 bytes from / to an address aligned to its elements only
template <class T>
__device__ __forceinline__ T ld_any(const void* p) {
  T v;
  __builtin_memcpy(&v, p, sizeof(T));
  return v;
}
// 16 bytes that are read once: the nontemporal hint keeps them from displacing what is read again
typedef uint32_t u32x4any __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  const u32x4any v = __builtin_nontemporal_load((const u32x4any*)p);
  return make_uint4(v.x, v.y, v.z, v.w);
}
template <class T>
__device__ __forceinline__ void st_any(void* p, const T v) {
  __builtin_memcpy(p, &v, sizeof(T));
}

// Scale of a block whose largest |v| has the bit pattern `top` (NaN patterns
// order above infinity, infinity above the finite values).  floor(log2) of a
// normal value is its exponent field less 127; zeros and subnormals fall below
// the smallest scale anyway.
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top) {
  constexpr int emax = FMT == kMxFp8 ? 8 : 2;
  const int b = (int)(top >> 23) - emax;
  return top >= 0x7F800000u ? kMxNan : (uint32_t)(b > 0 ? b : 0);
}
// 2^(byte - 127); byte 255 gives NaN
__device__ __forceinline__ float mx_unit(uint32_t byte) {
  return __builtin_bit_cast(float, byte == 0 ? 0x00400000u : byte == kMxNan ? 0x7FC00000u : byte << 23);
}

// Quantizes the 8 values of a lane; the block of 32 is an aligned group of 4
// lanes, all active.  Returns the scale byte; codes[0..1] hold 8 e4m3 codes or
// codes[0] 8 e2m1 codes.
template <int FMT>
__device__ __forceinline__ uint32_t mx_quantize8(float (&v)[8], uint32_t (&codes)[2]) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, __builtin_bit_cast(uint32_t, v[j]) & 0x7FFFFFFFu);
  top = max(top, dpp_u<0xB1>(top));
  top = max(top, dpp_u<0x4E>(top));
  const uint32_t byte = mx_scale_byte<FMT>(top);
  const bool bad = byte == kMxNan;
  const float unit = mx_unit(byte);
  if constexpr (FMT == kMxFp8) {
    const float lim = 448.0f * unit;  // the conversion does not saturate
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __builtin_amdgcn_fmed3f(v[j], -lim, lim);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      s16x2 r = {0, 0};
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, v[4 * j], v[4 * j + 1], unit, false);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, v[4 * j + 2], v[4 * j + 3], unit, true);
      codes[j] = bad ? 0u : __builtin_bit_cast(uint32_t, r);
    }
  } else {
    uint32_t r = 0;  // this conversion saturates at 6
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], unit, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], unit, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], unit, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], unit, 3);
    codes[0] = bad ? 0u : r;
  }
  return byte;
}

// Stores a lane's 8 codes and, from the first lane of each block, its scale.
// chunk: index of the 8 values in the contiguous [rows, cols] result.
template <int FMT>
__device__ __forceinline__ void mx_store8(const uint32_t (&codes)[2], uint32_t byte, uint8_t* __restrict__ out,
                                          uint8_t* __restrict__ scales, int64_t chunk) {
  if constexpr (FMT == kMxFp8) *(uint2*)(out + 8 * chunk) = make_uint2(codes[0], codes[1]);
  else *(uint32_t*)(out + 4 * chunk) = codes[0];
  if ((chunk & 3) == 0) scales[chunk >> 2] = (uint8_t)byte;
}

}  // namespace awq
