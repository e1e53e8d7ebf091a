// The RMS norm of a row that stays in registers.
#pragma once

#include "mx_device.h"

namespace awq {

__device__ __forceinline__ void load_weight8(const void* w, int dt, int64_t col, float (&f)[8]) {
  if (dt == 2) {
    *(float4*)&f[0] = ld_any<float4>((const float*)w + col);
    *(float4*)&f[4] = ld_any<float4>((const float*)w + col + 4);
  } else {
    const uint4 u = ld_any<uint4>((const uint16_t*)w + col);
    if (dt == 0) unpack8<0>(u, f);
    else unpack8<1>(u, f);
  }
}

// A row's lanes: with GL = 0 the block (blockDim.x of them), else GL lanes of a wave.  Their values, none of
// them below 0, joined by `f`; the same result in each of them.
template <int GL, class F>
__device__ __forceinline__ float row_total(float v, float* part, F f) {
  if constexpr (GL != 0) {
#pragma unroll
    for (int m = GL / 2; m >= 1; m >>= 1) v = f(v, __shfl_xor(v, m, kWave));
    return v;
  } else {
#pragma unroll
    for (int m = kWave / 2; m >= 1; m >>= 1) v = f(v, __shfl_xor(v, m, kWave));
    const int wave = (int)threadIdx.x >> 6, nw = (int)blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0) part[wave] = v;
    __syncthreads();
    v = 0.0f;
    for (int i = 0; i < nw; ++i) v = f(v, part[i]);
    return v;
  }
}

// The same for a block whose upper half has the second chunks: the result of half as many lanes that have two chunks
// each and join theirs first.  part: 16 floats, and one for each lane of the upper half.
template <class F>
__device__ __forceinline__ float row_total_halves(float v, float* part, F f) {
  const int half = (int)blockDim.x / 2, lane = (int)threadIdx.x;
  if (lane >= half) part[16 + lane - half] = v;
  __syncthreads();
  if (lane < half) {  // whole waves
    v = f(v, part[16 + lane]);
#pragma unroll
    for (int m = kWave / 2; m >= 1; m >>= 1) v = f(v, __shfl_xor(v, m, kWave));
    if ((lane & 63) == 0) part[lane >> 6] = v;
  }
  __syncthreads();
  v = 0.0f;
  for (int i = 0; i < half / kWave; ++i) v = f(v, part[i]);
  return v;
}

// Rows whose squares leave fp32's range: the mean is infinite, or so small that squares lost below the range count
// (those are off by at most 2^-150 each, 2^-134 for the longest row, 2^-34 of the least sum or eps taken).  They are
// brought to the middle of the range first, by the power of two of their largest value or, where that is less,
// of eps's root.  Rows that hold an infinity or a NaN stay as they are: 1 / sqrt(inf) = 0 times an infinity is NaN.
constexpr float kNormLeast = 0x1p-100f;

// 1 / sqrt(mean h^2 + eps) of a row whose lanes hold h and their sums of squares.  Where those leave fp32's range h
// is scaled, and what is returned goes with the scaled h.  N sums a lane: of all its chunks, or of each.  part: 16
// floats of LDS with GL = 0, and with HALVES as there.
template <int GL, int CH, bool HALVES = false, int N>
__device__ __forceinline__ float row_scale(float (&h)[CH][8], float (&sums)[N], bool live, int lane, int lanes, int cpr,
                                           int64_t cols, float eps, float* part) {
  static_assert(N == 1 || N == CH, "a sum for all of the lane's chunks or for each");
  auto total = [&](float v, auto f) {
    if constexpr (HALVES) return row_total_halves(v, part, f);
    else return row_total<GL>(v, part, f);
  };
  auto add = [](float x, float y) { return x + y; };
  auto joined = [&]() {
    float v = sums[0];
#pragma unroll
    for (int c = 1; c < N; ++c) v += sums[c];
    return v;
  };
  float sum = total(joined(), add);
  float mean = sum / (float)cols + eps;
  // the same for the whole row
  if (__builtin_expect(!(mean < HUGE_VALF) || (sum < kNormLeast && eps < kNormLeast), false)) {
    uint32_t top = 0;
    if constexpr (GL == 0) __syncthreads();  // the sum has been read
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (live && lane + c * lanes < cpr)
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, __builtin_bit_cast(uint32_t, h[c][j]) & 0x7FFFFFFFu);
    top = __builtin_bit_cast(uint32_t, total(__builtin_bit_cast(float, top), [](float x, float y) {
      return __builtin_bit_cast(float, max(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y)));
    }));
    if (top < 0x7F800000u) {
      int k2 = (int)(top >> 23) - 127;
      if (eps > 0.0f) k2 = max(k2, ((int)(__builtin_bit_cast(uint32_t, eps) >> 23) - 127) / 2);
#pragma unroll
      for (int c = 0; c < N; ++c) sums[c] = 0.0f;
      if constexpr (GL == 0) __syncthreads();
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if (live && lane + c * lanes < cpr)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            h[c][j] = __builtin_ldexpf(h[c][j], -k2);
            sums[N == 1 ? 0 : c] = __builtin_fmaf(h[c][j], h[c][j], sums[N == 1 ? 0 : c]);
          }
      sum = total(joined(), add);
      mean = sum / (float)cols + __builtin_ldexpf(eps, -2 * k2);
    }
  }
  return 1.0f / sqrtf(mean);
}

}  // namespace awq
