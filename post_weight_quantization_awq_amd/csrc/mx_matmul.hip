// Product of microscaled operands: Y [M, N] = A [M, K] W [N, K]^T, A in e4m3 or
// e2m1 blocks, W in e2m1 blocks, both row-major along K with one scale byte per
// 32 values.  The matrix cores take the codes and the scale bytes as they are
// (v_mfma_scale_f32_16x16x128_f8f6f4): no value is dequantized in registers.
#include "awq_launch.h"
#include "mx_device.h"

namespace awq {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// Operand registers of the 16x16x128 product, lane l of a wave: row l % 16,
// h = l / 16.  4-bit codes: the 32 values from 32 h on (16 bytes).  8-bit codes:
// the 16 values from 16 h on, then the 16 from 64 + 16 h on.  The scale of lane
// l is that of the row's block h for both.  W is the first operand, so a lane
// ends up with 4 consecutive outputs 4 h .. 4 h + 3 of token l % 16.
template <int AF>
__device__ __forceinline__ f32x4 mfma_mx(const i32x8 w, const i32x8 a, f32x4 c, int ws, int as) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, c, 4, AF == kMxFp8 ? 0 : 4, 0, ws, 0, as);
}
__device__ __forceinline__ i32x8 lo4(const uint4 u) {
  return (i32x8){(int)u.x, (int)u.y, (int)u.z, (int)u.w, 0, 0, 0, 0};
}
__device__ __forceinline__ i32x8 both4(const uint4 u, const uint4 v) {
  return (i32x8){(int)u.x, (int)u.y, (int)u.z, (int)u.w, (int)v.x, (int)v.y, (int)v.z, (int)v.w};
}

// y_dtype: 0 fp16, 1 bf16, 2 fp32
__device__ __forceinline__ void store_y(void* Y, int64_t at, float v, int y_dtype) {
  if (y_dtype == 2) ((float*)Y)[at] = v;
  else ((uint16_t*)Y)[at] = (uint16_t)(y_dtype == 0 ? f2x<0>(v) : f2x<1>(v));
}

// ---------------------------------------------------------------------------
// Few tokens: a block holds 16 outputs and 16 MT tokens; its 8 waves take K
// steps of 128 in turn and their sums are added in wave order through LDS.
// ---------------------------------------------------------------------------
constexpr int kFewWaves = 8;

template <int AF, int MT>
__global__ __launch_bounds__(kFewWaves * kWave) void mx_few_kernel(const uint8_t* __restrict__ A,
                                                                  const uint8_t* __restrict__ as, int64_t M,
                                                                  const uint8_t* __restrict__ W,
                                                                  const uint8_t* __restrict__ ws, int64_t N, int64_t K,
                                                                  void* __restrict__ Y, int64_t ld_y, int y_dtype) {
  __shared__ float red[kFewWaves][MT * 16][17];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, h = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * (16 * MT);
  const int64_t kb = K / kMxBlock;
  const int64_t n = n0 + r < N ? n0 + r : N - 1;  // rows past the end repeat the last one, unused
  const uint8_t* wr = W + n * (K / 2);
  const uint8_t* wsr = ws + n * kb;
  f32x4 acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = (f32x4){0, 0, 0, 0};
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int64_t b0 = 4 * wave; b0 < kb; b0 += 4 * kFewWaves) {
    const bool in = b0 + h < kb;
    const i32x8 w = lo4(in ? *(const uint4*)(wr + 16 * (b0 + h)) : zero);
    const int sw = in ? wsr[b0 + h] : 0;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int64_t m = m0 + 16 * t + r < M ? m0 + 16 * t + r : M - 1;
      const int sa = in ? as[m * kb + b0 + h] : 0;
      i32x8 a;
      if constexpr (AF == kMxFp8) {
        const uint8_t* p = A + m * K + 32 * b0 + 16 * h;
        const bool in0 = b0 + h / 2 < kb, in1 = b0 + 2 + h / 2 < kb;
        a = both4(in0 ? *(const uint4*)p : zero, in1 ? *(const uint4*)(p + 64) : zero);
      } else {
        a = lo4(in ? *(const uint4*)(A + m * (K / 2) + 16 * (b0 + h)) : zero);
      }
      acc[t] = mfma_mx<AF>(w, a, acc[t], sw, sa);
    }
  }
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[wave][16 * t + r][4 * h + e] = acc[t][e];
  __syncthreads();
  for (int i = threadIdx.x; i < MT * 256; i += kFewWaves * kWave) {
    const int t = i >> 4, o = i & 15;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) v += red[w][t][o];
    if (m0 + t < M && n0 + o < N) store_y(Y, (m0 + t) * ld_y + n0 + o, v, y_dtype);
  }
}

size_t mx_matmul_workspace(int a_fmt, int64_t M, int64_t N, int64_t K) {
  (void)a_fmt, (void)M, (void)N, (void)K;
  return 0;
}

template <int AF>
static void few_launch(const uint8_t* A, const uint8_t* as, int64_t M, const uint8_t* W, const uint8_t* ws, int64_t N,
                       int64_t K, void* Y, int64_t ld_y, int y_dtype, hipStream_t stream) {
  const unsigned gx = (unsigned)((N + 15) / 16);
#define AWQ_FEW(MT)                                                                                       \
  mx_few_kernel<AF, MT><<<dim3(gx, (unsigned)((M + 16 * MT - 1) / (16 * MT))), kFewWaves * kWave, 0, stream>>>( \
      A, as, M, W, ws, N, K, Y, ld_y, y_dtype)
  if (M <= 16) AWQ_FEW(1);
  else if (M <= 32) AWQ_FEW(2);
  else AWQ_FEW(4);
#undef AWQ_FEW
}

hipError_t launch_mx_matmul(const void* A, const uint8_t* as, int a_fmt, int64_t M, const void* W, const uint8_t* ws,
                            int64_t N, int64_t K, void* Y, int64_t ld_y, int y_dtype, void* work, hipStream_t stream) {
  (void)work;
  if (a_fmt == kMxFp8)
    few_launch<kMxFp8>((const uint8_t*)A, as, M, (const uint8_t*)W, ws, N, K, Y, ld_y, y_dtype, stream);
  else
    few_launch<kMxFp4>((const uint8_t*)A, as, M, (const uint8_t*)W, ws, N, K, Y, ld_y, y_dtype, stream);
  return hipGetLastError();
}

}  // namespace awq
