// Product of microscaled operands: Y [M, N] = A [M, K] W [N, K]^T, A in e4m3 or
// e2m1 blocks, W in e2m1 blocks, both row-major along K with one scale byte per
// 32 values.  The matrix cores take the codes and the scale bytes as they are
// (v_mfma_scale_f32_16x16x128_f8f6f4): no value is dequantized in registers.
#include "awq_launch.h"
#include "mx_product.h"

namespace awq {

// Y = sum over z, in order, of part[z] (fp32 [M, ld_p] each): 4 outputs a thread
template <int YT>
__global__ __launch_bounds__(256) void mx_reduce_kernel(const float* __restrict__ part, int n_split, int64_t M,
                                                        int64_t N, int64_t ld_p, void* __restrict__ Y, int64_t ld_y) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t m = i / (ld_p / 4), n = 4 * (i % (ld_p / 4));
  if (m >= M) return;
  float4 p[kMaxRanges];
#pragma unroll
  for (int z = 0; z < kMaxRanges; ++z)
    if (z < n_split) p[z] = *(const float4*)(part + (z * M + m) * ld_p + n);
  float4 v = p[0];
#pragma unroll
  for (int z = 1; z < kMaxRanges; ++z)
    if (z < n_split) v.x += p[z].x, v.y += p[z].y, v.z += p[z].z, v.w += p[z].w;
  const float f[4] = {v.x, v.y, v.z, v.w};
  const int64_t at = m * ld_y + n;
  if (n + 4 <= N) {
    if constexpr (YT == 2) st_any((float*)Y + at, v);
    else
      st_any((uint16_t*)Y + at,
             make_uint2(f2x<YT>(f[0]) | (f2x<YT>(f[1]) << 16), f2x<YT>(f[2]) | (f2x<YT>(f[3]) << 16)));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < N) store_y(Y, at + e, f[e], YT);
  }
}

static int64_t part_ld(int64_t N) { return (N + 3) / 4 * 4; }

static int64_t big_scale_words(int a_fmt, int64_t M, int64_t N, int64_t K) {
  const int64_t words = a_fmt == kMxFp8 ? (K + kMxStage - 1) / kMxStage : (K + kBigStage - 1) / kBigStage * 2;
  return (tiles_of(M, kBigTile) + tiles_of(N, kBigTile)) * kBigTile * words;
}

size_t mx_matmul_workspace(int a_fmt, int64_t M, int64_t N, int64_t K) {
  const MxTiling t = mx_tiling(a_fmt, M, N, K);
  if (t.tile == kBigTile) return (size_t)big_scale_words(a_fmt, M, N, K) * sizeof(uint32_t);
  return t.ranges > 1 ? (size_t)t.ranges * M * part_ld(N) * sizeof(float) : 0;
}

template <int AF>
static void few_launch(const uint8_t* A, const uint8_t* as, int64_t M, const uint8_t* W, const uint8_t* ws, int64_t N,
                       int64_t K, void* Y, int64_t ld_y, int y_dtype, hipStream_t stream) {
  const FewTile f = few_tile(AF, M, N);
  const int64_t a_row = AF == kMxFp8 ? K : K / 2, y_bytes = y_dtype == 2 ? 4 : 2;
  constexpr int64_t kRows = 65535 * 4;  // of a launch: the grid's second dimension holds 65535 blocks
  for (int64_t m = 0; m < M; m += kRows) {
    const int64_t n_rows = M - m < kRows ? M - m : kRows;
#define AWQ_FEW(AR, NT, ST, OCC)                                                                                   \
  mx_few_kernel<AF, AR, NT, ST, OCC><<<dim3((unsigned)((N + 16 * NT - 1) / (16 * NT)), (unsigned)((n_rows + AR - 1) / AR)), \
                                       kFewWaves * kWave, 0, stream>>>(A + m * a_row, as + m * (K / kMxBlock), n_rows, \
                                                                       W, ws, N, K, (uint8_t*)Y + m * ld_y * y_bytes, \
                                                                       ld_y, y_dtype)
    constexpr int kOcc32 = AF == kMxFp8 ? 2 : 4;  // the LDS of 32 rows holds one or two blocks
    if (f.rows == 4) AWQ_FEW(4, 1, 4, 4);
    else if (f.rows == 16 && f.tiles == 1) AWQ_FEW(16, 1, 2, 4);
    else if (f.rows == 16) AWQ_FEW(16, 2, 2, 4);
    else if (f.tiles == 2) AWQ_FEW(32, 2, 2, 2);
    else if (f.rows == 32) AWQ_FEW(32, 1, 2, kOcc32);
    else if constexpr (AF == kMxFp8) AWQ_FEW(24, 1, 2, 2);
  }
#undef AWQ_FEW
}

template <int AF, int YT>
static void tile_launch(const MxTiling& t, const uint8_t* A, const uint8_t* as, int64_t M, const uint8_t* W,
                        const uint8_t* ws, int64_t N, int64_t K, void* Y, int64_t ld_y, hipStream_t stream) {
  const int n_mt = (int)tiles_of(M, t.tile), n_nt = (int)tiles_of(N, t.tile);
  const dim3 g((unsigned)(n_mt * n_nt), (unsigned)t.ranges);
#define AWQ_TILE(BM, BN, WM, WN, NS, OCC)                                                                           \
  mx_tile_kernel<AF, YT, BM, BN, WM, WN, NS, OCC><<<g, WM * WN * kWave, 0, stream>>>(A, as, M, W, ws, N, K, n_mt, n_nt, 4, \
                                                                               t.split, Y, ld_y)
  if (t.tile == 64 && tile_slots(t, M, N) == 6) AWQ_TILE(64, 64, 2, 2, 6, 2);
  else if (t.tile == 64) AWQ_TILE(64, 64, 2, 2, 3, 4);
  else AWQ_TILE(128, 128, 2, 2, 3, 2);
#undef AWQ_TILE
}

template <int AF, int YT>
static void big_launch(const uint8_t* A, const uint8_t* as, int64_t M, const uint8_t* W, const uint8_t* ws, int64_t N,
                       int64_t K, void* Y, int64_t ld_y, uint32_t* sc, hipStream_t stream) {
  const int n_mt = (int)tiles_of(M, kBigTile), n_nt = (int)tiles_of(N, kBigTile), kb = (int)(K / kMxBlock);
  const int64_t m_pad = (int64_t)n_mt * kBigTile, rows = m_pad + (int64_t)n_nt * kBigTile;
  constexpr int SB = (AF == kMxFp8 ? kMxStage : kBigStage) / kMxBlock;
  stage_scales_kernel<SB><<<dim3((unsigned)(rows / 256), (unsigned)((kb + 15) / 16)), 256, 0, stream>>>(
      as, M, ws, N, kb, m_pad, rows, sc);
  if constexpr (AF == kMxFp8)
    mx_big8_kernel<YT><<<(unsigned)(n_mt * n_nt < 256 ? n_mt * n_nt : 256), 512, 0, stream>>>(
        A, M, W, N, K, sc, m_pad, rows, n_mt, n_nt, 4, Y, ld_y);
  else
    mx_big_kernel<YT><<<(unsigned)(n_mt * n_nt), 512, 0, stream>>>(A, M, W, N, K, sc, m_pad, rows, n_mt, n_nt, 4, Y,
                                                                   ld_y);
}

template <int AF, int YT>
static void product_launch(const uint8_t* A, const uint8_t* as, int64_t M, const uint8_t* W, const uint8_t* ws,
                           int64_t N, int64_t K, void* Y, int64_t ld_y, float* part, hipStream_t stream) {
  const MxTiling t = mx_tiling(AF, M, N, K);
  if (t.tile == 0) {
    few_launch<AF>(A, as, M, W, ws, N, K, Y, ld_y, YT, stream);
  } else if (t.tile == kBigTile) {
    if constexpr (AF == kMxFp4 || YT != 2) big_launch<AF, YT>(A, as, M, W, ws, N, K, Y, ld_y, (uint32_t*)part, stream);
  } else if (t.ranges == 1) {
    tile_launch<AF, YT>(t, A, as, M, W, ws, N, K, Y, ld_y, stream);
  } else {
    const int64_t ld_p = part_ld(N);
    tile_launch<AF, 2>(t, A, as, M, W, ws, N, K, part, ld_p, stream);
    mx_reduce_kernel<YT><<<(unsigned)((M * (ld_p / 4) + 255) / 256), 256, 0, stream>>>(part, t.ranges, M, N, ld_p, Y,
                                                                                      ld_y);
  }
}

hipError_t launch_mx_matmul(const void* A, const uint8_t* as, int a_fmt, int64_t M, const void* W, const uint8_t* ws,
                            int64_t N, int64_t K, void* Y, int64_t ld_y, int y_dtype, void* work, hipStream_t stream) {
#define AWQ_PRODUCT(F, T) \
  product_launch<F, T>((const uint8_t*)A, as, M, (const uint8_t*)W, ws, N, K, Y, ld_y, (float*)work, stream)
  if (a_fmt == kMxFp8) {
    if (y_dtype == 0) AWQ_PRODUCT(kMxFp8, 0); else AWQ_PRODUCT(kMxFp8, 1);
  } else {
    if (y_dtype == 0) AWQ_PRODUCT(kMxFp4, 0);
    else if (y_dtype == 1) AWQ_PRODUCT(kMxFp4, 1);
    else AWQ_PRODUCT(kMxFp4, 2);
  }
#undef AWQ_PRODUCT
  return hipGetLastError();
}

}  // namespace awq
