// Product of microscaled operands with bias, activation and residual in its
// epilogue: Y = act(A W^T + bias) + residual, rounded once, or quantized to blocks.
// The kernels and their choice are the product's (mx_product.h, mx_tiles.h); sums of
// K ranges are joined by a second launch, which then has the epilogue.
//
// One token, 6144 x 4096: 5.0 us (13 MB of weights; the product's time).  8192 x 4096 x
// 4096 in 4 bits with a residual: 100 us, the product alone 76 (the residual's 67 MB
// arrive while the last stages are multiplied, what is stored is waited for); 4096 x
// 12288 x 4096 in 8 bits with bias and GELU to 8 bits: 183-186 us (2.2 PFLOP/s), the
// product alone 156-175 (activation and quantization are 26 and 12 operations a value,
// for which the matrix cores wait).  A launch of its own for them would move 200 MB, 40
// us, and 150 MB, 30 us.  With the product's time, 8 bits: 256 x 4096 x 4096 with a residual
// 11.1 us (9.5), 256 x 12288 x 4096 with bias and GELU to 8 bits 24.5 (18.6), 1024 x 12288 x
// 4096 with them 63 (47), 1024 x 4096 x 12288 with a residual 54-58 (52).
#include <algorithm>

#include "awq_launch.h"
#include "mx_product.h"

namespace awq {

// Sum over z, in order, of part[z] (fp32 [M, ld_p] each), then the epilogue: 8 outputs a thread
__global__ __launch_bounds__(256) void mx_reduce_epi_kernel(const float* __restrict__ part, int n_split, int64_t M,
                                                            int64_t N, int64_t ld_p, void* __restrict__ Y,
                                                            int64_t ld_y, const Epilogue x) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t m = i / (ld_p / 8), n = 8 * (i % (ld_p / 8));
  if (m >= M) return;  // whole blocks of 32 together: ld_p = N where the result is quantized
  Raw8 bias = {};
  if (x.bias != nullptr) bias = load_raw8(x.bias, n, x.bias_dtype, N - n);
  uint4 r = make_uint4(0, 0, 0, 0);
  if (x.R != nullptr && x.r_dtype != 2) r = load_raw8(x.R, m * x.ld_r + n, x.r_dtype, N - n).lo;
  float4 p[kMaxRanges][2];
#pragma unroll
  for (int z = 0; z < kMaxRanges; ++z)
    if (z < n_split) {
      p[z][0] = *(const float4*)(part + (z * M + m) * ld_p + n);
      p[z][1] = *(const float4*)(part + (z * M + m) * ld_p + n + 4);
    }
  float v[8] = {p[0][0].x, p[0][0].y, p[0][0].z, p[0][0].w, p[0][1].x, p[0][1].y, p[0][1].z, p[0][1].w};
#pragma unroll
  for (int z = 1; z < kMaxRanges; ++z)
    if (z < n_split) {
      const float f[8] = {p[z][0].x, p[z][0].y, p[z][0].z, p[z][0].w, p[z][1].x, p[z][1].y, p[z][1].z, p[z][1].w};
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += f[j];
    }
  if (x.bias != nullptr) add_raw8(v, bias, x.bias_dtype);
  const OutRow o = out_row(x, Y, ld_y, m, n, N);
  if (x.R != nullptr) finish8<true>(x, v, r, o, N - n, n < N);
  else finish8<false>(x, v, r, o, N - n, n < N);
}

static int64_t part_ld8(int64_t N) { return (N + 7) / 8 * 8; }

size_t mx_linear_workspace(int a_fmt, int64_t M, int64_t N, int64_t K) {
  const MxTiling t = mx_tiling(a_fmt, M, N, K);
  return t.tile != kBigTile && t.ranges > 1 ? (size_t)t.ranges * M * part_ld8(N) * sizeof(float)
                                            : mx_matmul_workspace(a_fmt, M, N, K);
}

struct LinearArgs {
  const uint8_t *A, *as, *W, *ws;
  int64_t M, N, K;
  void* Y;
  int64_t ld_y;
  Epilogue x;
};

template <int AF>
static void linear_few(const LinearArgs& p, hipStream_t stream) {
  FewTile f = few_tile(AF, p.M, p.N);
  if (p.x.out > 2) f.tiles = 2;  // whole blocks of 32 outputs
  if (f.rows == 24 && f.tiles == 2) f.rows = 32;
  const int64_t a_row = AF == kMxFp8 ? p.K : p.K / 2, y_bytes = p.x.out == 2 ? 4 : 2;
  const int64_t r_bytes = p.x.r_dtype == 2 ? 4 : 2, c_row = p.x.out == kOutFp4 ? p.N / 2 : p.N;
  constexpr int64_t kRows = 65535 * 4;  // of a launch: the grid's second dimension holds 65535 blocks
  for (int64_t m = 0; m < p.M; m += kRows) {
    const int64_t n_rows = std::min(p.M - m, kRows);
    const dim3 grid((unsigned)tiles_of(p.N, 16 * f.tiles), (unsigned)tiles_of(n_rows, f.rows));
    Epilogue x = p.x;
    if (x.R != nullptr) x.R = (const uint8_t*)x.R + m * x.ld_r * r_bytes;
    if (x.out > 2) x.codes += m * c_row, x.scales += m * (p.N / kMxBlock);
    void* Y = x.out > 2 ? nullptr : (uint8_t*)p.Y + m * p.ld_y * y_bytes;
#define AWQ_FEW(AR, NT, ST, OCC)                                                                                    \
  mx_few_kernel<AF, AR, NT, ST, OCC, Epilogue><<<grid, kFewWaves * kWave, 0, stream>>>(                              \
      p.A + m * a_row, p.as + m * (p.K / kMxBlock), n_rows, p.W, p.ws, p.N, p.K, Y, p.ld_y, 0, x)
    constexpr int kOcc32 = AF == kMxFp8 ? 2 : 4;  // the LDS of 32 rows holds one or two blocks
    if (f.rows == 4 && f.tiles == 1) AWQ_FEW(4, 1, 4, 4);
    else if (f.rows == 4) AWQ_FEW(4, 2, 4, 2);
    else if (f.rows == 16 && f.tiles == 1) AWQ_FEW(16, 1, 2, 4);
    else if (f.rows == 16) AWQ_FEW(16, 2, 2, 4);
    else if (f.tiles == 2) AWQ_FEW(32, 2, 2, 2);
    else if (f.rows == 32) AWQ_FEW(32, 1, 2, kOcc32);
    else if constexpr (AF == kMxFp8) AWQ_FEW(24, 1, 2, 2);
#undef AWQ_FEW
  }
}

template <int AF, class X>
static void linear_tiles(const MxTiling& t, const LinearArgs& p, void* Y, int64_t ld_y, const X& x, hipStream_t stream) {
  const int n_mt = (int)tiles_of(p.M, t.tile), n_nt = (int)tiles_of(p.N, t.tile);
  const dim3 g((unsigned)(n_mt * n_nt), (unsigned)t.ranges);
#define AWQ_TILE(BM, NS, OCC)                                                                                    \
  mx_tile_kernel<AF, 2, BM, BM, 2, 2, NS, OCC, X><<<g, 4 * kWave, 0, stream>>>(p.A, p.as, p.M, p.W, p.ws, p.N, p.K, \
                                                                               n_mt, n_nt, 4, t.split, Y, ld_y, x)
  if (t.tile == 64 && tile_slots(t, p.M, p.N) == 6) AWQ_TILE(64, 6, 2);
  else if (t.tile == 64) AWQ_TILE(64, 3, 4);
  else AWQ_TILE(128, 3, 2);
#undef AWQ_TILE
}

template <int AF, class X>
static void linear_big(const LinearArgs& p, const uint32_t* sc, int n_mt, int n_nt, const X& x, hipStream_t stream) {
  const int64_t m_pad = (int64_t)n_mt * kBigTile, rows = m_pad + (int64_t)n_nt * kBigTile;
  if constexpr (AF == kMxFp8)
    mx_big8_kernel<0, X><<<(unsigned)std::min(n_mt * n_nt, 256), 512, 0, stream>>>(
        p.A, p.M, p.W, p.N, p.K, sc, m_pad, rows, n_mt, n_nt, 4, p.Y, p.ld_y, x);
  else
    mx_big_kernel<0, X><<<(unsigned)(n_mt * n_nt), 512, 0, stream>>>(p.A, p.M, p.W, p.N, p.K, sc, m_pad, rows, n_mt, n_nt,
                                                                     4, p.Y, p.ld_y, x);
}

template <int AF>
static void linear_launch(const LinearArgs& p, void* work, hipStream_t stream) {
  const MxTiling t = mx_tiling(AF, p.M, p.N, p.K);
  if (t.tile == 0) {
    linear_few<AF>(p, stream);
  } else if (t.tile == kBigTile) {
    const int n_mt = (int)tiles_of(p.M, kBigTile), n_nt = (int)tiles_of(p.N, kBigTile), kb = (int)(p.K / kMxBlock);
    const int64_t m_pad = (int64_t)n_mt * kBigTile, rows = m_pad + (int64_t)n_nt * kBigTile;
    constexpr int SB = (AF == kMxFp8 ? kMxStage : kBigStage) / kMxBlock;
    uint32_t* sc = (uint32_t*)work;
    stage_scales_kernel<SB><<<dim3((unsigned)(rows / 256), (unsigned)((kb + 15) / 16)), 256, 0, stream>>>(
        p.as, p.M, p.ws, p.N, kb, m_pad, rows, sc);
    if (p.x.R != nullptr) linear_big<AF, Epilogue>(p, sc, n_mt, n_nt, {p.x}, stream);
    else linear_big<AF, EpilogueAlone>(p, sc, n_mt, n_nt, {p.x}, stream);
  } else if (t.ranges == 1) {
    if (p.x.R != nullptr) linear_tiles<AF, Epilogue>(t, p, p.Y, p.ld_y, {p.x}, stream);
    else linear_tiles<AF, EpilogueAlone>(t, p, p.Y, p.ld_y, {p.x}, stream);
  } else {
    const int64_t ld_p = part_ld8(p.N);
    linear_tiles<AF, NoExtra>(t, p, work, ld_p, NoExtra(), stream);
    mx_reduce_epi_kernel<<<(unsigned)((p.M * (ld_p / 8) + 255) / 256), 256, 0, stream>>>((const float*)work, t.ranges, p.M,
                                                                                        p.N, ld_p, p.Y, p.ld_y, p.x);
  }
}

hipError_t launch_mx_linear(const void* A, const uint8_t* as, int a_fmt, int64_t M, const void* W, const uint8_t* ws,
                            int64_t N, int64_t K, const void* bias, int bias_dtype, int act, const void* residual,
                            int r_dtype, int64_t ld_r, void* Y, int64_t ld_y, int out, void* codes, uint8_t* scales,
                            void* work, hipStream_t stream) {
  const LinearArgs p = {(const uint8_t*)A, as, (const uint8_t*)W, ws, M, N, K, Y, ld_y,
                        {bias, bias_dtype, act, residual, r_dtype, ld_r, out, (uint8_t*)codes, scales}};
  if (a_fmt == kMxFp8) linear_launch<kMxFp8>(p, work, stream);
  else linear_launch<kMxFp4>(p, work, stream);
  return hipGetLastError();
}

}  // namespace awq
