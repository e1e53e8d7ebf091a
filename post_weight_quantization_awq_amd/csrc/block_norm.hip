// What stands between two blocks: the norm after the first with its gate, the
// residual's addition with its scale, and the norm before the second, quantized;
// for a block with experts the sum of each token's results, too.
//   y = X[t], or sum_j shares[t][j] X[places[t][j]]    in the order of j
//   z = y / sqrt(mean y^2 + eps) * post                (y without post)
//   h = residual_scale residual + gate z               residual_out = RN(h)
//   v = h / sqrt(mean h^2 + eps) * norm                -> codes, scales
// A row stays in registers from its loads to its codes, so that each input is
// read once: bound by memory, in one launch.  Lanes of a row as in rms_norm_mx:
// a wave or a part of it up to 512 columns, else a block.
#include "awq_launch.h"
#include "mx_device.h"
#include "mx_norm.h"

namespace awq {

// A row of X, or the weighted sum of its rows that a token's places name; places outside X name none.  Rows are
// loaded four at a time, ahead of their sums (one at a time from 16385 columns on, for want of registers).
template <int DT, int CH>
__device__ __forceinline__ void load_sum(const BlockNormArgs& a, int64_t row, int lane, int lanes, int cpr,
                                         float (&y)[CH][8]) {
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) y[c][j] = 0.0f;
  if (a.places == nullptr) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (lane + c * lanes < cpr) unpack8<DT>(ld_stream(a.X + row * a.ld_x + 8 * (lane + c * lanes)), y[c]);
    return;
  }
  constexpr int NP = CH >= 4 ? 1 : 4;
  for (int j0 = 0; j0 < a.top; j0 += NP) {
    uint32_t place[NP];
    float share[NP];
    uint4 x[NP][CH];
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const bool in = j0 + j < a.top;
      place[j] = in ? (uint32_t)a.places[row * a.top + j0 + j] : ~0u;
      share[j] = in ? a.shares[row * a.top + j0 + j] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < NP; ++j)
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if ((int64_t)place[j] < a.x_rows && lane + c * lanes < cpr)
          x[j][c] = ld_stream(a.X + (int64_t)place[j] * a.ld_x + 8 * (lane + c * lanes));
#pragma unroll
    for (int j = 0; j < NP; ++j)
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if ((int64_t)place[j] < a.x_rows && lane + c * lanes < cpr) {
          float f[8];
          unpack8<DT>(x[j][c], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[c][i] = __builtin_fmaf(share[j], f[i], y[c][i]);
        }
  }
}

template <int CH>
__device__ __forceinline__ float squares(const float (&h)[CH][8], int lane, int lanes, int cpr) {
  float sum = 0.0f;
#pragma unroll
  for (int c = 0; c < CH; ++c)
    if (lane + c * lanes < cpr)
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(h[c][j], h[c][j], sum);
  return sum;
}

template <int DT, int FMT, int GL, int CH>
__global__ __launch_bounds__(GL ? 256 : 1024) void block_norm_mx_kernel(const BlockNormArgs a) {
  const int lanes = GL ? GL : (int)blockDim.x;
  const int lane = GL ? (int)threadIdx.x % (GL ? GL : 1) : (int)threadIdx.x;
  const int64_t row = GL ? (int64_t)blockIdx.x * (256 / (GL ? GL : 1)) + (int)threadIdx.x / (GL ? GL : 1)
                         : (int64_t)blockIdx.x;
  const bool live = row < a.rows;
  const int cpr = live ? (int)(a.cols / 8) : 0;  // chunks of the row that there are
  __shared__ float part[2][GL ? 1 : 16];
  constexpr bool kEarly = CH < 8;  // the residual ahead of the sums, but for the longest rows, for want of registers
  uint4 res[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c)
    if (kEarly && lane + c * lanes < cpr) res[c] = ld_stream(a.R + row * a.ld_r + 8 * (lane + c * lanes));
  float h[CH][8];
  load_sum<DT, CH>(a, row, lane, lanes, cpr, h);
  if (a.post != nullptr) {
    const float r = row_scale<GL, CH>(h, squares<CH>(h, lane, lanes, cpr), live, lane, lanes, cpr, a.cols, a.eps,
                                      part[0]);
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (lane + c * lanes < cpr) {
        float w[8];
        load_weight8(a.post, a.post_dtype, 8 * (int64_t)(lane + c * lanes), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[c][j] = h[c][j] * r * w[j];
      }
  }
#pragma unroll
  for (int c = 0; c < CH; ++c)
    if (lane + c * lanes < cpr) {
      const int64_t col = 8 * (int64_t)(lane + c * lanes);
      if (a.gate != nullptr) {
        float g[8];
        load_weight8(a.gate, a.gate_dtype, row * a.ld_g + col, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[c][j] *= g[j];
      }
      if constexpr (!kEarly) res[c] = ld_stream(a.R + row * a.ld_r + col);
      float r[8];
      unpack8<DT>(res[c], r);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[c][j] = __builtin_fmaf(a.residual_scale, r[j], h[c][j]);
      st_any(a.RO + row * a.ld_ro + col, pack8<DT>(h[c]));
    }
  const float r =
      row_scale<GL, CH>(h, squares<CH>(h, lane, lanes, cpr), live, lane, lanes, cpr, a.cols, a.eps, part[1]);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int k = lane + c * lanes;
    if (k < cpr) {
      float w[8];
      load_weight8(a.norm, a.norm_dtype, 8 * (int64_t)k, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[c][j] = h[c][j] * r * w[j];
      uint32_t codes[2];
      const uint32_t byte = mx_quantize8<FMT>(h[c], codes);
      mx_store8<FMT>(codes, byte, a.codes, a.scales, row * cpr + k);
    }
  }
}

template <int DT, int FMT>
static void block_norm_launch(const BlockNormArgs& a, hipStream_t stream) {
  const int64_t cpr = a.cols / 8;
#define AWQ_NORM_W(GL, CH) \
  block_norm_mx_kernel<DT, FMT, GL, CH><<<(unsigned)((a.rows + 256 / GL - 1) / (256 / GL)), 256, 0, stream>>>(a)
#define AWQ_NORM_B(CH)                                                                                               \
  block_norm_mx_kernel<DT, FMT, 0, CH><<<(unsigned)a.rows, (unsigned)(((cpr + CH - 1) / CH + 63) / 64 * 64), 0, stream>>>( \
      a)
  if (cpr <= 4) AWQ_NORM_W(4, 1);
  else if (cpr <= 8) AWQ_NORM_W(8, 1);
  else if (cpr <= 16) AWQ_NORM_W(16, 1);
  else if (cpr <= 32) AWQ_NORM_W(32, 1);
  else if (cpr <= 64) AWQ_NORM_W(32, 2);
  else if (cpr <= 512) AWQ_NORM_B(2);
  else if (cpr <= 1024) AWQ_NORM_B(1);
  else if (cpr <= 2048) AWQ_NORM_B(2);
  else if (cpr <= 4096) AWQ_NORM_B(4);
  else AWQ_NORM_B(8);
#undef AWQ_NORM_W
#undef AWQ_NORM_B
}

hipError_t launch_block_norm_mx(const BlockNormArgs& a, int dt, int fmt, hipStream_t stream) {
  if (dt == 0) {
    if (fmt == kMxFp8) block_norm_launch<0, kMxFp8>(a, stream); else block_norm_launch<0, kMxFp4>(a, stream);
  } else {
    if (fmt == kMxFp8) block_norm_launch<1, kMxFp8>(a, stream); else block_norm_launch<1, kMxFp4>(a, stream);
  }
  return hipGetLastError();
}

}  // namespace awq
