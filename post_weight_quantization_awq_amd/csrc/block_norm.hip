// What stands between two blocks: the norm after the first with its gate, the
// residual's addition with its scale, and the norm before the second, quantized;
// for a block with experts the sum of each token's results, too.
//   y = X[t], or sum_j shares[t][j] X[places[t][j]]    in the order of j
//   z = y / sqrt(mean y^2 + eps) * post                (y without post)
//   h = residual_scale residual + gate z               residual_out = RN(h)
//   v = h / sqrt(mean h^2 + eps) * norm                -> codes, scales
// A row stays in registers from its loads to its codes, so that each input is
// read once: bound by memory, in one launch.  Lanes of a row as in rms_norm_mx:
// a wave or a part of it up to 512 columns, else a block.  6001 x 4096 with a norm
// and a gate 35.3 us (4.9 TB/s; a large copy 5.1), 4096 x 4096 with a sum of 4 rows
// 39.5 us (5.5 TB/s), one row with a sum of 8 4.6 us.  What the rows in flight leave
// of registers decides: the kernel without the sum has 58, and 88 (38.9 us for the
// first) with the sum's loads in it, so each has a kernel of its own; the weights'
// loads ahead of X cost more registers than they gain.
#include "awq_launch.h"
#include "mx_device.h"
#include "mx_norm.h"

namespace awq {

// A row of X, or the weighted sum of its rows that a token's places name; places outside X name none.  Rows are
// loaded eight at a time, ahead of their sums (four where a lane has two chunks, and one from 16385 columns on, for want
// of registers).
template <int DT, int CH, bool FULL, bool SUM>
__device__ __forceinline__ void load_sum(const BlockNormArgs& a, int64_t row, int lane, int lanes, int cpr,
                                         float (&y)[CH][8]) {
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) y[c][j] = 0.0f;
  if constexpr (!SUM) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (FULL || lane + c * lanes < cpr) unpack8<DT>(ld_stream(a.X + row * a.ld_x + 8 * (lane + c * lanes)), y[c]);
    return;
  }
  constexpr int NP = CH >= 4 ? 1 : CH == 2 ? 4 : 8;
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
        if ((int64_t)place[j] < a.x_rows && (FULL || lane + c * lanes < cpr))
          x[j][c] = ld_stream(a.X + (int64_t)place[j] * a.ld_x + 8 * (lane + c * lanes));
#pragma unroll
    for (int j = 0; j < NP; ++j)
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if ((int64_t)place[j] < a.x_rows && (FULL || lane + c * lanes < cpr)) {
          float f[8];
          unpack8<DT>(x[j][c], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[c][i] = __builtin_fmaf(share[j], f[i], y[c][i]);
        }
  }
}

// 8 weights as they lie in memory
struct Ahead8 {
  uint4 lo, hi;  // hi: of 32-bit ones
};
__device__ __forceinline__ Ahead8 load_ahead(const void* w, int dt, int64_t col) {
  Ahead8 r;
  if (dt == 2) {
    r.lo = ld_any<uint4>((const float*)w + col);
    r.hi = ld_any<uint4>((const float*)w + col + 4);
  } else {
    r.lo = ld_any<uint4>((const uint16_t*)w + col);
  }
  return r;
}
__device__ __forceinline__ void ahead_values(const Ahead8& r, int dt, float (&f)[8]) {
  if (dt == 2) {
    *(uint4*)&f[0] = r.lo;
    *(uint4*)&f[4] = r.hi;
  } else if (dt == 0) {
    unpack8<0>(r.lo, f);
  } else {
    unpack8<1>(r.lo, f);
  }
}

template <int CH, bool FULL, int N>
__device__ __forceinline__ void squares(const float (&h)[CH][8], int lane, int lanes, int cpr, float (&sums)[N]) {
#pragma unroll
  for (int c = 0; c < N; ++c) sums[c] = 0.0f;
#pragma unroll
  for (int c = 0; c < CH; ++c)
    if (FULL || lane + c * lanes < cpr)
#pragma unroll
      for (int j = 0; j < 8; ++j) sums[N == 1 ? 0 : c] = __builtin_fmaf(h[c][j], h[c][j], sums[N == 1 ? 0 : c]);
}

// FULL: every lane has CH chunks.  HALVES: twice the lanes of CH = 2 have a chunk each, for the same results
template <int DT, int FMT, int GL, int CH, bool FULL, bool SUM, bool HALVES>
__global__ __launch_bounds__(GL ? 256 : 1024) void block_norm_mx_kernel(const BlockNormArgs a) {
  const int lanes = GL ? GL : (int)blockDim.x;
  const int lane = GL ? (int)threadIdx.x % (GL ? GL : 1) : (int)threadIdx.x;
  const int64_t row = GL ? (int64_t)blockIdx.x * (256 / (GL ? GL : 1)) + (int)threadIdx.x / (GL ? GL : 1)
                         : (int64_t)blockIdx.x;
  const bool live = FULL || row < a.rows;
  const int cpr = FULL ? CH * lanes : live ? (int)(a.cols / 8) : 0;  // chunks of the row that there are
  // The sums of two chunks are kept apart and joined first, so that a row's total is the same with HALVES.
  constexpr int NS = GL == 0 && CH == 2 ? 2 : 1;
  __shared__ float part[2][GL ? 1 : HALVES ? 16 + 256 : 16];
  float sums[NS];
  constexpr bool kEarly = CH < 4;  // what is added ahead of the sums, but for the longest rows, for want of registers
  uint4 res[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c)
    if (kEarly && (FULL || lane + c * lanes < cpr)) res[c] = ld_stream(a.R + row * a.ld_r + 8 * (lane + c * lanes));
  float h[CH][8];
  load_sum<DT, CH, FULL, SUM>(a, row, lane, lanes, cpr, h);
  Ahead8 post[CH], gate[CH], norm[CH];
  auto each = [&](auto f) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (kEarly && (FULL || lane + c * lanes < cpr)) f(c, 8 * (int64_t)(lane + c * lanes));
  };
  auto get_post = [&]() { if (a.post != nullptr) each([&](int c, int64_t col) { post[c] = load_ahead(a.post, a.post_dtype, col); }); };
  auto get_gate = [&]() { if (a.gate != nullptr) each([&](int c, int64_t col) { gate[c] = load_ahead(a.gate, a.gate_dtype, row * a.ld_g + col); }); };
  auto get_norm = [&]() { each([&](int c, int64_t col) { norm[c] = load_ahead(a.norm, a.norm_dtype, col); }); };
  if (a.post != nullptr) {
    squares<CH, FULL>(h, lane, lanes, cpr, sums);
    const float r = row_scale<GL, CH, HALVES>(h, sums, live, lane, lanes, cpr, a.cols, a.eps, part[0]);
    get_post();
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (FULL || lane + c * lanes < cpr) {
        float w[8];
        if constexpr (kEarly) ahead_values(post[c], a.post_dtype, w);
        else load_weight8(a.post, a.post_dtype, 8 * (int64_t)(lane + c * lanes), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[c][j] = h[c][j] * r * w[j];
      }
  }
  get_gate();
#pragma unroll
  for (int c = 0; c < CH; ++c)
    if (FULL || lane + c * lanes < cpr) {
      const int64_t col = 8 * (int64_t)(lane + c * lanes);
      if (a.gate != nullptr) {
        float g[8];
        if constexpr (kEarly) ahead_values(gate[c], a.gate_dtype, g);
        else load_weight8(a.gate, a.gate_dtype, row * a.ld_g + col, g);
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
  squares<CH, FULL>(h, lane, lanes, cpr, sums);
  const float r = row_scale<GL, CH, HALVES>(h, sums, live, lane, lanes, cpr, a.cols, a.eps, part[1]);
  get_norm();
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int k = lane + c * lanes;
    if (FULL || k < cpr) {
      float w[8];
      if constexpr (kEarly) ahead_values(norm[c], a.norm_dtype, w);
      else load_weight8(a.norm, a.norm_dtype, 8 * (int64_t)k, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[c][j] = h[c][j] * r * w[j];
      uint32_t codes[2];
      const uint32_t byte = mx_quantize8<FMT>(h[c], codes);
      mx_store8<FMT>(codes, byte, a.codes, a.scales, row * cpr + k);
    }
  }
}

template <int DT, int FMT, bool SUM>
static void block_norm_launch(const BlockNormArgs& a, hipStream_t stream) {
  const int64_t cpr = a.cols / 8;
#define AWQ_NORM_W(GL, CH) \
  block_norm_mx_kernel<DT, FMT, GL, CH, false, SUM, false><<<(unsigned)((a.rows + 256 / GL - 1) / (256 / GL)), 256, 0, stream>>>(a)
#define AWQ_NORM_2(FULL)                                                                                             \
  block_norm_mx_kernel<DT, FMT, 0, 1, FULL, SUM, true><<<(unsigned)a.rows, (unsigned)(((cpr + 1) / 2 + 63) / 64 * 128), 0, \
                                                         stream>>>(a)
#define AWQ_NORM_B(CH, FULL)                                                                                         \
  block_norm_mx_kernel<DT, FMT, 0, CH, FULL, SUM, false><<<(unsigned)a.rows, (unsigned)(((cpr + CH - 1) / CH + 63) / 64 * 64), 0, \
                                               stream>>>(a)
  if constexpr (SUM) {
    // Few rows: twice the lanes have twice the sum's loads in flight (4096 columns, the sum of 8 rows: 1 row 4.6 us, with
    // two chunks a lane 5.3; 64 rows 6.3 both; without a sum nothing is gained).
    if (a.rows <= 32 && cpr > 64 && cpr <= 512) {
      if (cpr % 128 == 0) AWQ_NORM_2(true); else AWQ_NORM_2(false);
      return;
    }
  }
  if (cpr <= 4) AWQ_NORM_W(4, 1);
  else if (cpr <= 8) AWQ_NORM_W(8, 1);
  else if (cpr <= 16) AWQ_NORM_W(16, 1);
  else if (cpr <= 32) AWQ_NORM_W(32, 1);
  else if (cpr <= 64) AWQ_NORM_W(32, 2);
  else if (cpr <= 512 && cpr % 128 == 0) AWQ_NORM_B(2, true);
  else if (cpr <= 512) AWQ_NORM_B(2, false);
  else if (cpr <= 1024 && cpr % 64 == 0) AWQ_NORM_B(1, true);
  else if (cpr <= 1024) AWQ_NORM_B(1, false);
  else if (cpr <= 2048 && cpr % 128 == 0) AWQ_NORM_B(2, true);
  else if (cpr <= 2048) AWQ_NORM_B(2, false);
  else if (cpr <= 4096) AWQ_NORM_B(4, false);
  else AWQ_NORM_B(8, false);
#undef AWQ_NORM_W
#undef AWQ_NORM_B
#undef AWQ_NORM_2
}

hipError_t launch_block_norm_mx(const BlockNormArgs& a, int dt, int fmt, hipStream_t stream) {
#define AWQ_NORM(DT, FMT) \
  do { \
    if (a.places != nullptr) block_norm_launch<DT, FMT, true>(a, stream); \
    else block_norm_launch<DT, FMT, false>(a, stream); \
  } while (0)
  if (dt == 0) {
    if (fmt == kMxFp8) AWQ_NORM(0, kMxFp8); else AWQ_NORM(0, kMxFp4);
  } else {
    if (fmt == kMxFp8) AWQ_NORM(1, kMxFp8); else AWQ_NORM(1, kMxFp4);
  }
#undef AWQ_NORM
  return hipGetLastError();
}

}  // namespace awq
