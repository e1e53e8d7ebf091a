// Microscaled (MX) quantization, its inverse, and the two operators whose
// result is quantized as it is formed: RMS norm with the residual's addition,
// and SiLU gating.  All are bound by memory: each reads its inputs once and
// writes codes and scales once, in one launch.
//
// A lane holds 8 consecutive values (16 bytes of input), so a block of 32 is
// 4 neighbouring lanes and its maximum two lane permutations away.
#include "awq_launch.h"
#include "mx_device.h"
#include "mx_quotient.h"

namespace awq {

// ---------------------------------------------------------------------------
// quantize: v = x (or RN(x s[col])) -> codes, scales
// silu-mul: v = g / (1 + e^-g) u    -> codes, scales
// A lane takes four chunks of 8 values (two in the gating), all loads ahead of
// the arithmetic, nontemporal.  Measured: quantize 16384 x 4096 35.8 us, 5.7 TB/s
// (40.4 with ordinary loads, 37.3 at two chunks); gating 8192 x 12288 91 us,
// 5.6 TB/s (96 at four chunks, 121 with expf and a division: 34 VALU operations
// a value then bound it, 22 now).
// ---------------------------------------------------------------------------
constexpr int kEwThreads = 256, kEwUnroll = 4, kGateUnroll = 2;

// A lane's walk over the chunks of [rows, cpr]: its first one takes a division,
// the ones a block's width further on an addition and a wrap.
struct ChunkWalk {
  int64_t row;
  uint32_t col;
  const uint32_t cpr, rows_on, cols_on;
  __device__ __forceinline__ ChunkWalk(int64_t base, uint32_t cpr_)
      : cpr(cpr_), rows_on(kEwThreads / cpr_), cols_on(kEwThreads % cpr_) {
    const int64_t r0 = base / cpr;
    const uint32_t c = (uint32_t)(base - r0 * cpr) + threadIdx.x;
    row = r0 + c / cpr;
    col = c % cpr;
  }
  __device__ __forceinline__ int64_t at(int64_t ld) const { return row * ld + 8 * (int64_t)col; }
  __device__ __forceinline__ void next() {
    row += rows_on;
    col += cols_on;
    if (col >= cpr) col -= cpr, ++row;
  }
};

template <int DT, int FMT>
__global__ __launch_bounds__(kEwThreads) void mx_quantize_kernel(const uint16_t* __restrict__ X, int64_t n_chunks,
                                                                 uint32_t cpr, int64_t ld, uint8_t* __restrict__ out,
                                                                 uint8_t* __restrict__ scales) {
  const int64_t base = (int64_t)blockIdx.x * (kEwThreads * kEwUnroll);
  ChunkWalk p(base, cpr);
  uint4 x[kEwUnroll];
#pragma unroll
  for (int u = 0; u < kEwUnroll; ++u) {
    if (base + threadIdx.x + kEwThreads * u < n_chunks) x[u] = ld_stream(X + p.at(ld));
    p.next();
  }
#pragma unroll
  for (int u = 0; u < kEwUnroll; ++u) {
    const int64_t chunk = base + threadIdx.x + kEwThreads * u;
    if (chunk < n_chunks) {
      float v[8];
      unpack8<DT>(x[u], v);
      uint32_t codes[2];
      const uint32_t byte = mx_quantize8<FMT>(v, codes);
      mx_store8<FMT>(codes, byte, out, scales, chunk);
    }
  }
}

// With a scale of the columns a lane keeps its 8 columns over kColRows rows, so
// the scale is loaded (and, in the inverse, its reciprocal taken) once for them.
// A block is 2^tx chunks of columns (as many as a row has, rounded up to a power of
// two, from 4 to 64) by 256 / 2^tx x kColRows rows.  Measured at 4096 x 12288 to 4
// bits: 26.0 us, the inverse 24.3 us, 5 TB/s; on 48 million values (us, 16 / 64
// chunks a block, quantized): 128 columns 23.5 / 48, 480 columns 32.6 / 24.1, 4096
// columns 28.4 / 24.0.
constexpr int kColRows = 4;
struct ColPos {
  uint32_t col;
  int64_t row;
  int step;  // rows between the lane's rows
};
__device__ __forceinline__ ColPos col_pos(uint32_t cpr, int tx) {
  const uint32_t nx = (cpr + (1u << tx) - 1) >> tx;
  const uint32_t by = blockIdx.x / nx, bx = blockIdx.x - by * nx;
  const int step = kEwThreads >> tx;
  return {(bx << tx) + (threadIdx.x & ((1u << tx) - 1)), (int64_t)by * (step * kColRows) + (threadIdx.x >> tx), step};
}

template <int DT, int FMT>
__global__ __launch_bounds__(kEwThreads) void mx_quantize_scaled_kernel(const uint16_t* __restrict__ X, int64_t rows,
                                                                        uint32_t cpr, int tx, int64_t ld,
                                                                        const float* __restrict__ s,
                                                                        uint8_t* __restrict__ out,
                                                                        uint8_t* __restrict__ scales) {
  const ColPos p = col_pos(cpr, tx);
  const uint32_t col = p.col;
  const int64_t row = p.row;
  if (col >= cpr) return;  // whole groups of 4 lanes: cpr is a multiple of 4
  float sv[8];
  *(float4*)&sv[0] = ld_any<float4>(s + 8 * (int64_t)col);
  *(float4*)&sv[4] = ld_any<float4>(s + 8 * (int64_t)col + 4);
  uint4 x[kColRows];
#pragma unroll
  for (int u = 0; u < kColRows; ++u)
    if (row + p.step * u < rows) x[u] = ld_stream(X + (row + p.step * u) * ld + 8 * (int64_t)col);
#pragma unroll
  for (int u = 0; u < kColRows; ++u) {
    if (row + p.step * u < rows) {
      float v[8];
      unpack8<DT>(x[u], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= sv[j];
      uint32_t codes[2];
      const uint32_t byte = mx_quantize8<FMT>(v, codes);
      mx_store8<FMT>(codes, byte, out, scales, (row + p.step * u) * cpr + col);
    }
  }
}

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

template <int DT, int FMT>
__global__ __launch_bounds__(kEwThreads) void silu_mul_mx_kernel(const uint16_t* __restrict__ gate, int64_t ld_g,
                                                                 const uint16_t* __restrict__ up, int64_t ld_u,
                                                                 int64_t n_chunks, uint32_t cpr,
                                                                 uint8_t* __restrict__ out,
                                                                 uint8_t* __restrict__ scales) {
  const int64_t base = (int64_t)blockIdx.x * (kEwThreads * kGateUnroll);
  ChunkWalk p(base, cpr);
  uint4 g[kGateUnroll], w[kGateUnroll];
#pragma unroll
  for (int u = 0; u < kGateUnroll; ++u) {
    if (base + threadIdx.x + kEwThreads * u < n_chunks) {
      g[u] = ld_stream(gate + p.at(ld_g));
      w[u] = ld_stream(up + p.at(ld_u));
    }
    p.next();
  }
#pragma unroll
  for (int u = 0; u < kGateUnroll; ++u) {
    const int64_t chunk = base + threadIdx.x + kEwThreads * u;
    if (chunk < n_chunks) {
      float v[8], b[8];
      unpack8<DT>(g[u], v);
      unpack8<DT>(w[u], b);
      float gate_j[8];
      uint32_t far = 0;  // largest pattern: the least gate, if any is negative
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        gate_j[j] = v[j];
        far = max(far, __builtin_bit_cast(uint32_t, v[j]));
        v[j] = silu<DT>(v[j]) * b[j];
      }
      if (far > kFarGate) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (__builtin_bit_cast(uint32_t, gate_j[j]) > kFarGate) v[j] = far_silu_mul(gate_j[j], b[j]);
      }
      uint32_t codes[2];
      const uint32_t byte = mx_quantize8<FMT>(v, codes);
      mx_store8<FMT>(codes, byte, out, scales, chunk);
    }
  }
}

// a b, to be converted to output type OT.  The compiler makes one instruction of a product and its conversion to
// fp16, a b + 0, which loses the sign of a negative zero: there the product stays an operation of its own.
template <int OT>
__device__ __forceinline__ float product_for(float a, float b) {
  float p = a * b;
  if constexpr (OT == 0) asm("" : "+v"(p));
  return p;
}

// ---------------------------------------------------------------------------
// dequant: out = RN(RN32(code 2^e / s[col])), s optional.  code 2^e is exact in
// fp32 (unless it overflows); the quotient is rounded to fp32 and then to a
// 16-bit output, as unpack_dequant does.  Bound by the stores: 16384 x 4096 to
// bf16 takes 33 us from 4 bits (5.1 TB/s), 40 us from 8.
// ---------------------------------------------------------------------------
template <int FMT>
__device__ __forceinline__ void decode8(const uint2 c, float (&v)[8]) {  // elements, unscaled
  f32x2v t;
  if constexpr (FMT == kMxFp8) {
    t = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.x, false), v[0] = t[0], v[1] = t[1];
    t = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.x, true), v[2] = t[0], v[3] = t[1];
    t = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.y, false), v[4] = t[0], v[5] = t[1];
    t = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.y, true), v[6] = t[0], v[7] = t[1];
  } else {
    t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c.x, 1.0f, 0), v[0] = t[0], v[1] = t[1];
    t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c.x, 1.0f, 1), v[2] = t[0], v[3] = t[1];
    t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c.x, 1.0f, 2), v[4] = t[0], v[5] = t[1];
    t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c.x, 1.0f, 3), v[6] = t[0], v[7] = t[1];
  }
}
template <int FMT>
__device__ __forceinline__ uint2 load_codes8(const uint8_t* __restrict__ codes, int64_t chunk) {
  if constexpr (FMT == kMxFp8) return *(const uint2*)(codes + 8 * chunk);
  else return make_uint2(*(const uint32_t*)(codes + 4 * chunk), 0);
}
template <int OT>
__device__ __forceinline__ void store_values8(void* __restrict__ out, int64_t at, const float (&v)[8]) {
  if constexpr (OT == 2) {
    st_any((float*)out + at, make_float4(v[0], v[1], v[2], v[3]));
    st_any((float*)out + at + 4, make_float4(v[4], v[5], v[6], v[7]));
  } else {
    st_any((uint16_t*)out + at, pack8<OT>(v));
  }
}

template <int FMT, int OT>
__global__ __launch_bounds__(kEwThreads) void mx_dequant_kernel(const uint8_t* __restrict__ codes,
                                                                const uint8_t* __restrict__ scales, int64_t n_chunks,
                                                                uint32_t cpr, void* __restrict__ out, int64_t ld) {
  const int64_t base = (int64_t)blockIdx.x * (kEwThreads * kEwUnroll);
  ChunkWalk p(base, cpr);
  uint2 c[kEwUnroll];
  uint32_t e[kEwUnroll];
#pragma unroll
  for (int u = 0; u < kEwUnroll; ++u) {
    const int64_t chunk = base + threadIdx.x + kEwThreads * u;
    if (chunk < n_chunks) {
      c[u] = load_codes8<FMT>(codes, chunk);
      e[u] = scales[chunk >> 2];
    }
  }
#pragma unroll
  for (int u = 0; u < kEwUnroll; ++u) {
    if (base + threadIdx.x + kEwThreads * u < n_chunks) {
      const float unit = mx_unit(e[u]);
      float v[8];
      decode8<FMT>(c[u], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = product_for<OT>(v[j], unit);
      store_values8<OT>(out, p.at(ld), v);
    }
    p.next();
  }
}

// Divided by the columns' scale: mx_quotient (mx_quotient.h) with the reciprocal
// taken once for the lane's rows, where nothing leaves the normal range: |s| and
// 2^e within 2^+-60 and 2^+-40.  Elsewhere the division itself.
__device__ __forceinline__ bool mid_range(float x, uint32_t by) {
  const uint32_t e = __builtin_bit_cast(uint32_t, x) >> 23 & 255;
  return e - (127 - by) <= 2 * by;
}

template <int FMT, int OT>
__global__ __launch_bounds__(kEwThreads) void mx_dequant_scaled_kernel(const uint8_t* __restrict__ codes,
                                                                       const uint8_t* __restrict__ scales,
                                                                       int64_t rows, uint32_t cpr, int tx,
                                                                       const float* __restrict__ s,
                                                                       void* __restrict__ out, int64_t ld) {
  const ColPos p = col_pos(cpr, tx);
  const uint32_t col = p.col;
  const int64_t row = p.row;
  if (col >= cpr) return;
  uint2 c[kColRows];
  uint32_t e[kColRows];
#pragma unroll
  for (int u = 0; u < kColRows; ++u) {
    const int64_t chunk = (row + p.step * u) * cpr + col;
    if (row + p.step * u < rows) {
      c[u] = load_codes8<FMT>(codes, chunk);
      e[u] = scales[chunk >> 2];
    }
  }
  float sv[8], y[8];
  *(float4*)&sv[0] = ld_any<float4>(s + 8 * (int64_t)col);
  *(float4*)&sv[4] = ld_any<float4>(s + 8 * (int64_t)col + 4);
  bool usual = true;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    y[j] = 1.0f / sv[j];
    usual = usual && mid_range(sv[j], 60);
  }
#pragma unroll
  for (int u = 0; u < kColRows; ++u) {
    if (row + p.step * u < rows) {
      const float unit = mx_unit(e[u]);
      float v[8];
      decode8<FMT>(c[u], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= unit;
      if (usual && mid_range(unit, 40)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = mx_quotient(v[j], sv[j], y[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = v[j] / sv[j];
      }
      store_values8<OT>(out, (row + p.step * u) * ld + 8 * (int64_t)col, v);
    }
  }
}

// ---------------------------------------------------------------------------
// RMS norm: h = x + residual (fp32), residual_out = RN16(h),
// y = h / sqrt(mean h^2 + eps) * weight -> codes, scales.  The mean is taken
// over the unrounded fp32 h.  A row stays in registers between its sum of
// squares and its scaling, so the inputs are read once: 6001 x 4096 fp16 with a
// residual takes 30.6 us, 5.7 TB/s.  Lanes of a row: the GL lanes of a wave that
// its chunks of 8 need (several rows a wave) up to 256 columns, 32 lanes with two
// chunks each up to 512, else a whole block with one exchange of wave sums through
// LDS.  Measured on 24 million values in bf16 with a residual, us: 128 columns 30
// with 16 lanes, 78 with 64; 288 columns 37.6 with 2 x 32, 41 with a block of 64;
// 1024 columns 28.4 with a block (two chunks a lane), 29.2 with a wave; 4096
// columns 29.7 with two chunks a lane, 30.4 with one.  The split depends on the row
// length alone: a row's result is the same in every batch.
// ---------------------------------------------------------------------------
struct NormArgs {
  const uint16_t* X;
  int64_t ld_x;
  const uint16_t* R;  // may be null
  int64_t ld_r;
  uint16_t* RO;       // null with R
  int64_t ld_ro;
  const void* w;
  int w_dtype;        // 0 fp16, 1 bf16, 2 fp32
  float eps;
  int64_t rows;
  int64_t cols;
  uint8_t* codes;
  uint8_t* scales;
};

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

// Rows whose squares leave fp32's range: the mean is infinite, or so small that squares lost below the range count
// (those are off by at most 2^-150 each, 2^-134 for the longest row, 2^-34 of the least sum or eps taken).  They are
// brought to the middle of the range first, by the power of two of their largest value or, where that is less,
// of eps's root.  Rows that hold an infinity or a NaN stay as they are: 1 / sqrt(inf) = 0 times an infinity is NaN.
constexpr float kNormLeast = 0x1p-100f;

template <int DT, int FMT, int GL, int CH>
__global__ __launch_bounds__(GL ? 256 : 1024) void rms_norm_mx_kernel(const NormArgs a) {
  const int lanes = GL ? GL : (int)blockDim.x;
  const int lane = GL ? (int)threadIdx.x % (GL ? GL : 1) : (int)threadIdx.x;
  const int64_t row = GL ? (int64_t)blockIdx.x * (256 / (GL ? GL : 1)) + (int)threadIdx.x / (GL ? GL : 1)
                         : (int64_t)blockIdx.x;
  const int cpr = (int)(a.cols / 8);
  const bool live = row < a.rows;
  float h[CH][8];
  float sum = 0.0f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int k = lane + c * lanes;
    if (live && k < cpr) {
      unpack8<DT>(ld_stream(a.X + row * a.ld_x + 8 * k), h[c]);
      if (a.R != nullptr) {
        float r[8];
        unpack8<DT>(ld_stream(a.R + row * a.ld_r + 8 * k), r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[c][j] += r[j];
        st_any(a.RO + row * a.ld_ro + 8 * k, pack8<DT>(h[c]));
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(h[c][j], h[c][j], sum);
    }
  }
  __shared__ float part[GL ? 1 : 16];
  sum = row_total<GL>(sum, part, [](float x, float y) { return x + y; });
  float mean = sum / (float)a.cols + a.eps;
  // the same for the whole row
  if (__builtin_expect(!(mean < HUGE_VALF) || (sum < kNormLeast && a.eps < kNormLeast), false)) {
    uint32_t top = 0;
    if constexpr (GL == 0) __syncthreads();  // the sum has been read
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (live && lane + c * lanes < cpr)
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, __builtin_bit_cast(uint32_t, h[c][j]) & 0x7FFFFFFFu);
    top = __builtin_bit_cast(uint32_t, row_total<GL>(__builtin_bit_cast(float, top), part, [](float x, float y) {
      return __builtin_bit_cast(float, max(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y)));
    }));
    if (top < 0x7F800000u) {
      int k2 = (int)(top >> 23) - 127;
      if (a.eps > 0.0f) k2 = max(k2, ((int)(__builtin_bit_cast(uint32_t, a.eps) >> 23) - 127) / 2);
      sum = 0.0f;
      if constexpr (GL == 0) __syncthreads();
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if (live && lane + c * lanes < cpr)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            h[c][j] = __builtin_ldexpf(h[c][j], -k2);
            sum = __builtin_fmaf(h[c][j], h[c][j], sum);
          }
      sum = row_total<GL>(sum, part, [](float x, float y) { return x + y; });
      mean = sum / (float)a.cols + __builtin_ldexpf(a.eps, -2 * k2);
    }
  }
  const float r = 1.0f / sqrtf(mean);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int k = lane + c * lanes;
    if (live && k < cpr) {
      float w[8];
      load_weight8(a.w, a.w_dtype, 8 * (int64_t)k, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[c][j] = h[c][j] * r * w[j];
      uint32_t codes[2];
      const uint32_t byte = mx_quantize8<FMT>(h[c], codes);
      mx_store8<FMT>(codes, byte, a.codes, a.scales, row * cpr + k);
    }
  }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
static unsigned ew_blocks(int64_t n_chunks, int unroll) {
  return (unsigned)((n_chunks + kEwThreads * unroll - 1) / (kEwThreads * unroll));
}

static int col_tx(int64_t cols) {
  int tx = 2;
  while (tx < 6 && 8 << tx < cols) ++tx;
  return tx;
}
static unsigned col_blocks(int64_t rows, int64_t cols) {
  const int tx = col_tx(cols);
  const int64_t nx = (cols / 8 + (1 << tx) - 1) >> tx, per = (kEwThreads >> tx) * kColRows;
  return (unsigned)(nx * ((rows + per - 1) / per));
}

hipError_t launch_mx_quantize(const void* X, int dt, int64_t rows, int64_t cols, int64_t ld, const float* s, int fmt,
                              void* codes, uint8_t* scales, hipStream_t stream) {
  const int64_t n = rows * (cols / 8);
  const uint32_t cpr = (uint32_t)(cols / 8);
#define AWQ_MXQ(D, F)                                                                                                  \
  if (s)                                                                                                               \
    mx_quantize_scaled_kernel<D, F><<<col_blocks(rows, cols), kEwThreads, 0, stream>>>((const uint16_t*)X, rows, cpr, col_tx(cols), ld, \
                                                                                       s, (uint8_t*)codes, scales);    \
  else                                                                                                                 \
    mx_quantize_kernel<D, F><<<ew_blocks(n, kEwUnroll), kEwThreads, 0, stream>>>((const uint16_t*)X, n, cpr, ld, (uint8_t*)codes, \
                                                                      scales)
  if (dt == 0) {
    if (fmt == kMxFp8) { AWQ_MXQ(0, kMxFp8); } else { AWQ_MXQ(0, kMxFp4); }
  } else {
    if (fmt == kMxFp8) { AWQ_MXQ(1, kMxFp8); } else { AWQ_MXQ(1, kMxFp4); }
  }
#undef AWQ_MXQ
  return hipGetLastError();
}

hipError_t launch_silu_mul_mx(const void* gate, int64_t ld_g, const void* up, int64_t ld_u, int dt, int64_t rows,
                              int64_t cols, int fmt, void* codes, uint8_t* scales, hipStream_t stream) {
  const int64_t n = rows * (cols / 8);
  const unsigned g = ew_blocks(n, kGateUnroll);
#define AWQ_SILU(D, F)                                                                                         \
  silu_mul_mx_kernel<D, F><<<g, kEwThreads, 0, stream>>>((const uint16_t*)gate, ld_g, (const uint16_t*)up, ld_u, n, \
                                                         (uint32_t)(cols / 8), (uint8_t*)codes, scales)
  if (dt == 0) {
    if (fmt == kMxFp8) AWQ_SILU(0, kMxFp8); else AWQ_SILU(0, kMxFp4);
  } else {
    if (fmt == kMxFp8) AWQ_SILU(1, kMxFp8); else AWQ_SILU(1, kMxFp4);
  }
#undef AWQ_SILU
  return hipGetLastError();
}

hipError_t launch_mx_dequant(const void* codes, const uint8_t* scales, int fmt, int64_t rows, int64_t cols,
                             const float* s, void* out, int out_dtype, int64_t ld, hipStream_t stream) {
  const int64_t n = rows * (cols / 8);
  const uint32_t cpr = (uint32_t)(cols / 8);
#define AWQ_MXD(F, O)                                                                                                 \
  if (s)                                                                                                              \
    mx_dequant_scaled_kernel<F, O><<<col_blocks(rows, cols), kEwThreads, 0, stream>>>((const uint8_t*)codes, scales, rows, \
                                                                                      cpr, col_tx(cols), s, out, ld);               \
  else                                                                                                                \
    mx_dequant_kernel<F, O><<<ew_blocks(n, kEwUnroll), kEwThreads, 0, stream>>>((const uint8_t*)codes, scales, n, cpr, out, ld)
#define AWQ_MXD_O(F)                          \
  if (out_dtype == 0) { AWQ_MXD(F, 0); }      \
  else if (out_dtype == 1) { AWQ_MXD(F, 1); } \
  else { AWQ_MXD(F, 2); }
  if (fmt == kMxFp8) { AWQ_MXD_O(kMxFp8) } else { AWQ_MXD_O(kMxFp4) }
#undef AWQ_MXD_O
#undef AWQ_MXD
  return hipGetLastError();
}

int64_t rms_norm_mx_max_cols() { return 1024 * 8 * 8; }

template <int DT, int FMT>
static void rms_norm_launch(const NormArgs& a, hipStream_t stream) {
  const int64_t cpr = a.cols / 8;
#define AWQ_NORM_W(GL, CH) \
  rms_norm_mx_kernel<DT, FMT, GL, CH><<<(unsigned)((a.rows + 256 / GL - 1) / (256 / GL)), 256, 0, stream>>>(a)
#define AWQ_NORM_B(CH)                                                                                             \
  rms_norm_mx_kernel<DT, FMT, 0, CH><<<(unsigned)a.rows, (unsigned)(((cpr + CH - 1) / CH + 63) / 64 * 64), 0, stream>>>( \
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

hipError_t launch_rms_norm_mx(const void* X, int dt, int64_t rows, int64_t cols, int64_t ld_x, const void* residual,
                              int64_t ld_r, const void* norm, int norm_dtype, float eps, void* residual_out,
                              int64_t ld_ro, int fmt, void* codes, uint8_t* scales, hipStream_t stream) {
  const NormArgs a = {(const uint16_t*)X, ld_x, (const uint16_t*)residual, ld_r, (uint16_t*)residual_out, ld_ro,
                      norm, norm_dtype, eps, rows, cols, (uint8_t*)codes, scales};
  if (dt == 0) {
    if (fmt == kMxFp8) rms_norm_launch<0, kMxFp8>(a, stream); else rms_norm_launch<0, kMxFp4>(a, stream);
  } else {
    if (fmt == kMxFp8) rms_norm_launch<1, kMxFp8>(a, stream); else rms_norm_launch<1, kMxFp4>(a, stream);
  }
  return hipGetLastError();
}

}  // namespace awq
