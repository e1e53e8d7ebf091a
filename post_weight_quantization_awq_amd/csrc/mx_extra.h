// What a product does besides A W^T: nothing, an epilogue, or a choice of the
// weight by groups of rows.  The kernels of mx_product.h take one of these.
#pragma once

#include "mx_act.h"
#include "mx_device.h"

namespace awq {

struct NoExtra {
  static constexpr bool kGroups = false, kEpi = false;
};

// ---------------------------------------------------------------------------
// Epilogue: v = act(sum + bias[n]) + residual[m][n], in fp32; then rounded once or
// quantized.
// ---------------------------------------------------------------------------
struct Epilogue {
  static constexpr bool kGroups = false, kEpi = true, kRes = true;
  const void* bias;  // may be null
  int bias_dtype;    // 0 fp16, 1 bf16, 2 fp32
  int act;           // kAct*
  const void* R;     // may be null
  int r_dtype;
  int64_t ld_r;
  int out;           // 0 fp16, 1 bf16, 2 fp32; kOutFp8, kOutFp4: codes and scales
  uint8_t* codes;
  uint8_t* scales;
};
struct EpilogueAlone : Epilogue {  // without a residual
  static constexpr bool kRes = false;
};
constexpr int kOutFp8 = 3, kOutFp4 = 4;

__device__ __forceinline__ float load_float(const void* p, int64_t i, int dt) {
  if (dt == 2) return ((const float*)p)[i];
  const uint32_t v = ((const uint16_t*)p)[i];
  return dt == 0 ? x2f<0>(v) : x2f<1>(v);
}
// 8 values from i on as they lie in memory, the last `left` of them or all
struct Raw8 {
  uint4 lo, hi;  // hi: of 32-bit values
};
__device__ __forceinline__ Raw8 load_raw8(const void* p, int64_t i, int dt, int64_t left) {
  Raw8 r = {};
  if (left >= 8) {
    if (dt == 2) {
      r.lo = ld_any<uint4>((const float*)p + i);
      r.hi = ld_any<uint4>((const float*)p + i + 4);
    } else {
      r.lo = ld_any<uint4>((const uint16_t*)p + i);
    }
  } else {
    uint32_t w[8] = {};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) {
        if (dt == 2) w[j] = ((const uint32_t*)p)[i + j];
        else w[j / 2] |= (uint32_t)((const uint16_t*)p)[i + j] << (16 * (j % 2));
      }
    r.lo = make_uint4(w[0], w[1], w[2], w[3]);
    r.hi = make_uint4(w[4], w[5], w[6], w[7]);
  }
  return r;
}
__device__ __forceinline__ void add_raw8(float (&v)[8], const Raw8& r, int dt) {
  float f[8];
  if (dt == 0) {
    unpack8<0>(r.lo, f);
  } else if (dt == 1) {
    unpack8<1>(r.lo, f);
  } else {
    *(uint4*)&f[0] = r.lo;
    *(uint4*)&f[4] = r.hi;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] += f[j];
}
__device__ __forceinline__ void store_floats8(void* p, int64_t i, int dt, int64_t left, const float (&f)[8]) {
  if (left >= 8) {
    if (dt == 2) {
      st_any((float*)p + i, make_float4(f[0], f[1], f[2], f[3]));
      st_any((float*)p + i + 4, make_float4(f[4], f[5], f[6], f[7]));
    } else {
      st_any((uint16_t*)p + i, dt == 0 ? pack8<0>(f) : pack8<1>(f));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) {
        if (dt == 2) ((float*)p)[i + j] = f[j];
        else ((uint16_t*)p)[i + j] = (uint16_t)(dt == 0 ? f2x<0>(f[j]) : f2x<1>(f[j]));
      }
  }
}

// Where a lane's 8 outputs of a row go, and their residual; `on` rows further
struct OutRow {
  uint8_t* y;       // Y, or the codes
  uint8_t* scale;
  const uint8_t* r;
};
__device__ __forceinline__ OutRow out_row(const Epilogue& x, void* Y, int64_t ld_y, int64_t m, int64_t n, int64_t N) {
  OutRow o = {nullptr, nullptr, nullptr};
  if (x.out <= 2) {
    o.y = (uint8_t*)Y + (m * ld_y + n) * (x.out == 2 ? 4 : 2);
  } else {
    const int64_t at = m * N + n;
    o.y = x.codes + (x.out == kOutFp8 ? at : at / 2);
    o.scale = x.scales + at / 32;
  }
  if (x.R != nullptr) o.r = (const uint8_t*)x.R + (m * x.ld_r + n) * (x.r_dtype == 2 ? 4 : 2);
  return o;
}
__device__ __forceinline__ OutRow row_step(const Epilogue& x, int64_t ld_y, int on, int64_t N) {  // as offsets
  return {(uint8_t*)(on * (x.out == kOutFp8 ? N : x.out == kOutFp4 ? N / 2 : ld_y * (x.out == 2 ? 4 : 2))),
          (uint8_t*)(on * (N / 32)), (const uint8_t*)(on * x.ld_r * (x.r_dtype == 2 ? 4 : 2))};
}
__device__ __forceinline__ void go_on(OutRow& o, const OutRow& step) {
  o.y += (intptr_t)step.y, o.scale += (intptr_t)step.scale, o.r += (intptr_t)step.r;
}

// 8 outputs with their bias: activation, residual (`r` for 16-bit ones), store of the last `left` of them or all.
// Quantized results: the block of 32 is 4 neighbouring lanes, all active; `in`: the row is there.
template <bool RES>
__device__ __forceinline__ void finish8(const Epilogue& x, float (&v)[8], const uint4 r, const OutRow& o, int64_t left,
                                        bool in) {
  activate(v, x.act);
  if (RES && in) add_raw8(v, x.r_dtype == 2 ? load_raw8(o.r, 0, 2, left) : Raw8{r, r}, x.r_dtype);
  if (x.out <= 2) {
    if (in) store_floats8(o.y, 0, x.out, left, v);
  } else {
    uint32_t codes[2];
    uint32_t byte;
    if (x.out == kOutFp8) {
      byte = mx_quantize8<kMxFp8>(v, codes);
      if (in) *(uint2*)o.y = make_uint2(codes[0], codes[1]);
    } else {
      byte = mx_quantize8<kMxFp4>(v, codes);
      if (in) *(uint32_t*)o.y = codes[0];
    }
    if (in && threadIdx.x % 4 == 0) *o.scale = (uint8_t)byte;
  }
}

// The same for one output a lane; quantized: the block is an aligned half wave
__device__ __forceinline__ void finish1(const Epilogue& x, float v, int64_t m, int64_t n, int64_t N, bool in, void* Y,
                                        int64_t ld_y) {
  if (x.bias != nullptr && in) v += load_float(x.bias, n, x.bias_dtype);
  float one[1] = {v};
  activate(one, x.act);
  v = one[0];
  if (x.R != nullptr && in) v += load_float(x.R, m * x.ld_r + n, x.r_dtype);
  if (x.out <= 2) {
    if (!in) return;
    if (x.out == 2) ((float*)Y)[m * ld_y + n] = v;
    else ((uint16_t*)Y)[m * ld_y + n] = (uint16_t)(x.out == 0 ? f2x<0>(v) : f2x<1>(v));
    return;
  }
  uint32_t top = __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu;
  top = max(top, dpp_u<0xB1>(top));
  top = max(top, dpp_u<0x4E>(top));
  top = max(top, dpp_u<0x141>(top));
  top = max(top, dpp_u<0x140>(top));
  top = max(top, (uint32_t)__shfl_xor((int)top, 16, kWave));
  const int64_t at = m * N + n;
  uint32_t byte;
  if (x.out == kOutFp8) {
    byte = mx_scale_byte<kMxFp8>(top);
    const float unit = mx_unit(byte), lim = 448.0f * unit;  // the conversion does not saturate
    s16x2 r = {0, 0};
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, __builtin_amdgcn_fmed3f(v, -lim, lim), 0.0f, unit, false);
    if (in) x.codes[at] = byte == kMxNan ? 0 : (uint8_t)__builtin_bit_cast(uint32_t, r);
  } else {
    byte = mx_scale_byte<kMxFp4>(top);
    const float next = dpp_m<0xB1>(v);
    const uint32_t r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v, next, mx_unit(byte), 0);
    if (in && at % 2 == 0) x.codes[at / 2] = byte == kMxNan ? 0 : (uint8_t)r;
  }
  if (in && at % 32 == 0) x.scales[at / 32] = (uint8_t)byte;
}

// ---------------------------------------------------------------------------
// Groups: rows [offsets[e], offsets[e + 1]) of the result are products with
// matrix e of W.  The host knows no offsets: a launch has blocks for as many tiles
// of rows as there can be, and a block finds its own one, by a sum over the groups'
// tiles in its lanes.  Offsets are held inside [0, M] and row numbers inside A
// whatever they are.
// ---------------------------------------------------------------------------
struct Groups {
  static constexpr bool kGroups = true, kEpi = false;
  const int32_t* offsets;  // [n + 1]
  int n;
  const int32_t* rows;     // row of A for each row of the result, or null: its own
  int64_t a_rows;
  int first_tile;          // of the launch
};
struct GroupTile {
  int group;       // -1: none
  int first, end;  // rows
};

__device__ __forceinline__ int clamp_int(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// 64 groups in a wave's lanes: their rows and the sum of the tiles up to and with each
struct GroupSpan {
  int first, end, sum;
};
__device__ __forceinline__ GroupSpan group_span(const Groups& g, int M, int tile, int e0) {
  const int lane = threadIdx.x & 63, e = e0 + lane;
  GroupSpan s = {0, 0, 0};
  if (e < g.n) {
    s.first = clamp_int(g.offsets[e], 0, M);
    s.end = clamp_int(g.offsets[e + 1], s.first, M);
  }
  s.sum = (s.end - s.first + tile - 1) / tile;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int y = __shfl_up(s.sum, d, kWave);
    if (lane >= d) s.sum += y;
  }
  return s;
}
__device__ __forceinline__ int span_total(const GroupSpan& s) { return __builtin_amdgcn_readlane(s.sum, 63); }

__device__ __forceinline__ GroupTile span_tile(const GroupSpan& s, int e0, int tile, int at) {
  const int lane = __builtin_ctzll(__ballot(at < s.sum));
  const int first = __builtin_amdgcn_readlane(s.first, lane), end = __builtin_amdgcn_readlane(s.end, lane);
  const int tiles = (end - first + tile - 1) / tile;
  return {e0 + lane, first + (at - (__builtin_amdgcn_readlane(s.sum, lane) - tiles)) * tile, end};
}

// Tile `at` of all groups'; every lane of the wave takes part
__device__ __forceinline__ GroupTile group_tile(const Groups& g, int M, int tile, int at) {
  for (int e0 = 0; e0 < g.n; e0 += kWave) {
    const GroupSpan s = group_span(g, M, tile, e0);
    const int total = span_total(s);
    if (at < total) return span_tile(s, e0, tile, at);
    at -= total;
  }
  return {-1, 0, 0};
}

// The number of tiles, and the one that `pick` makes of it (-1: none)
template <class F>
__device__ __forceinline__ GroupTile group_pick(const Groups& g, int M, int tile, F pick) {
  const GroupSpan s = group_span(g, M, tile, 0);
  int total = span_total(s);
  for (int e0 = kWave; e0 < g.n; e0 += kWave) total += span_total(group_span(g, M, tile, e0));
  const int at = pick(total);
  if (at < 0 || at >= total) return {-1, 0, 0};
  if (at < span_total(s)) return span_tile(s, 0, tile, at);
  return group_tile(g, M, tile, at);
}

// Row of A for row m of the result; -1: none
__device__ __forceinline__ int64_t group_row(const Groups& g, int m) {
  if (g.rows == nullptr) return m;
  const int64_t r = g.rows[m];
  return (uint64_t)r < (uint64_t)g.a_rows ? r : -1;
}

}  // namespace awq
