// Kernels of the product of microscaled operands (mx_matmul.hip), which the product with an epilogue and the product
// grouped by expert share.
#pragma once

#include <stddef.h>

#include "mx_device.h"
#include "mx_extra.h"
#include "mx_tiles.h"

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

typedef __attribute__((address_space(3))) void* mx_lds_ptr;
constexpr uint32_t kMxOut = 0x80000000u;  // an offset past the range of every tile's buffer (256 rows of <= 2^22 bytes)

// 16-byte chunk c of an LDS row sits at slot c ^ swz(row): 8 consecutive rows
// spread over all positions of a 128-byte window and 16 over those of a 256-byte one
__device__ __forceinline__ int swz8(int row) { return (row & 7) ^ ((row >> 3) & 1); }         // 8 chunks a row
__device__ __forceinline__ int swz4(int row) { return ((row >> 1) & 3) ^ ((row >> 3) & 1); }  // 4 chunks a row

// s_waitcnt vmcnt(N) lgkmcnt(0)
template <int N>
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | ((N >> 4) << 14));
}

__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(0xC07F); }  // lgkmcnt(0)

// The compiler keeps memory accesses on their side of this point
__device__ __forceinline__ void hold_order() { asm volatile("" ::: "memory"); }
// The block's barrier, without waiting for the loads in flight as __syncthreads would
__device__ __forceinline__ void block_barrier() {
  hold_order();
  __builtin_amdgcn_s_barrier();
  hold_order();
}

// 16 bytes a lane from base + off + k_off straight into LDS, lane i to 16 i bytes past dst
__device__ __forceinline__ void load_lds16(const void* base, uint32_t bytes, uint8_t* dst, uint32_t off,
                                           uint32_t k_off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(
      __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000), (mx_lds_ptr)dst, 16,
      off, k_off, 0, 0);
}

// the same with 4 bytes a lane
__device__ __forceinline__ void load_lds4(const void* base, uint32_t bytes, uint8_t* dst, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(
      __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000), (mx_lds_ptr)dst, 4,
      off, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// Few tokens, bound by reading the weights: a block holds 16 NT outputs and AR
// tokens.  Its 8 waves take chunks of ST MFMA steps of 128 K in turn, and their
// sums are added in wave order through LDS.  A wave issues the next chunk's loads
// ahead of the products of the one at hand.  They are on their way meanwhile for
// every second chunk only: the loads of a row's ragged end stand under branches,
// where the compiler loses count of what is in flight, so in the first half of the
// loop it waits for all of it.  The matrix cores want 16 lanes side by side in 16 rows;
// loaded like that, every lane is an access of its own (measured at one token,
// 24576 x 4096: 14.3 us).  So the weights, used once, are read 64 bytes of a row by
// 4 lanes and turned by lane permutations (12.5 us), and the activations go through
// LDS, each wave's through buffers of its own and by direct loads of whole rows,
// which read nothing for rows past the last token (16 tokens, 4096 x 12288: 11.7 us
// loaded by the lanes, 8.3 us so, 8.1 through registers).  For up to 4 tokens 4 LDS
// rows leave room for more blocks (11.8 us, 4.5 TB/s).  With more, the path of the
// activations into LDS bounds it: 24 tokens, 4096 x 12288: 9.7 us, 295 KB a compute
// unit, its data unit busy 75% of the time.
// ---------------------------------------------------------------------------
constexpr int kFewWaves = 8;

// The scale bytes of the 4 ST blocks of a row's chunk c; zeros past the row's end
template <int ST>
struct FewScales {
  uint32_t v[ST];
};
template <int ST>
__device__ __forceinline__ FewScales<ST> few_scales(const uint8_t* row, int c, int kb) {
  if (4 * ST * (c + 1) <= kb) return ld_any<FewScales<ST>>(row + 4 * ST * c);
  FewScales<ST> s = {};
  for (int i = 0; i < kb - 4 * ST * c; ++i) {
    const uint32_t b = (uint32_t)row[4 * ST * c + i] << (8 * (i & 3));
#pragma unroll
    for (int d = 0; d < ST; ++d) s.v[d] |= d == i >> 2 ? b : 0;
  }
  return s;
}

// AR: LDS rows of activations (4, 16, 24 or 32); the lanes of rows past them read others, unused
template <int AF, int AR, int NT, int ST, int OCC, class X = NoExtra>
__global__ __launch_bounds__(kFewWaves * kWave, OCC) void mx_few_kernel(const uint8_t* __restrict__ A,
                                                                       const uint8_t* __restrict__ as, int64_t M,
                                                                       const uint8_t* __restrict__ W,
                                                                       const uint8_t* __restrict__ ws, int64_t N,
                                                                       int64_t K, void* __restrict__ Y, int64_t ld_y,
                                                                       int y_dtype, const X x = X()) {
  constexpr int MT = (AR + 15) / 16;                     // tiles of 16 tokens
  constexpr int RB = (AF == kMxFp8 ? 128 : 64) * ST;     // bytes of a row's chunk
  constexpr int CR = RB / 16;                            // 16-byte pieces of it
  constexpr int DI = AR * RB / 1024;                     // direct loads of a chunk, a KiB each
  static_assert(DI >= 1, "whole loads");
  // a wave's buffer: chunk, later sums
  constexpr int BS = AR * RB > 4 * NT * MT * 16 * 17 ? AR * RB : 4 * NT * MT * 16 * 17;
  __shared__ __attribute__((aligned(1024))) uint8_t b0[kFewWaves][(BS + 1023) / 1024 * 1024];
  __shared__ __attribute__((aligned(1024))) uint8_t b1[kFewWaves][AR * RB];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, h = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * NT);
  int64_t m0 = (int64_t)blockIdx.y * AR;
  const int kb = (int)(K / kMxBlock), nc = (kb + 4 * ST - 1) / (4 * ST);
  if constexpr (X::kGroups) {
    const GroupTile g = group_tile(x, (int)M, AR, x.first_tile + (int)blockIdx.y);
    if (g.group < 0) return;
    m0 = g.first;
    M = g.end;
    W += (int64_t)g.group * N * (K / 2);
    ws += (int64_t)g.group * N * kb;
  }
  const int m_rows = (int)(M - m0 < AR ? M - m0 : AR);
  const uint32_t a_row = (uint32_t)(AF == kMxFp8 ? K : K / 2);
  // weights: 4 lanes side by side read 64 bytes of a row, and turn() hands each lane the piece that the
  // matrix cores want of it.  Rows past the end repeat the last one, unused.
  // So are the scales, by 4 lanes side by side for a row's, which count as one access (64 accesses a load bound
  // 24 tokens, 4096 x 12288: 10.9 -> 10.2 us).  Up to 4 tokens wait for nothing but the weights: there each lane
  // loads its own row's (6.4 us, 6.8 turned).
  constexpr bool TURN = AR >= 16;
  const int sr = TURN ? lane / 4 : r;  // row of the scales that the lane loads
  const uint8_t* wr[NT];
  const uint8_t* wsr[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int64_t nl = n0 + 16 * i + lane / 4, n = n0 + 16 * i + sr;
    wr[i] = W + (nl < N ? nl : N - 1) * (K / 2) + 16 * (lane % 4);
    wsr[i] = ws + (n < N ? n : N - 1) * kb;
  }
  auto turn1 = [&](uint32_t v) { return (uint32_t)__builtin_amdgcn_ds_bpermute(4 * (4 * r + h), (int)v); };
  auto scale = [&](uint32_t v) { return (int)((TURN ? turn1(v) : v) >> (8 * h)); };
  auto turn = [&](const uint4 v) { return lo4(make_uint4(turn1(v.x), turn1(v.y), turn1(v.z), turn1(v.w))); };
  const uint8_t* asr[MT];
  bool no_row[MT];  // of A: its scales count as 0
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    int64_t row = m0 + min(16 * t + sr, m_rows - 1);
    no_row[t] = false;
    if constexpr (X::kGroups) {
      row = group_row(x, (int)row);
      no_row[t] = row < 0;
      row = row < 0 ? 0 : row;
    }
    asr[t] = as + row * kb;
  }
  const uint8_t* a_tile = A + m0 * a_row;
  uint32_t a_bytes = (uint32_t)m_rows * a_row;
  if constexpr (X::kGroups) {
    if (x.rows != nullptr) a_tile = A, a_bytes = (uint32_t)x.a_rows * a_row;
  }
  // piece c of row m sits at slot c ^ (m % 16) of its LDS row, or c ^ swz8(m) of one of 8 pieces
  uint32_t va[DI], vc[DI];  // offset of the lane's row (past the range for rows past the end), of its piece
#pragma unroll
  for (int j = 0; j < DI; ++j) {
    const int piece = kWave * j + lane, m = piece / CR;
    va[j] = m < m_rows ? (uint32_t)m * a_row : kMxOut;
    if constexpr (X::kGroups) {
      if (x.rows != nullptr && m < m_rows) {
        const int64_t row = group_row(x, (int)(m0 + m));
        va[j] = row < 0 ? kMxOut : (uint32_t)row * a_row;
      }
    }
    vc[j] = 16u * (uint32_t)(piece % CR ^ (CR >= 16 ? m & 15 : swz8(m)));
  }
  bool none[MT];  // the row that the lane multiplies is not in A
#pragma unroll
  for (int t = 0; t < MT; ++t) none[t] = X::kGroups && (TURN ? turn1(no_row[t]) : no_row[t]) != 0;
  f32x4 acc[MT][NT];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[t][i] = (f32x4){0, 0, 0, 0};

  struct Chunk {
    uint4 w[NT][ST];
    FewScales<ST> sw[NT], sa[MT];
  };
  constexpr int NL = DI + NT * (ST + 1) + MT;  // loads of a whole chunk (a row's last one may take others)
  auto load_chunk = [&](Chunk& f, uint8_t* buf, int c) {
    const uint32_t k = (uint32_t)c * RB;
#pragma unroll
    for (int j = 0; j < DI; ++j)  // past the row's end its last piece again: the weights there are 0
      load_lds16(a_tile, a_bytes, buf + 1024 * j, va[j] + min(k + vc[j], a_row - 16), 0);
    hold_order();
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int j = 0; j < ST; ++j) {
        f.w[i][j] = make_uint4(0, 0, 0, 0);
        if (4 * (ST * c + j) + lane % 4 < kb) f.w[i][j] = *(const uint4*)(wr[i] + 64 * (int64_t)(ST * c + j));
      }
      f.sw[i] = few_scales<ST>(wsr[i], c, kb);
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) f.sa[t] = few_scales<ST>(asr[t], c, kb);
    hold_order();
  };
  auto wait_chunk = [&](int next) {  // for all but the loads of chunk `next`, the youngest
    if (4 * ST * (next + 1) <= kb) wait_loads<NL>();
    else wait_loads<0>();
    hold_order();
  };
  auto multiply = [&](const Chunk& f, const uint8_t* buf) {
    i32x8 w[NT][ST];
    int sw[NT][ST];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < ST; ++j) {
        w[i][j] = turn(f.w[i][j]);
        sw[i][j] = scale(f.sw[i].v[j]);
      }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int m = 16 * t + (AR - 16 * t < 16 ? r % (AR - 16 * t) : r);
      auto piece = [&](int c) { return *(const uint4*)(buf + m * RB + 16 * (c ^ (CR >= 16 ? m & 15 : swz8(m)))); };
#pragma unroll
      for (int j = 0; j < ST; ++j) {
        i32x8 a;
        if constexpr (AF == kMxFp8) a = both4(piece(8 * j + h), piece(8 * j + 4 + h));
        else a = lo4(piece(4 * j + h));
        int sa = scale(f.sa[t].v[j]);
        if constexpr (X::kGroups) sa = none[t] ? 0 : sa;
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[t][i] = mfma_mx<AF>(w[i][j], a, acc[t][i], sw[i][j], sa);
      }
    }
  };
  Chunk f0, f1;
  int c = wave;
  if (c < nc) {
    load_chunk(f0, b0[wave], c);
    for (;;) {
      // chunk c in f0 / b0; before its buffer is filled again its reads are done (lgkmcnt 0)
      if (c + kFewWaves < nc) load_chunk(f1, b1[wave], c + kFewWaves);
      wait_chunk(c + kFewWaves);
      multiply(f0, b0[wave]);
      if ((c += kFewWaves) >= nc) break;
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
      hold_order();
      if (c + kFewWaves < nc) load_chunk(f0, b0[wave], c + kFewWaves);
      wait_chunk(c + kFewWaves);
      multiply(f1, b1[wave]);
      if ((c += kFewWaves) >= nc) break;
      __builtin_amdgcn_s_waitcnt(0xC07F);
      hold_order();
    }
  }
  // the wave's sums, in its first buffer's place
  float* sums = (float*)b0[wave];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) sums[((t * NT + i) * 16 + r) * 17 + 4 * h + e] = acc[t][i][e];
  __syncthreads();
  for (int i = threadIdx.x; i < MT * NT * 256; i += kFewWaves * kWave) {
    const int m = i / (16 * NT), o = i % (16 * NT);
    const int at = ((m / 16 * NT + o / 16) * 16 + m % 16) * 17 + o % 16;
    float v = 0.0f;
#pragma unroll
    for (int q = 0; q < kFewWaves; ++q) v += ((const float*)b0[q])[at];
    const bool in = m0 + m < M && m < AR && n0 + o < N;
    if constexpr (X::kEpi) finish1(x, v, m0 + m, n0 + o, N, in, Y, ld_y);
    else if (in) store_y(Y, (m0 + m) * ld_y + n0 + o, v, y_dtype);
  }
}

// ---------------------------------------------------------------------------
// Many tokens: tiles of BM tokens x BN outputs staged through LDS.
//
// K advances in stages of 128 through a ring of NS LDS slots (three or six), filled
// by direct loads (16 bytes a lane, no registers) NS - 1 stages ahead.  A stage is
// two steps of v_mfma_scale_f32_32x32x64_f8f6f4; the fragments of a step are read
// from LDS while the matrix cores work on the step before, across the stage
// boundary too: the block's one barrier a stage stands between the two steps, where
// the next stage's loads must have landed.
// ---------------------------------------------------------------------------
template <int AF>
__device__ __forceinline__ f32x16 mfma_mx32(const i32x8 w, const i32x8 a, f32x16 c, int ws, int as, int step) {
  // scale bytes 0 and 2 of the registers: the lane's block of step 0 and 1
  return step == 0
             ? __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, a, c, 4, AF == kMxFp8 ? 0 : 4, 0, ws, 0, as)
             : __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, a, c, 4, AF == kMxFp8 ? 0 : 4, 2, ws, 2, as);
}

// Issue order of half a stage: two LDS reads and one or two direct loads behind each MFMA, so that
// they are under way early and the matrix cores never wait for a burst of them
template <int READS, int LOADS>
__device__ __forceinline__ void interleave() {
#pragma unroll
  for (int i = 0; i < (READS + 1) / 2; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                           // MFMA
    __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);                           // LDS reads
    if (2 * i < LOADS) __builtin_amdgcn_sched_group_barrier(0x020, 2, 0);        // memory loads
  }
}

// 16 bytes of a result row, or as many of its elements as are left
template <int EB>
__device__ __forceinline__ void store_row16(uint8_t* p, const uint4 v, int64_t left) {
  if (left >= 16 / EB) {
    st_any(p, v);
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 16 / EB; ++e)
      if (e < left) {
        if constexpr (EB == 4) ((uint32_t*)p)[e] = w[e];
        else ((uint16_t*)p)[e] = (uint16_t)(w[e / 2] >> (16 * (e % 2)));
      }
  }
}

// Results of a wave's MT x NT tiles of 32 x 32 at (m0, n0): lane l holds outputs 8 (e / 4) + 4 h + e % 4 of
// token l % 32.  The wave turns 32 tokens at a time through its own part of the block's LDS arrays (SB
// bytes each), so that 16 bytes a lane and whole rows of its outputs go to memory together.
template <int YT, int MT, int NT, int NW, int SB, int NA = 3, bool WHOLE = false>
__device__ __forceinline__ void store_tile(const f32x16 (&acc)[NT][MT], uint8_t* s0, uint8_t* s1, uint8_t* s2,
                                           int wave, int lane, int64_t m0, int64_t n0, int64_t M, int64_t N, void* Y,
                                           int64_t ld_y) {
  constexpr int EB = YT == 2 ? 4 : 2;
  constexpr int CG = (EB == 2 && NA > 1) || NT == 1 ? NT : NT / 2;  // 32-output tiles per turn
  constexpr int RB = CG * 32 * EB;                           // bytes of a row
  constexpr int WS = (NW + NA - 1) / NA;                     // waves an array
  constexpr int RS = RB + (WS * 32 * (RB + 16) <= SB ? 16 : 0);  // stride: padded where there is room
  static_assert(WS * 32 * RS <= SB, "an array holds the rows of its waves");
  uint8_t* part = (wave < WS ? s0 : wave < 2 * WS ? s1 : s2) + wave % WS * (32 * RS);
  constexpr int LR = RB / 16, RI = kWave / LR;               // lanes a row, rows a store
  const int r = lane & 31, h = lane >> 5;
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int i0 = 0; i0 < NT; i0 += CG) {
#pragma unroll
      for (int i = 0; i < CG; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x16& v = acc[i0 + i][j];
          uint8_t* at = part + r * RS + (32 * i + 8 * g + 4 * h) * EB;
          if constexpr (YT == 2) *(float4*)at = make_float4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]);
          else
            *(uint2*)at = make_uint2(f2x<YT>(v[4 * g]) | (f2x<YT>(v[4 * g + 1]) << 16),
                                     f2x<YT>(v[4 * g + 2]) | (f2x<YT>(v[4 * g + 3]) << 16));
        }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
      for (int it = 0; it < 32 / RI; ++it) {
        const int row = it * RI + lane / LR, c = lane % LR;
        const uint4 v = *(const uint4*)(part + row * RS + 16 * c);
        const int64_t m = m0 + 32 * j + row, n = n0 + 32 * i0 + c * (16 / EB);
        if constexpr (WHOLE) st_any((uint8_t*)Y + (m * ld_y + n) * EB, v);
        else if (m < M) store_row16<EB>((uint8_t*)Y + (m * ld_y + n) * EB, v, N - n);
      }
      __builtin_amdgcn_wave_barrier();
    }
}

// The same with an epilogue: the sums go through LDS in fp32, 16 tokens x 64 outputs at a time (32 x 32 where a wave
// has no more), and come back 8 outputs a lane, so that 128 bytes of a row go to memory together.
// The turns are a loop, of which only the choice of the registers is unrolled: with all of it unrolled (60 KB of code,
// run once a tile) the blocks waited for instructions (8192 x 4096 x 4096 in 4 bits: 130 us, 72 without an
// epilogue).  A wait for a load is one for all earlier stores, too, so the bias lies in LDS, and with AHEAD, where the
// registers suffice, 16-bit residuals are loaded for all turns at first.
template <int MT, int NT, int NW, int SB, int NA, bool AHEAD, class X>
__device__ __forceinline__ void store_tile_epi(const f32x16 (&acc)[NT][MT], uint8_t* s0, uint8_t* s1, uint8_t* s2,
                                               int wave, int lane, int64_t m0, int64_t n0, int64_t M, int64_t N,
                                               void* Y, int64_t ld_y, const X& x) {
  constexpr int CG = NT > 1 ? 2 : 1;                              // 32-output tiles a turn
  constexpr int TR = 32 / CG, NS = MT * CG, LR = 4 * CG;          // tokens a turn, turns, lanes of a row
  constexpr int WS = (NW + NA - 1) / NA;                          // waves an array
  constexpr int RS = WS * TR * (CG * 128 + 16) <= SB ? CG * 128 + 16 : CG * 128;  // padded where there is room
  constexpr bool RES = X::kRes;
  static_assert(WS * TR * RS <= SB, "an array holds the rows of its waves");
  __shared__ __attribute__((aligned(16))) float biases[NW][32 * NT];
  uint8_t* part = (wave < WS ? s0 : wave < 2 * WS ? s1 : s2) + wave % WS * (TR * RS);
  const int r = lane & 31, h = lane >> 5, row = lane / LR, c = 8 * (lane % LR);
  const int rows = (int)(M - m0 < 32 * MT ? M - m0 : 32 * MT);  // of the wave's
  uint4 res[NT / CG][NS][2];  // with AHEAD
  const OutRow step = row_step(x, ld_y, TR / 2, N);
  auto load_res = [&](int ip, uint4 (&v)[NS][2]) {
    if (x.r_dtype == 2) return;
    const int64_t n = n0 + 32 * CG * ip + c;
    OutRow o = out_row(x, Y, ld_y, m0 + row, n, N);
#pragma unroll
    for (int t = 0; t < 2 * NS; ++t) {
      v[t / 2][t % 2] = make_uint4(0, 0, 0, 0);
      if (row + TR / 2 * t < rows && n < N) v[t / 2][t % 2] = load_raw8(o.r, 0, x.r_dtype, N - n).lo;
      o.r += (intptr_t)step.r;
    }
  };
  if constexpr (RES && AHEAD) {
#pragma unroll
    for (int ip = 0; ip < NT / CG; ++ip) load_res(ip, res[ip]);
  }
  if (x.bias != nullptr) {
#pragma unroll
    for (int i = 0; i < (NT + 1) / 2; ++i) {
      const int64_t n = n0 + 64 * i + lane;
      if ((NT > 1 || lane < 32) && n < N) biases[wave][64 * i + lane] = load_float(x.bias, n, x.bias_dtype);
    }
  }
#pragma unroll
  for (int ip = 0; ip < NT / CG; ++ip) {
    if (ip == 0) wait_loads<0>();
    const int64_t n = n0 + 32 * CG * ip + c;
    OutRow o = out_row(x, Y, ld_y, m0 + row, n, N);
    int at_row = row;
#pragma unroll 1
    for (int s = 0; s < NS; ++s) {
      uint4 now[2] = {};
      if constexpr (RES && !AHEAD) {
        if (x.r_dtype != 2) {
#pragma unroll
          for (int it = 0; it < 2; ++it)
            if (at_row + TR / 2 * it < rows && n < N)
              now[it] = load_raw8(o.r + it * (intptr_t)step.r, 0, x.r_dtype, N - n).lo;
        }
      }
#pragma unroll
      for (int k = 0; k < NS; ++k)
        if (s == k) {
          if (CG == 1 || r / 16 == k % 2) {
#pragma unroll
            for (int i = 0; i < CG; ++i)
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                const f32x16& v = acc[CG * ip + i][k / CG];
                *(float4*)(part + (CG == 1 ? r : r % 16) * RS + (32 * i + 8 * g + 4 * h) * 4) =
                    make_float4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]);
              }
          }
          if constexpr (RES && AHEAD) {
            now[0] = res[ip][k][0];
            now[1] = res[ip][k][1];
          }
        }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll 1
      for (int it = 0; it < 2; ++it) {
        const uint8_t* at = part + (TR / 2 * it + row) * RS + 4 * c;
        float v[8];
        *(float4*)&v[0] = *(const float4*)at;
        *(float4*)&v[4] = *(const float4*)(at + 16);
        if (x.bias != nullptr) {
          const float* b = &biases[wave][32 * CG * ip + c];
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] += b[j];
        }
        finish8<RES>(x, v, it == 0 ? now[0] : now[1], o, N - n, at_row < rows && n < N);
        go_on(o, step);
        at_row += TR / 2;
      }
      __builtin_amdgcn_wave_barrier();
    }
  }
}

// OCC: waves a SIMD that the registers are to leave room for.  blockIdx.y: one of gridDim.y ranges of
// `split` stages of K; range z's sums go to Y + z M ld_y (YT 2).
template <int AF, int YT, int BM, int BN, int WM, int WN, int NS, int OCC, class X = NoExtra>
__global__ __launch_bounds__(WM* WN* kWave, OCC) void mx_tile_kernel(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ as, int64_t M, const uint8_t* __restrict__ W,
    const uint8_t* __restrict__ ws, int64_t N, int64_t K, int n_mt, int n_nt, int group_m, int split,
    void* __restrict__ Y, int64_t ld_y, const X x = X()) {
  constexpr int NW = WM * WN;
  constexpr int MT = BM / WM / 32, NT = BN / WN / 32;
  constexpr int AB = AF == kMxFp8 ? 128 : 64;   // bytes of a row's stage
  constexpr int WB = 64;
  constexpr int AI = BM * AB / 1024 / NW, WI = BN * WB / 1024 / NW;  // direct loads a wave and stage
  constexpr int ND = AI + WI;
  constexpr int NR = NT + MT * (AF == kMxFp8 ? 2 : 1);               // LDS reads of a step's fragments
  // one array a slot (A tile, then W tile): fragment reads then visibly do not touch the loads in flight
  __shared__ __attribute__((aligned(1024))) uint8_t s0[BM * AB + BN * WB];
  __shared__ __attribute__((aligned(1024))) uint8_t s1[BM * AB + BN * WB];
  __shared__ __attribute__((aligned(1024))) uint8_t s2[BM * AB + BN * WB];
  __shared__ __attribute__((aligned(1024))) uint8_t s3[NS > 3 ? BM * AB + BN * WB : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t s4[NS > 3 ? BM * AB + BN * WB : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t s5[NS > 3 ? BM * AB + BN * WB : 16];
  __shared__ uint32_t sS[2 * (BM + BN) * 3];     // scale bytes of three stages, a row's side by side

  const int kb = (int)(K / kMxBlock);
  int mt = 0, nt;
  int64_t m0;
  if constexpr (X::kGroups) {  // n_mt: at least the tiles of rows that there are
    const GroupTile g = group_pick(x, (int)M, BM, [&](int total) {
      if (total > n_mt || (int)blockIdx.x >= total * n_nt) return -1;  // more than n_mt: offsets descend
      block_tile((int)blockIdx.x, total * n_nt, total, n_nt, group_m, &mt, &nt);
      return mt;
    });
    if (g.group < 0) return;
    m0 = g.first;
    M = g.end;
    W += (int64_t)g.group * N * (K / 2);
    ws += (int64_t)g.group * N * kb;
  } else {
    block_tile((int)blockIdx.x, (int)gridDim.x, n_mt, n_nt, group_m, &mt, &nt);
    m0 = (int64_t)mt * BM;
  }
  const int64_t n0 = (int64_t)nt * BN;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int k0 = (int)blockIdx.y * split;  // first stage
  const int nk = min((int)((K + kMxStage - 1) / kMxStage) - k0, split);
  const uint32_t a_row = (uint32_t)(AF == kMxFp8 ? K : K / 2), w_row = (uint32_t)(K / 2);
  const int m_rows = (int)(M - m0 < BM ? M - m0 : BM), n_rows = (int)(N - n0 < BN ? N - n0 : BN);

  // direct loads: lane i of load j fills 16 bytes i of the wave's j-th KiB.  Rows past the end are out of
  // the buffer's range and read as zeros (their results are not stored).  A last stage that K does not fill
  // takes the row's last 128 values instead: the scales of those already summed are 0 on both sides, so that
  // they add 0.
  const uint8_t* a_tile = A + m0 * a_row;
  const uint8_t* w_tile = W + n0 * w_row;
  uint32_t a_bytes = (uint32_t)m_rows * a_row;
  const uint32_t w_bytes = (uint32_t)n_rows * w_row;
  if constexpr (X::kGroups) {
    if (x.rows != nullptr) a_tile = A, a_bytes = (uint32_t)x.a_rows * a_row;
  }
  uint32_t va[AI], vw[WI];
#pragma unroll
  for (int j = 0; j < AI; ++j) {
    const int row = (wave * AI + j) * (1024 / AB) + lane / (AB / 16), slot = lane % (AB / 16);
    const uint32_t piece = 16u * (uint32_t)(slot ^ (AF == kMxFp8 ? swz8(row) : swz4(row)));
    va[j] = row < m_rows ? (uint32_t)row * a_row + piece : kMxOut;
    if constexpr (X::kGroups) {
      if (x.rows != nullptr && row < m_rows) {
        const int64_t of = group_row(x, (int)(m0 + row));
        va[j] = of < 0 ? kMxOut : (uint32_t)of * a_row + piece;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < WI; ++j) {
    const int row = (wave * WI + j) * 16 + lane / 4;
    vw[j] = row < n_rows ? (uint32_t)row * w_row + 16u * (uint32_t)((lane % 4) ^ swz4(row)) : kMxOut;
  }
  auto load_stage = [&](uint8_t* dst, int kt) {
    const uint32_t ka = min((uint32_t)(k0 + kt) * AB, a_row - AB), kw = min((uint32_t)(k0 + kt) * WB, w_row - WB);
#pragma unroll
    for (int j = 0; j < AI; ++j) load_lds16(a_tile, a_bytes, dst + (wave * AI + j) * 1024, va[j], ka);
#pragma unroll
    for (int j = 0; j < WI; ++j) load_lds16(w_tile, w_bytes, dst + BM * AB + (wave * WI + j) * 1024, vw[j], kw);
  };

  // scales: a thread carries the 12 bytes of its rows for the next three stages; near the row's end the
  // 12 last bytes are loaded and shifted down, with zeros behind them
  constexpr int SR = (BM + BN + NW * kWave - 1) / (NW * kWave);
  uint3 sc[SR];
  const uint8_t* srow[SR];
  int srow_i[SR];
  bool no_row[SR];  // not in A: its scales count as 0
#pragma unroll
  for (int q = 0; q < SR; ++q) {
    srow_i[q] = min(tid + q * NW * kWave, BM + BN - 1);
    int64_t a_of = m0 + min(srow_i[q], m_rows - 1);
    no_row[q] = false;
    if constexpr (X::kGroups) {
      if (srow_i[q] < BM) a_of = group_row(x, (int)a_of);
      no_row[q] = a_of < 0;
      a_of = a_of < 0 ? 0 : a_of;
    }
    srow[q] = srow_i[q] < BM ? as + a_of * kb : ws + (n0 + min(srow_i[q] - BM, n_rows - 1)) * kb;
  }
  auto load_scales = [&](int ss) {
#pragma unroll
    for (int q = 0; q < SR; ++q) sc[q] = ld_any<uint3>(srow[q] + min(4 * k0 + 12 * ss, kb - 12));
  };
  auto write_scales = [&](int ss) {
    const int b0 = 4 * k0 + 12 * ss, shift = b0 - min(b0, kb - 12);  // blocks, bytes
    const int words = shift >> 2, bits = 8 * (shift & 3);
#pragma unroll
    for (int q = 0; q < SR; ++q) {
      const uint32_t v[3] = {X::kGroups && no_row[q] ? 0 : sc[q].x, X::kGroups && no_row[q] ? 0 : sc[q].y,
                             X::kGroups && no_row[q] ? 0 : sc[q].z};
#pragma unroll
      for (int d = 0; d < 3; ++d) {
        uint32_t lo = 0, hi = 0;
#pragma unroll
        for (int e = d; e < 3; ++e) {
          lo = words == e - d ? v[e] : lo;
          hi = words == e - d - 1 ? v[e] : hi;
        }
        const int left = kb - b0 - 4 * d;  // blocks from the stage's first on
        sS[((ss & 1) * (BM + BN) + srow_i[q]) * 3 + d] =
            (uint32_t)((((uint64_t)hi << 32) | lo) >> bits) << (left > 0 && left < 4 ? 8 * (4 - left) : 0);
      }
    }
  };

  // fragments: lane l holds row l % 32 of a tile, h = l / 32
  const int r = lane & 31, h = lane >> 5;
  const int a_base = (wm * MT * 32 + r) * AB, w_base = BM * AB + (wn * NT * 32 + r) * WB;
  struct Frags {
    i32x8 a[MT];
    uint4 w[NT];
  };
  struct Scales {
    int a[MT], w[NT];
  };
  auto read_frags = [&](Frags& f, const uint8_t* tile, int step) {
#pragma unroll
    for (int i = 0; i < NT; ++i)
      f.w[i] = *(const uint4*)(tile + w_base + i * 32 * WB + 16 * ((2 * step + h) ^ swz4(r)));
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const uint8_t* p = tile + a_base + i * 32 * AB;
      if constexpr (AF == kMxFp8)
        f.a[i] = both4(*(const uint4*)(p + 16 * ((4 * step + h) ^ swz8(r))),
                       *(const uint4*)(p + 16 * ((4 * step + 2 + h) ^ swz8(r))));
      else
        f.a[i] = lo4(*(const uint4*)(p + 16 * ((2 * step + h) ^ swz4(r))));
    }
  };
  auto read_scales = [&](Scales& s, int ss, int d) {
    const uint32_t* p = sS + (ss & 1) * (BM + BN) * 3;
#pragma unroll
    for (int i = 0; i < MT; ++i) s.a[i] = (int)p[3 * (wm * MT * 32 + 32 * i + r) + d];
#pragma unroll
    for (int i = 0; i < NT; ++i) s.w[i] = (int)p[3 * (BM + wn * NT * 32 + 32 * i + r) + d];
  };
  auto own_bytes = [&](Scales& s, const Scales& raw) {  // the lane's blocks to bytes 0 and 2
#pragma unroll
    for (int i = 0; i < MT; ++i) s.a[i] = (int)((uint32_t)raw.a[i] >> (8 * h));
#pragma unroll
    for (int i = 0; i < NT; ++i) s.w[i] = (int)((uint32_t)raw.w[i] >> (8 * h));
  };
  f32x16 acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  auto products = [&](const Frags& f, const Scales& s, int step) {
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[i][j] = mfma_mx32<AF>(lo4(f.w[i]), f.a[j], acc[i][j], s.w[i], s.a[j], step);
  };

  load_scales(0);
  hold_order();
  load_stage(s0, 0);
  load_stage(s1, 1);
  if constexpr (NS > 3) {
    load_stage(s2, 2);
    load_stage(s3, 3);
    load_stage(s4, 4);
  }
  hold_order();
  write_scales(0);
  load_scales(1);
  wait_loads<(NS - 2) * ND>();
  block_barrier();
  Frags f0, f1;
  Scales c0, c1;
  read_frags(f0, s0, 0);
  read_scales(c1, 0, 0);

  // Stage kt in slot P = kt % NS (array C), its step-0 fragments read.  Before the barrier every wave has
  // read the rest of the stage (lgkmcnt 0), so its slot may be filled again by stage kt + NS; and stage
  // kt + 1 (array X) has landed: only the loads of the NS - 2 stages behind it are younger.  Loads past the
  // last stage repeat its last chunks.
#define AWQ_MX_STAGE(P, C, X, F)                      \
  {                                                   \
    own_bytes(c0, c1);                                \
    read_frags(f1, C, 1);                             \
    load_stage(F, kt + NS - 1);                       \
    if (P % 3 == 2) write_scales(ss + 1);             \
    products(f0, c0, 0);                              \
    interleave<NR, ND>();                             \
    __builtin_amdgcn_sched_barrier(0);                \
    wait_loads<(NS - 2) * ND>();                      \
    block_barrier();                                  \
    __builtin_amdgcn_sched_barrier(0);                \
    if (P % 3 == 2) load_scales(ss + 2);              \
    read_scales(c1, ss + (P % 3 == 2), (P + 1) % 3);  \
    read_frags(f0, X, 0);                             \
    products(f1, c0, 1);                              \
    interleave<NR + (MT + NT) / 2, 0>();              \
    __builtin_amdgcn_sched_barrier(0);                \
    ++kt;                                             \
    if (P % 3 == 2) ++ss;                             \
  }
  int kt = 0, ss = 0;  // ss = kt / 3
  if constexpr (NS == 3) {
    while (kt + 3 <= nk) {
      AWQ_MX_STAGE(0, s0, s1, s2)
      AWQ_MX_STAGE(1, s1, s2, s0)
      AWQ_MX_STAGE(2, s2, s0, s1)
    }
    if (kt < nk) AWQ_MX_STAGE(0, s0, s1, s2)
    if (kt < nk) AWQ_MX_STAGE(1, s1, s2, s0)
  } else {
    while (kt + 6 <= nk) {
      AWQ_MX_STAGE(0, s0, s1, s5)
      AWQ_MX_STAGE(1, s1, s2, s0)
      AWQ_MX_STAGE(2, s2, s3, s1)
      AWQ_MX_STAGE(3, s3, s4, s2)
      AWQ_MX_STAGE(4, s4, s5, s3)
      AWQ_MX_STAGE(5, s5, s0, s4)
    }
    if (kt < nk) AWQ_MX_STAGE(0, s0, s1, s5)
    if (kt < nk) AWQ_MX_STAGE(1, s1, s2, s0)
    if (kt < nk) AWQ_MX_STAGE(2, s2, s3, s1)
    if (kt < nk) AWQ_MX_STAGE(3, s3, s4, s2)
    if (kt < nk) AWQ_MX_STAGE(4, s4, s5, s3)
  }
#undef AWQ_MX_STAGE

  wait_loads<0>();  // none may land after the block has given its LDS back
  block_barrier();

  if constexpr (X::kEpi)
    store_tile_epi<MT, NT, NW, BM * AB + BN * WB, 3, true>(acc, s0, s1, s2, wave, lane, m0 + wm * MT * 32, n0 + wn * NT * 32, M,
                                                     N, Y, ld_y, x);
  else
    store_tile<YT, MT, NT, NW, BM * AB + BN * WB>(acc, s0, s1, s2, wave, lane, m0 + wm * MT * 32, n0 + wn * NT * 32, M, N,
                                                 YT == 2 ? (float*)Y + (int64_t)blockIdx.y * M * ld_y : Y, ld_y);
}

// ---------------------------------------------------------------------------
// Large products: 256 x 256 tiles.  The scale bytes of a stage lie in a line of
// their own for each row, so they are first laid out stage by stage
// (stage_scales_kernel): a stage then takes 16 or 32 lines of them instead of 512.
//
// 4-bit activations, stages of 256 K: the loads that reach the second-level cache
// bound them (8192^3 in stages of 128 K: 301 us, of which 252 remain with the loads
// alone), so every row of a stage is a whole 128-byte line, in two LDS slots.
// ---------------------------------------------------------------------------
constexpr int kBigStage = 256;

// Groups' tiles and row offsets, as stage_groups_kernel leaves them
struct StagedGroups {
  const int4* tab;
  const uint32_t* a_at;
};

// out[w][row] (rows: the A rows, then the W rows, each padded to whole tiles): word w of the row's scale bytes,
// SB / 4 words a stage.  A last stage that K does not fill holds the row's last SB blocks, 0 in the place of
// those of earlier stages; padded rows hold 0.
template <int SB>
__global__ __launch_bounds__(256) void stage_scales_kernel(const uint8_t* __restrict__ as, int64_t M,
                                                           const uint8_t* __restrict__ ws, int64_t N, int kb,
                                                           int64_t m_pad, int64_t rows, uint32_t* __restrict__ out) {
  const int64_t row = (int64_t)blockIdx.x * 256 + threadIdx.x;  // rows is a multiple of 256
  const bool is_a = row < m_pad;
  const int64_t r = is_a ? row : row - m_pad;
  const bool live = r < (is_a ? M : N);
  const uint8_t* p = (is_a ? as : ws) + (live ? r : 0) * kb;
  const int s0 = (int)blockIdx.y * (16 / SB), n_stage = (kb + SB - 1) / SB;  // 16 blocks a thread
  uint32_t v[4] = {0, 0, 0, 0};
  if (live) {
    if ((s0 + 16 / SB) * SB <= kb) {
      const uint4 u = ld_any<uint4>(p + s0 * SB);
      v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int b0 = (s0 + i / SB) * SB;                          // the stage's first block
        const int b = (b0 + SB <= kb ? b0 : kb - SB) + i % SB;      // the byte's
        if (b0 < kb && b >= b0) v[i / 4] |= (uint32_t)p[b] << (8 * (i % 4));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (s0 + i * 4 / SB < n_stage) out[(int64_t)(s0 * (SB / 4) + i) * rows + row] = v[i];
}

// Tile t of all groups' 256-row tiles, its place among them with those of more than 128 rows first, and the numbers of
// both kinds.  Every lane of a wave takes part.
struct GroupPlace {
  GroupTile tile;
  int place, full, half;
};
__device__ __forceinline__ GroupPlace group_place(const Groups& g, int M, int t) {
  GroupPlace p = {{-1, 0, 0}, 0, 0, 0};
  int tiles = 0, half = 0;  // of the groups before
  bool is_half = false;
  for (int e0 = 0; e0 < g.n; e0 += kWave) {
    const GroupSpan s = group_span(g, M, kBigTile, e0);
    const int last = (s.end - s.first) % kBigTile;
    const uint64_t halves = __ballot(last > 0 && last <= kHalfTile);  // groups whose last tile is half a one
    const int total = span_total(s);
    if (t >= tiles && t < tiles + total) {
      p.tile = span_tile(s, e0, kBigTile, t - tiles);
      const int l = p.tile.group - e0, before = half + __popcll(halves & ((1ull << l) - 1));
      is_half = p.tile.end - p.tile.first <= kHalfTile;
      p.place = is_half ? before : t - before;
    }
    tiles += total;
    half += __popcll(halves);
  }
  p.full = tiles - half;
  p.half = half;
  if (is_half) p.place += p.full;
  return p;
}

// The same for groups, with the rows of each group's tiles one after another (n_mt tiles at least) and the padded rows
// of every group's weight behind them; rows of no tile and of groups without rows are not written.  tab[place]: a
// tile's group, first row, end and scale rows; tab[n_mt]: the numbers of full and of half tiles.  a_at[row]: offset of
// the row's codes in A.
template <int SB>
__global__ __launch_bounds__(256) void stage_groups_kernel(const Groups g, const uint8_t* __restrict__ as, int M,
                                                           uint32_t a_row, const uint8_t* __restrict__ ws, int64_t N,
                                                           int64_t n_pad, int kb, int n_mt, int64_t rows,
                                                           uint32_t* __restrict__ out, int4* __restrict__ tab,
                                                           uint32_t* __restrict__ a_at) {
  // a block takes 128 bytes of 256 rows through LDS, so that both sides are read and written in whole lines (32 x 4096
  // x 128 bytes of weight scales: 25 us by threads that each take 16 bytes of a row, 12 us so)
  constexpr int CB = 128, LS = CB + 4;
  __shared__ __attribute__((aligned(16))) uint8_t bytes[256 * LS];
  __shared__ int64_t from[256];
  const int tid = (int)threadIdx.x;
  const int64_t row = (int64_t)blockIdx.x * 256 + tid;  // whole tiles
  const uint8_t* p;
  if ((int)blockIdx.x < n_mt) {
    const GroupPlace at = group_place(g, M, (int)blockIdx.x);
    const GroupTile& t = at.tile;
    // offsets that descend can name rows more than once, and more tiles than the table has places for: then none
    const bool over = at.full + at.half > n_mt;
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0)
      tab[n_mt] = over ? make_int4(0, 0, 0, 0) : make_int4(at.full, at.half, 0, 0);
    if (over || t.group < 0) return;
    const int m = t.first + tid;
    const int64_t of = m < t.end ? group_row(g, m) : -1;
    from[tid] = of;
    p = as;
    if (blockIdx.y == 0) {
      if (tid == 0) tab[at.place] = make_int4(t.group, t.first, t.end, (int)blockIdx.x * kBigTile);
      // the rows of each 32 in the order in which 8 lanes take every 8th of them
      const int place = (tid & ~31) | (tid & 7) << 2 | (tid >> 3 & 3);
      if (g.rows != nullptr) a_at[row - tid + place] = of >= 0 ? (uint32_t)of * a_row : kMxOut;
    }
  } else {
    const int64_t r = row - (int64_t)n_mt * kBigTile;
    const int e = (int)(r / n_pad);  // the same for the block
    const int first = clamp_int(g.offsets[e], 0, M);
    if (g.offsets[e + 1] <= first || first == M) return;
    from[tid] = r - e * n_pad < N ? e * N + (r - e * n_pad) : -1;
    p = ws;
  }
  __syncthreads();
  const int c0 = (int)blockIdx.y * CB;  // the first byte of each row
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = tid / 8 + 32 * i, c = 16 * (tid % 8);
    uint32_t v[4] = {0, 0, 0, 0};
    if (from[r] >= 0) {
      const uint8_t* at = p + from[r] * kb + c0 + c;
      if (c0 + c + 16 <= kb) {
        const uint4 u = ld_any<uint4>(at);
        v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
      } else {
#pragma unroll
        for (int b = 0; b < 16; ++b)
          if (c0 + c + b < kb) v[b / 4] |= (uint32_t)at[b] << (8 * (b % 4));
      }
    }
#pragma unroll
    for (int d = 0; d < 4; ++d) *(uint32_t*)(bytes + r * LS + c + 4 * d) = v[d];
  }
  __syncthreads();
  const uint8_t* mine = bytes + tid * LS;
  const int words = (kb + SB - 1) / SB * (SB / 4);
#pragma unroll 4
  for (int d = 0; d < CB / 4; ++d) {
    const int w = c0 / 4 + d, b0 = w * 4 / SB * SB;  // the word, its stage's first block
    if (w >= words) break;
    uint32_t v = 0;
    if (b0 + SB <= kb) {
      v = *(const uint32_t*)(mine + 4 * d);
    } else {  // the row's last SB blocks, 0 in the place of those of earlier stages
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int b = kb - SB + (4 * w - b0) + i;
        if (b >= b0) v |= (uint32_t)mine[b - c0] << (8 * i);
      }
    }
    out[(int64_t)w * rows + row] = v;
  }
}

template <int YT, class X = NoExtra>
__global__ __launch_bounds__(512, 2) void mx_big_kernel(const uint8_t* __restrict__ A, int64_t M,
                                                        const uint8_t* __restrict__ W, int64_t N, int64_t K,
                                                        const uint32_t* __restrict__ sc, int64_t m_pad, int64_t rows,
                                                        int n_mt, int n_nt, int group_m, void* __restrict__ Y,
                                                        int64_t ld_y, const X x = X(), const StagedGroups sg = {}) {
  constexpr int T = kBigTile;
  constexpr int WM = 4, WN = 2, NW = 8, MT = T / WM / 32, NT = T / WN / 32;
  constexpr int RB = kBigStage / 2;                    // bytes of a row's stage
  constexpr int DI = T * RB / 1024 / NW;               // direct loads of codes a wave and stage, for each operand
  constexpr int SW = 2;                                // scale words of a row's stage
  constexpr int NR = NT + MT;                          // LDS reads of a step's fragments
  constexpr int oW = T * RB, oS = 2 * T * RB, SB = oS + SW * 2 * T * 4;
  // one array a slot (A tile, W tile, scale words): fragment reads then visibly do not touch the loads in flight
  __shared__ __attribute__((aligned(1024))) uint8_t s0[SB];
  __shared__ __attribute__((aligned(1024))) uint8_t s1[SB];

  int mt, nt;
  if constexpr (X::kGroups) {
    const int4 n = sg.tab[n_mt];
    const int xcd = (int)blockIdx.x % kMxXcds, pos = (int)blockIdx.x / kMxXcds;
    if (pos >= group_tiles_of_xcd(xcd, n.x, n.y, n_nt)) return;
    group_tile_at(xcd, pos, n.x, n.y, n_nt, group_m, &mt, &nt);
  } else {
    block_tile((int)blockIdx.x, (int)gridDim.x, n_mt, n_nt, group_m, &mt, &nt);
  }
  int64_t m0 = (int64_t)mt * T;
  const int64_t n0 = (int64_t)nt * T;
  int64_t sc_m = m0, sc_n = m_pad + n0;  // the tile's scale rows
  if constexpr (X::kGroups) {
    const int4 g = sg.tab[mt];
    m0 = g.y;
    M = g.z;
    sc_m = g.w;
    W += (int64_t)g.x * N * (K / 2);
    sc_n += g.x * ((int64_t)n_nt * T);
  }
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int nk = (int)((K + kBigStage - 1) / kBigStage);
  const uint32_t row_bytes = (uint32_t)(K / 2);
  const int m_rows = (int)(M - m0 < T ? M - m0 : T), n_rows = (int)(N - n0 < T ? N - n0 : T);

  // direct loads: lane i of load j fills 16 bytes i of the wave's j-th KiB.  Rows past the end are out of
  // the buffer's range and read as zeros.  A last stage that K does not fill takes the row's last 256
  // values.
  const uint8_t* a_tile = A + m0 * row_bytes;
  const uint8_t* w_tile = W + n0 * row_bytes;
  uint32_t a_bytes = (uint32_t)m_rows * row_bytes;
  const uint32_t w_bytes = (uint32_t)n_rows * row_bytes;
  if constexpr (X::kGroups) {
    if (x.rows != nullptr) a_tile = A, a_bytes = (uint32_t)x.a_rows * row_bytes;
  }
  uint32_t va[DI], vw[DI];
#pragma unroll
  for (int j = 0; j < DI; ++j) {
    const int row = (wave * DI + j) * 8 + lane / 8;
    const uint32_t at = (uint32_t)row * row_bytes + 16u * (uint32_t)(lane % 8 ^ swz8(row));
    va[j] = row < m_rows ? at : kMxOut;
    vw[j] = row < n_rows ? at : kMxOut;
    if constexpr (X::kGroups) {
      if (x.rows != nullptr)
        va[j] = sg.a_at[sc_m + 32 * wave + 4 * (lane / 8) + j] + 16u * (uint32_t)(lane % 8 ^ swz8(row));
    }
  }
  // scales: the wave's 64 of the tile's 256 + 256 rows; words past the last stage's are not read
  const int64_t s_row = wave < 4 ? sc_m + 64 * wave : sc_n + 64 * (wave - 4);
  auto load_stage = [&](uint8_t* dst, int kt) {
    const uint32_t kt_off = min((uint32_t)kt * RB, row_bytes - RB);
#pragma unroll
    for (int j = 0; j < DI; ++j) load_lds16(a_tile, a_bytes, dst + (wave * DI + j) * 1024, va[j], kt_off);
#pragma unroll
    for (int j = 0; j < DI; ++j) load_lds16(w_tile, w_bytes, dst + oW + (wave * DI + j) * 1024, vw[j], kt_off);
#pragma unroll
    for (int j = 0; j < SW; ++j)
      load_lds4(sc + ((int64_t)min(kt, nk - 1) * SW + j) * rows + s_row, 256, dst + oS + (j * 2 * T + 64 * wave) * 4,
                4u * (uint32_t)lane);
  };

  // fragments: lane l holds row l % 32 of a tile, h = l / 32
  const int r = lane & 31, h = lane >> 5;
  const int a_base = (wm * MT * 32 + r) * RB, w_base = oW + (wn * NT * 32 + r) * RB;
  struct Frags {
    uint4 a[MT], w[NT];
  };
  struct Scales {
    uint32_t a[MT][SW], w[NT][SW];
  };
  auto read_frags = [&](Frags& f, const uint8_t* tile, int step) {
    const int c = 16 * ((2 * step + h) ^ swz8(r));
#pragma unroll
    for (int i = 0; i < NT; ++i) f.w[i] = *(const uint4*)(tile + w_base + i * 32 * RB + c);
#pragma unroll
    for (int i = 0; i < MT; ++i) f.a[i] = *(const uint4*)(tile + a_base + i * 32 * RB + c);
  };
  auto read_scales = [&](Scales& s, const uint8_t* tile) {
    const uint32_t* p = (const uint32_t*)(tile + oS);
#pragma unroll
    for (int w = 0; w < SW; ++w) {
#pragma unroll
      for (int i = 0; i < MT; ++i) s.a[i][w] = p[w * 2 * T + wm * MT * 32 + 32 * i + r];
#pragma unroll
      for (int i = 0; i < NT; ++i) s.w[i][w] = p[w * 2 * T + T + wn * NT * 32 + 32 * i + r];
    }
  };
  auto own_bytes = [&](Scales& s, const Scales& raw) {  // the lane's blocks to bytes 0 and 2
#pragma unroll
    for (int w = 0; w < SW; ++w) {
#pragma unroll
      for (int i = 0; i < MT; ++i) s.a[i][w] = raw.a[i][w] >> (8 * h);
#pragma unroll
      for (int i = 0; i < NT; ++i) s.w[i][w] = raw.w[i][w] >> (8 * h);
    }
  };
  f32x16 acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  auto products = [&](const Frags& f, const Scales& s, int step) {
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int i = 0; i < NT; ++i)
        acc[i][j] = mfma_mx32<kMxFp4>(lo4(f.w[i]), lo4(f.a[j]), acc[i][j], (int)s.w[i][step / 2],
                                      (int)s.a[j][step / 2], step % 2);
  };

  Frags f0, f1;
  Scales c0, c1;
  load_stage(s0, 0);
  load_stage(s1, 1);
  wait_loads<2 * DI + SW>();
  block_barrier();
  read_scales(c1, s0);
  read_frags(f0, s0, 0);

  // Stage kt (array C), its step-0 fragments and scales read.  At the barrier, ahead of the last step, every
  // wave has read the whole stage (lgkmcnt 0) and stage kt + 1 (array X) has landed: C may be filled again.
  // Loads past the last stage repeat it.
#define AWQ_MX_STEP(F, G, C, S)          \
  read_frags(G, C, S + 1);               \
  products(F, c0, S);                    \
  interleave<NR, 0>();                   \
  __builtin_amdgcn_sched_barrier(0);
  // waves without rows only load
  constexpr bool kParts = X::kGroups;
  const bool active = !kParts || m0 + wm * MT * 32 < M;
#define AWQ_MX_STAGE(C, X)                               \
  if (kParts && !active) {                               \
    wait_loads<0>();                                     \
    block_barrier();                                     \
    load_stage(C, kt + 2);                               \
    ++kt;                                                \
  } else {                                               \
    own_bytes(c0, c1);                                   \
    AWQ_MX_STEP(f0, f1, C, 0)                            \
    AWQ_MX_STEP(f1, f0, C, 1)                            \
    AWQ_MX_STEP(f0, f1, C, 2)                            \
    wait_loads<0>();                                     \
    block_barrier();                                     \
    __builtin_amdgcn_sched_barrier(0);                   \
    load_stage(C, kt + 2);                               \
    read_scales(c1, X);                                  \
    read_frags(f0, X, 0);                                \
    products(f1, c0, 3);                                 \
    interleave<NR + SW * (MT + NT) / 2, 2 * DI + SW>();  \
    __builtin_amdgcn_sched_barrier(0);                   \
    ++kt;                                                \
  }
  int kt = 0;
  while (kt + 2 <= nk) {
    AWQ_MX_STAGE(s0, s1)
    AWQ_MX_STAGE(s1, s0)
  }
  if (kt < nk) {
    AWQ_MX_STAGE(s0, s1)
  }
#undef AWQ_MX_STAGE
#undef AWQ_MX_STEP
  wait_loads<0>();  // none may land after the block has given its LDS back
  block_barrier();
  if constexpr (X::kEpi)
    store_tile_epi<MT, NT, NW, SB, 2, true>(acc, s0, s1, s1, wave, lane, m0 + wm * MT * 32, n0 + wn * NT * 32, M, N, Y, ld_y, x);
  else
    store_tile<YT, MT, NT, NW, SB / 2>(acc, s0, s1, s1 + SB / 2, wave, lane, m0 + wm * MT * 32, n0 + wn * NT * 32, M, N,
                                       Y, ld_y);
}

// The arguments of mx_big8_kernel as they lie in its argument block.  The epilogue reads its own ones there, behind a
// pointer that the compiler cannot see through: kept in scalar registers meanwhile they would push addresses of the
// stages into scratch memory, and each of those reloads waits for all loads in flight (4096 x 12288 x 4096: 1064 us).
template <class X>
struct Big8Args {
  const uint8_t* A;
  int64_t M;
  const uint8_t* W;
  int64_t N, K;
  const uint32_t* sc;
  int64_t m_pad, rows;
  int n_mt, n_nt, group_m;
  void* Y;
  int64_t ld_y;
  X x;
  StagedGroups sg;
};
template <class X>
__device__ __forceinline__ X own_extra() {
  typedef __attribute__((address_space(4))) const uint64_t* words;
  static_assert(sizeof(X) % 8 == 0 && offsetof(Big8Args<X>, x) % 8 == 0, "whole words");
  words p = (words)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  uint64_t w[sizeof(X) / 8];
#pragma unroll
  for (size_t i = 0; i < sizeof(X) / 8; ++i) w[i] = p[offsetof(Big8Args<X>, x) / 8 + i];
  X x;
  __builtin_memcpy(&x, w, sizeof(X));
  return x;
}

// 8-bit activations, stages of 128 K in three LDS slots as in mx_tile_kernel, each with its scale words.  At
// most a block for each compute unit: it goes on to its next tile without a stop, whose first two stages are
// loaded behind the last two of the one before.  A tile that starts in a block of its own costs 6.3 us, one
// that follows 3.6 (the results, stored by way of the slot that the last stage leaves, go out while all other
// blocks store theirs).  4096 x 24576 x 4096: 299-306 us, 315 with a block for each tile; 8192^3: 378 us, 2.9
// PFLOP/s (383); the matrix cores alone take 301 us there at the clock that they leave.
template <int YT, class X = NoExtra, bool GATHER = false>
__global__ __launch_bounds__(512, 2) void mx_big8_kernel(const uint8_t* __restrict__ A, int64_t M,
                                                         const uint8_t* __restrict__ W, int64_t N, int64_t K,
                                                         const uint32_t* __restrict__ sc, int64_t m_pad, int64_t rows,
                                                         int n_mt, int n_nt, int group_m, void* __restrict__ Y,
                                                         int64_t ld_y, const X x = X(), const StagedGroups sg = {}) {
  constexpr int T = kBigTile;
  constexpr int WM = 4, WN = 2, NW = 8, MT = T / WM / 32, NT = T / WN / 32;
  constexpr int AB = 128, WB = 64;                                    // bytes of a row's stage
  constexpr int AI = T * AB / 1024 / NW, WI = T * WB / 1024 / NW;     // direct loads of codes a wave and stage
  constexpr int ND = AI + WI + 1 + (GATHER ? 1 : 0);                  // one of scales, and one of row offsets
  constexpr int NR = NT + 2 * MT;                                     // LDS reads of a step's fragments
  constexpr int oW = T * AB, oS = oW + T * WB, oO = oS + 2 * T * 4, SB = oO + (GATHER ? NW * 256 : 0);
  __shared__ __attribute__((aligned(1024))) uint8_t s0[SB];
  __shared__ __attribute__((aligned(1024))) uint8_t s1[SB];
  __shared__ __attribute__((aligned(1024))) uint8_t s2[SB];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int nk = (int)((K + kMxStage - 1) / kMxStage);
  // the block's tiles: every `step`th of `tiles` from tile on; groups: of its XCD's
  int tile = (int)blockIdx.x, step = (int)gridDim.x, tiles = n_mt * n_nt;
  int n_full = 0, n_half = 0;
  const int xcd = (int)blockIdx.x % kMxXcds;
  if constexpr (X::kGroups) {
    const int4 n = sg.tab[n_mt];
    n_full = n.x, n_half = n.y;
    tiles = group_tiles_of_xcd(xcd, n_full, n_half, n_nt);
    tile = (int)blockIdx.x / kMxXcds, step = (int)gridDim.x / kMxXcds;
    if (tile >= tiles) return;
  }
  const uint32_t a_row = (uint32_t)K, w_row = (uint32_t)(K / 2);

  // loads: the tile and stage that come next
  uint32_t va[AI], vw[WI];
#pragma unroll
  for (int j = 0; j < AI; ++j) {
    const int row = (wave * AI + j) * (1024 / AB) + lane / (AB / 16);
    va[j] = (uint32_t)row * a_row + 16u * (uint32_t)(lane % (AB / 16) ^ swz8(row));
  }
#pragma unroll
  for (int j = 0; j < WI; ++j) {
    const int row = (wave * WI + j) * 16 + lane / 4;
    vw[j] = (uint32_t)row * w_row + 16u * (uint32_t)((lane % 4) ^ swz4(row));
  }
  // where a tile is: its group, first row and end, the first output, its scale rows
  struct Place {
    int m0, n0, end, group, sc;
  };
  auto tile_at = [&](int id) {
    if constexpr (X::kGroups) {
      int mt, nt;
      const bool some = id < tiles;
      group_tile_at(xcd, some ? id : 0, n_full, n_half, n_nt, group_m, &mt, &nt);
      const int4 g = sg.tab[mt];
      return Place{some ? g.y : g.z, some ? nt * T : (int)N, g.z, g.x, g.w};
    } else {
      const TileAt t = big_tile_at(id, n_mt, n_nt, group_m, (int)M, (int)N);
      return Place{t.m0, t.n0, (int)M, 0, t.m0};
    }
  };
  Place now = tile_at(tile), then = tile_at(tile + step);  // computed, computed next
  Place src = now;  // loaded
  int l_k = 0;     // and its stage that is loaded next
  // GATHER: the offsets of a tile's rows, 32 of each wave, come with the stage that is computed when they are needed,
  // two stages ahead of the one that they are for (a tile has at least four).  at: where the first ones come from
  auto load_stage = [&](uint8_t* dst, const void* at) {
    if constexpr (GATHER) {
      const uint4 v = *(const uint4*)at;
      const uint32_t piece = 16u * (uint32_t)(lane % 8 ^ lane / 8);
      va[0] = v.x + piece, va[1] = v.y + (piece ^ 16), va[2] = v.z + piece, va[3] = v.w + (piece ^ 16);
    }
    const int m0 = __builtin_amdgcn_readfirstlane(src.m0), n0 = __builtin_amdgcn_readfirstlane(src.n0);
    const int k = __builtin_amdgcn_readfirstlane(l_k);
    const int end = X::kGroups ? __builtin_amdgcn_readfirstlane(src.end) : (int)M;
    const int group = X::kGroups ? __builtin_amdgcn_readfirstlane(src.group) : 0;
    const int sc_m = X::kGroups ? __builtin_amdgcn_readfirstlane(src.sc) : m0;
    const uint8_t* a_tile = GATHER ? A : A + (int64_t)m0 * a_row;
    const uint8_t* w_tile = W + ((int64_t)group * N + n0) * w_row;
    StageSpan a = stage_span<AB>(m0, end, a_row, k);
    const StageSpan w = stage_span<WB>(n0, (int)N, w_row, k);
    if constexpr (GATHER) a.bytes = a.bytes > 0 ? (uint32_t)x.a_rows * a_row : 0;
    const int64_t sc_n = m_pad + (X::kGroups ? (int64_t)group * n_nt * T : 0) + n0;
#pragma unroll
    for (int j = 0; j < AI; ++j) load_lds16(a_tile, a.bytes, dst + (wave * AI + j) * 1024, va[j], a.k_off);
#pragma unroll
    for (int j = 0; j < WI; ++j) load_lds16(w_tile, w.bytes, dst + oW + (wave * WI + j) * 1024, vw[j], w.k_off);
    load_lds4(sc + k * rows + (wave < 4 ? sc_m + 64 * wave : sc_n + 64 * (wave - 4)), a.bytes > 0 ? 256 : 0,
              dst + oS + 256 * wave, 4u * (uint32_t)lane);
    if constexpr (GATHER)
      load_lds4(sg.a_at + (k + 2 >= nk ? __builtin_amdgcn_readfirstlane(then.sc) : sc_m) + 32 * wave, a.bytes > 0 ? 128 : 0,
                dst + oO + 256 * wave, 4u * (uint32_t)(lane % 32));
    const bool wrap = k + 1 == nk;  // without a branch, which would part the stage's products
    l_k = wrap ? 0 : k + 1;
    src.m0 = wrap ? then.m0 : m0;
    src.n0 = wrap ? then.n0 : n0;
    if constexpr (X::kGroups) {
      src.end = wrap ? then.end : end;
      src.group = wrap ? then.group : group;
      src.sc = wrap ? then.sc : sc_m;
    }
  };

  const int r = lane & 31, h = lane >> 5;
  const int a_base = (wm * MT * 32 + r) * AB, w_base = oW + (wn * NT * 32 + r) * WB;
  int kt = 0;
  // An offset that the compiler takes for one of this stage: it then adds the slot's place to it here instead of
  // keeping the sums of all slots in registers
  auto here = [&](int off) {
    asm("" : "+v"(off) : "s"(kt));
    return off;
  };
  struct Frags {
    i32x8 a[MT];
    uint4 w[NT];
  };
  struct Scales {
    uint32_t a[MT], w[NT];
  };
  auto read_frags = [&](Frags& f, const uint8_t* tile, int step) {
    const int ow = here(w_base + 16 * ((2 * step + h) ^ swz4(r)));
    const int oa0 = here(a_base + 16 * ((4 * step + h) ^ swz8(r)));
    const int oa1 = here(a_base + 16 * ((4 * step + 2 + h) ^ swz8(r)));
#pragma unroll
    for (int i = 0; i < NT; ++i)
      f.w[i] = *(const uint4*)(tile + ow + i * 32 * WB);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      f.a[i] = both4(*(const uint4*)(tile + oa0 + i * 32 * AB), *(const uint4*)(tile + oa1 + i * 32 * AB));
    }
  };
  auto read_scales = [&](Scales& s, const uint8_t* tile) {
    const uint32_t* pa = (const uint32_t*)(tile + here(oS + 4 * (wm * MT * 32 + r)));
    const uint32_t* pw = (const uint32_t*)(tile + here(oS + 4 * (T + wn * NT * 32 + r)));
#pragma unroll
    for (int i = 0; i < MT; ++i) s.a[i] = pa[32 * i];
#pragma unroll
    for (int i = 0; i < NT; ++i) s.w[i] = pw[32 * i];
  };
  auto own_bytes = [&](Scales& s, const Scales& raw) {  // the lane's blocks to bytes 0 and 2
#pragma unroll
    for (int i = 0; i < MT; ++i) s.a[i] = raw.a[i] >> (8 * h);
#pragma unroll
    for (int i = 0; i < NT; ++i) s.w[i] = raw.w[i] >> (8 * h);
  };
  f32x16 acc[NT][MT];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  };
  auto products = [&](const Frags& f, const Scales& s, int step) {
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int i = 0; i < NT; ++i)
        acc[i][j] = mfma_mx32<kMxFp8>(lo4(f.w[i]), f.a[j], acc[i][j], (int)s.w[i], (int)s.a[j], step);
  };

  auto offsets = [&](const uint8_t* slot) { return (const void*)(slot + oO + 256 * wave + 16 * (lane / 8)); };
  const void* first = GATHER ? (const void*)(sg.a_at + now.sc + 32 * wave + 4 * (lane / 8)) : nullptr;
  // waves without rows only load
  constexpr bool kParts = X::kGroups;
  auto has_rows = [&]() { return !X::kGroups || now.m0 + wm * MT * 32 < now.end; };
  bool active = has_rows();
  Frags f0, f1;
  Scales c0, c1;
  clear();

  // A stage in slot C (its step-0 fragments and scales read), the next one in X, loading the one after into F.
  // Before the barrier every wave has read the rest of C (lgkmcnt 0), so that it may be filled again, and X has
  // landed: only the loads into F are younger.
#define AWQ_MX_STAGE(C, X, F)            \
  if (kParts && !active) {               \
    load_stage(F, offsets(C));           \
    wait_loads<ND>();                    \
    block_barrier();                     \
    ++kt;                                \
  } else {                               \
    own_bytes(c0, c1);                   \
    read_frags(f1, C, 1);                \
    load_stage(F, offsets(C));           \
    products(f0, c0, 0);                 \
    interleave<NR, ND>();                \
    __builtin_amdgcn_sched_barrier(0);   \
    wait_loads<ND>();                    \
    block_barrier();                     \
    __builtin_amdgcn_sched_barrier(0);   \
    read_scales(c1, X);                  \
    read_frags(f0, X, 0);                \
    products(f1, c0, 1);                 \
    interleave<NR + (MT + NT) / 2, 0>(); \
    __builtin_amdgcn_sched_barrier(0);   \
    ++kt;                                \
  }
  // The end of a tile, whose last stage was in C: its results go out by way of C
#define AWQ_MX_STORE(C)                                                                                    \
  int own = lane; /* opaque, so that nothing made of it is kept in registers meanwhile */                  \
  asm volatile("" : "+v"(own));                                                                            \
  const int64_t ym = now.m0 + wm * MT * 32, yn = now.n0 + wn * NT * 32;                                    \
  const int64_t ye = X::kGroups ? now.end : M;                                                             \
  if constexpr (X::kEpi)                                                                                   \
    store_tile_epi<MT, NT, NW, SB, 1, false>(acc, C, C, C, wave, own, ym, yn, M, N, Y, ld_y, own_extra<X>());     \
  else if (now.m0 + T <= ye && now.n0 + T <= N)                                                            \
    store_tile<YT, MT, NT, NW, SB, 1, true>(acc, C, C, C, wave, own, ym, yn, ye, N, Y, ld_y);              \
  else                                                                                                     \
    store_tile<YT, MT, NT, NW, SB, 1>(acc, C, C, C, wave, own, ym, yn, ye, N, Y, ld_y);                    \
  tile += step;
#define AWQ_MX_NEXT(X)                   \
  kt = 0;                                \
  now = then;                            \
  then = tile_at(tile + step);           \
  active = has_rows();                   \
  clear();                               \
  wait_lds();                            \
  block_barrier();                       \
  read_scales(c1, X);                    \
  read_frags(f0, X, 0);
#define AWQ_MX_START(C, X) \
  load_stage(C, first);    \
  load_stage(X, first);    \
  wait_loads<ND>();        \
  block_barrier();         \
  read_scales(c1, C);      \
  read_frags(f0, C, 0);

  // The block's last stage is to be the third of the loop, its only way out: the stages over are done ahead
  const int over = (int)((int64_t)((tiles - 1 - tile) / step + 1) * nk % 3);
  if (over == 0) {
    AWQ_MX_START(s0, s1)
  } else if (over == 1) {
    AWQ_MX_START(s2, s0)
    AWQ_MX_STAGE(s2, s0, s1)
  } else {
    AWQ_MX_START(s1, s2)
    AWQ_MX_STAGE(s1, s2, s0)
    AWQ_MX_STAGE(s2, s0, s1)
  }
  // the epilogue's loops are not to look hotter to the register allocation than the stages
#define AWQ_MX_IF_ENDED if (X::kEpi ? __builtin_expect(kt == nk, false) : kt == nk)
  for (;;) {
    AWQ_MX_STAGE(s0, s1, s2)
    AWQ_MX_IF_ENDED {
      AWQ_MX_STORE(s0)
      AWQ_MX_NEXT(s1)
    }
    AWQ_MX_STAGE(s1, s2, s0)
    AWQ_MX_IF_ENDED {
      AWQ_MX_STORE(s1)
      AWQ_MX_NEXT(s2)
    }
    AWQ_MX_STAGE(s2, s0, s1)
    AWQ_MX_IF_ENDED {
      AWQ_MX_STORE(s2)
      if (tile >= tiles) break;
      AWQ_MX_NEXT(s0)
    }
  }
#undef AWQ_MX_IF_ENDED
#undef AWQ_MX_START
#undef AWQ_MX_NEXT
#undef AWQ_MX_STORE
#undef AWQ_MX_STAGE
  wait_loads<0>();  // none may land after the block has given its LDS back
  block_barrier();
}

}  // namespace awq
