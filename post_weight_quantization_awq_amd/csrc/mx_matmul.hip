// Product of microscaled operands: Y [M, N] = A [M, K] W [N, K]^T, A in e4m3 or
// e2m1 blocks, W in e2m1 blocks, both row-major along K with one scale byte per
// 32 values.  The matrix cores take the codes and the scale bytes as they are
// (v_mfma_scale_f32_16x16x128_f8f6f4): no value is dequantized in registers.
#include <math.h>

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
// Few tokens: a block holds 16 outputs and 16 MT tokens.  Its 8 waves take chunks
// of 512 K in turn (four MFMA steps; 64 lanes read 16 rows of 64 bytes a load),
// the next chunk's weights on their way while one is multiplied; their sums are
// added in wave order through LDS.
// ---------------------------------------------------------------------------
constexpr int kFewWaves = 8;
constexpr int kFewBlocks = 16;  // scale blocks of a chunk

// The 16 scale bytes of a row's chunk c; zeros past the row's end
__device__ __forceinline__ uint4 few_scales(const uint8_t* row, int c, int kb) {
  if (kFewBlocks * (c + 1) <= kb) return ld_any<uint4>(row + kFewBlocks * c);
  uint32_t v[4] = {0, 0, 0, 0};
  for (int i = 0; i < kb - kFewBlocks * c; ++i) {
    const uint32_t b = (uint32_t)row[kFewBlocks * c + i] << (8 * (i & 3));
#pragma unroll
    for (int d = 0; d < 4; ++d) v[d] |= d == i >> 2 ? b : 0;
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}
// 16 bytes of codes that hold values of block b, zeros past the row's end
__device__ __forceinline__ uint4 few_codes(const uint8_t* p, int b, int kb) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (b < kb) v = *(const uint4*)p;
  return v;
}

template <int AF, int MT>
__global__ __launch_bounds__(kFewWaves * kWave, 2) void mx_few_kernel(const uint8_t* __restrict__ A,
                                                                     const uint8_t* __restrict__ as, int64_t M,
                                                                     const uint8_t* __restrict__ W,
                                                                     const uint8_t* __restrict__ ws, int64_t N,
                                                                     int64_t K, void* __restrict__ Y, int64_t ld_y,
                                                                     int y_dtype) {
  __shared__ float red[kFewWaves][MT * 16][17];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, h = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * (16 * MT);
  const int kb = (int)(K / kMxBlock), nc = (kb + kFewBlocks - 1) / kFewBlocks;
  const int64_t n = n0 + r < N ? n0 + r : N - 1;  // rows past the end repeat the last one, unused
  const uint8_t* wr = W + n * (K / 2) + 16 * h;
  const uint8_t* wsr = ws + n * kb;
  const uint8_t* ar[MT];
  const uint8_t* asr[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int64_t m = m0 + 16 * t + r < M ? m0 + 16 * t + r : M - 1;
    ar[t] = A + m * (AF == kMxFp8 ? K : K / 2) + 16 * h;
    asr[t] = as + m * kb;
  }
  f32x4 acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = (f32x4){0, 0, 0, 0};

  uint4 w[4], sw;
  auto load_w = [&](int c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = few_codes(wr + 256 * (int64_t)c + 64 * j, kFewBlocks * c + 4 * j + h, kb);
    sw = few_scales(wsr, c, kb);
  };
  if (wave < nc) load_w(wave);
  for (int c = wave; c < nc; c += kFewWaves) {
    uint4 wc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) wc[j] = w[j];
    const uint32_t swc[4] = {sw.x >> (8 * h), sw.y >> (8 * h), sw.z >> (8 * h), sw.w >> (8 * h)};
    if (c + kFewWaves < nc) load_w(c + kFewWaves);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const uint4 sa = few_scales(asr[t], c, kb);
      const uint32_t sac[4] = {sa.x >> (8 * h), sa.y >> (8 * h), sa.z >> (8 * h), sa.w >> (8 * h)};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int b = kFewBlocks * c + 4 * j;
        i32x8 a;
        if constexpr (AF == kMxFp8) {
          const uint8_t* p = ar[t] + 32 * (int64_t)b;
          a = both4(few_codes(p, b + h / 2, kb), few_codes(p + 64, b + 2 + h / 2, kb));
        } else {
          a = lo4(few_codes(ar[t] + 16 * (int64_t)b, b + h, kb));
        }
        acc[t] = mfma_mx<AF>(lo4(wc[j]), a, acc[t], (int)swc[j], (int)sac[j]);
      }
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
    for (int q = 0; q < kFewWaves; ++q) v += red[q][t][o];
    if (m0 + t < M && n0 + o < N) store_y(Y, (m0 + t) * ld_y + n0 + o, v, y_dtype);
  }
}

// ---------------------------------------------------------------------------
// Many tokens: tiles of BM tokens x BN outputs staged through LDS.
//
// K advances in stages of 128 through a ring of three LDS slots, filled by direct
// loads (16 bytes a lane, no registers) two stages ahead.  A stage is two steps of
// v_mfma_scale_f32_32x32x64_f8f6f4; the fragments of a step are read from LDS
// while the matrix cores work on the step before, across the stage boundary too:
// the block's one barrier a stage stands between the two steps, where the next
// stage's loads must have landed.
// ---------------------------------------------------------------------------
template <int AF>
__device__ __forceinline__ f32x16 mfma_mx32(const i32x8 w, const i32x8 a, f32x16 c, int ws, int as, int step) {
  // scale bytes 0 and 2 of the registers: the lane's block of step 0 and 1
  return step == 0
             ? __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, a, c, 4, AF == kMxFp8 ? 0 : 4, 0, ws, 0, as)
             : __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, a, c, 4, AF == kMxFp8 ? 0 : 4, 2, ws, 2, as);
}

typedef __attribute__((address_space(3))) void* mx_lds_ptr;
constexpr int kMxXcds = 8;
constexpr int kMxStage = 128;   // K per stage
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
template <int YT, int MT, int NT, int NW, int SB>
__device__ __forceinline__ void store_tile(const f32x16 (&acc)[NT][MT], uint8_t* s0, uint8_t* s1, uint8_t* s2,
                                           int wave, int lane, int64_t m0, int64_t n0, int64_t M, int64_t N, void* Y,
                                           int64_t ld_y) {
  constexpr int EB = YT == 2 ? 4 : 2;
  constexpr int CG = EB == 2 || NT == 1 ? NT : NT / 2;       // 32-output tiles per turn
  constexpr int RB = CG * 32 * EB;                           // bytes of a row
  constexpr int WS = (NW + 2) / 3;                           // waves an array
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
        if (m < M) store_row16<EB>((uint8_t*)Y + (m * ld_y + n) * EB, v, N - n);
      }
      __builtin_amdgcn_wave_barrier();
    }
}

// The tile of a block: each XCD owns a contiguous range of tiles, walked in groups of group_m token tiles
__device__ __forceinline__ void block_tile(int n_mt, int n_nt, int group_m, int* mt, int* nt) {
  const int nblk = (int)gridDim.x, bid = (int)blockIdx.x;
  const int xcd = bid % kMxXcds, pos = bid / kMxXcds, q = nblk / kMxXcds, rr = nblk % kMxXcds;
  const int id = xcd * q + (xcd < rr ? xcd : rr) + pos;
  const int per_group = group_m * n_nt;
  const int first_m = id / per_group * group_m;
  const int gsz = n_mt - first_m < group_m ? n_mt - first_m : group_m;
  *mt = first_m + id % per_group % gsz;
  *nt = id % per_group / gsz;
}

// OCC: waves a SIMD that the registers are to leave room for.  blockIdx.y: one of gridDim.y ranges of
// `split` stages of K; range z's sums go to Y + z M ld_y (YT 2).
template <int AF, int YT, int BM, int BN, int WM, int WN, int OCC>
__global__ __launch_bounds__(WM* WN* kWave, OCC) void mx_tile_kernel(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ as, int64_t M, const uint8_t* __restrict__ W,
    const uint8_t* __restrict__ ws, int64_t N, int64_t K, int n_mt, int n_nt, int group_m, int split,
    void* __restrict__ Y, int64_t ld_y) {
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
  __shared__ uint32_t sS[2 * (BM + BN) * 3];     // scale bytes of three stages, a row's side by side

  int mt, nt;
  block_tile(n_mt, n_nt, group_m, &mt, &nt);
  const int64_t m0 = (int64_t)mt * BM, n0 = (int64_t)nt * BN;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int kb = (int)(K / kMxBlock);
  const int k0 = (int)blockIdx.y * split;  // first stage
  const int nk = min((int)((K + kMxStage - 1) / kMxStage) - k0, split);
  const uint32_t a_row = (uint32_t)(AF == kMxFp8 ? K : K / 2), w_row = (uint32_t)(K / 2);
  const int m_rows = (int)(M - m0 < BM ? M - m0 : BM), n_rows = (int)(N - n0 < BN ? N - n0 : BN);

  // direct loads: lane i of load j fills 16 bytes i of the wave's j-th KiB.  Rows past the end are out of
  // the buffer's range and read as zeros (their results are not stored).  A last stage that K does not fill takes the row's last
  // 128 values instead: the scales of those already summed are 0 on both sides, so that they add 0.
  const uint8_t* a_tile = A + m0 * a_row;
  const uint8_t* w_tile = W + n0 * w_row;
  const uint32_t a_bytes = (uint32_t)m_rows * a_row, w_bytes = (uint32_t)n_rows * w_row;
  uint32_t va[AI], vw[WI];
#pragma unroll
  for (int j = 0; j < AI; ++j) {
    const int row = (wave * AI + j) * (1024 / AB) + lane / (AB / 16), slot = lane % (AB / 16);
    va[j] = row < m_rows ? (uint32_t)row * a_row + 16u * (uint32_t)(slot ^ (AF == kMxFp8 ? swz8(row) : swz4(row))) : kMxOut;
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
#pragma unroll
  for (int q = 0; q < SR; ++q) {
    srow_i[q] = min(tid + q * NW * kWave, BM + BN - 1);
    srow[q] = srow_i[q] < BM ? as + (m0 + min(srow_i[q], m_rows - 1)) * kb
                             : ws + (n0 + min(srow_i[q] - BM, n_rows - 1)) * kb;
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
      const uint32_t v[3] = {sc[q].x, sc[q].y, sc[q].z};
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

  load_stage(s0, 0);
  load_stage(s1, 1);
  load_scales(0);
  write_scales(0);
  load_scales(1);
  wait_loads<0>();
  __builtin_amdgcn_s_barrier();
  Frags f0, f1;
  Scales c0, c1;
  read_frags(f0, s0, 0);
  read_scales(c1, 0, 0);

  // Stage kt in slot P = kt % 3 (array C), its step-0 fragments read.  Before the barrier every wave has
  // read the rest of the stage (lgkmcnt 0), so its slot may be filled again by stage kt + 3; and stage
  // kt + 1 (array X) has landed: only the loads of stage kt + 2 (array F) are younger.  Loads past the
  // last stage repeat its last chunks.
#define AWQ_MX_STAGE(P, C, X, F)                  \
  {                                               \
    own_bytes(c0, c1);                            \
    read_frags(f1, C, 1);                         \
    load_stage(F, kt + 2);                        \
    if (P == 2) write_scales(ss + 1);             \
    products(f0, c0, 0);                          \
    interleave<NR, ND>();                         \
    __builtin_amdgcn_sched_barrier(0);            \
    wait_loads<ND>();                             \
    __builtin_amdgcn_s_barrier();                 \
    __builtin_amdgcn_sched_barrier(0);            \
    if (P == 2) load_scales(ss + 2);              \
    read_scales(c1, ss + (P == 2), (P + 1) % 3);  \
    read_frags(f0, X, 0);                         \
    products(f1, c0, 1);                          \
    interleave<NR + (MT + NT) / 2, 0>();          \
    __builtin_amdgcn_sched_barrier(0);            \
    ++kt;                                         \
  }
  int kt = 0, ss = 0;  // ss = kt / 3
  for (; kt + 3 <= nk; ++ss) {
    AWQ_MX_STAGE(0, s0, s1, s2)
    AWQ_MX_STAGE(1, s1, s2, s0)
    AWQ_MX_STAGE(2, s2, s0, s1)
  }
  if (kt < nk) AWQ_MX_STAGE(0, s0, s1, s2)
  if (kt < nk) AWQ_MX_STAGE(1, s1, s2, s0)
#undef AWQ_MX_STAGE

  wait_loads<0>();  // none may land after the block has given its LDS back
  __builtin_amdgcn_s_barrier();

  store_tile<YT, MT, NT, NW, BM * AB + BN * WB>(acc, s0, s1, s2, wave, lane, m0 + wm * MT * 32, n0 + wn * NT * 32, M, N,
                                               YT == 2 ? (float*)Y + (int64_t)blockIdx.y * M * ld_y : Y, ld_y);
}

// ---------------------------------------------------------------------------
// Large products: 256 x 256 tiles, where the loads that reach the second-level
// cache bound the kernel (measured with everything else left out: 297 us of the
// 388 us of an 8-bit 8192^3 product, 252 of 301 us of a 4-bit one).  So every row
// of a stage is a whole 128-byte line where LDS allows it: a stage is 128 K in
// three slots for 8-bit activations (W rows then half a line) and 256 K in two
// slots for 4-bit ones; and the scales, whose bytes of a stage lie in a line of
// their own for each row, are first laid out stage by stage (stage_scales), so
// that a stage takes 16 or 32 lines of them instead of 512.
// ---------------------------------------------------------------------------
template <int AF>
constexpr int kBigStage = AF == kMxFp8 ? 128 : 256;
template <int AF>
constexpr int kBigSlots = AF == kMxFp8 ? 3 : 2;
constexpr int kBigTile = 256;

// out[w][row] (rows: the A rows, then the W rows, each padded to whole tiles): word w % (SB / 4) of stage
// w / (SB / 4), the scale bytes of SB = K / 32 blocks.  A last stage that K does not fill holds the row's
// last SB blocks, 0 in the place of those of earlier stages; padded rows hold 0.
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

template <int AF, int YT>
__global__ __launch_bounds__(512, 2) void mx_big_kernel(const uint8_t* __restrict__ A, int64_t M,
                                                        const uint8_t* __restrict__ W, int64_t N, int64_t K,
                                                        const uint32_t* __restrict__ sc, int64_t m_pad, int64_t rows,
                                                        int n_mt, int n_nt, int group_m, void* __restrict__ Y,
                                                        int64_t ld_y) {
  constexpr int KS = kBigStage<AF>, SL = kBigSlots<AF>, T = kBigTile;
  constexpr int WM = 4, WN = 2, NW = 8, MT = T / WM / 32, NT = T / WN / 32;
  constexpr int AB = 128, WB = KS / 2;                 // bytes of a row's stage
  constexpr int SW = KS / 128;                         // scale words of a row's stage
  constexpr int AI = T * AB / 1024 / NW, WI = T * WB / 1024 / NW, SI = SW;  // direct loads a wave and stage
  constexpr int ND = AI + WI + SI;
  constexpr int ST = KS / 64;                          // MFMA steps a stage
  constexpr int NR = NT + MT * (AF == kMxFp8 ? 2 : 1);  // LDS reads of a step's fragments
  constexpr int oW = T * AB, oS = oW + T * WB, SB = oS + SW * 2 * T * 4;
  // one array a slot (A tile, W tile, scale words): fragment reads then visibly do not touch the loads in flight
  __shared__ __attribute__((aligned(1024))) uint8_t s0[SB];
  __shared__ __attribute__((aligned(1024))) uint8_t s1[SB];
  __shared__ __attribute__((aligned(1024))) uint8_t s2[SL == 3 ? SB : 16];

  int mt, nt;
  block_tile(n_mt, n_nt, group_m, &mt, &nt);
  const int64_t m0 = (int64_t)mt * T, n0 = (int64_t)nt * T;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int nk = (int)((K + KS - 1) / KS);
  const uint32_t a_row = (uint32_t)(AF == kMxFp8 ? K : K / 2), w_row = (uint32_t)(K / 2);
  const int m_rows = (int)(M - m0 < T ? M - m0 : T), n_rows = (int)(N - n0 < T ? N - n0 : T);

  // direct loads: lane i of load j fills 16 bytes i of the wave's j-th KiB.  Rows past the end are out of
  // the buffer's range and read as zeros.  A last stage that K does not fill takes the row's last KS values.
  const uint8_t* a_tile = A + m0 * a_row;
  const uint8_t* w_tile = W + n0 * w_row;
  const uint32_t a_bytes = (uint32_t)m_rows * a_row, w_bytes = (uint32_t)n_rows * w_row;
  uint32_t va[AI], vw[WI];
#pragma unroll
  for (int j = 0; j < AI; ++j) {
    const int row = (wave * AI + j) * (1024 / AB) + lane / (AB / 16);
    va[j] = row < m_rows ? (uint32_t)row * a_row + 16u * (uint32_t)(lane % (AB / 16) ^ swz8(row)) : kMxOut;
  }
#pragma unroll
  for (int j = 0; j < WI; ++j) {
    const int row = (wave * WI + j) * (1024 / WB) + lane / (WB / 16), c = lane % (WB / 16);
    vw[j] = row < n_rows ? (uint32_t)row * w_row + 16u * (uint32_t)(c ^ (WB == 128 ? swz8(row) : swz4(row))) : kMxOut;
  }
  // scales: the wave's 64 of the tile's 256 + 256 rows; words past the last stage's are not read
  const int64_t s_row = wave < 4 ? m0 + 64 * wave : m_pad + n0 + 64 * (wave - 4);
  auto load_stage = [&](uint8_t* dst, int kt) {
    const uint32_t ka = min((uint32_t)kt * AB, a_row - AB), kw = min((uint32_t)kt * WB, w_row - WB);
#pragma unroll
    for (int j = 0; j < AI; ++j) load_lds16(a_tile, a_bytes, dst + (wave * AI + j) * 1024, va[j], ka);
#pragma unroll
    for (int j = 0; j < WI; ++j) load_lds16(w_tile, w_bytes, dst + oW + (wave * WI + j) * 1024, vw[j], kw);
#pragma unroll
    for (int j = 0; j < SI; ++j)
      load_lds4(sc + ((int64_t)min(kt, nk - 1) * SW + j) * rows + s_row, 256, dst + oS + (j * 2 * T + 64 * wave) * 4,
                4u * (uint32_t)lane);
  };

  // fragments: lane l holds row l % 32 of a tile, h = l / 32
  const int r = lane & 31, h = lane >> 5;
  const int a_base = (wm * MT * 32 + r) * AB, w_base = oW + (wn * NT * 32 + r) * WB;
  struct Frags {
    i32x8 a[MT];
    uint4 w[NT];
  };
  struct Scales {
    uint32_t a[MT][SW], w[NT][SW];
  };
  auto read_frags = [&](Frags& f, const uint8_t* tile, int step) {
#pragma unroll
    for (int i = 0; i < NT; ++i)
      f.w[i] = *(const uint4*)(tile + w_base + i * 32 * WB +
                               16 * ((2 * step + h) ^ (WB == 128 ? swz8(r) : swz4(r))));
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const uint8_t* p = tile + a_base + i * 32 * AB;
      if constexpr (AF == kMxFp8)
        f.a[i] = both4(*(const uint4*)(p + 16 * ((4 * step + h) ^ swz8(r))),
                       *(const uint4*)(p + 16 * ((4 * step + 2 + h) ^ swz8(r))));
      else
        f.a[i] = lo4(*(const uint4*)(p + 16 * ((2 * step + h) ^ swz8(r))));
    }
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
        acc[i][j] = mfma_mx32<AF>(lo4(f.w[i]), f.a[j], acc[i][j], (int)s.w[i][step / 2], (int)s.a[j][step / 2],
                                  step % 2);
  };

  Frags f0, f1;
  Scales c0, c1;
  load_stage(s0, 0);
  load_stage(s1, 1);
  if constexpr (SL == 3) load_stage(s2, 2);
  wait_loads<ND*(SL - 1)>();
  __builtin_amdgcn_s_barrier();
  read_scales(c1, s0);
  read_frags(f0, s0, 0);

  // Stage kt (array C), its step-0 fragments and scales read.  At the barrier, ahead of the last step, every
  // wave has read the whole stage (lgkmcnt 0) and stage kt + 1 (array X) has landed, only loads of later
  // stages being younger: C may be filled again.  Loads past the last stage repeat it.
#define AWQ_MX_STEP(F, G, C, S)          \
  read_frags(G, C, S + 1);               \
  products(F, c0, S);                    \
  interleave<NR, 0>();                   \
  __builtin_amdgcn_sched_barrier(0);
#define AWQ_MX_STAGE(C, X)                       \
  {                                              \
    own_bytes(c0, c1);                           \
    AWQ_MX_STEP(f0, f1, C, 0)                    \
    if constexpr (ST == 4) {                     \
      AWQ_MX_STEP(f1, f0, C, 1)                  \
      AWQ_MX_STEP(f0, f1, C, 2)                  \
    }                                            \
    wait_loads<ND*(SL - 2)>();                   \
    __builtin_amdgcn_s_barrier();                \
    __builtin_amdgcn_sched_barrier(0);           \
    load_stage(C, kt + SL);                      \
    read_scales(c1, X);                          \
    read_frags(f0, X, 0);                        \
    products(f1, c0, ST - 1);                    \
    interleave<NR + SW * (MT + NT) / 2, ND>();   \
    __builtin_amdgcn_sched_barrier(0);           \
    ++kt;                                        \
  }
  int kt = 0;
  if constexpr (SL == 3) {
    while (kt + 3 <= nk) {
      AWQ_MX_STAGE(s0, s1)
      AWQ_MX_STAGE(s1, s2)
      AWQ_MX_STAGE(s2, s0)
    }
    if (kt < nk) AWQ_MX_STAGE(s0, s1)
    if (kt < nk) AWQ_MX_STAGE(s1, s2)
  } else {
    while (kt + 2 <= nk) {
      AWQ_MX_STAGE(s0, s1)
      AWQ_MX_STAGE(s1, s0)
    }
    if (kt < nk) AWQ_MX_STAGE(s0, s1)
  }
#undef AWQ_MX_STAGE
#undef AWQ_MX_STEP
  wait_loads<0>();  // none may land after the block has given its LDS back
  __builtin_amdgcn_s_barrier();
  if constexpr (SL == 3)
    store_tile<YT, MT, NT, NW, SB>(acc, s0, s1, s2, wave, lane, m0 + wm * MT * 32, n0 + wn * NT * 32, M, N, Y, ld_y);
  else  // the second half of the second array takes the third's place
    store_tile<YT, MT, NT, NW, SB / 2>(acc, s0, s1, s1 + SB / 2, wave, lane, m0 + wm * MT * 32, n0 + wn * NT * 32, M,
                                       N, Y, ld_y);
}

// Y = sum over z, in order, of part[z] (fp32 [M, ld_p] each): 4 outputs a thread
template <int YT>
__global__ __launch_bounds__(256) void mx_reduce_kernel(const float* __restrict__ part, int n_split, int64_t M,
                                                        int64_t N, int64_t ld_p, void* __restrict__ Y, int64_t ld_y) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t m = i / (ld_p / 4), n = 4 * (i % (ld_p / 4));
  if (m >= M) return;
  float4 v = *(const float4*)(part + m * ld_p + n);
  for (int z = 1; z < n_split; ++z) {
    const float4 p = *(const float4*)(part + (z * M + m) * ld_p + n);
    v.x += p.x, v.y += p.y, v.z += p.z, v.w += p.w;
  }
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

// The kernel, its tile and the number of K ranges of a product: the ones with the least estimated time.
// Measured on 8-bit activations (4-bit ones rank alike), in us: a stage of K costs 0.27 / 0.5 / 1.3 a
// block of 64 / 128 / 256 squared while no compute unit has more than one, and 0.21 / 0.5 / 1.3 for each
// 256 blocks beyond; K ranges add 2.5 for the second launch and their fp32 sums written and read at 5 TB/s;
// the few-token kernel reads the weights at 4.2 TB/s and the activations once per 16 outputs at 12 TB/s.
// E.g. 24 x 4096 x 12288: few tokens 15.7, 64-tiles 29, in 4 ranges 12.6; 512 x 24576 x 4096: 82 / 52 / 46;
// 2048 x 4096 x 4096: 55 / 34 / 38; 256 x 4096 x 4096: 12 / 16 / 23.
struct MxTiling {
  int tile;   // outputs and tokens a tile: 64, 128 or 256; 0: few tokens
  int split;  // stages a range
  int ranges;
};
static MxTiling mx_tiling(int a_fmt, int64_t M, int64_t N, int64_t K) {
  const int nk = (int)((K + kMxStage - 1) / kMxStage);
  const double w_bytes = (double)N * K * (17.0 / 32), a_bytes = (double)M * K * (a_fmt == kMxFp8 ? 1.0 : 0.5);
  MxTiling best = {0, nk, 1};
  if (K < 3 * kMxStage) return best;  // a tile's scales are taken three stages at a time
  double least = 2.5 + w_bytes / 4.2e6 + (double)((N + 15) / 16) * a_bytes / 12e6;
  for (int tile = 64; tile <= 256; tile *= 2) {
    const double per = tile == 64 ? 0.21 : tile == 128 ? 0.5 : 1.3;
    const double blocks = (double)((M + tile - 1) / tile) * (double)((N + tile - 1) / tile);
    for (int s = 1; s <= 8 && nk / s >= 6; ++s) {
      const int split = (nk + s - 1) / s, ranges = (nk + split - 1) / split;
      if (s > 1 && (ranges != s || blocks * s > 512 || tile == 256)) continue;
      const double rounds = ceil(blocks * ranges / 256);
      double t = 3 + split * (tile == 64 && rounds == 1 ? 0.27 : per * rounds);
      if (ranges > 1) t += 2.5 + ranges * (double)M * (double)N * 8 / 5e6;
      if (t < least) least = t, best = {tile, split, ranges};
    }
  }
  return best;
}
static int64_t part_ld(int64_t N) { return (N + 3) / 4 * 4; }

static int64_t tiles_of(int64_t n, int tile) { return (n + tile - 1) / tile; }
static int64_t big_scale_words(int a_fmt, int64_t M, int64_t N, int64_t K) {
  const int64_t ks = a_fmt == kMxFp8 ? kBigStage<kMxFp8> : kBigStage<kMxFp4>;
  return (tiles_of(M, kBigTile) + tiles_of(N, kBigTile)) * kBigTile * ((K + ks - 1) / ks * (ks / 128));
}

size_t mx_matmul_workspace(int a_fmt, int64_t M, int64_t N, int64_t K) {
  const MxTiling t = mx_tiling(a_fmt, M, N, K);
  if (t.tile == kBigTile) return (size_t)big_scale_words(a_fmt, M, N, K) * sizeof(uint32_t);
  return t.ranges > 1 ? (size_t)t.ranges * M * part_ld(N) * sizeof(float) : 0;
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

template <int AF, int YT>
static void tile_launch(const MxTiling& t, const uint8_t* A, const uint8_t* as, int64_t M, const uint8_t* W,
                        const uint8_t* ws, int64_t N, int64_t K, void* Y, int64_t ld_y, hipStream_t stream) {
  const int n_mt = (int)tiles_of(M, t.tile), n_nt = (int)tiles_of(N, t.tile);
  const dim3 g((unsigned)(n_mt * n_nt), (unsigned)t.ranges);
#define AWQ_TILE(BM, BN, WM, WN, OCC)                                                                               \
  mx_tile_kernel<AF, YT, BM, BN, WM, WN, OCC><<<g, WM * WN * kWave, 0, stream>>>(A, as, M, W, ws, N, K, n_mt, n_nt, 8, \
                                                                               t.split, Y, ld_y)
  if (t.tile == 64) AWQ_TILE(64, 64, 2, 2, 4);
  else AWQ_TILE(128, 128, 2, 2, 2);
#undef AWQ_TILE
}

template <int AF, int YT>
static void big_launch(const uint8_t* A, const uint8_t* as, int64_t M, const uint8_t* W, const uint8_t* ws, int64_t N,
                       int64_t K, void* Y, int64_t ld_y, uint32_t* sc, hipStream_t stream) {
  constexpr int SB = kBigStage<AF> / kMxBlock;
  const int n_mt = (int)tiles_of(M, kBigTile), n_nt = (int)tiles_of(N, kBigTile), kb = (int)(K / kMxBlock);
  const int64_t m_pad = (int64_t)n_mt * kBigTile, rows = m_pad + (int64_t)n_nt * kBigTile;
  stage_scales_kernel<SB><<<dim3((unsigned)(rows / 256), (unsigned)((kb + 15) / 16)), 256, 0, stream>>>(
      as, M, ws, N, kb, m_pad, rows, sc);
  mx_big_kernel<AF, YT><<<(unsigned)(n_mt * n_nt), 512, 0, stream>>>(A, M, W, N, K, sc, m_pad, rows, n_mt, n_nt,
                                                                    AF == kMxFp8 ? 4 : 8, Y, ld_y);
}

template <int AF, int YT>
static void product_launch(const uint8_t* A, const uint8_t* as, int64_t M, const uint8_t* W, const uint8_t* ws,
                           int64_t N, int64_t K, void* Y, int64_t ld_y, float* part, hipStream_t stream) {
  const MxTiling t = mx_tiling(AF, M, N, K);
  if (t.tile == 0) {
    few_launch<AF>(A, as, M, W, ws, N, K, Y, ld_y, YT, stream);
  } else if (t.tile == kBigTile) {
    big_launch<AF, YT>(A, as, M, W, ws, N, K, Y, ld_y, (uint32_t*)part, stream);
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
