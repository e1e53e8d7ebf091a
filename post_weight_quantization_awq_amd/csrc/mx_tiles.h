// The kernel and tile that a microscaled product takes, which tile a block
// computes, and which part of the operands a stage of K reads for it.  Host and
// device: host tests ask and walk them.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "mx_format.h"

namespace awq {

constexpr int kMxXcds = 8;
constexpr int kMxStage = 128;  // K per stage
constexpr int kBigTile = 256;  // outputs and tokens of the largest tiles

// The tile of a block: each XCD owns a contiguous range of tiles, walked in groups of group_m token tiles
__host__ __device__ __forceinline__ void block_tile(int bid, int nblk, int n_mt, int n_nt, int group_m, int* mt,
                                                    int* nt) {
  const int xcd = bid % kMxXcds, pos = bid / kMxXcds, q = nblk / kMxXcds, rr = nblk % kMxXcds;
  const int id = xcd * q + (xcd < rr ? xcd : rr) + pos;
  const int per_group = group_m * n_nt;
  const int first_m = id / per_group * group_m;
  const int gsz = n_mt - first_m < group_m ? n_mt - first_m : group_m;
  *mt = first_m + id % per_group % gsz;
  *nt = id % per_group / gsz;
}

// First token and output of tile `id` of the persistent blocks; past the last tile the place behind all rows
struct TileAt {
  int m0, n0;
};
__host__ __device__ __forceinline__ TileAt big_tile_at(int id, int n_mt, int n_nt, int group_m, int M, int N) {
  const int tiles = n_mt * n_nt;
  int mt, nt;
  block_tile(id < tiles ? id : 0, tiles, n_mt, n_nt, group_m, &mt, &nt);
  return TileAt{id < tiles ? mt * kBigTile : M, id < tiles ? nt * kBigTile : N};
}

// The bytes of the rows that a tile at `first` has of an operand's `rows`, and where in each row stage k of SB
// bytes begins (the last one a row holds, for stages past its end).  Behind all rows both are 0: the hardware
// compares an offset with the buffer's size less the scalar offset, which must not pass that size.
struct StageSpan {
  uint32_t bytes, k_off;
};
template <int SB>
__host__ __device__ __forceinline__ StageSpan stage_span(int first, int rows, uint32_t row_bytes, int k) {
  const int left = rows - first;
  const uint32_t off = (uint32_t)k * SB, last = row_bytes - SB;
  return StageSpan{(uint32_t)(left < kBigTile ? left : kBigTile) * row_bytes, left <= 0 ? 0 : off < last ? off : last};
}

constexpr int kMaxRanges = 8;
inline int64_t tiles_of(int64_t n, int tile) { return (n + tile - 1) / tile; }

// Few tokens: LDS rows of activations, and 16-output tiles a block: two where that still leaves every
// compute unit a block (16 tokens, us: 24576 x 4096 14.8 -> 11.9, 6144 x 4096 6.5 -> 5.5; but 4096 x 12288,
// 256 tiles, 8.3 -> 10.5), one for up to 4 tokens (24576 x 4096 11.8, 12.9 with two).  24 rows save what the 8
// others cost with 8-bit activations and one tile (24 tokens, 4096 x 12288: 10.3 -> 9.9; 14.4 both at 24576 x
// 4096, two tiles; 8.1 -> 8.3 in 4 bits).
struct FewTile {
  int rows, tiles;
};
inline FewTile few_tile(int a_fmt, int64_t M, int64_t N) {
  if (M <= 4) return {4, 1};
  const int rows = M <= 16 ? 16 : 32;
  const int tiles = (N + 15) / 16 * ((M + rows - 1) / rows) > 256 ? 2 : 1;
  return {a_fmt == kMxFp8 && rows == 32 && M <= 24 && tiles == 1 ? 24 : rows, tiles};
}

// The kernel, its tile and the number of K ranges of a product: the ones with the least estimated time.
// The estimates are fitted to measurements of N, K in {4096, 12288, 24576} x {1024, 4096, 12288} at 1 to 4096
// tokens.  E.g. (us, 8 bits; few tokens / tiles of 64 / 128 / 256) 16 x 24576 x 4096: 11.6 / 14.4 / - / -;
// 24 x 4096 x 12288: 9.9 / 11.3 in 8 ranges / - / -; 256 x 4096 x 4096: - / 10 / 15 / 40; 256 x 4096 x 12288:
// - / 29 / 23 in 4 ranges / 104; 512 x 24576 x 4096: - / 82 / 54 / 50; 2048 x 4096 x 4096: - / 55 / 34 / 44;
// (4 bits) 512 x 24576 x 4096: - / - / 46 / 35; 2048 x 4096 x 12288: - / - / 87 / 73.
struct MxTiling {
  int tile;   // outputs and tokens a tile: 64, 128 or 256; 0: few tokens
  int split;  // stages a range
  int ranges;
};
// us: the weights at 5 TB/s, for every further block row at 10 TB/s, and the activations that all blocks read
// at 50 TB/s for 16 rows, 20 or (4 bits) 29 TB/s and 0.3 more above, these in whole rounds of 256 blocks of at
// least 2.2 us
inline double few_time(int a_fmt, int64_t M, int64_t N, int64_t K) {
  const FewTile f = few_tile(a_fmt, M, N);
  const double w_mb = (double)N * (double)K * (17.0 / 32) * 1e-6;
  const double a_mb = (double)M * (double)K * (a_fmt == kMxFp8 ? 1.0 : 0.5) * 1e-6;
  const double cols = (double)((N + 16 * f.tiles - 1) / (16 * f.tiles)), rows = (double)((M + f.rows - 1) / f.rows);
  const double a_cost = f.rows == 4 ? 0.0 : f.rows == 16 ? 0.02 : a_fmt == kMxFp8 ? 0.05 : 0.035;
  double t = w_mb / 5 + (rows - 1) * w_mb / 10 + a_cost * cols * a_mb;
  if (f.rows >= 24) {
    const double rounds = ceil(cols * rows / 256);
    t += 0.3;
    if (rounds > 1) t *= rounds * 256 / (cols * rows);
    t = t < 2.2 * rounds ? 2.2 * rounds : t;
  }
  return 1.1 + t;
}
// us: for each stage, and for a few more that stand for a tile's start and end, `one` + `more` x load while
// no compute unit has more than one block (load: blocks for each of the 256), else `full` for a load of 1, a
// third of it by whole rounds (half of it for the persistent blocks)
inline double tile_time(int a_fmt, int tile, double blocks, int stages) {
  struct Cost {
    double base, ends, one, more, full, whole;
  };
  static const Cost cost[2][3] = {
      {{3, 0, 0.18, 0.04, 0.20, 1. / 3}, {3, 1.5, 0.30, 0.20, 0.50, 1. / 3}, {6, 2.5, 0.95, 0.45, 1.40, 1. / 2}},
      {{3.3, 0, 0.125, 0.05, 0.18, 1. / 3}, {3, 1.5, 0.26, 0.17, 0.43, 1. / 3}, {7, 3.5, 0.50, 0.40, 1.02, 1. / 3}}};
  const Cost& c = cost[a_fmt == kMxFp8 ? 0 : 1][tile == 64 ? 0 : tile == 128 ? 1 : 2];
  const double load = blocks / 256;
  return c.base + (stages + c.ends) * (load <= 1 ? c.one + c.more * load
                                                 : c.full * (c.whole * ceil(load) + (1 - c.whole) * load));
}
inline MxTiling mx_tiling(int a_fmt, int64_t M, int64_t N, int64_t K) {
  const int nk = (int)((K + kMxStage - 1) / kMxStage);
  MxTiling best = {0, nk, 1};
  // A tile's scales are taken three stages at a time, so shorter rows go to the few-token kernel however many tokens
  // there are.  A row is one or two chunks then, for one or two of a block's 8 waves: 4096 x 4096 x 256 takes 131 us
  // in 8 bits and 121 in 4, 4096 x 4096 x 384 on the tiles 16 and 13.
  if (K < 3 * kMxStage) return best;
  double least = M <= 64 ? few_time(a_fmt, M, N, K) : HUGE_VAL;
  for (int tile = 64; tile <= 256; tile *= 2) {
    const double blocks = (double)((M + tile - 1) / tile) * (double)((N + tile - 1) / tile);
    if (blocks > (1 << 22)) continue;  // a launch holds fewer than 2^32 lanes
    for (int s = 1; s == 1 || (s <= kMaxRanges && nk / s >= 6); ++s) {
      const int split = (nk + s - 1) / s, ranges = (nk + split - 1) / split;
      if (s > 1 && (ranges != s || blocks * s > 512 || tile == 256)) continue;
      double t = tile_time(a_fmt, tile, blocks * ranges, split);
      // a second launch, and the ranges' fp32 sums written and read at 5 TB/s
      if (ranges > 1) t += 2.3 + ranges * (double)M * (double)N * 8 / 5e6;
      if (t < least) least = t, best = {tile, split, ranges};
    }
  }
  return best;
}

// Slots of the 64 x 64 tiles: six, for loads five stages ahead, where no compute unit has more than one block
// and there are stages to load ahead (256 x 4096 x 4096, us: 8 bits 11.9 -> 10.1, 4 bits 11.1 -> 8.6); else three,
// which leave room for more blocks (512 x 4096 x 4096 in 8 bits: 16.4, 17.0 with six; 32 x 12288 x 1024, 8
// stages: 4.2, 4.6 with six).  Six slots of 128 x 128 tiles gain 0 to 6% there and lose 15 to 30% of larger
// products.
inline int tile_slots(const MxTiling& t, int64_t M, int64_t N) {
  return t.tile == 64 && tiles_of(M, 64) * tiles_of(N, 64) * t.ranges <= 256 && t.split >= 12 ? 6 : 3;
}

}  // namespace awq
