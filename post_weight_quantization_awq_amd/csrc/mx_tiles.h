// Which tile of a microscaled product a block computes, and which part of the
// operands a stage of K reads for it.  Host and device: a host test walks them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

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

}  // namespace awq
