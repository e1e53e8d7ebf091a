// Product of microscaled operands grouped by expert: rows [offsets[e],
// offsets[e + 1]) of Y are rows of A (their own, or those that `rows` names) times
// matrix e of W.  The kernels are the product's (mx_product.h); a block finds its
// tile of rows by itself, from the offsets on the device, so that the host waits
// for nothing and a captured graph takes whatever offsets there are.
//
// Few rows a group are bound by reading the weights: the 8 groups of 4096 x 4096 of
// one token 16.4 us (4.4 TB/s with the launch), 64 groups of 4096 x 2048 for 512 rows
// 63 us (4.6).  Large groups are bound by the matrix cores and by tiles that no group fills:
// 16384 rows of 32 uneven groups of 4096 x 4096 276 us (2.0 PFLOP/s; one group of all
// 209, the plain product 195-203, and reading A through `rows` adds 13), in 4 bits
// 204-220 us (2.6 PFLOP/s): a group's last tile of fewer than 128 rows takes 0.95 of a full
// one, since its stages wait for their loads either way.
#include <algorithm>

#include "awq_launch.h"
#include "mx_product.h"

namespace awq {

struct GroupedWork {
  int n_mt, n_nt;
  int64_t m_pad, n_pad, rows;        // scale rows: of A, of one group's weight, of all
  size_t scales, tab, offsets, all;  // bytes up to the tiles' table, the row offsets, the end
};
static GroupedWork grouped_work(int a_fmt, int64_t M, int64_t N, int64_t K, int n_groups) {
  GroupedWork w;
  w.n_mt = (int)group_tiles_most(M, n_groups, kBigTile);
  w.n_nt = (int)tiles_of(N, kBigTile);
  w.m_pad = (int64_t)w.n_mt * kBigTile;
  w.n_pad = (int64_t)w.n_nt * kBigTile;
  w.rows = w.m_pad + n_groups * w.n_pad;
  const int64_t words = a_fmt == kMxFp8 ? (K + kMxStage - 1) / kMxStage : (K + kBigStage - 1) / kBigStage * 2;
  w.scales = (size_t)(w.rows * words) * 4;
  w.tab = w.scales;  // a multiple of 1024
  w.offsets = w.tab + ((size_t)w.n_mt + 1) * sizeof(int4);
  w.all = w.offsets + (size_t)w.m_pad * 4;
  return w;
}

size_t mx_grouped_workspace(int a_fmt, int64_t M, int64_t N, int64_t K, int n_groups) {
  if (group_tiling(a_fmt, M, N, K, n_groups).tile != kBigTile) return 0;
  return grouped_work(a_fmt, M, N, K, n_groups).all;
}

struct GroupedArgs {
  const uint8_t *A, *as, *W, *ws;
  int64_t M, N, K;
  void* Y;
  int64_t ld_y;
  Groups g;
};

template <int AF>
static void grouped_few(const GroupedArgs& p, int y_dtype, hipStream_t stream) {
  const int64_t most = group_tiles_most(p.M, p.g.n, kFewGroupRows), cols = tiles_of(p.N, 16 * kFewGroupTiles);
  // of a launch: the grid's second dimension, and fewer than 2^32 lanes
  const int64_t step = std::min<int64_t>(65535, std::max<int64_t>(1, ((int64_t)1 << 22) / cols));
  Groups g = p.g;
  for (int64_t m = 0; m < most; m += step) {
    g.first_tile = (int)m;
    mx_few_kernel<AF, kFewGroupRows, kFewGroupTiles, 2, 4, Groups>
        <<<dim3((unsigned)cols, (unsigned)std::min(step, most - m)), kFewWaves * kWave, 0, stream>>>(
            p.A, p.as, p.M, p.W, p.ws, p.N, p.K, p.Y, p.ld_y, y_dtype, g);
  }
}

template <int AF, int YT>
static void grouped_launch(const GroupedArgs& p, uint8_t* work, hipStream_t stream) {
  const GroupTiling t = group_tiling(AF, p.M, p.N, p.K, p.g.n);
  if (t.tile == 0) {
    grouped_few<AF>(p, YT, stream);
  } else if (t.tile < kBigTile) {
    const int n_mt = (int)group_tiles_most(p.M, p.g.n, t.tile), n_nt = (int)tiles_of(p.N, group_tile_outs(t.tile));
    const int nk = (int)((p.K + kMxStage - 1) / kMxStage);
#define AWQ_TILE(BM, BN, WM, WN, NS, OCC)                                                                            \
  mx_tile_kernel<AF, YT, BM, BN, WM, WN, NS, OCC, Groups><<<(unsigned)(n_mt * n_nt), WM * WN * kWave, 0, stream>>>( \
      p.A, p.as, p.M, p.W, p.ws, p.N, p.K, n_mt, n_nt, 4, nk, p.Y, p.ld_y, p.g)
    if (t.tile == 32 && t.slots == 6) AWQ_TILE(32, 128, 1, 2, 6, 1);
    else if (t.tile == 32) AWQ_TILE(32, 128, 1, 2, 3, 2);
    else if (t.tile == 64) AWQ_TILE(64, 64, 2, 2, 3, 4);
    else AWQ_TILE(128, 128, 2, 2, 3, 2);
#undef AWQ_TILE
  } else if constexpr (AF == kMxFp4 || YT != 2) {
    const GroupedWork w = grouped_work(AF, p.M, p.N, p.K, p.g.n);
    constexpr int SB = (AF == kMxFp8 ? kMxStage : kBigStage) / kMxBlock;
    const int kb = (int)(p.K / kMxBlock);
    uint32_t* sc = (uint32_t*)work;
    const StagedGroups sg = {(const int4*)(work + w.tab), (const uint32_t*)(work + w.offsets)};
    stage_groups_kernel<SB><<<dim3((unsigned)(w.rows / 256), (unsigned)((kb + 127) / 128)), 256, 0, stream>>>(
        p.g, p.as, (int)p.M, (uint32_t)(AF == kMxFp8 ? p.K : p.K / 2), p.ws, p.N, w.n_pad, kb, w.n_mt, w.rows, sc,
        (int4*)(work + w.tab), (uint32_t*)(work + w.offsets));
    if constexpr (AF == kMxFp8) {
#define AWQ_BIG8(GATHER)                                                                                             \
  mx_big8_kernel<YT, Groups, GATHER><<<256, 512, 0, stream>>>(p.A, p.M, p.W, p.N, p.K, sc, w.m_pad, w.rows, w.n_mt, w.n_nt, \
                                                              4, p.Y, p.ld_y, p.g, sg)
      if (p.g.rows != nullptr) AWQ_BIG8(true); else AWQ_BIG8(false);
#undef AWQ_BIG8
    } else {
      mx_big_kernel<YT, Groups><<<(unsigned)(w.n_mt * w.n_nt + 2 * kMxXcds), 512, 0, stream>>>(
          p.A, p.M, p.W, p.N, p.K, sc, w.m_pad, w.rows, w.n_mt, w.n_nt, 4, p.Y, p.ld_y, p.g, sg);
    }
  }
}

hipError_t launch_mx_matmul_grouped(const void* A, const uint8_t* as, int a_fmt, int64_t a_rows, const int32_t* rows,
                                    int64_t M, const void* W, const uint8_t* ws, int n_groups, int64_t N, int64_t K,
                                    const int32_t* offsets, void* Y, int64_t ld_y, int y_dtype, void* work,
                                    hipStream_t stream) {
  const GroupedArgs p = {(const uint8_t*)A, as, (const uint8_t*)W, ws, M, N, K, Y, ld_y,
                         {offsets, n_groups, rows, a_rows, 0}};
  if (a_fmt == kMxFp8) {
    if (y_dtype == 0) grouped_launch<kMxFp8, 0>(p, (uint8_t*)work, stream);
    else grouped_launch<kMxFp8, 1>(p, (uint8_t*)work, stream);
  } else {
    if (y_dtype == 0) grouped_launch<kMxFp4, 0>(p, (uint8_t*)work, stream);
    else if (y_dtype == 1) grouped_launch<kMxFp4, 1>(p, (uint8_t*)work, stream);
    else grouped_launch<kMxFp4, 2>(p, (uint8_t*)work, stream);
  }
  return hipGetLastError();
}

}  // namespace awq
