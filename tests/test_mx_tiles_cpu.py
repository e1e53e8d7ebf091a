"""The host side of the product's tiles, compiled from the kernels' own header
(csrc/mx_tiles.h) and run without a GPU."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "post_weight_quantization_awq_amd", "csrc")

SOURCE = r"""
#include "mx_tiles.h"
#include <vector>
using namespace awq;

// One direct load of 16 bytes at offset v of a buffer of `bytes`, with scalar offset s.  The hardware drops it if
// v >= bytes - s in 32 bits, or, by another reading of the rule, if v >= bytes; under both it must stay inside, and
// the difference must not wrap.  left: bytes that are really there behind the buffer's start.
static int bad_load(uint32_t v, StageSpan s, int64_t left) {
  if (s.k_off > s.bytes) return 1;
  const bool in1 = v < s.bytes - s.k_off, in2 = v < s.bytes;
  return (in1 || in2) && (int64_t)v + s.k_off + 16 > left;
}

template <int SB>
static int64_t bad_operand(int first, int rows, uint32_t row_bytes, int k) {
  const StageSpan s = stage_span<SB>(first, rows, row_bytes, k);
  const int64_t left = (int64_t)(rows - first) * row_bytes;
  int64_t bad = 0;
  for (int r = 0; r < kBigTile; ++r)
    for (int c = 0; c < SB; c += 16) bad += bad_load((uint32_t)r * row_bytes + c, s, left);
  return bad;
}

// Every load of 8-bit (128 bytes a stage) and 4-bit (64) codes by the persistent blocks of an M x N x K product:
// all stages of a block's tiles, then the first two of what lies behind its last tile.
extern "C" int64_t bad_loads(int M, int N, int K, int units, int* visits) {
  const int n_mt = (M + kBigTile - 1) / kBigTile, n_nt = (N + kBigTile - 1) / kBigTile, tiles = n_mt * n_nt;
  const int nk = (K + kMxStage - 1) / kMxStage, grid = tiles < units ? tiles : units;
  int64_t bad = 0;
  for (int i = 0; i < tiles; ++i) visits[i] = 0;
  for (int b = 0; b < grid; ++b) {
    int id = b;
    for (; id < tiles; id += grid) {
      const TileAt t = big_tile_at(id, n_mt, n_nt, 4, M, N);
      if (t.m0 % kBigTile || t.n0 % kBigTile || t.m0 >= M || t.n0 >= N) return -1;
      ++visits[t.m0 / kBigTile * n_nt + t.n0 / kBigTile];
      for (int k = 0; k < nk; ++k) bad += bad_operand<128>(t.m0, M, K, k) + bad_operand<64>(t.n0, N, K / 2, k);
    }
    const TileAt t = big_tile_at(id, n_mt, n_nt, 4, M, N);
    if (t.m0 != M || t.n0 != N) return -2;
    for (int k = 0; k < 2; ++k) bad += bad_operand<128>(t.m0, M, K, k) + bad_operand<64>(t.n0, N, K / 2, k);
  }
  return bad;
}
"""


@pytest.fixture(scope="module")
def tiles(tmp_path_factory):
    from post_weight_quantization_awq_amd.build import HIPCC
    d = tmp_path_factory.mktemp("mx_tiles")
    src, lib = d / "tiles.cpp", d / "libtiles.so"
    src.write_text(SOURCE)
    r = subprocess.run([HIPCC, "-x", "hip", "--offload-host-only", "-O2", "-std=c++17", "-fPIC", "-shared", "-I", CSRC,
                        str(src), "-o", str(lib)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    L = ctypes.CDLL(str(lib))
    L.bad_loads.restype = ctypes.c_int64
    return L


@pytest.mark.parametrize("M,N,K,units", [
    (4096, 24576, 416, 256), (1000, 12250, 384, 256), (1, 1, 384, 256), (257, 255, 4096, 2), (4000, 16001, 544, 256),
    (300, 70000, 1056, 256), (769, 2049, 736, 3), (256, 256, 1 << 22, 1),
])
def test_persistent_blocks_load_inside_their_operands(tiles, M, N, K, units):
    """Every tile once, and no load past an operand's end, those behind a block's last tile included: there the
    scalar offset is 0, as the buffer's size is."""
    n = -(-M // 256) * -(-N // 256)
    visits = (ctypes.c_int * n)()
    assert tiles.bad_loads(M, N, K, units, visits) == 0
    assert list(visits) == [1] * n
