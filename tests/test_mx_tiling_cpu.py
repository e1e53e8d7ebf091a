"""Which kernel, tile, number of K ranges and LDS slots the products of the GPU tests
take: the selection (csrc/mx_tiles.h) compiled for the host, asked for each of their shapes."""
import ctypes
import os
import subprocess

import pytest

from tests.mx_shapes import FORMS, PRODUCTS, REACHED

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "post_weight_quantization_awq_amd", "csrc")

SOURCE = r"""
#include "mx_tiles.h"
using namespace awq;
extern "C" void tiling(int fmt, int64_t M, int64_t N, int64_t K, int* out) {
  const MxTiling t = mx_tiling(fmt, M, N, K);
  const FewTile f = few_tile(fmt, M, N);
  out[0] = t.tile, out[1] = t.tile ? t.ranges : f.rows, out[2] = t.tile ? tile_slots(t, M, N) : f.tiles;
  out[3] = t.split, out[4] = (int)((K + kMxStage - 1) / kMxStage);
}
"""


@pytest.fixture(scope="module")
def tiling(tmp_path_factory):
    from post_weight_quantization_awq_amd.build import HIPCC
    d = tmp_path_factory.mktemp("mx_tiling")
    src, lib = d / "tiling.cpp", d / "libtiling.so"
    src.write_text(SOURCE)
    r = subprocess.run([HIPCC, "-x", "hip", "--offload-host-only", "-O2", "-std=c++17", "-fPIC", "-shared", "-I", CSRC,
                        str(src), "-o", str(lib)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    L = ctypes.CDLL(str(lib))

    def ask(fmt, M, N, K):
        out = (ctypes.c_int * 5)()
        L.tiling(0 if fmt == "fp8" else 1, ctypes.c_int64(M), ctypes.c_int64(N), ctypes.c_int64(K), out)
        kind = {0: "few", 256: "largest"}.get(out[0], f"tile {out[0]}")
        if kind == "few":
            return kind, out[1], out[2]                                     # LDS rows, tiles of 16 outputs
        return kind, out[1] > 1, out[2] if kind == "tile 64" else 0         # K ranges, slots
    return ask


@pytest.mark.parametrize("M,N,K,fmt,form", PRODUCTS)
def test_shape_takes_the_form_it_is_there_for(tiling, M, N, K, fmt, form):
    assert tiling(fmt, M, N, K) == FORMS[form]


def test_every_form_is_there_in_both_formats():
    seen = {(form, fmt) for _, _, _, fmt, form in PRODUCTS}
    for form in FORMS:
        for fmt in ("fp8", "fp4"):
            assert (form, fmt) in seen or (form, fmt) == ("few 24 x 1", "fp4"), (form, fmt)


@pytest.mark.parametrize("M,N,K,fmt,form", REACHED)
def test_shapes_of_the_stream_tests(tiling, M, N, K, fmt, form):
    assert tiling(fmt, M, N, K)[:2] == form
