"""Operators of a block with experts without a GPU: the oracle's routing and activations pinned by hand, the forms
that the GPU tests' grouped products take, and every refusal of the C ABI and of the Python binding.  Device
pointers are fake: each call fails validation on the host or has an empty size."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from oracle import awq_oracle as O
from tests.moe_shapes import GROUPED
from tests.test_mx_cpu import A, FAKE, ODD, err, mx, raises  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "post_weight_quantization_awq_amd", "csrc")
INF = float("inf")


# ---- the oracle ------------------------------------------------------------
def test_route_by_hand():
    l = np.array([[0.0, 2.0, 2.0, 1.0], [-INF, -INF, -INF, -INF], [-INF, 3.0, -INF, -INF], [1.0, np.nan, 5.0, 0.0]])
    experts, weights, rows, places, offsets = O.moe_route(l, 2)
    assert experts.tolist() == [[1, 2], [-1, -1], [1, -1], [1, 2]]
    assert weights[:3].tolist() == [[0.5, 0.5], [0, 0], [1, 0]] and np.isnan(weights[3]).all()
    assert offsets.tolist() == [0, 0, 3, 5, 5]
    assert rows.tolist() == [0, 2, 3, 0, 3, -1, -1, -1]
    assert places.tolist() == [[0, 3], [-1, -1], [1, -1], [2, 4]]
    w = O.moe_route(l[:1], 2, renormalize=False, scale=2.0)[1]
    assert np.allclose(w, 2 * np.exp(2.0) / (1 + 2 * np.exp(2.0) + np.exp(1.0)))


def test_activations_by_hand():
    x = np.array([-1.0, 0.0, 1.0])
    assert O.activation(x, "relu").tolist() == [0, 0, 1]
    assert np.allclose(O.activation(x, "silu"), [-0.2689414213699951, 0, 0.7310585786300049])
    assert np.allclose(O.activation(x, "gelu"), [-0.15865525393145707, 0, 0.8413447460685429])
    assert np.allclose(O.activation(x, "gelu_tanh"), [-0.15880800939172324, 0, 0.8411919906082768])


def test_block_norm_by_hand():
    x, r = np.array([[3.0, 4.0], [1.0, 1.0]]), np.array([[1.0, 0.0]])
    h, v = O.block_norm(x, r, np.ones(2), 0.0, residual_scale=2.0, places=np.array([[1, 0, -1]]),
                        shares=np.array([[2.0, 0.5, 9.0]]), gate=np.array([1.0, -1.0]))
    assert h.tolist() == [[5.5, -4.0]]
    assert np.allclose(v, h / np.sqrt((5.5 ** 2 + 16) / 2))
    h, _ = O.block_norm(x[:1], r, np.ones(2), 0.0, post=np.array([2.0, 1.0]))
    assert np.allclose(h, [[1 + 6 / np.sqrt(12.5), 4 / np.sqrt(12.5)]])


# ---- the forms of the grouped product -----------------------------------------
SOURCE = r"""
#include "mx_tiles.h"
using namespace awq;
extern "C" void grouped(int fmt, int64_t M, int64_t N, int64_t K, int groups, int* out) {
  const GroupTiling t = group_tiling(fmt, M, N, K, groups);
  out[0] = t.tile, out[1] = kFewGroupRows, out[2] = t.tile ? t.slots : kFewGroupTiles;
}
// How often each tile of 256 rows x outputs is some XCD's; -1: a place out of range, a full tile behind a half one, or
// shares of full or half tiles that differ by more than one
extern "C" int walk(int n_full, int n_half, int n_nt, int* visits) {
  const int n_mt = n_full + n_half;
  int least[2] = {1 << 30, 1 << 30}, most[2] = {0, 0};
  for (int i = 0; i < n_mt * n_nt; ++i) visits[i] = 0;
  for (int x = 0; x < kMxXcds; ++x) {
    const int n = group_tiles_of_xcd(x, n_full, n_half, n_nt);
    int kind[2] = {0, 0};
    for (int pos = 0; pos < n; ++pos) {
      int mt, nt;
      group_tile_at(x, pos, n_full, n_half, n_nt, 4, &mt, &nt);
      if (mt < 0 || mt >= n_mt || nt < 0 || nt >= n_nt) return -1;
      const int half = mt >= n_full;
      if (!half && kind[1]) return -1;
      ++kind[half];
      ++visits[mt * n_nt + nt];
    }
    for (int k = 0; k < 2; ++k) {
      least[k] = kind[k] < least[k] ? kind[k] : least[k];
      most[k] = kind[k] > most[k] ? kind[k] : most[k];
    }
  }
  return most[0] - least[0] > 1 || most[1] - least[1] > 1 ? -1 : 0;
}
extern "C" int64_t most(int64_t M, int groups, int tile) { return group_tiles_most(M, groups, tile); }
"""


@pytest.fixture(scope="module")
def tiles(tmp_path_factory):
    from post_weight_quantization_awq_amd.build import HIPCC
    d = tmp_path_factory.mktemp("moe_tiles")
    src, lib = d / "tiles.cpp", d / "libtiles.so"
    src.write_text(SOURCE)
    r = subprocess.run([HIPCC, "-x", "hip", "--offload-host-only", "-O2", "-std=c++17", "-fPIC", "-shared", "-I", CSRC,
                        str(src), "-o", str(lib)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lib = ctypes.CDLL(str(lib))
    lib.most.restype = ctypes.c_int64
    return lib


def form_of(tiles, M, E, N, K, fmt):
    out = (ctypes.c_int * 3)()
    tiles.grouped(0 if fmt == "fp8" else 1, ctypes.c_int64(M), ctypes.c_int64(N), ctypes.c_int64(K), E, out)
    return f"few {out[1]} x {out[2]}" if out[0] == 0 else f"32, {out[2]} slots" if out[0] == 32 else str(out[0])


@pytest.mark.parametrize("M,E,N,K,fmt,form", GROUPED)
def test_grouped_forms(tiles, M, E, N, K, fmt, form):
    assert form_of(tiles, M, E, N, K, fmt) == form


def test_grouped_forms_are_all_reached():
    for fmt in ("fp8", "fp4"):
        assert {f for *_, g, f in GROUPED if g == fmt} == {"few 16 x 2", "32, 3 slots", "32, 6 slots", "64", "128", "256"}


def test_grouped_tiles_are_enough(tiles):
    """The launches' bound of row tiles holds for any shares of the rows, and is met."""
    rng = np.random.default_rng(0)
    for _ in range(3000):
        E, tile = int(rng.integers(1, 40)), int(rng.choice([4, 16, 32, 64, 128, 256]))
        M = int(rng.integers(1, 40 * tile))
        cuts = np.sort(rng.integers(0, M + 1, E - 1))
        if rng.random() < 0.3:                       # one row for many, the rest for one
            cuts = np.arange(1, E) if M >= E else np.minimum(np.arange(1, E), M)
        counts = np.diff(np.concatenate([[0], cuts, [M]]))
        most = tiles.most(ctypes.c_int64(M), E, tile)
        assert (-(-counts // tile)).sum() <= most
    assert tiles.most(ctypes.c_int64(100), 1, 64) == 2 and tiles.most(ctypes.c_int64(3), 8, 64) == 3


def test_grouped_walk(tiles):
    """Every tile of the largest kind is computed once, and the XCDs' shares of full and half tiles are equal."""
    rng = np.random.default_rng(1)
    cases = [(0, 1, 1), (1, 0, 1), (3, 5, 1), (0, 9, 7), (47, 34, 16), (1000, 3, 33)]
    cases += [(int(rng.integers(0, 60)), int(rng.integers(1, 60)), int(rng.integers(1, 40))) for _ in range(200)]
    for full, half, nt in cases:
        visits = (ctypes.c_int * ((full + half) * nt))()
        assert tiles.walk(full, half, nt, visits) == 0, (full, half, nt)
        assert all(v == 1 for v in visits), (full, half, nt)


# ---- the C ABI's refusals ---------------------------------------------------
def test_linear_validation(A):
    n = ctypes.c_size_t()

    def m(a=FAKE, a_s=FAKE, fmt=A.AWQ_MX_FP8, M=3, w=FAKE, w_s=FAKE, N=64, K=64, b=None, bdt=0, act=0, r=None, rdt=0,
          ld_r=64, Y=FAKE, ld=64, dt=A.AWQ_F16, yf=-1, codes=None, scales=None, ws=FAKE, nb=1 << 40):
        return A.lib().awq_mx_linear(a, a_s, fmt, M, w, w_s, N, K, b, bdt, act, r, rdt, ld_r, Y, ld, dt, yf, codes, scales,
                                     ws, nb, None)
    assert m(fmt=3) == A.AWQ_EDTYPE and m(dt=4) == A.AWQ_EDTYPE and m(yf=2) == A.AWQ_EDTYPE
    assert m(dt=A.AWQ_F32) == A.AWQ_EDTYPE and "fp32 result" in err(A)
    assert m(act=5) == A.AWQ_EINVAL and m(act=-1) == A.AWQ_EINVAL
    assert m(b=FAKE, bdt=3) == A.AWQ_EDTYPE and m(r=FAKE, rdt=-1) == A.AWQ_EDTYPE
    assert m(K=40) == A.AWQ_ESHAPE and m(K=0) == A.AWQ_ESHAPE and m(ld=63) == A.AWQ_ESHAPE and m(r=FAKE, ld_r=63) == A.AWQ_ESHAPE
    assert m(M=-1) == A.AWQ_EINVAL and m(M=2 ** 27) == A.AWQ_ESHAPE
    q = dict(yf=A.AWQ_MX_FP4, codes=FAKE, scales=FAKE)
    assert m(N=48, **q) == A.AWQ_ESHAPE and "multiple of 32" in err(A)
    assert m(M=2 ** 26, N=128, **q) == A.AWQ_ESHAPE and "2^33" in err(A)
    assert m(yf=A.AWQ_MX_FP8, codes=None, scales=FAKE) == A.AWQ_EINVAL
    assert m(yf=A.AWQ_MX_FP8, codes=FAKE, scales=None) == A.AWQ_EINVAL
    for k in ("a", "a_s", "w", "w_s", "Y"):
        assert m(**{k: None}) == A.AWQ_EINVAL
    assert m(r=FAKE, rdt=A.AWQ_BF16) == A.AWQ_EINVAL and "residual is Y" in err(A)
    assert m(r=FAKE, ld_r=80) == A.AWQ_EINVAL
    assert m(a=FAKE + 8) == A.AWQ_EALIGN and m(w=FAKE + 8) == A.AWQ_EALIGN and m(Y=ODD) == A.AWQ_EALIGN
    assert m(b=FAKE + 2, bdt=A.AWQ_F32) == A.AWQ_EALIGN and m(r=FAKE + 1) == A.AWQ_EALIGN
    assert m(yf=A.AWQ_MX_FP8, codes=FAKE + 4, scales=FAKE) == A.AWQ_EALIGN
    assert m(M=0, a=None, a_s=None, Y=None) == A.AWQ_OK and m(N=0, w=None, w_s=None, Y=None) == A.AWQ_OK
    L = A.lib()
    assert L.awq_mx_linear_workspace(A.AWQ_MX_FP8, 200, 544, 4096, ctypes.byref(n)) == A.AWQ_OK and n.value > 0
    need = n.value
    big = dict(M=200, N=544, K=4096, ld=544)
    assert m(ws=None, nb=need, **big) == A.AWQ_EWORKSPACE and m(nb=need - 1, **big) == A.AWQ_EWORKSPACE
    assert m(ws=FAKE + 128, **big) == A.AWQ_EALIGN
    assert L.awq_mx_linear_workspace(A.AWQ_MX_FP8, 1, 1, 32, None) == A.AWQ_EINVAL
    assert L.awq_mx_linear_workspace(A.AWQ_MX_FP8, 1, 1, 31, ctypes.byref(n)) == A.AWQ_ESHAPE


def test_route_validation(A):
    n = ctypes.c_size_t()

    def r(l=FAKE, dt=A.AWQ_F32, T=100, E=16, ld=16, top=2, renorm=1, scale=1.0, ex=FAKE, w=FAKE, rows=FAKE, pl=FAKE,
          off=FAKE, ws=FAKE, nb=1 << 30):
        return A.lib().awq_moe_route(l, dt, T, E, ld, top, renorm, scale, ex, w, rows, pl, off, ws, nb, None)
    assert r(dt=3) == A.AWQ_EDTYPE
    assert r(T=-1) == A.AWQ_EINVAL and r(E=0) == A.AWQ_ESHAPE and r(E=1025, ld=1025) == A.AWQ_ESHAPE
    assert r(T=2 ** 24 + 1) == A.AWQ_ESHAPE
    assert r(top=0) == A.AWQ_ESHAPE and r(top=17) == A.AWQ_ESHAPE and r(E=64, ld=64, top=33) == A.AWQ_ESHAPE
    assert r(ld=15) == A.AWQ_ESHAPE
    for k in ("l", "ex", "w", "rows", "pl", "off"):
        assert r(**{k: None}) == A.AWQ_EINVAL
        assert r(**{k: FAKE + 2}) == A.AWQ_EALIGN
    assert r(ws=None) == A.AWQ_EWORKSPACE and r(nb=31) == A.AWQ_EWORKSPACE and r(ws=FAKE + 64) == A.AWQ_EALIGN
    L = A.lib()
    assert L.awq_moe_route_workspace(100, 16, None) == A.AWQ_EINVAL
    assert L.awq_moe_route_workspace(64, 1024, ctypes.byref(n)) == A.AWQ_OK and n.value == 0
    assert L.awq_moe_route_workspace(65, 16, ctypes.byref(n)) == A.AWQ_OK and n.value >= 64
    assert L.awq_moe_route_workspace(2 ** 24, 1024, ctypes.byref(n)) == A.AWQ_OK and n.value == 512 * 2048


def test_grouped_validation(A):
    n = ctypes.c_size_t()

    def m(a=FAKE, a_s=FAKE, fmt=A.AWQ_MX_FP8, ar=9, rows=None, M=9, w=FAKE, w_s=FAKE, E=4, N=48, K=64, off=FAKE, Y=FAKE,
          ld=48, dt=A.AWQ_F16, ws=FAKE, nb=1 << 40):
        return A.lib().awq_mx_matmul_grouped(a, a_s, fmt, ar, rows, M, w, w_s, E, N, K, off, Y, ld, dt, ws, nb, None)
    assert m(fmt=3) == A.AWQ_EDTYPE and m(dt=4) == A.AWQ_EDTYPE
    assert m(dt=A.AWQ_F32) == A.AWQ_EDTYPE and "fp32 result" in err(A)
    assert m(K=40) == A.AWQ_ESHAPE and m(K=0) == A.AWQ_ESHAPE and m(ld=47) == A.AWQ_ESHAPE
    assert m(E=0) == A.AWQ_ESHAPE and m(E=1025) == A.AWQ_ESHAPE and m(N=2 ** 20 + 1, ld=2 ** 20 + 1) == A.AWQ_ESHAPE
    assert m(M=-1) == A.AWQ_EINVAL and m(ar=-1) == A.AWQ_EINVAL and m(M=2 ** 27, ar=2 ** 27) == A.AWQ_ESHAPE
    assert m(ar=8) == A.AWQ_ESHAPE and "rows is NULL" in err(A)
    assert m(ar=0, rows=FAKE) == A.AWQ_ESHAPE and m(ar=2 ** 26 + 1, rows=FAKE) == A.AWQ_ESHAPE
    assert m(ar=2 ** 25, rows=FAKE) == A.AWQ_ESHAPE and "2^31" in err(A)
    for k in ("a", "a_s", "w", "w_s", "off", "Y"):
        assert m(**{k: None}) == A.AWQ_EINVAL
    assert m(a=FAKE + 8) == A.AWQ_EALIGN and m(w=FAKE + 8) == A.AWQ_EALIGN and m(Y=ODD) == A.AWQ_EALIGN
    assert m(off=FAKE + 2) == A.AWQ_EALIGN and m(rows=FAKE + 1) == A.AWQ_EALIGN
    assert m(M=0, ar=0, a=None, Y=None) == A.AWQ_OK and m(N=0, w=None, Y=None) == A.AWQ_OK
    L = A.lib()
    assert L.awq_mx_matmul_grouped_workspace(A.AWQ_MX_FP8, 9, 9, 64, 4, None) == A.AWQ_EINVAL
    assert L.awq_mx_matmul_grouped_workspace(A.AWQ_MX_FP8, 4096, 4096, 1184, 4, ctypes.byref(n)) == A.AWQ_OK and n.value > 0
    big = dict(M=4096, ar=4096, N=4096, K=1184, ld=4096)
    assert m(ws=None, **big) == A.AWQ_EWORKSPACE and m(nb=n.value - 1, **big) == A.AWQ_EWORKSPACE
    assert m(ws=FAKE + 128, **big) == A.AWQ_EALIGN


def test_block_norm_validation(A):
    def n(X=FAKE, dt=A.AWQ_BF16, xr=4, ld=64, pl=None, sh=None, top=0, rows=4, cols=64, post=None, pdt=0, gate=None, gdt=0,
          ld_g=0, r=FAKE, ld_r=64, c=1.0, w=FAKE, wdt=A.AWQ_BF16, eps=1e-6, ro=FAKE, ld_ro=64, fmt=A.AWQ_MX_FP8, codes=FAKE,
          scales=FAKE):
        return A.lib().awq_block_norm_mx(X, dt, xr, ld, pl, sh, top, rows, cols, post, pdt, gate, gdt, ld_g, r, ld_r, c, w,
                                         wdt, eps, ro, ld_ro, fmt, codes, scales, None)
    assert n(dt=A.AWQ_F32) == A.AWQ_EDTYPE and n(wdt=5) == A.AWQ_EDTYPE and n(fmt=7) == A.AWQ_EDTYPE
    assert n(post=FAKE, pdt=3) == A.AWQ_EDTYPE and n(gate=FAKE, gdt=-1) == A.AWQ_EDTYPE
    assert n(cols=80) == A.AWQ_ESHAPE
    big = 65568
    assert n(cols=big, ld=big, ld_r=big, ld_ro=big) == A.AWQ_ESHAPE and "65536" in err(A)
    assert n(eps=-1.0) == A.AWQ_EINVAL and n(eps=float("nan")) == A.AWQ_EINVAL
    assert n(pl=FAKE, top=2) == A.AWQ_EINVAL and n(sh=FAKE) == A.AWQ_EINVAL and "go together" in err(A)
    assert n(pl=FAKE, sh=FAKE, top=0, ro=FAKE + 64) == A.AWQ_ESHAPE and n(pl=FAKE, sh=FAKE, top=33) == A.AWQ_ESHAPE
    assert n(xr=5) == A.AWQ_ESHAPE and "places is NULL" in err(A) and n(xr=-1) == A.AWQ_ESHAPE
    assert n(ld=63) == A.AWQ_ESHAPE and n(ld_r=32) == A.AWQ_ESHAPE and n(ld_ro=0) == A.AWQ_ESHAPE
    assert n(gate=FAKE, ld_g=63) == A.AWQ_ESHAPE
    for k in ("X", "r", "w", "ro", "codes", "scales"):
        assert n(**{k: None}) == A.AWQ_EINVAL
    assert n(pl=FAKE, sh=FAKE, top=2) == A.AWQ_EINVAL and "other tokens" in err(A)
    for other in ("ld", "ld_r", "ld_ro"):  # residual_out is X and residual here
        assert n(**{other: 72}) == A.AWQ_EINVAL and "row stride" in err(A)
    assert n(X=ODD) == A.AWQ_EALIGN and n(w=FAKE + 2, wdt=A.AWQ_F32) == A.AWQ_EALIGN and n(codes=FAKE + 4) == A.AWQ_EALIGN
    assert n(r=ODD) == A.AWQ_EALIGN and n(post=ODD) == A.AWQ_EALIGN and n(gate=FAKE + 2, gdt=A.AWQ_F32) == A.AWQ_EALIGN
    assert n(pl=FAKE + 2, sh=FAKE, top=2, ro=FAKE + 64) == A.AWQ_EALIGN
    assert n(rows=0, xr=0, X=None, w=None, codes=None, scales=None) == A.AWQ_OK


# ---- the binding's refusals ---------------------------------------------------
def test_binding_rejects_bad_tensors(A):
    c, s = mx(4, 64, "fp8")
    w = mx(32, 64, "fp4")
    raises(lambda: A.mx_linear(c, s, *mx(32, 64, "fp8")), "4-bit codes")
    raises(lambda: A.mx_linear(c, s, *w, activation="tanh"), "activation 'tanh'")
    raises(lambda: A.mx_linear(c, s, *w, bias=torch.ones(31)), r"bias must have shape \[32\]")
    raises(lambda: A.mx_linear(c, s, *w, bias=torch.ones(32, dtype=torch.float64)), "bias must have dtype")
    raises(lambda: A.mx_linear(c, s, *w, residual=torch.ones((4, 31))), "residual must have shape")
    raises(lambda: A.mx_linear(c, s, *w, residual=torch.ones((4, 64))[:, ::2]), "unit column stride")
    raises(lambda: A.mx_linear(c, s, *w, fmt="fp6"), "fmt 'fp6'")
    raises(lambda: A.mx_linear(c, s, *mx(48, 64, "fp4"), fmt="fp8"), "whole blocks of 32")
    raises(lambda: A.mx_linear(c, s, *w, fmt="fp8", out=mx(4, 32, "fp4")), "codes must have dtype")
    raises(lambda: A.mx_linear(c, s, *w, out_dtype=torch.float64), "out_dtype")
    raises(lambda: A.mx_linear(c, s, *w), "a_codes must be a device tensor")

    L = torch.zeros((6, 16))
    raises(lambda: A.moe_route(L.double(), 2), "logits must have dtype")
    raises(lambda: A.moe_route(L, 0), "top must be in")
    raises(lambda: A.moe_route(L, 17), "top must be in")
    i = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    raises(lambda: A.moe_route(L, 2, out=A.MoeRouting(i(6, 2), torch.zeros((6, 2)), i(12), i(6, 2), i(16))),
           "offsets must have shape")
    raises(lambda: A.moe_route(L, 2), "logits must be a device tensor")

    W, S = torch.stack([w[0]] * 3), torch.stack([w[1].view(torch.uint8)] * 3).view(torch.float8_e8m0fnu)
    raises(lambda: A.mx_matmul_grouped(c, s, W, S, i(3)), r"offsets must have shape \[4\]")
    raises(lambda: A.mx_matmul_grouped(c, s, W, S, i(4).long()), "offsets must have dtype")
    raises(lambda: A.mx_matmul_grouped(c, s, W[0], S, i(4)), "w_codes must have shape")
    raises(lambda: A.mx_matmul_grouped(c, s, W, S[:2], i(4)), "w_scales must have shape")
    raises(lambda: A.mx_matmul_grouped(c, s, W, S, i(4), rows=i(4, 1)), "rows must have shape")
    raises(lambda: A.mx_matmul_grouped(c, s, W, S, i(4), rows=i(7), out=torch.zeros((4, 32))), "out must have shape")
    raises(lambda: A.mx_matmul_grouped(c, s, W, S, i(4), out_dtype=torch.int32), "out_dtype")
    raises(lambda: A.mx_matmul_grouped(c, s, W, S, i(4)), "a_codes must be a device tensor")

    X, o = torch.zeros((4, 64), dtype=torch.bfloat16), torch.ones(64)
    raises(lambda: A.block_norm_mx(X, X.half(), o), "residual must have dtype")
    raises(lambda: A.block_norm_mx(X, X[:2], o), "X must have shape")
    raises(lambda: A.block_norm_mx(X, X, o[:32]), "weight must have shape")
    raises(lambda: A.block_norm_mx(X, X, o, post_weight=o[:32]), "post_weight must have shape")
    raises(lambda: A.block_norm_mx(X, X, o, gate=o[:32]), "gate must have shape")
    raises(lambda: A.block_norm_mx(X, X, o, gate=torch.ones((3, 64))), "gate must have shape")
    raises(lambda: A.block_norm_mx(X, X, o, gate=torch.ones(1).expand(4, 64)), "gate must be")
    raises(lambda: A.block_norm_mx(X, X, o, places=i(4, 2)), "go together")
    raises(lambda: A.block_norm_mx(X, X, o, places=i(4, 2), shares=torch.zeros((4, 3))), "shares must have shape")
    raises(lambda: A.block_norm_mx(X, X, o, places=i(3, 2), shares=torch.zeros((3, 2))), "places must have shape")
    raises(lambda: A.block_norm_mx(X, X, o, residual_out=X[:2]), "residual_out must have shape")
    raises(lambda: A.block_norm_mx(X[:, :40], X[:, :40], o[:40]), "whole blocks of 32")
    raises(lambda: A.block_norm_mx(X, X, o), "X must be a device tensor")
