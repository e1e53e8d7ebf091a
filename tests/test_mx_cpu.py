"""Microscaled operators without a GPU: the oracle's formats pinned by hand, and
every refusal of the C ABI and of the Python binding.  Device pointers are fake:
each call fails validation on the host or has an empty size."""
import numpy as np
import pytest
import torch

from oracle import awq_oracle as O


@pytest.fixture(scope="module")
def A():
    import os
    from post_weight_quantization_awq_amd import LIB_PATH
    if not os.path.exists(LIB_PATH):
        from post_weight_quantization_awq_amd import build
        build.build()
    import post_weight_quantization_awq_amd as A
    A.lib()
    return A


# ---- the oracle ------------------------------------------------------------
def test_element_tables():
    assert O.mx_element_table("fp4").tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]
    t = O.mx_element_table("fp8")
    ref = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, ref, equal_nan=True)
    assert t[0x7E] == 448 and t[1] == 2.0 ** -9 and np.isnan(t[0x7F])


def test_quantize_by_hand():
    v = np.zeros((1, 64))
    v[0, :12] = [8.0, 7.0, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.75, -0.2, 5.0000001]
    codes, scales = O.mx_quantize(v, "fp4")
    # max 8 = 2^3: e = 1, elements v / 2: 4, 3.5 -> 4 (even), 2.5 -> 2 (even), 1.75 -> 2, 1.25 -> 1, .875 -> 1,
    # .625 -> .5, .375 -> .5, .125 -> 0, -.375 -> -.5, -.1 -> -0, 2.50000005 -> 3
    assert scales.tolist() == [[128, 0]]
    assert O.mx_values(codes, scales, "fp4")[0, :12].tolist() == [8, 8, 4, 4, 2, 2, 1, 1, 0, -1, 0, 6]
    v = np.zeros((1, 32))
    v[0, :5] = [511.0, 449.0, -17.0, 2.0 ** -10, 3 * 2.0 ** -10]
    codes, scales = O.mx_quantize(v, "fp8")
    assert scales.tolist() == [[127]]
    assert O.mx_values(codes, scales, "fp8")[0, :5].tolist() == [448, 448, -16, 0, 2.0 ** -8]


def test_quantize_edges():
    v = np.zeros((1, 128))
    v[0, 3] = np.nan
    v[0, 40] = -np.inf
    v[0, 70] = 2.0 ** -140      # below the smallest scale: e = -127, rounds to 0
    v[0, 100] = 3e38
    for fmt, top in (("fp8", 254 - 8), ("fp4", 254 - 2)):
        codes, scales = O.mx_quantize(v, fmt)
        assert scales.tolist() == [[255, 255, 0, top]]
        got = O.mx_values(codes, scales, fmt)
        assert np.isnan(got[0, :64]).all() and not got[0, 64:96].any()
    assert np.array_equal(O.mx_quantize(np.zeros((2, 32)), "fp8")[1], [[0], [0]])


# ---- the C ABI's refusals ---------------------------------------------------
FAKE, ODD = 1 << 20, (1 << 20) + 1


def err(A):
    return A.lib().awq_last_error().decode()


def test_quantize_validation(A):
    def q(X=FAKE, dt=A.AWQ_BF16, rows=4, cols=64, ld=64, s=None, fmt=A.AWQ_MX_FP8, codes=FAKE, scales=FAKE):
        return A.lib().awq_mx_quantize(X, dt, rows, cols, ld, s, fmt, codes, scales, None)
    assert q(dt=A.AWQ_F32) == A.AWQ_EDTYPE
    assert q(fmt=2) == A.AWQ_EDTYPE and "format 2" in err(A)
    assert q(cols=48) == A.AWQ_ESHAPE and "multiple of 32" in err(A)
    assert q(rows=-1) == A.AWQ_EINVAL
    assert q(ld=63) == A.AWQ_ESHAPE
    assert q(rows=2 ** 27, cols=64) == A.AWQ_ESHAPE and "2^33" in err(A)
    assert q(rows=2 ** 62, cols=64) == A.AWQ_ESHAPE
    assert q(rows=2 ** 27 + 1, cols=32, ld=32) == A.AWQ_ESHAPE and "2^27" in err(A)
    assert q(X=None) == A.AWQ_EINVAL and q(codes=None) == A.AWQ_EINVAL and q(scales=None) == A.AWQ_EINVAL
    assert q(X=ODD) == A.AWQ_EALIGN and q(s=FAKE + 2) == A.AWQ_EALIGN and q(codes=FAKE + 8) == A.AWQ_EALIGN
    assert q(rows=0, X=None, codes=None, scales=None) == A.AWQ_OK and err(A) == ""
    assert q(cols=0, X=None, codes=None, scales=None) == A.AWQ_OK


def test_dequant_validation(A):
    def d(codes=FAKE, scales=FAKE, fmt=A.AWQ_MX_FP4, rows=4, cols=64, s=None, out=FAKE, dt=A.AWQ_F32, ld=64):
        return A.lib().awq_mx_dequant(codes, scales, fmt, rows, cols, s, out, dt, ld, None)
    assert d(dt=3) == A.AWQ_EDTYPE and d(fmt=-1) == A.AWQ_EDTYPE
    assert d(cols=33) == A.AWQ_ESHAPE and d(ld=32) == A.AWQ_ESHAPE
    assert d(codes=None) == A.AWQ_EINVAL and d(scales=None) == A.AWQ_EINVAL and d(out=None) == A.AWQ_EINVAL
    assert d(out=FAKE + 2) == A.AWQ_EALIGN and d(dt=A.AWQ_F16, out=ODD) == A.AWQ_EALIGN
    assert d(codes=FAKE + 4) == A.AWQ_EALIGN and d(s=ODD) == A.AWQ_EALIGN
    assert d(rows=0, codes=None, scales=None, out=None) == A.AWQ_OK


def test_norm_validation(A):
    def n(X=FAKE, dt=A.AWQ_BF16, rows=4, cols=64, ld=64, r=None, ld_r=64, w=FAKE, wdt=A.AWQ_BF16, eps=1e-6, ro=None,
          ld_ro=64, fmt=A.AWQ_MX_FP8, codes=FAKE, scales=FAKE):
        return A.lib().awq_rms_norm_mx(X, dt, rows, cols, ld, r, ld_r, w, wdt, eps, ro, ld_ro, fmt, codes, scales, None)
    assert n(dt=A.AWQ_F32) == A.AWQ_EDTYPE and n(wdt=5) == A.AWQ_EDTYPE and n(fmt=7) == A.AWQ_EDTYPE
    assert n(cols=80) == A.AWQ_ESHAPE and n(cols=65568, ld=65568) == A.AWQ_ESHAPE and "65536" in err(A)
    assert n(eps=-1.0) == A.AWQ_EINVAL and n(eps=float("nan")) == A.AWQ_EINVAL
    assert n(r=FAKE) == A.AWQ_EINVAL and n(ro=FAKE) == A.AWQ_EINVAL and "go together" in err(A)
    assert n(r=FAKE, ro=FAKE, ld_r=32) == A.AWQ_ESHAPE and n(r=FAKE, ro=FAKE, ld_ro=63) == A.AWQ_ESHAPE
    assert n(ld=0) == A.AWQ_ESHAPE
    assert n(X=None) == A.AWQ_EINVAL and n(w=None) == A.AWQ_EINVAL and n(scales=None) == A.AWQ_EINVAL
    assert n(X=ODD) == A.AWQ_EALIGN and n(w=FAKE + 2, wdt=A.AWQ_F32) == A.AWQ_EALIGN
    assert n(r=ODD, ro=FAKE) == A.AWQ_EALIGN and n(codes=FAKE + 4) == A.AWQ_EALIGN
    assert n(rows=0, X=None, w=None, codes=None, scales=None) == A.AWQ_OK


def test_silu_validation(A):
    def g(gate=FAKE, ld_g=64, up=FAKE, ld_u=64, dt=A.AWQ_F16, rows=2, cols=64, fmt=A.AWQ_MX_FP4, codes=FAKE,
          scales=FAKE):
        return A.lib().awq_silu_mul_mx(gate, ld_g, up, ld_u, dt, rows, cols, fmt, codes, scales, None)
    assert g(dt=A.AWQ_F32) == A.AWQ_EDTYPE and g(fmt=9) == A.AWQ_EDTYPE
    assert g(cols=16) == A.AWQ_ESHAPE and g(ld_g=32) == A.AWQ_ESHAPE and g(ld_u=32) == A.AWQ_ESHAPE
    assert g(gate=None) == A.AWQ_EINVAL and g(up=None) == A.AWQ_EINVAL and g(codes=None) == A.AWQ_EINVAL
    assert g(gate=ODD) == A.AWQ_EALIGN and g(codes=FAKE + 2) == A.AWQ_EALIGN
    assert g(rows=0, gate=None, up=None, codes=None, scales=None) == A.AWQ_OK


def test_matmul_validation(A):
    import ctypes
    n = ctypes.c_size_t()

    def m(a=FAKE, a_s=FAKE, fmt=A.AWQ_MX_FP8, M=3, w=FAKE, w_s=FAKE, N=48, K=64, Y=FAKE, ld=48, dt=A.AWQ_F16,
          ws=FAKE, nb=1 << 40):
        return A.lib().awq_mx_matmul(a, a_s, fmt, M, w, w_s, N, K, Y, ld, dt, ws, nb, None)
    assert m(fmt=3) == A.AWQ_EDTYPE and m(dt=4) == A.AWQ_EDTYPE
    assert m(dt=A.AWQ_F32) == A.AWQ_EDTYPE and "fp32 result" in err(A)
    assert m(K=40) == A.AWQ_ESHAPE and m(K=0) == A.AWQ_ESHAPE and m(ld=47) == A.AWQ_ESHAPE
    assert m(M=-1) == A.AWQ_EINVAL and m(M=2 ** 27) == A.AWQ_ESHAPE and m(K=2 ** 22 + 32) == A.AWQ_ESHAPE
    assert m(M=2 ** 20, N=2 ** 18, ld=2 ** 18) == A.AWQ_ESHAPE and "2^37" in err(A)
    for k in ("a", "a_s", "w", "w_s", "Y"):
        assert m(**{k: None}) == A.AWQ_EINVAL
    assert m(a=FAKE + 8) == A.AWQ_EALIGN and m(w=FAKE + 8) == A.AWQ_EALIGN and m(Y=ODD) == A.AWQ_EALIGN
    assert m(fmt=A.AWQ_MX_FP4, dt=A.AWQ_F32, Y=FAKE + 2) == A.AWQ_EALIGN
    assert m(M=0, a=None, a_s=None, Y=None) == A.AWQ_OK and m(N=0, w=None, w_s=None, Y=None) == A.AWQ_OK
    L = A.lib()
    assert L.awq_mx_matmul_workspace(A.AWQ_MX_FP8, 1, 1, 32, None) == A.AWQ_EINVAL
    assert L.awq_mx_matmul_workspace(A.AWQ_MX_FP8, 1, 1, 31, ctypes.byref(n)) == A.AWQ_ESHAPE
    assert L.awq_mx_matmul_workspace(A.AWQ_MX_FP8, 0, 64, 64, ctypes.byref(n)) == A.AWQ_OK and n.value == 0


# ---- the binding's refusals ---------------------------------------------------
def raises(fn, match):
    with pytest.raises(ValueError, match=match):
        fn()


def mx(rows, cols, fmt):
    codes = torch.zeros((rows, cols), dtype=torch.float8_e4m3fn) if fmt == "fp8" else \
        torch.zeros((rows, cols // 2), dtype=torch.uint8)
    return codes, torch.zeros((rows, cols // 32), dtype=torch.uint8).view(torch.float8_e8m0fnu)


def test_binding_rejects_bad_tensors(A):
    X = torch.zeros((4, 64), dtype=torch.bfloat16)
    raises(lambda: A.mx_quantize(X.float()), "X must have dtype")
    raises(lambda: A.mx_quantize(X[:, ::2]), "unit column stride")
    raises(lambda: A.mx_quantize(X[:, :40]), "whole blocks of 32")
    raises(lambda: A.mx_quantize(X, "fp6"), "fmt 'fp6'")
    raises(lambda: A.mx_quantize(X, s=torch.ones(32)), r"s must have shape \[64\]")
    raises(lambda: A.mx_quantize(X, out=mx(4, 64, "fp4")), "codes must have dtype")
    raises(lambda: A.mx_quantize(X, "fp4", out=mx(3, 64, "fp4")), "codes must have shape")
    raises(lambda: A.mx_quantize(X), "X must be a device tensor")
    c, s = mx(4, 64, "fp8")
    raises(lambda: A.mx_dequant(c, s[:, :1].contiguous()), "scales must have shape")
    raises(lambda: A.mx_dequant(c, s.view(torch.uint8)), "scales must have dtype")
    raises(lambda: A.mx_dequant(c, s, out_dtype=torch.float64), "out_dtype")
    raises(lambda: A.mx_dequant(c, s, out=torch.zeros((4, 32))), "out must have shape")
    raises(lambda: A.mx_dequant(c, s), "codes must be a device tensor")
    w = torch.ones(64)
    raises(lambda: A.rms_norm_mx(X, w[:32]), "weight must have shape")
    raises(lambda: A.rms_norm_mx(X, w, residual=X.half()), "residual must have dtype")
    raises(lambda: A.rms_norm_mx(X, w, residual_out=X), "residual_out without residual")
    raises(lambda: A.rms_norm_mx(X, w, residual=X, residual_out=X[:2]), "residual_out must have shape")
    raises(lambda: A.rms_norm_mx(X, w), "X must be a device tensor")
    raises(lambda: A.silu_mul_mx(X, X[:2]), "up must have shape")
    raises(lambda: A.silu_mul_mx(X, X.half()), "up must have dtype")
    raises(lambda: A.silu_mul_mx(X, X), "gate must be a device tensor")
    wc, wsc = mx(16, 64, "fp4")
    raises(lambda: A.mx_matmul(c, s, *mx(16, 64, "fp8")), "4-bit codes")
    raises(lambda: A.mx_matmul(c, s, *mx(16, 96, "fp4")), "64 columns, w_codes 96")
    raises(lambda: A.mx_matmul(c.t(), s, wc, wsc), "contiguous")
    raises(lambda: A.mx_matmul(c, s, wc, wsc, out=torch.zeros((4, 17), dtype=torch.float16)), "out must have shape")
    raises(lambda: A.mx_matmul(c, s, wc, wsc, out_dtype=torch.float64), "out_dtype")
    raises(lambda: A.mx_matmul(c, s, wc, wsc), "a_codes must be a device tensor")
