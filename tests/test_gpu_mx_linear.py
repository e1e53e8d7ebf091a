"""The microscaled product with bias, activation and residual against the oracle, on the GPU.

Tolerances (u = 2^-24).  The sum is within T of the exact one, as for the plain product (tests/test_gpu_mx.py); the
bias adds u (|sum + bias| + T).  An activation's slope is at most 1.13 (gelu's, at 1.4), so it hands on 1.13 times
that, and adds its own error: an exponential errs by u |argument| for each rounding of its argument; silu 2^-17, gelu_tanh
2^-15, gelu 2^-16 of the value, as documented.  The residual's addition rounds once, and so does the result.  A quantized
result is at most half a step of its element from a value within that error, or saturates."""
import numpy as np
import pytest

from oracle import awq_oracle as O
from tests._util import say
from tests.mx_shapes import PRODUCTS
from tests.test_gpu_mx import (A, STEP, U, dev_mx, fmt_of, product_tol, quantized, random_mx, tdt, to_dev,  # noqa: F401
                               values)

pytestmark = pytest.mark.gpu
ACT = {None: 0.0, "relu": 0.0, "silu": 2.0 ** -17, "gelu_tanh": 2.0 ** -15, "gelu": 2.0 ** -16}


def check_codes(out, fmt, y, e):
    """Quantized `out` against exact values y, each known to the kernel within e."""
    codes, scales = quantized(out)
    emax, most, mbits, emin = {"fp8": (8, 448.0, 3, -6), "fp4": (2, 6.0, 1, 0)}[fmt]
    rows = y.shape[0]
    sc = scales.astype(np.int64)
    for top, le in ((np.maximum(np.abs(y) - e, 0), False), (np.abs(y) + e, True)):
        t = top.reshape(rows, -1, 32).max(axis=2)
        b = np.where(t == 0, 0, np.maximum(np.frexp(t)[1] - 1 - emax, -127) + 127)
        assert np.all(sc <= b) if le else np.all(sc >= b), "scale"
    unit = np.repeat(np.exp2(sc - 127.0), 32, axis=1)
    got = O.mx_values(codes, scales, fmt)
    x = np.minimum((np.abs(y) + e) / unit, most)
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(x, 1e-30))), emin) - mbits)
    want = np.sign(y) * np.minimum(np.abs(y), most * unit)
    assert np.all(np.abs(got - want) <= unit * step / 2 + e), "element"


def check(A, M, N, K, fmt, dtype="f16", bias="f32", act=None, residual=None, out_fmt=None, ld=None, seed=0,
          in_place=False, scale=1.0):
    import torch
    rng = np.random.default_rng(seed + M + 3 * N + 7 * K)
    ac, asc = random_mx(rng, M, K, fmt)
    wc, wsc = O.mx_quantize(scale * values(rng, N, K, 0.5) / np.sqrt(K), "fp4")
    a, w = O.mx_values(ac, asc, fmt), O.mx_values(wc, wsc, "fp4")
    B, b = to_dev(rng.standard_normal((1, N)), bias) if bias else (None, np.zeros((1, N), np.float32))
    R, r = to_dev(2 * rng.standard_normal((M, N)), residual, ld, 1) if residual else (None, np.zeros((M, N), np.float32))
    out, buf = None, None
    if out_fmt is None and in_place:
        out = R
    elif out_fmt is None and ld:
        buf = torch.full((M * ld + 1,), 7.0, dtype=tdt(dtype), device="cuda")
        out = buf[1:].view(M, ld)[:, :N]
    Y = A.mx_linear(*dev_mx(ac, asc, fmt), *dev_mx(wc, wsc, "fp4"), bias=None if B is None else B[0].contiguous(),
                    activation=act, residual=R, out_dtype=tdt(dtype), fmt=out_fmt, out=out)
    torch.cuda.synchronize()
    p = a @ w.T
    T = product_tol(a, w, K, fmt, np.zeros_like(p), "f32")
    p, T = p + b, T + (U * (np.abs(p + b) + T) if bias else 0)
    y = O.activation(p, act)
    e = 1.13 * T + (ACT[act] * np.abs(y) + 2.0 ** -126 if act else 0)
    y = y + r
    e = e + (U * (np.abs(y) + e) if residual else 0)
    if out_fmt:
        check_codes(Y, out_fmt, y, e)
        return
    e = e + STEP[dtype] * (np.abs(y) + e) + (2.0 ** -25 if dtype == "f16" else 0)
    err = np.abs(Y.double().cpu().numpy() - y)
    assert np.all(err <= e), (float((err / e).max()), np.argwhere(err > e)[:4].tolist())
    if buf is not None:
        assert buf[0] == 7 and buf[1:].view(M, ld)[:, N:].eq(7).all()


SHAPES = sorted({(M, N, K, fmt) for M, N, K, fmt, _ in PRODUCTS if M * N < 9_000_000})


@pytest.mark.parametrize("M,N,K,fmt", SHAPES)
def test_every_form(A, M, N, K, fmt):
    """The shapes that reach every form of the product's kernels; what the epilogue does goes round with them."""
    i = SHAPES.index((M, N, K, fmt))
    act = [None, "relu", "silu", "gelu", "gelu_tanh"][i % 5]
    dtype = ["f16", "bf16", "f32" if fmt == "fp4" else "bf16"][i % 3]
    say(f"mx_linear {M}x{N}x{K} {fmt} {act} {dtype}")
    check(A, M, N, K, fmt, dtype, ["f32", "bf16", None, "f16"][i % 4], act, ["bf16", None, "f16", "f32"][i % 4],
          ld=N + 3 if i % 2 else None)


@pytest.mark.parametrize("out_fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("M,N,K,fmt", [
    (1, 32, 32, "fp8"), (1, 4096, 160, "fp4"), (3, 96, 4128, "fp8"), (16, 2080, 544, "fp8"), (20, 512, 1184, "fp8"),
    (30, 320, 416, "fp4"), (40, 4128, 352, "fp8"), (100, 352, 384, "fp8"), (333, 992, 2080, "fp4"),
    (200, 544, 4096, "fp8"), (130, 64, 4640, "fp4"), (512, 992, 12288, "fp8"), (1500, 2080, 544, "fp4"),
    (333, 12256, 768, "fp8"), (200, 2080, 12288, "fp4"), (1024, 8224, 768, "fp8"), (1500, 4128, 1184, "fp4"),
    (300, 4096, 96, "fp8"),
])
def test_quantized_result(A, M, N, K, fmt, out_fmt):
    say(f"mx_linear {M}x{N}x{K} {fmt} -> {out_fmt}")
    check(A, M, N, K, fmt, bias="bf16", act="gelu_tanh" if M % 2 else "silu", out_fmt=out_fmt)
    check(A, M, N, K, fmt, bias=None, act=None, residual="bf16", out_fmt=out_fmt, seed=1)


@pytest.mark.parametrize("act", [None, "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M,fmt", [(1, "fp8"), (33, "fp4"), (150, "fp8"), (700, "fp4")])
def test_activations(A, M, fmt, act):
    say(f"mx_linear activation {act} M {M} {fmt}")
    check(A, M, 520, 1056, fmt, "bf16", "f32", act, None, scale=4.0)
    check(A, M, 520, 1056, fmt, "f16", None, act, "f16", in_place=True, ld=523)
    if fmt == "fp4":
        check(A, M, 520, 1056, fmt, "f32", "f16", act, "f32", in_place=True)


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M", [3, 100])
def test_activation_over_the_whole_range(A, M, act):
    """Products that are 0, so that the bias alone goes through the activation: every bf16 value, to bf16 and fp32."""
    import torch
    say(f"mx_linear every bf16 through {act}, M {M}")
    N, K = 65536, 512
    bits = np.arange(N, dtype=np.uint32) << 16
    b = bits.view(np.float32)
    a = dev_mx(np.zeros((M, K // 2), np.uint8), np.full((M, K // 32), 127, np.uint8), "fp4")
    w = dev_mx(np.zeros((N, K // 2), np.uint8), np.full((N, K // 32), 127, np.uint8), "fp4")
    B = torch.from_numpy(b.copy()).cuda().bfloat16()
    y = O.activation(b.astype(np.float64), act)
    if act == "relu":
        y = np.where(np.isnan(b), np.nan, y)
    for dtype in ("f32", "bf16"):
        got = A.mx_linear(*a, *w, bias=B, activation=act, out_dtype=tdt(dtype)).double().cpu().numpy()
        assert np.array_equal(got, np.repeat(got[:1], M, axis=0), equal_nan=True)
        got = got[0]
        nan = np.isnan(b) | (np.isneginf(b) & (act != "relu"))
        assert np.array_equal(np.isnan(got), nan)
        ok = np.isfinite(y) & ~nan
        assert np.array_equal(got[~ok & ~nan], y[~ok & ~nan])
        top = {"f32": 3.4028235677973366e38, "bf16": 3.3895313892515355e38 * (1 + 2.0 ** -9)}[dtype]
        over = ok & (np.abs(y) >= top)
        tol = (ACT[act] + STEP[dtype] * 1.01) * np.abs(y) + 2.0 ** -126
        err = np.where(ok & ~over, np.abs(got - np.where(ok, y, 0)), 0)
        assert np.all(err <= np.where(ok, tol, np.inf)), (act, dtype, b[np.argmax(err / np.where(ok, tol, 1))])


@pytest.mark.parametrize("M,fmt", [(2, "fp8"), (90, "fp4"), (600, "fp8")])
def test_nan_and_infinities(A, M, fmt):
    """A NaN bias makes its column NaN, an infinite residual its value; a quantized block with one of them is NaN."""
    import torch
    say(f"mx_linear NaN M {M} {fmt}")
    rng = np.random.default_rng(M)
    N, K = 128, 544
    a, w = dev_mx(*random_mx(rng, M, K, fmt), fmt), dev_mx(*random_mx(rng, N, K, "fp4"), "fp4")
    bias = torch.zeros(N, device="cuda")
    ref = A.mx_linear(*a, *w, bias=bias, activation="silu")
    bias[70] = float("nan")
    R = torch.zeros((M, N), dtype=torch.float16, device="cuda")
    R[M - 1, 5] = -float("inf")
    got = A.mx_linear(*a, *w, bias=bias, activation="silu", residual=R)
    keep = torch.ones_like(got, dtype=torch.bool)
    keep[:, 70] = False
    keep[M - 1, 5] = False
    assert got[:, 70].isnan().all() and got[M - 1, 5] == -float("inf")
    assert torch.equal(got[keep], ref[keep])
    codes, scales = A.mx_linear(*a, *w, bias=bias, activation="silu", residual=R, fmt="fp8")
    s = scales.view(torch.uint8)
    assert s[:, 2].eq(255).all() and s[M - 1, 0] == 255 and s[:, [1, 3]].ne(255).all()
    assert s[:M - 1, 0].ne(255).all()
    assert not codes.view(torch.uint8)[:, 64:96].any()


def test_plain_epilogue_is_the_product(A):
    """Without bias, activation and residual the result is that of mx_matmul, bit for bit, in every form."""
    import torch
    say("mx_linear plain = mx_matmul")
    rng = np.random.default_rng(2)
    for M, N, K, fmt, form in PRODUCTS:
        if M * N > 3_000_000:
            continue
        a, w = dev_mx(*random_mx(rng, M, K, fmt), fmt), dev_mx(*random_mx(rng, N, K, "fp4"), "fp4")
        for t in (torch.float16, torch.bfloat16):
            assert torch.equal(A.mx_linear(*a, *w, out_dtype=t), A.mx_matmul(*a, *w, out_dtype=t)), (M, N, K, fmt, form)


def test_empty(A):
    import torch
    say("mx_linear empty")
    w = A.mx_quantize(torch.zeros((32, 64), dtype=torch.bfloat16, device="cuda"), "fp4")
    c, s = A.mx_quantize(torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda"))
    assert A.mx_linear(c, s, *w, activation="gelu").shape == (0, 32)
    q = A.mx_linear(c, s, *w, fmt="fp4")
    assert q[0].shape == (0, 16) and q[1].shape == (0, 1)
    with pytest.raises(A.AwqError, match="fp32 result"):
        A.mx_linear(*A.mx_quantize(torch.zeros((5, 64), dtype=torch.bfloat16, device="cuda")), *w,
                    out_dtype=torch.float32)


@pytest.mark.parametrize("M,N,K", [(1, 520, 1056), (200, 544, 4096), (1024, 8224, 768)])
def test_captured_and_replayed(A, M, N, K):
    """Plans captured and replayed on new activations; two plans with workspaces of their own on two streams."""
    import torch
    say(f"mx_linear captured {M}x{N}x{K}")
    rng = np.random.default_rng(M)
    a, w = dev_mx(*random_mx(rng, M, K, "fp8"), "fp8"), dev_mx(*random_mx(rng, N, K, "fp4"), "fp4")
    bias, R = torch.ones(N, device="cuda"), torch.ones((M, N), dtype=torch.float16, device="cuda")
    plan = A.MxLinearPlan(*a, *w, bias=bias, activation="gelu", residual=R)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Y = plan.run()
    for i in range(3):
        for t, n in zip(a, random_mx(np.random.default_rng(i), M, K, "fp8")):
            t.view(torch.uint8).copy_(torch.from_numpy(n))
        R.fill_(i)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, A.mx_linear(*a, *w, bias=bias, activation="gelu", residual=R))
    streams = [torch.cuda.Stream() for _ in range(2)]
    plans = [A.MxLinearPlan(*a, *w, bias=bias, activation="gelu", residual=R, stream=s) for s in streams]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [p.run() for p in plans]
    torch.cuda.synchronize()
    assert all(torch.equal(x, Y) for x in got)
