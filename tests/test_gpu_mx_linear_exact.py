"""Products with an epilogue that round nowhere but in the result, so that equality is the bar, in every form of the
kernels: the largest tiles too, whose persistent blocks read the epilogue's arguments by themselves.

The products are those of tests/test_gpu_mx_exact.py: their sums are multiples of 1/8 below 2^17.  The bias and the
residual are multiples of 1/8 below 16 (7 bits, which fp16 and bf16 hold), and ReLU keeps what it keeps, so every value
on the way is a multiple of 1/8 below 2^18: 21 bits, which fp32 holds."""
import numpy as np
import pytest

from oracle import awq_oracle as O
from tests._util import say
from tests.linear_shapes import QUANTIZED
from tests.mx_shapes import PRODUCTS
from tests.test_gpu_mx import A, tdt  # noqa: F401
from tests.test_gpu_mx_exact import exact_product, operand

pytestmark = pytest.mark.gpu
KINDS = ["f16", "bf16", "f32"]


def eighths(g, dtype, *shape):
    """Random multiples of 1/8 in (-16, 16)."""
    import torch
    return (torch.randint(-127, 128, shape, generator=g, device="cuda").double() / 8).to(tdt(dtype))


def strided(t, ld):
    """`t` in rows `ld` apart, an odd number of elements into its memory, which holds 7 elsewhere: (view, memory)."""
    import torch
    M, N = t.shape
    buf = torch.full((M * ld + 1,), 7.0, dtype=t.dtype, device="cuda")
    view = buf[1:].view(M, ld)[:, :N]
    view.copy_(t)
    return view, buf


def untouched(view, buf, ld):
    M, N = view.shape
    return bool(buf[0] == 7) and bool(buf[1:].view(M, ld)[:, N:].eq(7).all())


def quantize(v, fmt):
    """(codes, scale bytes) of values that fp32 holds: the largest power of two in a block less the format's, elements
    to nearest even, saturated."""
    import torch
    b = v.float().reshape(v.shape[0], -1, 32)
    top = b.abs().amax(2)
    e = torch.where(top == 0, -127, (torch.frexp(top)[1] - 1 - {"fp8": 8, "fp4": 2}[fmt]).clamp(-127, 127))
    x = torch.ldexp(b, -e[..., None]).reshape(v.shape)
    scales = (e + 127).to(torch.uint8)
    if fmt == "fp8":
        return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scales
    m = x.abs()
    c = sum((m > t if i % 2 == 0 else m >= t).int() for i, t in enumerate((.25, .75, 1.25, 1.75, 2.5, 3.5, 5)))
    c += 8 * torch.signbit(x).int()
    return (c[:, 0::2] | c[:, 1::2] << 4).to(torch.uint8), scales


def finish(y, bias, act, residual):
    v = y if bias is None else y + bias.double()
    v = v.clamp(min=0) if act == "relu" else v
    return v if residual is None else v + residual.double()


@pytest.mark.parametrize("M,N,K,fmt,form", PRODUCTS)
def test_every_form(A, M, N, K, fmt, form):
    """With a residual of each type, in place and apart, and without; every type of result and bias."""
    import torch
    say(f"mx_linear exact {form} {M}x{N}x{K} {fmt}")
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    for i, dtype in enumerate(KINDS[:2 if fmt == "fp8" else 3]):
        a, w, y = exact_product(M, N, K, fmt, dtype, M + 3 * N + 7 * K + i)
        bias = eighths(g, KINDS[(i + 1) % 3], N)
        # no residual
        out, buf = strided(torch.full((M, N), float("nan"), dtype=tdt(dtype), device="cuda"), N + 3)
        A.mx_linear(*a, *w, bias=bias, activation="relu", out=out)
        assert torch.equal(out, finish(y, bias, "relu", None).to(tdt(dtype))), dtype
        assert untouched(out, buf, N + 3)
        # the result in the residual's place
        r = eighths(g, dtype, M, N)
        out, buf = strided(r, N + 5)
        A.mx_linear(*a, *w, residual=out, out=out)
        assert torch.equal(out, finish(y, None, None, r).to(tdt(dtype))), dtype
        assert untouched(out, buf, N + 5)
        # a residual of every type, apart
        for kind in KINDS:
            r = eighths(g, kind, M, N)
            R, buf = strided(r, N + 1)
            Y = A.mx_linear(*a, *w, bias=bias, activation="relu", residual=R, out_dtype=tdt(dtype))
            assert torch.equal(Y, finish(y, bias, "relu", r).to(tdt(dtype))), (dtype, kind)
            assert torch.equal(R, r) and untouched(R, buf, N + 1)
        assert bool((y.abs() > 2).any())


def test_the_quantizer_is_the_oracles():
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    v = torch.randint(-2000, 2000, (64, 256), generator=g, device="cuda") / 8
    v[:, 32:64] *= 0
    v[:, 64:96].clamp_(min=0)
    for fmt in ("fp8", "fp4"):
        codes, scales = O.mx_quantize(v.double().cpu().numpy(), fmt)
        got = quantize(v, fmt)
        assert np.array_equal(got[0].cpu().numpy(), codes) and np.array_equal(got[1].cpu().numpy(), scales)


@pytest.mark.parametrize("M,N,K,fmt,form", QUANTIZED)
def test_every_quantized_form(A, M, N, K, fmt, form):
    """Codes and scales, with a residual of each type and without, and nothing behind them."""
    import torch
    say(f"mx_linear exact {form} {M}x{N}x{K} {fmt} quantized")
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    a, w, y = exact_product(M, N, K, fmt, "f16", M + 3 * N + 7 * K)
    bias = eighths(g, "bf16", N)
    for out_fmt, width in (("fp8", N), ("fp4", N // 2)):
        for kind in (None, *KINDS):
            r = None if kind is None else eighths(g, kind, M, N)
            R = None if r is None else strided(r, N + 1)[0]
            c = torch.full((M * width + 64,), 0xA5, dtype=torch.uint8, device="cuda")
            s = torch.full((M * (N // 32) + 64,), 0xA5, dtype=torch.uint8, device="cuda")
            codes, scales = c[:M * width].view(M, width), s[:M * (N // 32)].view(M, N // 32)
            out = (codes.view(torch.float8_e4m3fn) if out_fmt == "fp8" else codes, scales.view(torch.float8_e8m0fnu))
            A.mx_linear(*a, *w, bias=bias, residual=R, fmt=out_fmt, out=out)
            want = quantize(finish(y, bias, None, r), out_fmt)
            assert torch.equal(scales, want[1]) and torch.equal(codes, want[0]), (out_fmt, kind)
            assert c[M * width:].eq(0xA5).all() and s[M * (N // 32):].eq(0xA5).all()


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M,N,K,fmt", [(1024, 16001, 768, "fp8"), (2100, 12250, 1088, "fp8"), (1500, 8209, 1184, "fp4")])
def test_activations_of_the_largest_tiles(A, M, N, K, fmt, act):
    """Each is elementwise, so that the same sums, taken one by one from the exact ones, have the same activation as
    in the form for few tokens: the result of a row is equal to that of the row alone."""
    import torch
    say(f"mx_linear {act} largest {M}x{N}x{K} {fmt}")
    a, w, y = exact_product(M, N, K, fmt, "f16", M + N)
    bias = eighths(torch.Generator(device="cuda").manual_seed(M), "f32", N)
    Y = A.mx_linear(*a, *w, bias=bias, activation=act, out_dtype=torch.bfloat16)
    for m in sorted({0, 1, 31, 32, 255, 256, 257, M // 2, M - 2, M - 1}):
        one = A.mx_linear(a[0][m:m + 1].clone(), a[1][m:m + 1].clone(), *w, bias=bias, activation=act,
                          out_dtype=torch.bfloat16)
        assert torch.equal(Y[m], one[0]), m


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_rows_past_the_first_launch(A, fmt):
    """More rows than a launch of the few-token kernel holds (262140)."""
    import torch
    M, N, K = 600_001, 17, 64
    say(f"mx_linear exact {M}x{N}x{K} {fmt}")
    g = torch.Generator(device="cuda").manual_seed(5)
    a, w, y = exact_product(M, N, K, fmt, "bf16", 5)
    bias, r = eighths(g, "f32", N), eighths(g, "f32", M, N)
    out, buf = strided(torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda"), N + 3)
    R, _ = strided(r, N + 1)
    A.mx_linear(*a, *w, bias=bias, activation="relu", residual=R, out=out)
    assert torch.equal(out, finish(y, bias, "relu", r).bfloat16()) and untouched(out, buf, N + 3)
    N = 96
    a, w, y = exact_product(M, N, K, fmt, "f16", 6)
    bias, r = eighths(g, "f16", N), eighths(g, "f16", M, N)
    R, _ = strided(r, N + 1)
    for out_fmt in ("fp8", "fp4"):
        codes, scales = A.mx_linear(*a, *w, bias=bias, residual=R, fmt=out_fmt)
        want = quantize(finish(y, bias, None, r), out_fmt)
        assert torch.equal(codes.view(torch.uint8), want[0]) and torch.equal(scales.view(torch.uint8), want[1])


@pytest.mark.parametrize("M,N,K,fmt", [(1024, 16032, 768, "fp8"), (1500, 8224, 1184, "fp4"), (200, 2080, 12288, "fp8")])
def test_workspaces_in_graphs_and_on_two_streams(A, M, N, K, fmt):
    """Forms that use their workspace (laid out scales, K ranges): two plans captured and replayed at once on new
    inputs, with eager calls between the replays, then two streams at once."""
    import torch
    say(f"mx_linear exact graphs {M}x{N}x{K} {fmt}")
    g = torch.Generator(device="cuda").manual_seed(K)
    assert A.mx_linear_workspace_bytes(fmt, M, N, K) > 0
    bias = [eighths(g, "f32", N) for _ in range(2)]
    R = [eighths(g, "f16", M, N) for _ in range(2)]
    ops = [exact_product(M, N, K, fmt, "f16", i) for i in (1, 2)]
    a = [tuple(t.clone() for t in o[0]) for o in ops]
    w = [o[1] for o in ops]
    plans = [A.MxLinearPlan(*a[0], *w[0], bias=bias[0], activation="relu", residual=R[0]),
             A.MxLinearPlan(*a[1], *w[1], bias=bias[1], residual=R[1], fmt="fp8")]
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in plans]
    for p, graph in zip(plans, graphs):
        with torch.cuda.graph(graph):
            p.run()
    streams = [torch.cuda.Stream() for _ in graphs]

    def check():
        y = [x[2] @ v for x, v in zip(now, exact)]
        assert torch.equal(plans[0].out, finish(y[0], bias[0], "relu", R[0]).half())
        want = quantize(finish(y[1], bias[1], None, R[1]), "fp8")
        assert all(torch.equal(p.view(torch.uint8), q) for p, q in zip(plans[1].out, want))

    exact = [A.mx_dequant(*v).double().t().contiguous() for v in w]
    for i in range(3):
        now = []
        for j in range(2):
            codes, scales, _ = new = operand(g, M, K, fmt, 15, min(1.0, 60 / K))
            now.append(new)
            a[j][0].view(torch.uint8).copy_(codes.view(torch.uint8))
            a[j][1].view(torch.uint8).copy_(scales.view(torch.uint8))
            R[j].copy_(eighths(g, "f16", M, N))
        for t in (plans[0].out, *plans[1].out):
            t.view(torch.uint8).fill_(0xA5)
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        check()
        A.mx_linear(*a[0], *w[0], bias=bias[0])
    apart = [A.MxLinearPlan(*a[j], *w[j], bias=bias[j], residual=R[j], stream=s) for j, s in enumerate(streams)]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [p.run() for p in apart]
    torch.cuda.synchronize()
    for j in range(2):
        assert torch.equal(got[j], finish(now[j][2] @ exact[j], bias[j], None, R[j]).half())
