"""Microscaled products that have no rounding but the result's, so that equality is the bar.

Activations are small integers, weights any of the sixteen 4-bit codes and block
scales 1/2, 1 or 2.  Within 8 consecutive products the largest is at most
15 x 6 / (1 x 1/2) = 180 < 2^13 times the smallest that is not 0, so that nothing
is dropped where the matrix cores align 8-bit products to the largest.  All sums
are multiples of 1/8 and below 180 x 2 K < 2^23 for K <= 12288: 26 bits at the
very most and, with random signs, under 2^17 x 8 = 2^20 steps, which fp32 holds
exactly in any order.  The sums' spread is set by the number of activations that
are not 0: small enough that a wrong or missing product shows in a 16-bit result.
"""
import pytest

from tests._util import say
from tests.mx_shapes import PRODUCTS, REACHED
from tests.test_gpu_mx import A, tdt  # noqa: F401

pytestmark = pytest.mark.gpu
FP4 = [0, .5, 1, 1.5, 2, 3, 4, 6]


def operand(g, rows, cols, fmt, top, density):
    """(codes, scales, fp64 values) on the device."""
    import torch
    r = lambda *s: torch.rand(s, generator=g, device="cuda")
    scales = torch.randint(126, 129, (rows, cols // 32), generator=g, device="cuda", dtype=torch.uint8)
    if fmt == "fp8":
        v = torch.randint(1, top + 1, (rows, cols), generator=g, device="cuda").float()
        v *= torch.where(r(rows, cols) < 0.5, -1.0, 1.0)
        v *= r(rows, cols) < density
        codes, v = v.to(torch.float8_e4m3fn), v.double()
    else:
        c = torch.randint(0, 16, (rows, cols), generator=g, device="cuda", dtype=torch.uint8)
        if density < 1:
            c = torch.where(r(rows, cols) < density, c, c & 8)
        t = torch.tensor(FP4, device="cuda", dtype=torch.float64)
        v = torch.cat([t, -t])[c.long()]
        codes = c[:, 0::2] | (c[:, 1::2] << 4)
    v *= torch.exp2(scales.double() - 127).repeat_interleave(32, dim=1)
    return codes, scales.view(torch.float8_e8m0fnu), v


def exact_product(M, N, K, fmt, dtype, seed):
    """Operands and the exact product, of a spread that dtype shows."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    target, top = {"f16": (400, 15), "bf16": (60, 3), "f32": (1e9, 15)}[dtype]
    a_rms = (top * (top + 1) * (2 * top + 1) / 6 / top) ** 0.5 if fmt == "fp8" else 2.93
    n = max(8, (target / (a_rms * 2.93 * 1.75)) ** 2)
    a, w = operand(g, M, K, fmt, top, min(1.0, n / K)), operand(g, N, K, "fp4", 0, 1.0)
    y = a[2] @ w[2].t().contiguous()
    assert bool((y.abs() < 2.0 ** 17).all())
    return a[:2], w[:2], y


@pytest.mark.parametrize("M,N,K,fmt,form,dtype", [(*p, dtype) for p in PRODUCTS for dtype in ("f16", "bf16", "f32")
                                                  if (p[3], dtype) != ("fp8", "f32")])     # refused
def test_product_equals_the_exact_one(A, M, N, K, fmt, form, dtype):
    """Every form of the kernels and type of result, rows of the result an odd stride apart, and nothing else
    written."""
    import torch
    say(f"mx_matmul exact {form} {M}x{N}x{K} {fmt} {dtype}")
    a, w, y = exact_product(M, N, K, fmt, dtype, M + 3 * N + 7 * K)
    buf = torch.full((M * (N + 3) + 1,), 7.0, dtype=tdt(dtype), device="cuda")
    out = buf[1:].view(M, N + 3)[:, :N]
    out.fill_(float("nan"))
    Y = A.mx_matmul(*a, *w, out=out)
    same = Y == y.to(tdt(dtype))
    assert bool(same.all()), (int((~same).sum()), (~same).nonzero()[:4].tolist())
    assert buf[0] == 7 and buf[1:].view(M, N + 3)[:, N:].eq(7).all()
    assert bool((Y.abs() > 2).any())


@pytest.mark.parametrize("M,N,K,fmt", [(M, N, K, fmt) for M, N, K, fmt, _ in REACHED])
def test_products_with_workspaces_on_two_streams(A, M, N, K, fmt):
    """Two products at once, each with a workspace of its own that it uses: K ranges or laid out scales."""
    import torch
    say(f"mx_matmul two streams {M}x{N}x{K} {fmt}")
    ops = [exact_product(M, N, K, fmt, "f16", i) for i in (1, 2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ops]
    plans = [A.MxMatmulPlan(*a, *w, stream=s) for (a, w, _), s in zip(ops, streams)]
    need = A.mx_matmul_workspace_bytes(fmt, M, N, K)
    p, q = (plan.ws.data_ptr() for plan in plans)
    assert need > 0 and abs(p - q) >= need
    for _ in range(5):
        got = [plan.run() for plan in plans]
    torch.cuda.synchronize()
    for Y, (_, _, y) in zip(got, ops):
        assert torch.equal(Y, y.half())
