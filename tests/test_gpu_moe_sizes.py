"""The operators of a block with experts at the ends of what awq.h allows: the most tokens, blocks of many chunks in
the kernel for many experts, operands and results of more than 4 GiB."""
import numpy as np
import pytest

from tests._util import say
from tests.test_gpu_block_norm import EPS, case
from tests.test_gpu_block_norm import check as check_norm
from tests.test_gpu_moe_route import logits, route
from tests.test_gpu_mx import A  # noqa: F401
from tests.test_gpu_mx_exact import operand
from tests.test_gpu_mx_linear_exact import eighths, finish, quantize

pytestmark = pytest.mark.gpu


def check_route(r, L, top):
    """Against a sort instead of the oracle's loops; shares within the tolerance of tests/test_gpu_moe_route.py for
    logits less than 100 apart."""
    import torch
    v, ids = torch.sort(L.float(), dim=1, descending=True, stable=True)
    v, ids = v[:, :top], ids[:, :top]
    assert torch.equal(r.experts, ids.int())
    p = torch.exp((v - v[:, :1]).double())
    p /= p.sum(1, keepdim=True)
    assert float((v[:, 0] - v[:, -1]).max()) < 100
    assert bool(((r.weights - p).abs() <= 200 * 2.0 ** -24 * p).all())
    order = torch.sort(ids.reshape(-1), stable=True)[1]
    assert torch.equal(r.rows, (order // top).int())
    back = torch.empty_like(order)
    back[order] = torch.arange(order.numel(), device="cuda")
    assert torch.equal(r.places.reshape(-1), back.int())
    assert not r.offsets[0]
    assert torch.equal(r.offsets[1:], torch.bincount(ids.reshape(-1), minlength=L.shape[1]).cumsum(0).int())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,top", [(33000, 300, 8), (40001, 40, 9), (70001, 128, 20), (33001, 1024, 32)])
def test_route_many_chunks_of_many_experts(A, T, E, top, dtype):
    """Blocks of more than 64 tokens in the kernel for many experts or places."""
    say(f"moe_route chunks T {T} E {E} top {top} {dtype}")
    L, _ = logits(6, T, E, dtype)
    check_route(route(A, L, top), L, top)


def test_route_the_most_tokens(A):
    """2^24 tokens, of random logits, and of equal ones, which all go to the first experts."""
    import torch
    T, top = 1 << 24, 2
    say(f"moe_route T {T}")
    g = torch.Generator(device="cuda").manual_seed(1)
    L = torch.randn((T, 24), generator=g, device="cuda").bfloat16()
    check_route(route(A, L, top), L, top)
    L.fill_(3.0)
    r = route(A, L, top)
    t = torch.arange(T, dtype=torch.int32, device="cuda")
    assert torch.equal(r.places, torch.stack([t, t + T], 1)) and torch.equal(r.rows, torch.cat([t, t]))
    assert r.experts[:, 0].eq(0).all() and r.experts[:, 1].eq(1).all() and r.weights.eq(0.5).all()
    assert r.offsets.tolist() == [0, T] + [2 * T] * 23
    with pytest.raises(A.AwqError, match="T 16777217"):
        A.moe_route(torch.zeros((T + 1, 1), device="cuda"), 1)


@pytest.mark.parametrize("E,top", [(16, 3), (270, 10)])
def test_route_rows_past_4_gib(A, E, top):
    import torch
    T, ld = 300_000, 9001                                    # 5.4 GB
    say(f"moe_route strided past 4 GiB E {E} top {top}")
    buf = torch.zeros(T * ld, dtype=torch.bfloat16, device="cuda").view(T, ld)
    L = buf[:, 7:7 + E]
    L.copy_(logits(2, T, E, "bf16")[0])
    check_route(route(A, L, top), L, top)


def test_block_norm_past_4_gib(A):
    """Rows of X behind 2^32 bytes that places name, and rows of the residual and the results behind them."""
    import torch
    rows, cols, top = (1 << 20) + 5, 2080, 3
    say("block_norm_mx past 4 GiB")
    rng = np.random.default_rng(3)
    t, n = case(rng, 5, cols, "bf16", top, "f32", ("f32", "rows"), x_rows=9)
    X = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    R, G = torch.zeros_like(X), torch.zeros((rows, cols), device="cuda")
    X[-9:], R[-5:], G[-5:] = t["X"], t["residual"], t["gate"]
    places = torch.zeros((rows, top), dtype=torch.int32, device="cuda")
    shares = torch.zeros((rows, top), device="cuda")
    places[-5:], shares[-5:] = t["places"] + rows - 9, t["shares"]
    out = A.block_norm_mx(X, R, t["weight"], EPS, t["post_weight"], G, places=places, shares=shares)
    check_norm([o[-5:] for o in out], n, "fp8", "bf16")
    assert not out[2][:-5].any() and not out[0][:-5].view(torch.uint8).any() and not out[1][:-5].view(torch.uint8).any()
    # without places, in place
    t, n = case(rng, 5, cols, "bf16", 0, None, None)
    X.zero_(), R.zero_()
    X[-5:], R[-5:] = t["X"], t["residual"]
    out = A.block_norm_mx(X, R, t["weight"], EPS, residual_out=X)
    check_norm([o[-5:] for o in out], n, "fp8", "bf16")
    assert not X[:-5].any() and not out[0][:-5].view(torch.uint8).any()


@pytest.mark.parametrize("M,N,K,fmt", [(70_000, 65_568, 384, "fp8"), (70_000, 65_568, 384, "fp4"),   # the largest tiles
                                       (70, 33_000_032, 32, "fp8"), (300_000, 15_008, 96, "fp4")])   # few tokens
def test_linear_past_4_gib(A, M, N, K, fmt):
    """Residual, result and codes of more than 4 GiB, on operands whose sums round nowhere."""
    import torch
    say(f"mx_linear past 4 GiB {M}x{N}x{K} {fmt}")
    g = torch.Generator(device="cuda").manual_seed(M)
    a, w = operand(g, M, K, fmt, 15, min(1.0, 300 / K)), operand(g, N, K, "fp4", 0, 1.0)
    wt = w[2].t().contiguous()
    bias, R = eighths(g, "f32", N), torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    step = max(1, (1 << 28) // N)
    for m in range(0, M, step):
        R[m:m + step] = eighths(g, "bf16", min(step, M - m), N)
    Q = A.mx_linear(*a[:2], *w[:2], bias=bias, residual=R, fmt="fp8")
    Y = A.mx_linear(*a[:2], *w[:2], bias=bias, activation="relu", residual=R, out_dtype=torch.float16)
    for m in range(0, M, step):
        s = slice(m, min(M, m + step))
        y = a[2][s] @ wt
        assert torch.equal(Y[s], finish(y, bias, "relu", R[s]).half()), m
        codes, scales = quantize(finish(y, bias, None, R[s]), "fp8")
        assert torch.equal(Q[0][s].view(torch.uint8), codes) and torch.equal(Q[1][s].view(torch.uint8), scales), m
    tail = R[-3:].clone()
    A.mx_linear(*a[:2], *w[:2], residual=R, out=R)            # in place
    assert torch.equal(R[-3:], finish(a[2][-3:] @ wt, None, None, tail).bfloat16())


@pytest.mark.parametrize("M,N,fmt", [(M, N, fmt) for M, N in ((7, 100), (100, 4100), (900, 1000), (1500, 2000),
                                                                  (3000, 4100)) for fmt in ("fp8", "fp4")])
def test_grouped_rows_up_to_2_gib(A, M, N, fmt):
    """Row numbers up to the last row of the largest A that can be read through them; one row more is refused."""
    import torch
    K, E = 4096, 3
    width = K if fmt == "fp8" else K // 2
    a_rows = (1 << 31) // width - 1
    say(f"mx_matmul_grouped rows up to 2 GiB {M} rows {N} {fmt}")
    g = torch.Generator(device="cuda").manual_seed(M)
    last = 50
    a, w = operand(g, last, K, fmt, 15, 300 / K), operand(g, E * N, K, "fp4", 0, 1.0)
    codes = torch.zeros((a_rows + 1, width), dtype=torch.uint8, device="cuda")
    scales = torch.full((a_rows + 1, K // 32), 255, dtype=torch.uint8, device="cuda")      # NaN where no row is named
    codes[a_rows - last:a_rows], scales[a_rows - last:a_rows] = a[0].view(torch.uint8), a[1].view(torch.uint8)
    codes = codes.view(torch.float8_e4m3fn) if fmt == "fp8" else codes
    scales = scales.view(torch.float8_e8m0fnu)
    rng = np.random.default_rng(M)
    at = torch.from_numpy(rng.integers(0, last, M)).cuda()
    at[-1] = last - 1
    rows = (at + a_rows - last).int()
    rows[0] = a_rows                                          # the first that is not there: a row of zeros
    off = torch.tensor([0, M // 3, M // 2, M], dtype=torch.int32, device="cuda")
    W = tuple(t.view(E, N, -1) for t in w)
    Y = A.mx_matmul_grouped(codes[:a_rows], scales[:a_rows], *W[:2], off, rows=rows, out_dtype=torch.float16)
    x = a[2][at]
    x[0] = 0
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        assert torch.equal(Y[lo:hi], (x[lo:hi] @ W[2][e].t().contiguous()).half()), e
    with pytest.raises(A.AwqError, match="2\\^31 bytes"):
        A.mx_matmul_grouped(codes, scales, *W[:2], off, rows=rows)


@pytest.mark.parametrize("M,N,K,fmt", [(1_100_000, 40, 4128, "fp8"), (700_000, 300, 6240, "fp8"),
                                       (700_000, 3300, 6240, "fp4")])
def test_grouped_activations_and_results_past_4_gib(A, M, N, K, fmt):
    """Rows in order behind 2^32 bytes of A and of the result: zeros but for the last rows of each group."""
    import torch
    E = 4
    say(f"mx_matmul_grouped past 4 GiB {M} rows {N}x{K} {fmt}")
    g = torch.Generator(device="cuda").manual_seed(M)
    width = K if fmt == "fp8" else K // 2
    w = operand(g, E * N, K, "fp4", 0, 1.0)
    W = tuple(t.view(E, N, -1) for t in w)
    codes = torch.zeros((M, width), dtype=torch.uint8, device="cuda")
    scales = torch.full((M, K // 32), 127, dtype=torch.uint8, device="cuda")
    cuts = [0, M // 5, M // 5 + 3, M - 100_001, M]
    values = []
    for e in range(E):
        a = operand(g, 3, K, fmt, 15, 300 / K)
        codes[cuts[e + 1] - 3:cuts[e + 1]], scales[cuts[e + 1] - 3:cuts[e + 1]] = a[0].view(torch.uint8), a[1].view(torch.uint8)
        values.append(a[2])
    Y = A.mx_matmul_grouped(codes.view(torch.float8_e4m3fn) if fmt == "fp8" else codes, scales.view(torch.float8_e8m0fnu),
                            *W[:2], torch.tensor(cuts, dtype=torch.int32, device="cuda"), out_dtype=torch.float16)
    for e in range(E):
        rows = slice(cuts[e + 1] - 3, cuts[e + 1])
        assert torch.equal(Y[rows], (values[e] @ W[2][e].t().contiguous()).half()), e
        Y[rows] = 0
    step = (1 << 28) // N
    assert not any(bool(Y[m:m + step].any()) for m in range(0, M, step))
