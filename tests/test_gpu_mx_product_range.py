"""Microscaled products at the ends of what awq.h allows: scales far apart, NaN element codes, operands and results
of more than 4 GiB."""
import numpy as np
import pytest

from oracle import awq_oracle as O
from tests._util import say
from tests.test_gpu_mx import A, check_near, codes_np, dev_mx, product_tol, random_mx, tdt, to_dev, values  # noqa: F401

pytestmark = pytest.mark.gpu
# few tokens (4, 16, 24 or 32 rows), tiles of 64 with three and six slots and in ranges, of 128, the largest
SHAPES = [(3, 65, 544), (16, 65, 544), (20, 65, 544), (40, 65, 544), (100, 333, 544), (65, 48, 2080), (130, 49, 4640),
          (1500, 2051, 544), (1024, 16001, 800)]


def within(Y, y, tol, dtype):
    """Y is y to the tolerance, or infinite of its sign where y to the tolerance reaches past fp16's range: results
    of 65520 and more round to infinity there."""
    Y = Y.double().cpu().numpy()
    past = (np.abs(y) + tol >= 65520) if dtype == "f16" else np.zeros(y.shape, bool)
    with np.errstate(invalid="ignore"):
        near = np.abs(Y - y) <= tol
    return bool(np.all(near | (past & np.isinf(Y) & (np.sign(Y) == np.sign(y)))))


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_scales_of_opposite_ends(A, M, N, K, fmt):
    """2^127 times 2^-127 and the like: the product of the scales is an ordinary one, neither is."""
    import torch
    say(f"mx_matmul opposite scales {M}x{N}x{K} {fmt}")
    rng = np.random.default_rng(M + K)
    (ac, asc), (wc, wsc) = random_mx(rng, M, K, fmt), random_mx(rng, N, K, "fp4")
    ends = rng.integers(0, 4, K // 32)
    far = np.choose(ends, [0, 254, 30, 224])
    asc[:] = np.clip(far + rng.integers(0, 2, asc.shape), 0, 254)
    wsc[:] = 254 - far
    a, w = O.mx_values(ac, asc, fmt), O.mx_values(wc, wsc, "fp4")
    # the terms of a block are of ordinary size: the bound is taken on operands scaled to the middle
    f = np.repeat(np.exp2(far - 127.0), 32)
    a, w = a / f, w * f
    y = a @ w.T
    for dtype in ("f16", "bf16") + (("f32",) if fmt == "fp4" else ()):
        Y = A.mx_matmul(*dev_mx(ac, asc, fmt), *dev_mx(wc, wsc, "fp4"), out_dtype=tdt(dtype))
        assert within(Y, y, product_tol(a, w, K, fmt, y, dtype), dtype), dtype


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_nan_codes_stay_in_their_row(A, M, N, K):
    """An e4m3 NaN makes the results of its row NaN and no others."""
    import torch
    say(f"mx_matmul NaN codes {M}x{N}x{K}")
    rng = np.random.default_rng(M)
    (ac, asc), w = random_mx(rng, M, K, "fp8"), dev_mx(*random_mx(rng, N, K, "fp4"), "fp4")
    ref = A.mx_matmul(*dev_mx(ac, asc, "fp8"), *w)
    rows = {0: 0, M // 2: K - 1, M - 1: K // 2}
    for r, c in rows.items():
        ac[r, c] = 0x7F if r else 0xFF
    Y = A.mx_matmul(*dev_mx(ac, asc, "fp8"), *w)
    keep = [i for i in range(M) if i not in rows]
    assert Y[list(rows)].isnan().all() and torch.equal(Y[keep], ref[keep])
    v = A.mx_dequant(*dev_mx(ac, asc, "fp8"))
    assert int(v.isnan().sum()) == len(rows)


def tail_check(A, M, N, K, fmt, dtype):
    """All zero but the last rows of A and W (and some in the middle): there the oracle's, elsewhere 0."""
    import torch
    rng = np.random.default_rng(K)
    at_m = sorted({0, 1, M // 2, M - 3, M - 1} & set(range(M)))
    at_n = sorted({0, 1, N // 2 + 1, N - 2, N - 1} & set(range(N)))
    width = {"fp8": K, "fp4": K // 2}
    ac = torch.zeros((M, width[fmt]), dtype=torch.uint8, device="cuda")
    wc = torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda")
    asc = torch.full((M, K // 32), 127, dtype=torch.uint8, device="cuda")
    wsc = torch.full((N, K // 32), 127, dtype=torch.uint8, device="cuda")
    ca, sa = random_mx(rng, len(at_m), K, fmt)
    cw, sw = random_mx(rng, len(at_n), K, "fp4")
    for dst, idx, src in ((ac, at_m, ca), (asc, at_m, sa), (wc, at_n, cw), (wsc, at_n, sw)):
        dst[idx] = torch.from_numpy(src).cuda()
    e8 = torch.float8_e8m0fnu
    Y = A.mx_matmul(ac.view(torch.float8_e4m3fn) if fmt == "fp8" else ac, asc.view(e8), wc, wsc.view(e8),
                    out_dtype=tdt(dtype))
    a, w = O.mx_values(ca, sa, fmt), O.mx_values(cw, sw, "fp4")
    y = a @ w.T
    assert within(Y[at_m][:, at_n], y, product_tol(a, w, K, fmt, y, dtype), dtype)
    for m in at_m:
        Y[m, at_n] = 0
    step = max(1, (1 << 28) // N)
    assert not any(bool(Y[i:i + step].any()) for i in range(0, M, step))


@pytest.mark.parametrize("M,N,K,fmt,dtype", [
    (1_100_000, 40, 4128, "fp8", "f16"),          # activations of 4.5 GB
    (2_100_000, 72, 4128, "fp4", "bf16"),         # 4.3 GB in 4 bits
    (3, 2_100_000, 4128, "fp8", "f16"),           # weights of 4.3 GB
    (100, 2_100_000, 4128, "fp4", "f32"),
    (2, 2100, 1 << 22, "fp8", "bf16"),            # the longest rows, 4.4 GB of them: few tokens
    (2, 2100, 1 << 22, "fp4", "f32"),             # and tiles in ranges
    (70_000, 40_003, 384, "fp8", "bf16"),         # a result of 5.6 GB
    (70_000, 40_003, 384, "fp4", "f16"),
    (50_000, 24_001, 160, "fp4", "f32"),          # of 4.8 GB, on the few-token kernel
    (300_000, 15_000, 96, "fp8", "f16"),          # of 9 GB, in more than one launch
])
def test_more_than_4_gib(A, M, N, K, fmt, dtype):
    say(f"mx_matmul past 4 GiB {M}x{N}x{K} {fmt} {dtype}")
    tail_check(A, M, N, K, fmt, dtype)


def test_norm_and_gating_past_4_gib(A):
    """Rows of more than 4 GiB, by length and by stride: their last rows."""
    import torch
    say("rms_norm_mx and silu_mul_mx past 4 GiB")
    rng = np.random.default_rng(2)
    rows, cols = (1 << 20) + 5, 2080
    tail, x = to_dev(values(rng, 5, cols), "bf16")
    X = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    X[-5:] = tail
    w = torch.ones(cols, device="cuda")
    out = A.rms_norm_mx(X, w, residual=X)
    assert torch.equal(out[2][-5:], 2 * tail) and not out[2][:-5].any() and not out[0][:-5].view(torch.uint8).any()
    check_near([t[-5:] for t in out[:2]], "fp8", O.rms_norm(x, np.ones(cols, np.float32), 1e-6, x)[1], 64 * 2.0 ** -24)
    out = A.silu_mul_mx(X, X, "fp4")
    assert not out[0][:-5].any()
    check_near([t[-5:] for t in out], "fp4", O.silu_mul(x, x), 8 * 2.0 ** -24)
    del X, out
    # few columns of very long rows
    ld = 3_000_000
    buf = torch.zeros(999 * ld + 64, dtype=torch.float16, device="cuda")
    V = buf.as_strided((1000, 64), (ld, 1))
    V[-1] = to_dev(values(rng, 1, 64), "f16")[0][0]
    one = V[-1:].clone()
    for whole, alone in ((A.mx_quantize(V), A.mx_quantize(one)), (A.silu_mul_mx(V, V), A.silu_mul_mx(one, one)),
                         (A.rms_norm_mx(V, w[:64].contiguous())[:2], A.rms_norm_mx(one, w[:64].contiguous())[:2])):
        for t, u in zip(whole, alone):
            assert torch.equal(t[-1:].view(torch.uint8), u.view(torch.uint8))
    back = torch.zeros(999 * ld + 64, dtype=torch.float16, device="cuda").as_strided((1000, 64), (ld, 1))
    q = A.mx_quantize(V)
    A.mx_dequant(*q, out=back)
    assert torch.equal(back, A.mx_dequant(*q, out_dtype=torch.float16))


def test_one_plan_in_two_graphs(A):
    """Graphs of one plan share its workspace and result: replayed one after the other, each is right."""
    import torch
    say("mx plan in two graphs")
    rng = np.random.default_rng(6)
    X = torch.zeros((200, 4640), dtype=torch.float16, device="cuda")
    w = dev_mx(*random_mx(rng, 520, 4640, "fp4"), "fp4")
    q = A.MxQuantPlan(X)
    p = A.MxMatmulPlan(*q.out, *w)
    assert A.mx_matmul_workspace_bytes("fp8", 200, 520, 4640) > 0
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            q.run()
            p.run()
    for i in range(4):
        X.copy_(to_dev(values(rng, 200, 4640), "f16")[0])
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(p.out, A.mx_matmul(*A.mx_quantize(X), *w))
