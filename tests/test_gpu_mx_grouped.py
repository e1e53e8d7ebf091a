"""Products grouped by expert against the oracle, on the GPU: each group's rows are a product of their own, with the
tolerances of the plain product (tests/test_gpu_mx.py)."""
import numpy as np
import pytest

from oracle import awq_oracle as O
from tests._util import say
from tests.moe_shapes import GROUPED
from tests.test_gpu_mx import A, dev_mx, product_tol, random_mx, tdt  # noqa: F401

pytestmark = pytest.mark.gpu


def counts_of(rng, M, E, how):
    """Rows of each group, M in all."""
    if how == "even":
        return np.bincount(np.arange(M) % E, minlength=E)
    if how == "one":                                     # one group has them all
        c = np.zeros(E, np.int64)
        c[rng.integers(E)] = M
        return c
    p = rng.dirichlet(np.full(E, 0.7))                   # "skewed": some have none, some several times the mean
    return np.bincount(rng.choice(E, size=M, p=p), minlength=E)


def weights(rng, E, N, K):
    import torch
    w = [O.mx_quantize(rng.standard_normal((N, K)) / np.sqrt(K), "fp4") for _ in range(E)]
    codes = torch.from_numpy(np.stack([c for c, _ in w])).cuda()
    scales = torch.from_numpy(np.stack([s for _, s in w])).cuda().view(torch.float8_e8m0fnu)
    return (codes, scales), [O.mx_values(*x, "fp4") for x in w]


def check(A, M, E, N, K, fmt, how="skewed", gather=True, dtype=None, behind=0, before=0, ld=None, seed=0):
    import torch
    rng = np.random.default_rng(seed + M + 3 * N + 7 * K + E)
    dtype = dtype or ("f32" if fmt == "fp4" else "bf16")
    counts = counts_of(rng, M, E, how)
    offsets = before + np.concatenate([[0], np.cumsum(counts)])
    room = before + M + behind
    a_rows = max(1, room // 2) if gather else room
    ac, asc = random_mx(rng, a_rows, K, fmt)
    rows = rng.integers(0, a_rows, room) if gather else np.arange(room)
    w, wv = weights(rng, E, N, K)
    buf = torch.full((room * (ld or N) + 1,), 7.0, dtype=tdt(dtype), device="cuda")
    out = buf[1:].view(room, ld or N)[:, :N]
    A.mx_matmul_grouped(*dev_mx(ac, asc, fmt), *w, torch.from_numpy(offsets.astype(np.int32)).cuda(),
                        rows=torch.from_numpy(rows.astype(np.int32)).cuda() if gather else None, out=out)
    torch.cuda.synchronize()
    got = out.double().cpu().numpy()
    a = O.mx_values(ac, asc, fmt)
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        if lo == hi:
            continue
        x = a[rows[lo:hi]]
        y = x @ wv[e].T
        tol = product_tol(x, wv[e], K, fmt, y, dtype)
        err = np.abs(got[lo:hi] - y)
        assert np.all(err <= tol), (e, lo, hi, float((err / tol).max()), np.argwhere(err > tol)[:4].tolist())
    assert np.all(got[:before] == 7) and np.all(got[before + M:] == 7)
    if ld:
        assert buf[0] == 7 and buf[1:].view(room, ld)[:, N:].eq(7).all()


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("M,E,N,K,fmt,form", GROUPED)
def test_every_form(A, M, E, N, K, fmt, form, gather):
    say(f"mx_matmul_grouped {M} rows {E} groups {N}x{K} {fmt} {form} gather {gather}")
    check(A, M, E, N, K, fmt, "skewed", gather)


@pytest.mark.parametrize("how", ["even", "one", "skewed"])
@pytest.mark.parametrize("M,E,N,K,fmt", [(5, 3, 72, 160, "fp8"), (100, 7, 200, 544, "fp4"), (300, 2, 333, 1056, "fp8"),
                                         (700, 5, 520, 416, "fp8"), (1500, 3, 272, 800, "fp4")])
def test_shares(A, M, E, N, K, fmt, how):
    say(f"mx_matmul_grouped {how} {M} rows {E} groups {N}x{K} {fmt}")
    check(A, M, E, N, K, fmt, how, True, "f16", seed=1)
    check(A, M, E, N, K, fmt, how, False, "bf16", behind=37, before=5, ld=N + 3, seed=2)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("K", [32, 64, 96, 128, 288, 384, 416, 640, 2080, 4128])
@pytest.mark.parametrize("M", [1, 40, 400])
def test_lengths(A, M, K, fmt):
    say(f"mx_matmul_grouped lengths {M} rows K {K} {fmt}")
    check(A, M, 4, 49, K, fmt, seed=3)


@pytest.mark.parametrize("M,E,N,K", [(50, 64, 48, 160), (50, 65, 48, 160), (300, 130, 33, 416), (900, 1024, 17, 64),
                                     (2000, 200, 64, 512), (5, 1024, 40, 96), (70, 1, 300, 544), (4000, 129, 256, 768)])
def test_group_counts(A, M, E, N, K):
    """More groups than a wave has lanes, more groups than rows, one group."""
    say(f"mx_matmul_grouped {E} groups {M} rows {N}x{K}")
    check(A, M, E, N, K, "fp8", behind=3, seed=4)


@pytest.mark.parametrize("M,N,K,fmt", [(6, 64, 160, "fp8"), (90, 64, 544, "fp4"), (200, 256, 512, "fp8"),
                                       (1500, 4096, 800, "fp8"), (3000, 4096, 800, "fp4")])
def test_rows_and_offsets_out_of_range(A, M, N, K, fmt):
    """Row numbers outside A stand for rows of zeros, also where A's first row is NaN; offsets are held inside [0, M]."""
    import torch
    say(f"mx_matmul_grouped out of range {M} rows {N}x{K} {fmt}")
    rng = np.random.default_rng(M)
    E, a_rows = 3, 50
    ac, asc = random_mx(rng, a_rows, K, fmt)
    asc[0] = 255
    w, wv = weights(rng, E, N, K)
    rows = rng.integers(1, a_rows, M).astype(np.int32)
    bad = rng.random(M) < 0.3
    rows[bad] = rng.choice([-1, -2 ** 31, a_rows, 2 ** 31 - 1], bad.sum())
    rows[M // 3], bad[M // 3] = 0, False
    a = O.mx_values(ac, asc, fmt)
    x = np.where(bad[:, None], 0.0, a[np.clip(rows, 0, a_rows - 1)])
    offsets = np.array([-5, M // 3, M // 3, 2 ** 31 - 1], np.int32)
    Y = A.mx_matmul_grouped(*dev_mx(ac, asc, fmt), *w, torch.from_numpy(offsets).cuda(),
                            rows=torch.from_numpy(rows).cuda(), out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    got = Y.double().cpu().numpy()
    assert np.isnan(got[M // 3]).all()
    keep = np.arange(M) != M // 3
    for e, lo, hi in ((0, 0, M // 3), (2, M // 3, M)):
        k = keep[lo:hi]
        y = x[lo:hi][k] @ wv[e].T
        assert np.all(np.abs(got[lo:hi][k] - y) <= product_tol(x[lo:hi][k], wv[e], K, fmt, y, "bf16"))
    assert not got[bad].any()


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("M,E,N,K", [(500, 3, 333, 352), (61, 8, 4100, 2208), (900, 5, 1000, 416), (2000, 6, 2054, 800),
                                     (3000, 3, 8209, 800), (4096, 7, 8196, 1184)])
def test_offsets_that_descend(A, M, E, N, K, fmt):
    """Values of rows that several groups name are left or are one group's, with more tiles than there are places for
    and with as many; nothing behind the workspace is written."""
    import torch
    say(f"mx_matmul_grouped descending {M} {E} {N} {K} {fmt}")
    rng = np.random.default_rng(K + E)
    # activations of -1, 0 and 1, scales of 1: the sums are multiples of 1/2 below 2^14 and round nowhere
    if fmt == "fp8":
        ac = torch.from_numpy(rng.integers(-1, 2, (M, K)).astype(np.float32)).cuda().to(torch.float8_e4m3fn)
    else:
        nibble = np.array([0x0, 0x2, 0xA], np.uint8)[rng.integers(0, 3, (2, M, K // 2))]
        ac = torch.from_numpy(nibble[0] | nibble[1] << 4).cuda()
    a = ac, torch.full((M, K // 32), 127, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
    codes = torch.from_numpy(rng.integers(0, 256, (E, N, K // 2)).astype(np.uint8)).cuda()
    scales = torch.full((E, N, K // 32), 127, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
    need = A.mx_matmul_grouped_workspace_bytes(fmt, M, N, K, E)
    ws = torch.full((need + 65536,), 0xA5, dtype=torch.uint8, device="cuda")
    for cuts in ([0, M] * E, [0, 40, 20] + [20] * E, [M] + [0] * E, [0, M, 0] + [5] * E, [M // 2, M, 0, M // 2] + [M // 2] * E):
        offsets = torch.tensor(cuts[:E + 1], dtype=torch.int32, device="cuda")
        out = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
        plan = A.MxMatmulGroupedPlan(*a, codes, scales, offsets, out=out, ws=ws)
        plan.run()
        torch.cuda.synchronize()
        assert plan.ws is ws and ws[need:].eq(0xA5).all()
        left = out.eq(7)
        for e in range(E):
            lo, hi = max(0, cuts[e]), min(M, cuts[e + 1])
            if lo < hi:
                y = A.mx_matmul(a[0][lo:hi], a[1][lo:hi], codes[e], scales[e], out_dtype=torch.bfloat16)
                left[lo:hi] |= out[lo:hi].eq(y)
        assert left.all()


def test_nothing_to_do(A):
    import torch
    say("mx_matmul_grouped empty")
    rng = np.random.default_rng(0)
    w, _ = weights(rng, 3, 40, 64)
    a = dev_mx(*random_mx(rng, 9, 64, "fp8"), "fp8")
    zero = torch.zeros(4, dtype=torch.int32, device="cuda")
    out = torch.full((9, 40), 7.0, dtype=torch.float16, device="cuda")
    A.mx_matmul_grouped(*a, *w, zero, out=out)
    A.mx_matmul_grouped(*a, *w, zero + 9, out=out)
    assert out.eq(7).all()
    rows = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert A.mx_matmul_grouped(*a, *w, zero, rows=rows).shape == (0, 40)
    with pytest.raises(A.AwqError, match="fp32 result"):
        A.mx_matmul_grouped(*a, *w, zero, out_dtype=torch.float32)


def test_one_group_is_the_product(A):
    """With one group the result is within a bf16 step of mx_matmul's: the same products, summed in the same type."""
    import torch
    say("mx_matmul_grouped one group")
    rng = np.random.default_rng(1)
    for M, N, K in ((3, 520, 1184), (300, 520, 1024), (1500, 4128, 1184)):
        a, w = random_mx(rng, M, K, "fp4"), random_mx(rng, N, K, "fp4")
        ad, wd = dev_mx(*a, "fp4"), dev_mx(*w, "fp4")
        off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
        got = A.mx_matmul_grouped(*ad, wd[0][None], wd[1][None], off, out_dtype=torch.float32)
        ref = A.mx_matmul(*ad, *wd, out_dtype=torch.float32)
        B = np.abs(O.mx_values(*a, "fp4")) @ np.abs(O.mx_values(*w, "fp4")).T
        tol = (K // 128 + 16) * 4 * 2.0 ** -24 * B
        assert np.all(np.abs((got.double() - ref.double()).cpu().numpy()) <= tol)


def test_weights_past_4_gib(A):
    """Matrices behind 2^32 bytes of codes."""
    import torch
    say("mx_matmul_grouped past 4 GiB")
    E, N, K = 5, 131072, 16384                      # 2^30 bytes a matrix
    codes = torch.zeros((E, N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((E, N, K // 32), 127, dtype=torch.uint8, device="cuda")
    codes[4, 131071] = 0x22                         # the last output of the last matrix: ones
    codes[3, 0] = 0x44                              # twos
    a = torch.ones((40, K), device="cuda").to(torch.float8_e4m3fn)
    s = torch.full((40, K // 32), 127, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
    off = torch.tensor([0, 0, 0, 1, 3, 40], dtype=torch.int32, device="cuda")
    Y = A.mx_matmul_grouped(a, s, codes, scales.view(torch.float8_e8m0fnu), off, out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    want = torch.zeros_like(Y)
    want[1:3, 0] = 2.0 * K
    want[3:, 131071] = K
    assert torch.equal(Y, want)


@pytest.mark.parametrize("M,N,K", [(30, 96, 544), (300, 520, 1024), (4000, 4128, 1184)])
def test_captured_with_new_offsets(A, M, N, K):
    """The offsets and rows are read in each replay; two graphs with workspaces of their own."""
    import torch
    say(f"mx_matmul_grouped captured {M}x{N}x{K}")
    rng = np.random.default_rng(M)
    E = 6
    a = dev_mx(*random_mx(rng, M, K, "fp8"), "fp8")
    w, _ = weights(rng, E, N, K)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    rows = torch.zeros(M, dtype=torch.int32, device="cuda")
    plans = [A.MxMatmulGroupedPlan(*a, *w, off, rows=rows) for _ in range(2)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for p in plans:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(p.run())
        graphs.append(g)
    for i in range(4):
        c = counts_of(rng, M - i, E, ["even", "skewed", "one", "skewed"][i])
        off.copy_(torch.from_numpy(np.concatenate([[0], np.cumsum(c)]).astype(np.int32)))
        rows.copy_(torch.from_numpy(rng.integers(0, M, M).astype(np.int32)))
        for o in outs:
            o.fill_(-1)
        streams = [torch.cuda.Stream() for _ in graphs]
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        ref = torch.full_like(outs[0], -1)
        A.mx_matmul_grouped(*a, *w, off, rows=rows, out=ref)
        assert all(torch.equal(o, ref) for o in outs), i
        assert ref[M - i:].eq(-1).all()


def test_two_streams(A):
    import torch
    say("mx_matmul_grouped two streams")
    rng = np.random.default_rng(8)
    w, _ = weights(rng, 4, 4128, 1184)
    ops = [dev_mx(*random_mx(rng, 3000, 1184, "fp8"), "fp8") for _ in range(2)]
    off = torch.tensor([0, 100, 1500, 1500, 3000], dtype=torch.int32, device="cuda")
    ref = [A.mx_matmul_grouped(*a, *w, off) for a in ops]
    torch.cuda.synchronize()
    plans = [A.MxMatmulGroupedPlan(*a, *w, off, stream=torch.cuda.Stream()) for a in ops]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [p.run() for p in plans]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
