"""Products grouped by expert that round nowhere but in the result, so that equality is the bar.  Operands as in
tests/test_gpu_mx_exact.py: sums are multiples of 1/8 below 2^17."""
import numpy as np
import pytest

from tests._util import say
from tests.moe_shapes import GROUPED
from tests.test_gpu_mx import A, tdt  # noqa: F401
from tests.test_gpu_mx_exact import operand
from tests.test_gpu_mx_grouped import counts_of

pytestmark = pytest.mark.gpu


def operands(a_rows, E, N, K, fmt, dtype, seed):
    """(codes, scales, fp64 values) of A [a_rows, K] and W [E, N, K], for sums of a spread that dtype shows."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    target, top = {"f16": (400, 15), "bf16": (60, 3), "f32": (1e9, 15)}[dtype]
    a_rms = (top * (top + 1) * (2 * top + 1) / 6 / top) ** 0.5 if fmt == "fp8" else 2.93
    n = max(8, (target / (a_rms * 2.93 * 1.75)) ** 2)
    a, w = operand(g, a_rows, K, fmt, top, min(1.0, n / K)), operand(g, E * N, K, "fp4", 0, 1.0)
    return a, tuple(t.view(E, N, -1) for t in w)


def check(A, room, E, N, K, fmt, dtype, gather, before, behind, ld, how="skewed", seed=0):
    """`room` rows of the result, of which `before` and `behind` belong to no group."""
    import torch
    rng = np.random.default_rng(seed + room + 3 * N + 7 * K + E)
    a_rows = max(1, room // 2) if gather else room
    a, w = operands(a_rows, E, N, K, fmt, dtype, seed + room + K)
    offsets = before + np.concatenate([[0], np.cumsum(counts_of(rng, room - before - behind, E, how))])
    rows = torch.from_numpy(rng.integers(0, a_rows, room).astype(np.int32)).cuda() if gather else None
    buf = torch.full((room * ld + 1,), 7.0, dtype=tdt(dtype), device="cuda")
    out = buf[1:].view(room, ld)[:, :N]
    out[before:room - behind] = float("nan")
    A.mx_matmul_grouped(*a[:2], *w[:2], torch.from_numpy(offsets.astype(np.int32)).cuda(), rows=rows, out=out)
    large = 0.0
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if lo == hi:
            continue
        x = a[2][rows[lo:hi].long()] if gather else a[2][lo:hi]
        wt = w[2][e].t().contiguous()
        step = max(1, (1 << 27) // N)                       # a GiB of exact values at a time
        for m in range(0, hi - lo, step):
            y = x[m:m + step] @ wt
            assert bool((y.abs() < 2.0 ** 17).all())
            same = out[lo + m:min(hi, lo + m + step)] == y.to(tdt(dtype))
            assert bool(same.all()), (e, lo, hi, int((~same).sum()), (~same).nonzero()[:4].tolist())
            large = max(large, float(y.abs().max()))
    assert large > 2
    assert out[:before].eq(7).all() and out[room - behind:].eq(7).all()
    assert buf[0] == 7 and (ld == N or buf[1:].view(room, ld)[:, N:].eq(7).all())


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("M,E,N,K,fmt,form", GROUPED)
def test_every_form(A, M, E, N, K, fmt, form, gather):
    """Every type of result, rows an odd stride apart, before and behind the groups."""
    say(f"mx_matmul_grouped exact {form} {M} rows {E} groups {N}x{K} {fmt} gather {gather}")
    for i, dtype in enumerate(("f16", "bf16") if fmt == "fp8" else ("f16", "bf16", "f32")):
        check(A, M, E, N, K, fmt, dtype, gather, min(5, M // 8), min(37, M // 8), N + 3, seed=i)


@pytest.mark.parametrize("how", ["even", "one"])
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("M,E,N,K", [(4096, 2, 8196, 1184), (4096, 7, 4100, 1184), (2500, 3, 8192, 1024)])
def test_shares_of_the_largest_tiles(A, M, E, N, K, fmt, gather, how):
    say(f"mx_matmul_grouped exact {how} {M} rows {E} groups {N}x{K} {fmt} gather {gather}")
    check(A, M, E, N, K, fmt, "f16", gather, 0, 0, N, how)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("M,E,N,K", [(500, 3, 333, 352), (61, 8, 4100, 2208), (900, 5, 1000, 416), (2000, 6, 2054, 800),
                                     (3000, 3, 8209, 800), (4096, 7, 8196, 1184)])
def test_descending_offsets_that_fit(A, M, E, N, K, fmt):
    """Offsets that descend, with no more tiles than the launch has places for: the rows that one group names are its
    products, the others are left."""
    import torch
    say(f"mx_matmul_grouped exact descending {M} {E} {N} {K} {fmt}")
    a, w = operands(M, E, N, K, fmt, "f16", K + E)
    h = M // 2
    for cuts in ([0, 40, 20] + [20] * E, [M] + [0] * E, [0, M, 0] + [5] * E, [h, M, 0, h] + [h] * E):
        offsets = torch.tensor(cuts[:E + 1], dtype=torch.int32, device="cuda")
        out = torch.full((M, N), 7.0, dtype=torch.float16, device="cuda")
        A.mx_matmul_grouped(*a[:2], *w[:2], offsets, out=out)
        named = np.zeros(M, np.int64)
        for e in range(E):
            named[cuts[e]:cuts[e + 1]] += 1
        for e in range(E):
            lo, hi = cuts[e], min(M, cuts[e + 1])
            if lo >= hi:
                continue
            once = torch.from_numpy(named[lo:hi] == 1).cuda()
            y = (a[2][lo:hi] @ w[2][e].t().contiguous()).half()
            assert torch.equal(out[lo:hi][once], y[once]), (cuts[:5], e)
        left = torch.from_numpy(named == 0).cuda()
        assert out[left].eq(7).all(), cuts[:5]


@pytest.mark.parametrize("M,fmt", [(100, "fp8"), (100, "fp4"), (1300, "fp8"), (1300, "fp4")])
def test_weights_past_4_gib(A, M, fmt):
    """Matrices behind 2^32 bytes of codes, for tiles of 128 and the largest ones."""
    import torch
    say(f"mx_matmul_grouped exact past 4 GiB {M} rows {fmt}")
    E, N, K = 5, 131072, 16384                              # 2^30 bytes a matrix
    codes = torch.zeros((E, N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((E, N, K // 32), 127, dtype=torch.uint8, device="cuda")
    codes[4, 131071] = 0x22                                 # the last output of the last matrix: ones
    codes[4, 70000, -16:] = 0x44                            # twos in a row's last 32 values,
    scales[4, 70000, -1] = 128                              # whose scale is 2
    codes[3, 0] = 0x44
    if fmt == "fp8":
        a = torch.ones((M, K), device="cuda").to(torch.float8_e4m3fn)
    else:
        a = torch.full((M, K // 2), 0x22, dtype=torch.uint8, device="cuda")
    s = torch.full((M, K // 32), 127, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
    off = torch.tensor([0, 0, 0, 1, M // 3, M], dtype=torch.int32, device="cuda")
    for rows in (None, torch.arange(M, dtype=torch.int32, device="cuda")):
        Y = A.mx_matmul_grouped(a, s, codes, scales.view(torch.float8_e8m0fnu), off, rows=rows, out_dtype=torch.bfloat16)
        want = torch.zeros_like(Y)
        want[1:M // 3, 0] = 2.0 * K
        want[M // 3:, 131071] = K
        want[M // 3:, 70000] = 32 * 2 * 2
        assert torch.equal(Y, want)


@pytest.mark.parametrize("M,E,N,K,fmt,dtype", [
    (1_100_000, 3, 17, 32, "fp8", "f16"), (1_100_000, 3, 17, 32, "fp4", "f32"),   # more than 65535 tiles of 16 rows
    (2300, 3, 1_000_003, 32, "fp8", "bf16"),                # more tiles than 2^22 / 31251, and a result of 4.6 GB
])
def test_tiles_past_the_first_launch(A, M, E, N, K, fmt, dtype):
    """More tiles of the few-row kernel than one launch of it holds."""
    say(f"mx_matmul_grouped exact launches {M} rows {E} groups {N}x{K} {fmt}")
    for gather in (True, False):
        check(A, M, E, N, K, fmt, dtype, gather, 5, 37, N, "even" if gather else "skewed")


@pytest.mark.parametrize("how", ["even", "skewed"])
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("M,E,N,K", [(5000, 70, 1030, 544), (9000, 1024, 1030, 544), (20000, 130, 520, 544),
                                     (30000, 70, 1030, 512), (60000, 200, 1030, 544)])
def test_more_groups_than_lanes(A, M, E, N, K, fmt, how):
    """More groups than a wave's lanes hold at once, on the tiles of 32 to 256 rows."""
    say(f"mx_matmul_grouped exact {how} {M} rows {E} groups {N}x{K} {fmt}")
    for gather in (True, False):
        check(A, M, E, N, K, fmt, "f16", gather, 11, 300, N + 1, how)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("M,E,N,K", [(5000, 70, 130, 544), (60000, 200, 1030, 544)])
def test_empty_groups_between_full_ones(A, M, E, N, K, fmt):
    """All rows in the last groups of each 64, and in the last group of all."""
    import torch
    say(f"mx_matmul_grouped exact sparse {M} rows {E} groups {N}x{K} {fmt}")
    a, w = operands(M, E, N, K, fmt, "f16", M)
    for full in ([63], [E - 1], [63, 64, E - 1], [0, E - 1]):
        counts = np.zeros(E, np.int64)
        counts[full] = M // len(full)
        counts[full[-1]] += M - counts.sum()
        cuts = np.concatenate([[0], np.cumsum(counts)])
        Y = A.mx_matmul_grouped(*a[:2], *w[:2], torch.from_numpy(cuts.astype(np.int32)).cuda(), out_dtype=torch.float16)
        for e in full:
            s = slice(int(cuts[e]), int(cuts[e + 1]))
            assert torch.equal(Y[s], (a[2][s] @ w[2][e].t().contiguous()).half()), (full, e)
