"""RMS norm of rows whose sum of squares leaves fp32's range, next to ordinary rows.

The tolerance is the ordinary one (64 u, tests/test_gpu_mx.py): a row brought to
the middle of the range by a power of two takes the same roundings.
"""
import numpy as np
import pytest

from oracle import awq_oracle as O
from tests._util import say
from tests.test_gpu_mx import U, A, check_near, tdt, to_dev, values  # noqa: F401

pytestmark = pytest.mark.gpu
# one of each split of a row over lanes
COLS = [32, 64, 96, 160, 288, 1024, 2080, 8192, 16416, 40960]


def rows_of(rng, cols, powers):
    x = rng.standard_normal((len(powers), cols))
    return (x / np.abs(x).max(axis=1, keepdims=True) * np.exp2(np.array(powers, float))[:, None]).astype(np.float32)


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("eps", [1e-5, 0.0, 1e-30, 1e-36])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_of_huge_and_tiny_rows(A, cols, eps, residual):
    import torch
    say(f"rms_norm_mx range cols {cols} eps {eps} residual {residual}")
    rng = np.random.default_rng(cols)
    powers = [127, 0, 126, 90, 64, 63, 62, 0, 50, -40, -50, -55, -60, -64, -75, -100, -126, 10, 127, -118]
    if residual:
        powers = [min(p, 125) for p in powers]      # the sum stays finite
    X, x = to_dev(rows_of(rng, cols, powers), "bf16")
    R, r = to_dev(rows_of(rng, cols, powers), "bf16") if residual else (None, None)
    W, w = to_dev(1 + 0.2 * rng.standard_normal((1, cols)), "f32")
    out = A.rms_norm_mx(X, W[0].contiguous(), eps, residual=R)
    h, y = O.rms_norm(x, w[0], float(np.float32(eps)), r)
    big = np.abs(y).max(axis=1) >= 2.0 ** -100      # rows that eps does not drown
    assert big[:9].all() and (eps > 0 or big.all())
    sel = torch.from_numpy(big).cuda()
    check_near([t.view(torch.uint8)[sel].view(t.dtype) for t in out[:2]], "fp8", y[big], 64 * U)
    if residual:
        assert torch.equal(out[2].cpu(), torch.from_numpy(x + r).to(torch.bfloat16))


@pytest.mark.parametrize("cols", COLS)
def test_ordinary_rows_among_others(A, cols):
    """Rows are as they are alone, bit for bit, whatever lies next to them; NaN, infinite and zero rows as ever."""
    import torch
    say(f"rms_norm_mx mixed rows cols {cols}")
    rng = np.random.default_rng(cols + 1)
    powers = [0, 127, 3, -100, 1, 90, -2, 5, 100, 0, 0, 7]
    X, _ = to_dev(rows_of(rng, cols, powers), "bf16")
    X[2, 5], X[6, 7], X[9] = float("nan"), float("inf"), 0
    w = torch.ones(cols, device="cuda")
    got = A.rms_norm_mx(X, w, 1e-30)
    for i in range(len(powers)):
        one = A.rms_norm_mx(X[i:i + 1], w, 1e-30)
        assert all(torch.equal(a.view(torch.uint8), b[i:i + 1].view(torch.uint8)) for a, b in zip(one[:2], got[:2]))
    v = A.mx_dequant(*got[:2])
    assert v[2].isnan().all() and v[6, :32].isnan().all() and not v[6, 32:].any() and not v[9].any()
    assert v[[0, 1, 3, 4, 5, 7, 8, 10, 11]].isfinite().all()
    assert A.mx_dequant(*A.rms_norm_mx(X, w, 0.0)[:2])[9].isnan().all()      # 0 / 0


def test_norm_sum_overflow_by_count_alone(A):
    """Squares that fit one by one and not together, and a mean that fits only without eps."""
    import torch
    say("rms_norm_mx sums past the range")
    for cols, p in ((65536, 60), (4096, 61), (32, 62)):
        X = torch.full((3, cols), 2.0 ** p, dtype=torch.bfloat16, device="cuda")
        v = A.mx_dequant(*A.rms_norm_mx(X, torch.ones(cols, device="cuda"))[:2])
        assert bool((v == 1).all()), (cols, p)
    X = torch.full((1, 64), 1.5 * 2.0 ** 63, dtype=torch.bfloat16, device="cuda")
    h, y = O.rms_norm(X.double().cpu().numpy(), np.ones(64), float(np.float32(3e38)))
    check_near(A.rms_norm_mx(X, torch.ones(64, device="cuda"), 3e38), "fp8", y, 64 * U)
