"""SiLU gating where e^-gate passes fp32's range or nearly does, with large and small `up`.

Tolerance (u = 2^-24): below -87 the value is gate up e^gate.  The exponential is
taken as four factors of at most 1 ulp, 2 u, each; six products follow: 14 u, and
the correction of its argument's rounding adds less than u.  d = 16 u.
"""
import numpy as np
import pytest

from oracle import awq_oracle as O
from tests._util import say
from tests.test_gpu_mx import U, A, check_near, quantized, tdt, to_dev  # noqa: F401

pytestmark = pytest.mark.gpu
SMALL = 2.0 ** -118         # the least value whose element is at least a normal one at the smallest block scale


def far(A, dtype, g, up, fmt):
    """One gate a block, at a column of its own; the rest 0."""
    import torch
    n = g.size
    G, Up = np.zeros((n, 32), np.float32), np.ones((n, 32), np.float32)
    at = np.arange(n) % 32
    G[np.arange(n), at], Up[np.arange(n), at] = g, up
    (Gd, gv), (Ud, uv) = to_dev(G, dtype), to_dev(Up, dtype)
    y = O.silu_mul(gv, uv)
    out = A.silu_mul_mx(Gd, Ud, fmt)
    codes, scales = quantized(out)
    got = O.mx_values(codes, scales, fmt)
    big = np.abs(y).max(axis=1) >= SMALL
    # below: elements in steps of the smallest block's, and fp32 subnormals' own step three times over
    step = 2.0 ** -127 * (2.0 ** -9 if fmt == "fp8" else 0.5)
    assert np.all(np.abs(got[~big] - y[~big]) <= step / 2 + 3 * 2.0 ** -149 + np.abs(y[~big]) / 4)
    if not big.any():
        return big
    sel = torch.from_numpy(big).cuda()
    check_near([t.view(torch.uint8)[sel].view(t.dtype) for t in out], fmt, y[big], 16 * U)
    return big


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("dtype,up", [("bf16", 3.3e38), ("bf16", -1e38), ("bf16", 1e30), ("bf16", 1.0),
                                      ("bf16", 1e-30), ("f16", 65504.0), ("f16", -3.0), ("f16", 2.0 ** -14)])
def test_far_gates(A, dtype, up, fmt):
    """Gates from -60 down to -200, with one `up` for all."""
    say(f"silu_mul_mx far gates {dtype} up {up} {fmt}")
    g = -np.concatenate([np.linspace(60, 100, 333), np.linspace(100, 200, 222), [87.0, 87.5, 88.0, 88.5, 89.0]])
    big = far(A, dtype, g, up, fmt)
    if abs(up) > 1e4:
        assert big[g <= -87.5].any()


def test_far_and_near_gates_in_one_block(A):
    """The others of a block are as they are without the far ones."""
    import torch
    say("silu_mul_mx far and near gates")
    rng = np.random.default_rng(1)
    G, Up = 3 * rng.standard_normal((64, 256)), rng.standard_normal((64, 256))
    G[:, 3::32], Up[:, 3::32] = -90, 1e37
    G[::2, 40], G[1::2, 41] = -3e38, 3e38
    Up[1::2, 41] = 1e-38
    (Gd, gv), (Ud, uv) = to_dev(G, "bf16"), to_dev(Up, "bf16")
    check_near(A.silu_mul_mx(Gd, Ud, "fp8"), "fp8", O.silu_mul(gv, uv), 16 * U)


def test_infinite_and_nan_gates(A):
    """-inf / (1 + inf) and NaN are NaN, in their blocks alone."""
    import torch
    say("silu_mul_mx infinite gates")
    for dtype in ("f16", "bf16"):
        G = torch.full((1, 160), -90.0, dtype=tdt(dtype), device="cuda")
        G[0, 3], G[0, 40], G[0, 70] = float("-inf"), float("nan"), float("inf")
        v = A.mx_dequant(*A.silu_mul_mx(G, torch.ones_like(G)))
        assert v[0, :96].isnan().all() and v[0, 96:].isfinite().all()
