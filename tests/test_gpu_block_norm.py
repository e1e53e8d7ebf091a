"""The norms after and before a block, with the experts' sum, gate and residual, against the oracle on the GPU.

Tolerances (u = 2^-24), each step's error handed on by the next to first order, 1% added for the rest:
* y: top roundings of partial sums, each at most u sum_j |share x| (no error without places).
* a norm: within 64 u of its value (tests/test_gpu_mx.py), and an error d of its input moves it by
  |w| / rms (d + |x| rms(d) / rms), rms including eps.
* h: gate's product and the fused sum round once each: u |gate z| + u |h|.
* residual_out: half a step of its type from a value within that error (2^-25 more for fp16's subnormals).
"""
import numpy as np
import pytest

from oracle import awq_oracle as O
from tests._util import say
from tests.test_gpu_mx import A, STEP, U, tdt, to_dev, values  # noqa: F401
from tests.test_gpu_mx_linear import check_codes

pytestmark = pytest.mark.gpu
EPS = 1e-5


def rms(v, eps=0.0):
    return np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)


def normed(x, dx, w, eps=EPS):
    """(value, error) of a norm whose input is within dx of x."""
    r = rms(x, eps)
    v = x / r * w
    return v, 1.01 * np.abs(w) / r * (dx + np.abs(x) * rms(dx) / r) + 64 * U * np.abs(v)


def case(rng, rows, cols, dtype, top=0, post=None, gate=None, wdtype="f32", ld=None, offset=0, x_rows=None, lost=False):
    import torch
    k = dict(x_rows=x_rows or (rows * max(1, top)))
    X, x = to_dev(values(rng, k["x_rows"] if top else rows, cols), dtype, ld, offset)
    R, r = to_dev(2 * values(rng, rows, cols), dtype, ld, offset)
    W, w = to_dev(1 + 0.2 * rng.standard_normal((1, cols)), wdtype)
    t, n = {"X": X, "residual": R, "weight": W[0].contiguous()}, {"x": x, "residual": r, "norm": w[0]}
    if post:
        P, p = to_dev(1 + 0.2 * rng.standard_normal((1, cols)), post)
        t["post_weight"], n["post"] = P[0].contiguous(), p[0]
    if gate:
        G, g = to_dev(0.5 * rng.standard_normal((1 if gate[1] == "cols" else rows, cols)), gate[0],
                      ld if gate[1] == "rows" else None)
        t["gate"], n["gate"] = (G[0].contiguous(), g[0]) if gate[1] == "cols" else (G, g)
    if top:
        places = rng.integers(0, k["x_rows"], (rows, top)).astype(np.int32)
        shares = rng.random((rows, top)).astype(np.float32)
        if lost:
            gone = rng.random((rows, top)) < 0.4
            places[gone] = rng.choice([-1, -2 ** 31, k["x_rows"], 2 ** 31 - 1], gone.sum())
            places[0] = -1
        t["places"], t["shares"] = torch.from_numpy(places).cuda(), torch.from_numpy(shares).cuda()
        n["places"], n["shares"] = places, shares
    return t, n


def check(out, n, fmt, dtype, scale=1.0):
    import torch
    torch.cuda.synchronize()
    h, v = O.block_norm(n["x"], n["residual"], n["norm"], EPS, n.get("post"), n.get("gate"), scale, n.get("places"),
                        n.get("shares"))
    if "places" in n:
        ok = (n["places"] >= 0) & (n["places"] < n["x"].shape[0])
        p = np.where(ok, n["places"], 0)
        d = n["places"].shape[1] * U * (np.abs(n["x"][p].astype(np.float64)) * (n["shares"] * ok)[..., None]).sum(1)
        y = (n["x"][p].astype(np.float64) * (n["shares"].astype(np.float64) * ok)[..., None]).sum(1)
    else:
        y, d = n["x"].astype(np.float64), np.zeros(n["x"].shape)
    if "post" in n:
        y, d = normed(y, d, n["post"].astype(np.float64))
    if "gate" in n:
        g = n["gate"].astype(np.float64)
        y, d = g * y, np.abs(g) * d + U * np.abs(g * y)
    dh = d + U * (np.abs(h) + d)
    ro = out[2].double().cpu().numpy()
    assert np.all(np.abs(ro - h) <= dh + STEP[dtype] * (np.abs(h) + dh) + (2.0 ** -25 if dtype == "f16" else 0)), "residual"
    _, dv = normed(h, dh, n["norm"].astype(np.float64))
    check_codes(out[:2], fmt, v, dv)


@pytest.mark.parametrize("rows,cols,dtype,top,post,gate,wdtype,fmt,ld,offset,scale", [
    (1, 32, "f16", 0, None, None, "f16", "fp8", None, 0, 1.0),
    (1, 4096, "bf16", 8, None, None, "bf16", "fp8", None, 0, 1.0),
    (5, 96, "bf16", 0, "f32", None, "f32", "fp8", 99, 1, 1.0),
    (67, 128, "bf16", 3, "bf16", ("f32", "cols"), "bf16", "fp4", None, 0, 0.75),
    (33, 160, "f16", 0, "f16", ("f16", "rows"), "f32", "fp8", 163, 0, -1.5),
    (19, 512, "f16", 5, None, ("bf16", "cols"), "bf16", "fp8", 517, 5, 0.0),
    (9, 1024, "bf16", 4, "f32", ("bf16", "rows"), "bf16", "fp8", None, 0, 1.0),
    (130, 4096, "f16", 0, "bf16", ("f32", "cols"), "f16", "fp4", 4104, 0, 0.5),
    (21, 2080, "bf16", 32, None, None, "f32", "fp8", 2081, 3, 1.0),
    (3, 8192, "f16", 2, "f16", None, "f16", "fp8", None, 0, 1.0),
    (3, 8224, "bf16", 1, "f32", ("f32", "rows"), "bf16", "fp8", None, 0, 1.0),
    (2, 20000, "bf16", 6, "bf16", ("f16", "cols"), "f32", "fp8", 20001, 1, 2.0),
    (2, 65536, "f16", 3, "f32", ("f32", "cols"), "f32", "fp4", None, 0, 1.0),
    (2, 40032, "bf16", 0, None, None, "f32", "fp8", None, 0, 1.0),
    (131, 64, "bf16", 2, "f32", None, "f32", "fp4", 67, 1, 1.0),
    (35, 256, "f16", 0, None, ("f16", "cols"), "bf16", "fp8", None, 0, 1.0),
    (140, 4096, "bf16", 8, "bf16", None, "bf16", "fp8", None, 0, 1.0),
    (139, 2080, "f16", 5, None, ("f32", "rows"), "bf16", "fp4", 2083, 1, 0.5),
    (129, 1056, "bf16", 0, "f16", None, "f32", "fp8", None, 0, 1.0),
    (17, 288, "bf16", 7, "f16", ("f32", "cols"), "f16", "fp8", 291, 1, 1.0),
])
def test_block_norm(A, rows, cols, dtype, top, post, gate, wdtype, fmt, ld, offset, scale):
    import torch
    say(f"block_norm_mx {rows}x{cols} {dtype} top {top} post {post} gate {gate} w {wdtype} {fmt} ld {ld} scale {scale}")
    rng = np.random.default_rng(rows + cols)
    t, n = case(rng, rows, cols, dtype, top, post, gate, wdtype, ld, offset)
    before = {k: v.clone() for k, v in t.items()}
    check(A.block_norm_mx(**t, eps=EPS, residual_scale=scale, fmt=fmt), n, fmt, dtype, scale)
    assert all(torch.equal(t[k], before[k]) for k in t)


@pytest.mark.parametrize("cols", [96, 416, 2080])
def test_places_outside(A, cols):
    """Places outside X add nothing, whatever stands in X; a token without any keeps its scaled residual."""
    import torch
    say(f"block_norm_mx places outside, {cols}")
    rng = np.random.default_rng(cols)
    t, n = case(rng, 40, cols, "bf16", 4, x_rows=50, lost=True)
    out = A.block_norm_mx(**t, eps=EPS)
    check(out, n, "fp8", "bf16")
    assert torch.equal(out[2][0], t["residual"][0])
    # an X without rows
    t["X"] = t["X"][:0]
    out = A.block_norm_mx(**t, eps=EPS, residual_scale=0.5)
    assert torch.equal(out[2], (0.5 * t["residual"].float()).bfloat16())


def test_broadcast_gate_is_the_columns_gate(A):
    import torch
    say("block_norm_mx broadcast gate")
    t, n = case(np.random.default_rng(3), 40, 544, "f16", 0, "f32", ("f32", "cols"))
    a = A.block_norm_mx(**t)
    t["gate"] = t["gate"].expand(40, 544)
    b = A.block_norm_mx(**t)
    t["gate"] = t["gate"].contiguous()
    c = A.block_norm_mx(**t)
    for x in (b, c):
        assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(a, x))


@pytest.mark.parametrize("cols", [160, 4096])
def test_in_place_and_batch_independent(A, cols):
    import torch
    say(f"block_norm_mx in place {cols}")
    t, n = case(np.random.default_rng(5), 37, cols, "bf16", 0, "f32", ("f32", "rows"))
    ref = A.block_norm_mx(**t)

    def same(got, want):
        return all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
    for i in (0, 17, 36):
        one = {k: (v[i:i + 1] if v.dim() == 2 else v) for k, v in t.items()}
        assert same(A.block_norm_mx(**one), [r[i:i + 1] for r in ref])
    for which in ("residual", "X"):
        u = {k: v.clone() for k, v in t.items()}
        assert same(A.block_norm_mx(**u, residual_out=u[which]), ref)
    t, n = case(np.random.default_rng(6), 37, cols, "bf16", 3)
    ref = A.block_norm_mx(**t)
    u = {k: v.clone() for k, v in t.items()}
    assert same(A.block_norm_mx(**u, residual_out=u["residual"]), ref)
    with pytest.raises(A.AwqError, match="other tokens"):
        A.block_norm_mx(**t, residual_out=t["X"][:37])


@pytest.mark.parametrize("cols,top", [(4096, 0), (4096, 5), (2080, 0), (2080, 2), (1056, 3), (544, 6), (8192, 0)])
@pytest.mark.parametrize("size", [1.0, 2.0 ** 70])
def test_many_rows_as_one(A, cols, top, size):
    """More rows than take one chunk a lane: each as by itself, bit for bit, squares beyond fp32's range or not."""
    import torch
    say(f"block_norm_mx many rows {cols} top {top} size {size}")
    t, n = case(np.random.default_rng(8), 150, cols, "bf16", top, "f32", ("f16", "rows"))
    t["X"].mul_(size)
    ref = A.block_norm_mx(**t)
    for i in (0, 77, 149):
        one = {k: v[i:i + 1] if v.dim() == 2 and not (k == "X" and top) else v for k, v in t.items()}
        for a, b in zip(A.block_norm_mx(**one), ref):
            assert torch.equal(a.view(torch.uint8), b[i:i + 1].contiguous().view(torch.uint8))


@pytest.mark.parametrize("cols", [64, 1056])
def test_bad_rows_stay_alone(A, cols):
    """A row with a NaN is NaN, one with an infinity in its block's result too; the others are as without them."""
    import torch
    say(f"block_norm_mx bad rows {cols}")
    t, n = case(np.random.default_rng(7), 6, cols, "f16", 0, "f32")
    ref = A.mx_dequant(*A.block_norm_mx(**t)[:2])
    t["X"][1, 7], t["X"][3, 0], t["residual"][4, 2] = float("nan"), float("inf"), float("nan")
    t["X"][5] = 0
    out = A.block_norm_mx(**t)
    got = A.mx_dequant(*out[:2])
    assert got[1].isnan().all() and got[3].isnan().all() and got[4].isnan().all()
    assert torch.equal(got[[0, 2]], ref[[0, 2]])
    assert torch.equal(out[2][5], t["residual"][5])


@pytest.mark.parametrize("cols", [96, 512, 4096])
@pytest.mark.parametrize("size", [2.0 ** 100, 2.0 ** -80])
def test_rows_whose_squares_leave_the_range(A, cols, size):
    """Both norms keep values whose squares overflow or vanish."""
    import torch
    say(f"block_norm_mx far rows {cols} {size}")
    rng = np.random.default_rng(cols)
    x = (values(rng, 9, cols) * size).astype(np.float32)
    X, xv = to_dev(x, "bf16")
    R, r = to_dev(x[::-1] * 0.5, "bf16")
    w = torch.ones(cols, device="cuda")
    out = A.block_norm_mx(X, R, w, eps=0.0)
    h, v = O.block_norm(xv, r, np.ones(cols), 0.0)
    dh = U * np.abs(h)
    check_codes(out[:2], "fp8", v, normed(h, dh, 1.0, 0.0)[1])
    P, p = to_dev(1 + 0.1 * rng.standard_normal((1, cols)), "f32")
    out = A.block_norm_mx(X, R, w, eps=0.0, post_weight=P[0].contiguous(), residual_scale=0.0)
    h, v = O.block_norm(xv, r, np.ones(cols), 0.0, post=p[0], residual_scale=0.0)
    z, dz = normed(xv.astype(np.float64), np.zeros_like(h), p.astype(np.float64), 0.0)
    check_codes(out[:2], "fp8", v, normed(h, dz + U * np.abs(z), 1.0, 0.0)[1])


def test_empty(A):
    import torch
    say("block_norm_mx empty")
    X = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    c, s, h = A.block_norm_mx(X, X, torch.ones(64, device="cuda"))
    assert c.shape == (0, 64) and s.shape == (0, 2) and h.shape == (0, 64)
