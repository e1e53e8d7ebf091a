"""Routing of tokens to experts against the oracle, on the GPU.

Whole numbers are equal.  Weights (u = 2^-24): the difference d = l - max is rounded (u |d| in the exponential's
argument, which is the exponential's relative error), exp is within 2 u, a sum of up to 1024 of them takes up to 64
additions in a lane and 6 across lanes (70 u, and the terms' own errors), then quotient and scale (2 u): within
(|d| + 100) u of the value, |d| the token's largest among the experts that count, or it vanishes below 2^-126.
"""
import numpy as np
import pytest

from oracle import awq_oracle as O
from tests._util import say
from tests.test_gpu_mx import A, tdt  # noqa: F401

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def route(A, L, top, **kw):
    import torch
    r = A.moe_route(L, top, **kw)
    torch.cuda.synchronize()
    return r


def check(r, l, top, renormalize=True, scale=1.0):
    experts, weights, rows, places, offsets = O.moe_route(l, top, renormalize, scale)
    assert np.array_equal(r.experts.cpu().numpy(), experts)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.places.cpu().numpy(), places)
    assert np.array_equal(r.rows.cpu().numpy(), rows)
    got = r.weights.cpu().numpy().astype(np.float64)
    bad = np.isnan(weights)
    assert np.array_equal(np.isnan(got), bad)
    finite = np.where(np.isfinite(l), l, np.nan).astype(np.float64)
    with np.errstate(all="ignore"):
        d = np.nan_to_num(np.nanmax(finite, axis=1, initial=-np.inf, keepdims=True) -
                          np.nanmin(finite, axis=1, initial=np.inf, keepdims=True), nan=0, neginf=0, posinf=0)
    tol = (np.maximum(d, 0) + 100) * U * np.abs(weights) + 2.0 ** -126
    assert np.all((np.abs(got - weights) <= tol) | bad), float(np.nanmax(np.abs(got - weights) / tol))


def logits(seed, T, E, dtype, spread=2.0):
    import torch
    l = torch.from_numpy((spread * np.random.default_rng(seed).standard_normal((T, E))).astype(np.float32)).to(tdt(dtype))
    return l.cuda(), l.float().numpy()


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("T,E,top", [
    (1, 1, 1), (1, 8, 2), (3, 5, 5), (17, 64, 8), (64, 65, 6), (65, 64, 1), (63, 128, 8), (24, 256, 32), (7, 1024, 32),
    (40, 200, 8), (300, 256, 7), (500, 250, 2), (129, 128, 8), (1000, 10, 3), (257, 600, 16), (70, 1000, 32), (333, 9, 9), (2049, 40, 4),
])
def test_route(A, T, E, top, dtype):
    say(f"moe_route T {T} E {E} top {top} {dtype}")
    L, l = logits(T + E, T, E, dtype)
    check(route(A, L, top), l, top)
    check(route(A, L, top, renormalize=False, scale=2.5), l, top, False, 2.5)


@pytest.mark.parametrize("T,E,top", [(32769, 8, 2), (70001, 16, 4)])
def test_route_more_than_a_chunk_a_block(A, T, E, top):
    """Blocks of more than 64 tokens: checked against a sort instead of the oracle's loops."""
    import torch
    say(f"moe_route large T {T} E {E} top {top}")
    L, _ = logits(5, T, E, "bf16")
    r = route(A, L, top)
    v, ids = torch.sort(L.float(), dim=1, descending=True, stable=True)
    assert torch.equal(r.experts, ids[:, :top].int())
    assert torch.allclose(r.weights, torch.softmax(v[:, :top].double(), 1).float(), rtol=2e-5, atol=0)
    order = torch.sort(ids[:, :top].reshape(-1), stable=True)[1]
    assert torch.equal(r.rows, (order // top).int())
    back = torch.empty_like(order)
    back[order] = torch.arange(order.numel(), device="cuda")
    assert torch.equal(r.places.reshape(-1), back.int())
    assert torch.equal(r.offsets[1:], torch.bincount(ids[:, :top].reshape(-1), minlength=E).cumsum(0).int())


@pytest.mark.parametrize("T", [5, 64, 200])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_ties_masks_and_nan(A, T, dtype):
    """Many equal logits, +0 and -0, experts and whole tokens masked by -inf, +inf and NaN."""
    import torch
    say(f"moe_route ties T {T} {dtype}")
    rng = np.random.default_rng(T)
    E, top = 70, 6
    l = rng.integers(-2, 3, (T, E)).astype(np.float32) * 0.5
    l[l == 0] *= rng.choice([1.0, -1.0], (l == 0).sum())
    l[rng.random((T, E)) < 0.3] = -np.inf
    l[1] = -np.inf                                 # no expert
    l[2] = -np.inf
    l[2, [69, 3]] = [1.0, 1.0]                     # fewer than top
    l[3, 11] = np.nan
    l[4, [60, 5]] = np.inf
    l[0] = torch.finfo(tdt(dtype)).min             # the type's lowest value is not a mask
    L = torch.from_numpy(l).to(tdt(dtype)).cuda()
    check(route(A, L, top), L.float().cpu().numpy(), top)
    check(route(A, L, top, renormalize=False), L.float().cpu().numpy(), top, False)


def test_no_token_has_an_expert(A):
    import torch
    say("moe_route all masked")
    for T in (3, 100):
        r = route(A, torch.full((T, 16), -float("inf"), device="cuda"), 2)
        assert r.experts.eq(-1).all() and r.rows.eq(-1).all() and r.places.eq(-1).all()
        assert not r.offsets.any() and not r.weights.any()
    r = route(A, torch.zeros((0, 16), device="cuda"), 2)
    assert r.offsets.shape == (17,) and not r.offsets.any() and r.experts.shape == (0, 2)


@pytest.mark.parametrize("T", [20, 300])
def test_strided_logits_and_given_outputs(A, T):
    import torch
    say(f"moe_route strided T {T}")
    _, l = logits(9, T, 33, "f16")
    buf = torch.full((T * 41 + 3,), 9.0, dtype=torch.float16, device="cuda")
    L = buf[3:].view(T, 41)[:, :33]
    L.copy_(torch.from_numpy(l).half())
    out = A.MoeRouting(torch.full((T, 4), 77, dtype=torch.int32, device="cuda"), torch.zeros((T, 4), device="cuda"),
                       torch.full((T * 4,), 77, dtype=torch.int32, device="cuda"),
                       torch.full((T, 4), 77, dtype=torch.int32, device="cuda"),
                       torch.full((34,), 77, dtype=torch.int32, device="cuda"))
    r = route(A, L, 4, out=out)
    assert r.rows.data_ptr() == out.rows.data_ptr()
    check(out, l, 4)


@pytest.mark.parametrize("T", [40, 700])
def test_captured_and_replayed(A, T):
    """A plan in a captured graph, replayed on new logits between eager calls."""
    import torch
    say(f"moe_route captured T {T}")
    L, _ = logits(1, T, 48, "bf16")
    plan = A.MoeRoutePlan(L, 4)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = plan.run()
    for i in range(4):
        L.copy_(logits(60 + i, T, 48, "bf16")[0])
        for t in out:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        ref = route(A, L, 4)
        assert all(torch.equal(a, b) for a, b in zip(out, ref)), i


def test_two_streams(A):
    import torch
    say("moe_route two streams")
    Ls = [logits(i, 900, 100, "f32")[0] for i in range(2)]
    ref = [route(A, L, 8) for L in Ls]
    streams = [torch.cuda.Stream() for _ in Ls]
    plans = [A.MoeRoutePlan(L, 8, stream=s) for L, s in zip(Ls, streams)]
    for _ in range(5):
        got = [p.run() for p in plans]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for x, y in zip(got, ref) for a, b in zip(x, y))
