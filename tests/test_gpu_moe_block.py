"""A block with experts, its operators one after the other as a program runs them: router, gate/up by expert, gating,
down by expert, the experts' sum with the residual and the next norm; and an attention projection before it."""
import numpy as np
import pytest

from oracle import awq_oracle as O
from tests._util import say
from tests.test_gpu_block_norm import case  # noqa: F401
from tests.test_gpu_mx import A, U, check_near, product_tol, quantized, tdt, to_dev, values  # noqa: F401
from tests.test_gpu_moe_route import check as check_route

pytestmark = pytest.mark.gpu
D, F, E, TOP = 416, 544, 11, 3


def weights(A, T):
    import torch
    rng = np.random.default_rng(T)
    q = lambda n, k: A.mx_quantize(to_dev(rng.standard_normal((n, k)) / np.sqrt(k), "f16")[0], "fp4")  # noqa: E731
    stack = lambda w: (torch.stack([c for c, _ in w]),  # noqa: E731
                       torch.stack([s.view(torch.uint8) for _, s in w]).view(torch.float8_e8m0fnu))
    return {"o": q(D, D), "gu": stack([q(2 * F, D) for _ in range(E)]), "down": stack([q(D, F) for _ in range(E)]),
            "router": torch.from_numpy((rng.standard_normal((D, E)) / 20).astype(np.float32)).cuda(),
            "norm": torch.ones(D, device="cuda"), "post": torch.full((D,), 0.5, device="cuda")}


def block(A, x, h, w, stream=None):
    """x: attention's output, h: the residual stream."""
    a = A.mx_quantize(x, stream=stream)
    h = A.mx_linear(*a, *w["o"], residual=h, out_dtype=x.dtype, stream=stream)
    c, s, _ = A.rms_norm_mx(h, w["norm"], stream=stream)
    logits = h.float() @ w["router"]
    r = A.moe_route(logits, TOP, stream=stream)
    gu = A.mx_matmul_grouped(c, s, *w["gu"], r.offsets, rows=r.rows, out_dtype=x.dtype, stream=stream)
    d = A.silu_mul_mx(gu[:, :F], gu[:, F:], stream=stream)
    y = A.mx_matmul_grouped(*d, *w["down"], r.offsets, out_dtype=x.dtype, stream=stream)
    out = A.block_norm_mx(y, h, w["norm"], post_weight=w["post"], places=r.places, shares=r.weights, stream=stream)
    return out, (a, h, logits, (c, s), r, gu, d, y)


@pytest.mark.parametrize("T", [1, 20, 300])
def test_block(A, T):
    """Each operator against the oracle on the kernels' own inputs."""
    import torch
    say(f"moe block T {T}")
    w = weights(A, T)
    rng = np.random.default_rng(T + 1)
    X, _ = to_dev(values(rng, T, D, 0.5), "bf16")
    H, h0 = to_dev(values(rng, T, D, 0.5), "bf16")
    out, (a, h, logits, n, r, gu, d, y) = block(A, X, H, w)
    torch.cuda.synchronize()
    av, wv = O.mx_values(*quantized(a), "fp8"), O.mx_values(*quantized(w["o"]), "fp4")
    p = av @ wv.T
    tol = product_tol(av, wv, D, "fp8", p + h0, "bf16") + U * np.abs(p + h0)
    assert np.all(np.abs(h.double().cpu().numpy() - (p + h0)) <= tol)
    check_route(r, logits.cpu().numpy(), TOP)
    off, rows = r.offsets.cpu().numpy(), r.rows.cpu().numpy()
    for x, src, ww, k, got in ((n, rows, w["gu"], D, gu), (d, np.arange(T * TOP), w["down"], F, y)):
        xv = O.mx_values(*quantized(x), "fp8")[src]
        for e in range(E):
            s = slice(off[e], off[e + 1])
            if off[e] == off[e + 1]:
                continue
            we = O.mx_values(*quantized((ww[0][e], ww[1][e])), "fp4")
            want = xv[s] @ we.T
            assert np.all(np.abs(got[s].double().cpu().numpy() - want) <= product_tol(xv[s], we, k, "fp8", want, "bf16"))
    g = gu.double().cpu().numpy()
    check_near(d, "fp8", O.silu_mul(g[:, :F], g[:, F:]), 8 * U)
    from tests.test_gpu_block_norm import check as check_norm
    import tests.test_gpu_block_norm as bn
    old, bn.EPS = bn.EPS, 1e-6
    try:
        check_norm(out, {"x": y.float().cpu().numpy(), "residual": h.float().cpu().numpy(), "norm": np.ones(D),
                         "post": np.full(D, 0.5), "places": r.places.cpu().numpy(), "shares": r.weights.cpu().numpy()},
                   "fp8", "bf16")
    finally:
        bn.EPS = old


@pytest.mark.parametrize("T", [1, 20, 300])
def test_block_captured_and_replayed(A, T):
    """The chain in a captured graph, replayed on new inputs (and so new routes) between eager calls; and on a
    stream of its own."""
    import torch
    say(f"moe block captured T {T}")
    w = weights(A, T)
    X, H = (torch.zeros((T, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):                      # the router's library product is set up outside the capture
        block(A, X, H, w)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, _ = block(A, X, H, w)
    for i in range(4):
        rng = np.random.default_rng(90 + i)
        X.copy_(to_dev(values(rng, T, D, 0.5), "bf16")[0])
        H.copy_(to_dev(values(rng, T, D, 0.5), "bf16")[0])
        for o in out:
            o.view(torch.uint8).zero_()
        g.replay()
        torch.cuda.synchronize()
        ref, _ = block(A, X, H, w)
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(out, ref)), i
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, _ = block(A, X, H, w, stream=s)
    s.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, ref))
