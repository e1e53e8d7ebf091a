"""Prepared calls of the microscaled operators: on the stream that is current when they
run, in captured graphs, and on a stream of their own."""
import numpy as np
import pytest

from tests._util import say
from tests.test_gpu_mx import A, dev_mx, random_mx, to_dev, values  # noqa: F401

pytestmark = pytest.mark.gpu


def plans(A, T, D=4640, N=520):
    """A prepared call of each operator on X (200 rows: the product in K ranges, with a workspace and two launches),
    and a function that computes the same by functional calls."""
    import torch
    rng = np.random.default_rng(T)
    X = torch.zeros((T, D), dtype=torch.bfloat16, device="cuda")
    R = to_dev(values(rng, T, D), "bf16")[0]
    norm = torch.ones(D, device="cuda")
    w = dev_mx(*random_mx(rng, N, D, "fp4"), "fp4")
    p = [A.RmsNormMxPlan(X, norm, residual=R), A.MxQuantPlan(X, "fp4"), A.SiluMulMxPlan(X, R)]
    p += [A.MxDequantPlan(*p[1].out), A.MxMatmulPlan(*p[0].out[:2], *w), A.MxMatmulPlan(*p[1].out, *w)]

    def eager():
        n, q, g = A.rms_norm_mx(X, norm, residual=R), A.mx_quantize(X, "fp4"), A.silu_mul_mx(X, R)
        return [n, q, g, A.mx_dequant(*q), A.mx_matmul(*n[:2], *w), A.mx_matmul(*q, *w)]
    return X, p, eager


def flat(outs):
    for o in outs:
        yield from (o if isinstance(o, tuple) else (o,))


def same(a, b):
    import torch
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
               for x, y in zip(flat(a), flat(b)))


@pytest.mark.parametrize("T", [1, 30, 200])
def test_plans_built_before_the_capture(A, T):
    """Plans built on the ordinary stream, run inside a capture: their launches are the graph's, and every replay
    takes the inputs of that moment."""
    import torch
    say(f"mx plans captured T {T}")
    X, p, eager = plans(A, T)
    assert T < 200 or A.mx_matmul_workspace_bytes("fp8", T, 520, 4640) > 0
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = [q.run() for q in p]
    for i in range(4):
        X.copy_(to_dev(values(np.random.default_rng(70 + i), T, X.shape[1]), "bf16")[0])
        for o in flat(outs):
            o.view(torch.uint8).zero_()
        g.replay()
        torch.cuda.synchronize()
        assert same(outs, eager()), i
        assert any(o.view(torch.uint8).any() for o in flat(outs))


def test_plans_run_on_the_current_stream(A):
    """A plan run under another stream is in that stream's order: behind a long wait and a copy into its input."""
    import torch
    say("mx plans on the current stream")
    X, p, eager = plans(A, 60)
    new = to_dev(values(np.random.default_rng(5), *X.shape), "bf16")[0]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        X.copy_(new)
        outs = [q.run() for q in p]
    s.synchronize()
    assert same(outs, eager())
    # and in the first one's order again
    X.zero_()
    outs = [q.run() for q in p]
    torch.cuda.synchronize()
    assert same(outs, eager())


@pytest.mark.parametrize("which", ["ws", "out"])
def test_plan_keeps_its_memory_for_the_stream_that_used_it(A, which):
    """A plan dropped while another stream still runs it: its memory is not handed out before that stream is done."""
    import torch
    say(f"mx plan dropped while its stream runs, {which}")
    rng = np.random.default_rng(3)
    a, w = dev_mx(*random_mx(rng, 200, 4096, "fp8"), "fp8"), dev_mx(*random_mx(rng, 520, 4096, "fp4"), "fp4")
    plan = A.MxMatmulPlan(*a, *w)
    assert plan.ws.numel() > 256
    plan.run()
    t = getattr(plan, which)
    at, n = t.data_ptr(), t.numel() * t.element_size()
    del t
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(400_000_000)
        plan.run()
    del plan
    assert not s.query(), "the wait was too short"
    q = torch.empty(n, dtype=torch.uint8, device="cuda").data_ptr()
    assert q + n <= at or at + n <= q
    s.synchronize()


def test_plan_with_a_stream_stays_on_it(A):
    """stream= holds whatever is current; captured on that stream, the plan is in the graph."""
    import torch
    say("mx plan with a stream of its own")
    rng = np.random.default_rng(4)
    X = torch.zeros((40, 1024), dtype=torch.float16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    plan = A.MxQuantPlan(X, "fp8", stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = plan.run()
    for i in range(3):
        X.copy_(to_dev(values(rng, 40, 1024), "f16")[0])
        g.replay()
        torch.cuda.synchronize()
        assert same([out], [A.mx_quantize(X, "fp8")])
    X.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        X.copy_(to_dev(values(rng, 40, 1024), "f16")[0])
    plan.run()                                     # the current stream is another one
    s.synchronize()
    assert same([out], [A.mx_quantize(X, "fp8")])
