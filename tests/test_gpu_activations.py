"""The activations of the product with an epilogue over fp32 arguments, against fp64: products that are 0, so that the
bias alone goes through them.  The bounds are the documented ones (include/awq.h), down to fp32's smallest normal
number; below it an absolute 2^-126."""
import pytest

from tests._util import say
from tests.test_gpu_mx import A  # noqa: F401

pytestmark = pytest.mark.gpu
BOUND = {"silu": (2.0 ** -17, -95.0), "gelu": (2.0 ** -16, -14.5), "gelu_tanh": (2.0 ** -15, -11.0)}


def exact(x, act):
    import torch
    if act == "silu":
        return x / (1 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * torch.erfc(x * -0.5 ** 0.5)
    return x / (1 + torch.exp(-2 * (2 / torch.pi) ** 0.5 * (x + 0.044715 * x ** 3)))


@pytest.mark.parametrize("act", sorted(BOUND))
@pytest.mark.parametrize("M,K", [(1, 32), (100, 384)])
def test_bound_over_fp32_arguments(A, M, K, act):
    """Random arguments over the range where the result is not rounded away, most of them in its lower part, and of
    every size around 0; the form of one value a lane and the one of eight."""
    import torch
    say(f"mx_linear fp32 arguments through {act}, M {M}")
    N = 1 << 20
    e8 = torch.float8_e8m0fnu
    a = torch.zeros((M, K // 2), dtype=torch.uint8, device="cuda")
    w = torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda")
    one = [torch.full((r, K // 32), 127, dtype=torch.uint8, device="cuda").view(e8) for r in (M, N)]
    g = torch.Generator(device="cuda").manual_seed(M)
    bound, least = BOUND[act]
    for i in range(3):
        u = torch.rand(N, generator=g, device="cuda", dtype=torch.float64)
        v = (least + (20 - least) * u, least * (1 - 0.35 * u),
             (2 * u - 1) * torch.exp2(-60 * torch.rand(N, generator=g, device="cuda", dtype=torch.float64)))[i].float()
        Y = A.mx_linear(a, one[0], w, one[1], bias=v, activation=act, out_dtype=torch.float32)
        assert torch.equal(Y[0], Y[-1])
        y = exact(v.double(), act)
        err = (Y[0].double() - y).abs()
        worst = float((err / (bound * y.abs() + 2.0 ** -126)).max())
        assert worst <= 1, (i, worst)
