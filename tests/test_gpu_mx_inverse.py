"""The inverse of the microscaled quantization bit for bit, the signs of its zeros included."""
import numpy as np
import pytest

from oracle import awq_oracle as O
from tests._util import say
from tests.test_gpu_mx import A, dev_mx, tdt  # noqa: F401

pytestmark = pytest.mark.gpu


def bits(t):
    """Bit patterns, every NaN the same."""
    import torch
    v = t.cpu()
    i = v.view(torch.int32 if v.dtype == torch.float32 else torch.int16)
    return torch.where(v.isnan(), torch.full_like(i, -1), i)


def signed_zeros(rng, rows, cols, fmt):
    """Random codes, a quarter of them zeros of both signs."""
    zero = 128 if fmt == "fp8" else 8
    c = rng.integers(0, 2 * zero, (rows, cols))
    c = np.where(rng.random((rows, cols)) < 0.25, rng.integers(0, 2, (rows, cols)) * zero, c).astype(np.uint8)
    return c if fmt == "fp8" else c[:, 0::2] | (c[:, 1::2] << 4)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("rows,cols", [(40, 96), (5, 32), (130, 544)])
def test_dequant_bit_patterns(A, fmt, rows, cols):
    import torch
    say(f"mx_dequant bits {fmt} {rows}x{cols}")
    rng = np.random.default_rng(rows + cols)
    codes, blocks = signed_zeros(rng, rows, cols, fmt), rng.integers(0, 256, (rows, cols // 32)).astype(np.uint8)
    with np.errstate(over="ignore"):
        v = O.mx_values(codes, blocks, fmt).astype(np.float32)
    assert np.signbit(v[v == 0]).any() and not np.signbit(v[v == 0]).all()
    for odt in ("f32", "f16", "bf16"):
        got = A.mx_dequant(*dev_mx(codes, blocks, fmt), out_dtype=tdt(odt))
        assert torch.equal(bits(got), bits(torch.from_numpy(v).to(tdt(odt)))), odt


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("scales", ["usual", "negative", "far"])
@pytest.mark.parametrize("rows,cols", [(40, 96), (5, 32), (130, 544)])
def test_scaled_dequant_bit_patterns(A, fmt, scales, rows, cols):
    """The IEEE quotient: usual scales and block exponents, scales of both signs, and far ones."""
    import torch
    say(f"mx_dequant scaled bits {fmt} {scales} {rows}x{cols}")
    rng = np.random.default_rng(rows + cols)
    codes = signed_zeros(rng, rows, cols, fmt)
    blocks = rng.integers(*((0, 256) if scales == "far" else (100, 150)), (rows, cols // 32)).astype(np.uint8)
    s = np.exp(rng.standard_normal(cols))
    if scales == "negative":
        s *= np.where(rng.random(cols) < 0.5, -1, 1)
    if scales == "far":
        s *= np.exp2(rng.uniform(-120, 120, cols))
    s = s.astype(np.float32)
    with np.errstate(over="ignore"):
        v = O.mx_values(codes, blocks, fmt).astype(np.float32) / s
    assert np.signbit(v[v == 0]).any() and not np.signbit(v[v == 0]).all()
    for odt in ("f32", "f16", "bf16"):
        got = A.mx_dequant(*dev_mx(codes, blocks, fmt), s=torch.from_numpy(s).cuda(), out_dtype=tdt(odt))
        assert torch.equal(bits(got), bits(torch.from_numpy(v).to(tdt(odt)))), odt
