"""The forms that the products with an epilogue of the GPU tests take: the selection (csrc/mx_tiles.h), which the
linear shares with the plain product, asked for each of their shapes."""
import pytest

from tests.linear_shapes import QUANTIZED
from tests.mx_shapes import FORMS
from tests.test_mx_tiling_cpu import tiling  # noqa: F401


@pytest.mark.parametrize("M,N,K,fmt,form", QUANTIZED)
def test_shape_takes_the_form_it_is_there_for(tiling, M, N, K, fmt, form):  # noqa: F811
    assert N % 32 == 0 and tiling(fmt, M, N, K) == FORMS[form]


def test_every_form_is_there_in_both_formats():
    seen = {(form, fmt) for _, _, _, fmt, form in QUANTIZED}
    assert seen == {(form, fmt) for form in FORMS for fmt in ("fp8", "fp4") if (form, fmt) != ("few 24 x 1", "fp4")}
