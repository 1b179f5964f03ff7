"""The 4-bit cache's scale, max / 7, is computed without a division: it has to be the IEEE quotient."""
import numpy as np
import pytest

from tests.test_kv4_host import wq  # noqa: F401  (fixture)


@pytest.mark.parametrize("exponent", [-100, -1, 0, 1, 2, 99])
def test_every_mantissa_is_rounded_as_the_division_rounds_it(wq, exponent):  # noqa: F811
    """All 2^23 values of a binade (powers of two change nothing between the ends: no product is subnormal there)."""
    bits = np.arange(1 << 23, dtype=np.uint32) | np.uint32((exponent + 127) << 23)
    x = bits.view(np.float32)
    out = np.empty_like(x)
    wq.wq_debug_kv4_seventh(x.ctypes.data, out.ctypes.data, len(x))
    assert np.array_equal(out, x / np.float32(7))
