"""The scale of the 4-bit cache's attention, on the host."""
import pytest

from tests.test_kv4_host import A, _batch, _cache, _rows, wq  # noqa: F401  (fixture)


@pytest.mark.parametrize("scale,status", [(2.1e38, "WQ_ERR_SHAPE"), (3e38, "WQ_ERR_SHAPE"), (float("inf"), "WQ_ERR_SHAPE"),
                                          (0.0, "WQ_ERR_SHAPE"), (2e38, "WQ_OK"), (1e-38, "WQ_OK")])
def test_scales_whose_base_2_form_overflows_are_refused(wq, scale, status):  # noqa: F811
    """scale * log2(e) above fp32's range would make even a zero query's scores NaN."""
    got = wq.wq_kv4_attention(_cache(wq), _batch(wq, T=0), _rows(wq), _rows(wq), 4, scale, 0, A, 1 << 30, 0)
    assert got == getattr(wq, status)
