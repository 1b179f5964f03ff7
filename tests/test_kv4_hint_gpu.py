"""Which kernel the 4-bit cache's attention takes where the caller does not say how many new tokens a sequence has."""
import numpy as np
import pytest
import torch

from tests import kv4_ref
from tests.gpu_util import bf16_to_dev
from tests.test_kv4_gpu import Step, _no_error, wq  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


def _both(wq, st, Hq, hints):  # noqa: F811
    bits = kv4_ref.bf16(np.random.default_rng(1).normal(size=(st.T, Hq, st.D)))
    Q = bf16_to_dev(bits).view(st.T, Hq, st.D)
    out = []
    for hint in hints:
        batch = wq.kv4_batch(st.batch.page_table, st.batch.cu_q, st.batch.kv_len, st.T, max_q=hint)
        out.append(wq.kv4_attention(Q, st.cache, batch))
    return bits, out


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q,hint", [
    ([1] * 24, 1),            # a decoding step: 4 rows a sequence, 96 in all
    ([3] + [1] * 15, 3),      # one short block among single tokens
    ([40], 40),               # one sequence: all tokens are its own
])
def test_without_a_hint_the_same_kernel_runs(wq, D, q, hint):  # noqa: F811
    """The kernels round weights differently, so equal bits of rows over some hundred keys show which one ran."""
    kv = [n + 37 * i % 300 + 200 for i, n in enumerate(q)]
    st = Step(wq, q, kv, D=D, group=64, page=32, Hkv=2, seed=60)
    bits, (without, with_hint) = _both(wq, st, 8, (0, hint))
    assert torch.equal(without, with_hint)
    st.check(bits, without, 8, D ** -0.5, many_rows=True)


def test_any_hint_is_right(wq):  # noqa: F811
    """Hints below what a sequence has, above what the batch has, and so large that their products would overflow."""
    st = Step(wq, [30, 0, 2], [300, 10, 129], D=128, group=128, page=16, Hkv=1, seed=61)
    hints = (0, 1, 5, 31, 1000, 2 ** 40, 2 ** 62)
    bits, outs = _both(wq, st, 4, hints)
    for O in outs:
        st.check(bits, O, 4, 128 ** -0.5, many_rows=True)
