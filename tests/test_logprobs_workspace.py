"""One workspace for the log probabilities of a batch whose size changes from step to step."""
import numpy as np
import pytest
import torch

from tests.gpu_util import dev


@pytest.fixture(scope="module")
def wq():
    import __graft_entry__
    __graft_entry__.build()
    import w4a16_weight_only_wq_gb300 as m
    return m


def test_a_larger_call_needs_no_less(wq):
    n = wq.wq_logprobs_workspace_bytes
    rows, vocab, ks = (1, 2, 7, 15, 16, 64, 65, 76, 100, 128, 152, 227, 228, 229, 456, 457, 4096, 1 << 30), \
        (1, 1000, 16384, 32767, 32768, 50000, 131071, 248000, 2 ** 31 - 1), (0, 1, 5, 20, 32)
    for V in vocab:
        for k in ks:
            if k <= V:
                sizes = [n(T, V, k) for T in rows]
                assert sizes == sorted(sizes) and sizes[0] > 0
    for T in rows:
        for k in ks:
            sizes = [n(T, V, k) for V in vocab if k <= V]
            assert sizes == sorted(sizes)
        for V in vocab[1:]:
            sizes = [n(T, V, k) for k in ks]
            assert sizes == sorted(sizes)


@pytest.mark.gpu
def test_one_workspace_for_calls_of_any_size(wq):
    """Outputs are filled before each call, so that a row that is not written shows; every result equals a fresh
    workspace's."""
    most, rng = (228, 131071, 20), np.random.default_rng(3)
    x = {t: (torch.randn(most[0], most[1], generator=torch.Generator("cuda").manual_seed(1), device=dev()) * 3).to(t)
         for t in (torch.bfloat16, torch.float32)}
    ws = wq.logprobs_workspace(*most)
    steps = [(100, 131071, 5), (1, 131071, 5), (100, 131071, 5), (16, 131071, 20), (228, 131071, 1), (1, 40000, 20),
             (128, 131071, 5), (16, 131071, 0), (200, 65537, 20), (3, 131071, 20), (65, 131071, 7), (228, 131071, 20)]
    steps += [(int(rng.integers(1, 229)), int(rng.integers(33000, 131072)), int(rng.integers(0, 21))) for _ in range(20)]
    for i, (T, V, k) in enumerate(steps):
        dtype = torch.float32 if i % 3 == 2 else torch.bfloat16
        logits = x[dtype][:T, :V]
        tok = torch.from_numpy(rng.integers(0, V, size=T)).to(dev())
        want = wq.token_logprobs(logits, tok, k=k)
        got = [torch.full_like(w, -77) for w in want]
        assert wq.wq_token_logprobs(logits.data_ptr(), wq.WQ_F32 if dtype is torch.float32 else wq.WQ_BF16, T, V,
                                    logits.stride(0), tok.data_ptr(), None, k, *(g.data_ptr() for g in got),
                                    ws.data_ptr(), ws.nbytes, torch.cuda.current_stream().cuda_stream) == wq.WQ_OK
        assert all(torch.equal(g, w) for g, w in zip(got, want)), (T, V, k, dtype)
    assert not ws[:4 * 228].any()  # the counters
