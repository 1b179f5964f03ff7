"""The 4-bit cache when a batch's lengths do not fit its buffers."""
import numpy as np
import pytest
import torch

from tests import kv4_ref
from tests.gpu_util import bf16_to_dev, dev
from tests.test_kv4_gpu import Step, _i32, _no_error, wq  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cu,kv,slots", [
    # per token: (sequence, slot), or None where it has none
    ([0, 2, 3], [64, 65], [(0, 62), (0, 63), None]),              # one past the second's table of 64 slots
    ([0, 2, 3], [65, 40], [(0, 63), None, (1, 39)]),              # the second new token alone is past it
    ([0, 2, 3], [2000, 40], [None, None, (1, 39)]),
    ([0, 2, 3], [2 ** 31 - 1, 40], [None, None, (1, 39)]),
    ([0, 2, 3], [-5, 40], [None, None, (1, 39)]),
    ([0, 1, 9], [20, 40], [(0, 19), (1, 32), (1, 33)]),           # cu_q past the tokens: those there keep their slots
    ([0, 1, 60], [20, 40], [(0, 19), None, None]),
    ([0, 1, 2 ** 31 - 1], [20, 40], [(0, 19), None, None]),
    ([-3, 1, 3], [20, 40], [(0, 19), (1, 38), (1, 39)]),          # and before them
    ([-2 ** 31, 1, 3], [20, 40], [(0, 19), (1, 38), (1, 39)]),
])
def test_append_and_read_touch_the_tokens_own_slots_only(wq, cu, kv, slots):  # noqa: F811
    st = Step(wq, [2, 1], [64, 64], D=64, group=32, page=16, Hkv=2, seed=50)
    batch = wq.kv4_batch(st.batch.page_table, _i32(cu), _i32(kv), 3, max_q=2)
    bits = kv4_ref.bf16(st.rng.normal(size=(2, 3, 2, 64)))
    K, V = (bf16_to_dev(b).view(3, 2, 64) for b in bits)
    Q = torch.ones((3, 2, 64), dtype=torch.bfloat16, device=dev())
    rope = wq.rope_table(64, 64)
    Qo = wq.kv4_append(st.cache, batch, K, V, Q=Q, rope=rope)
    torch.cuda.synchronize()
    assert wq.wq_last_device_error() == wq.WQ_ERR_DEVICE_BOUNDS
    wq.wq_clear_device_error()
    want, turn = st.pool.copy(), rope.cpu().numpy()
    for i, place in enumerate(slots):
        assert bool(Qo[i].any()) == (place is not None)
        if place is None:
            continue
        b, slot = place
        k = kv4_ref.rotate(kv4_ref.widen(bits[0, i]).reshape(2, 64), turn[slot], False).astype(np.float32)
        v = kv4_ref.widen(bits[1, i]).reshape(2, 64).astype(np.float32)
        for value, rows in ((0, k), (1, v)):
            codes, scales = kv4_ref.grid(rows, 32)
            for h in range(2):
                kv4_ref.put(want, 16, 64, 32, st.table[b, slot // 16], h, slot % 16, codes[h], scales[h], value)
    assert np.array_equal(st.cache.pool.cpu().numpy(), want)
    for value, got in enumerate(wq.kv4_read(st.cache, batch)):
        got = got.float().cpu().numpy()
        for i, place in enumerate(slots):
            ref = np.zeros((2, 64))
            if place is not None:
                ref = kv4_ref.rows(want[st.table[place[0], place[1] // 16]][None], 16, 64, 32, value)[0, :, place[1] % 16]
            assert np.array_equal(got[i], kv4_ref.widen(kv4_ref.bf16(ref)))
    torch.cuda.synchronize()
    assert wq.wq_last_device_error() == wq.WQ_ERR_DEVICE_BOUNDS
    wq.wq_clear_device_error()


@pytest.mark.parametrize("cu,kv", [
    ([0, 1, 1], [20, -1]),          # sequences without new tokens: a length below zero,
    ([0, 1, 1], [20, 65]),          # one past the table's 64 slots,
    ([0, 1, 0], [20, 30]),          # entries that descend
])
def test_sequences_without_new_tokens_are_checked_too(wq, cu, kv):  # noqa: F811
    st = Step(wq, [1, 0], [64, 64], D=64, group=32, page=16, Hkv=1, seed=51)
    batch = wq.kv4_batch(st.batch.page_table, _i32(cu), _i32(kv), 1, max_q=1)
    x = torch.ones((1, 1, 64), dtype=torch.bfloat16, device=dev())
    for call in (lambda: wq.kv4_append(st.cache, batch, x, x), lambda: wq.kv4_read(st.cache, batch),
                 lambda: wq.kv4_attention(x, st.cache, batch)):
        call()
        torch.cuda.synchronize()
        assert wq.wq_last_device_error() == wq.WQ_ERR_DEVICE_BOUNDS
        wq.wq_clear_device_error()
