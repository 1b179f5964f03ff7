"""The many-row attention over the 4-bit cache (more than 16 rows of a head of 128
and sequence, or 64 of a head of 64) where its own paths can go wrong."""
import numpy as np
import pytest
import torch

from tests import kv4_ref
from tests.gpu_util import bf16_to_dev, dev
from tests.test_kv4_gpu import Step, _no_error, wq  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


def _codes(st, value, b, h, keys, codes):
    """Sets the codes of some of a sequence's keys (or values), leaving their scales."""
    n = st.page * st.D // 2
    for j in keys:
        blk = st.pool[st.table[b, j // st.page], h]
        row = np.zeros(st.D // 8, dtype=np.uint32)
        place = kv4_ref.value_place if value else kv4_ref.key_place
        for d in range(st.D):
            w, nib = place(st.D, d)
            row[w] |= np.uint32(int(codes[d]) + 8) << np.uint32(4 * nib)
        at = value * n + j % st.page * st.D // 2
        blk[at:at + st.D // 2] = row.astype("<u4").view(np.uint8)


def _scales(st, value, b, h, keys, scale):
    n, G = st.page * st.D // 2, st.D // st.group
    for j in keys:
        s = st.pool[st.table[b, j // st.page], h][2 * n + value * st.page * 2 * G:][:st.page * 2 * G]
        s.view("<u2").reshape(st.page, G)[j % st.page] = kv4_ref.bf16(np.float32(scale))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("tokens", [10, 25, 60])       # 40 and 100 rows (one tile), 240 (two)
@pytest.mark.parametrize("per_key", [False, True])     # keys that share their factors, and keys that do not
@pytest.mark.parametrize("column", [5, 40, 70, 100, 127])
def test_a_larger_score_late_in_a_block(wq, D, tokens, per_key, column):  # noqa: F811
    """Keys of equal weight, but one in the third block of 128 that weighs 2^10.8 as much: the reference moves while
    the weights of the block's earlier pieces are on their way, and the other keys together still are a tenth of the
    result.  160 sequences that share their pages, so that a CTA has several of an item's blocks."""
    B = 160
    st = Step(wq, [tokens], [128 * 3 + tokens], D=D, group=D, page=32, Hkv=1, seed=column)
    m = st.kv[0]
    rng = np.random.default_rng(column + tokens)
    half = np.arange(D) % 2 * 2 - 1
    for j in range(m):
        # opposite codes in neighbouring dimensions: nothing of a query that is the same in all dimensions
        _codes(st, 0, 0, 0, [j], np.repeat(rng.integers(-7, 8, size=D // 2), 2) * half)
    _scales(st, 0, 0, 0, range(m), 2.0 ** -6)
    late = 256 + column
    _codes(st, 0, 0, 0, [late], np.ones(D))
    _scales(st, 0, 0, 0, [late], 1.0)
    _scales(st, 1, 0, 0, range(m), 0.25)
    if per_key:  # within a warp's sixteen keys, further apart than 2^12
        _scales(st, 0, 0, 0, [3, 131, 259, 258 + 64], 2.0 ** -20)
    st.upload(wq)
    base = 10.8 * np.log(2) / D ** 0.5
    bits = kv4_ref.bf16(base * np.ones((tokens, 4, D)) + rng.normal(size=(tokens, 4, D)) * 2.0 ** -10)
    Q = kv4_ref.widen(bits).reshape(tokens, 4, D)
    batch = wq.kv4_batch(st.batch.page_table.expand(B, -1).contiguous(),
                         torch.arange(B + 1, dtype=torch.int32, device=dev()) * tokens,
                         torch.full((B,), m, dtype=torch.int32, device=dev()), B * tokens, max_q=tokens)
    queries = bf16_to_dev(bits).view(1, tokens, 4, D).expand(B, -1, -1, -1).reshape(B * tokens, 4, D)
    O = wq.kv4_attention(queries, st.cache, batch)
    assert torch.equal(O, wq.kv4_attention(queries, st.cache, batch))
    got = O.float().cpu().numpy().astype(np.float64).reshape(B, tokens, 4, D)
    K, V = st.keys_values(0, 0)
    pos = np.arange(m - tokens, m)
    for h in range(4):
        ref, A, big = kv4_ref.attention(Q[:, h], K, V, pos, D ** -0.5, 0)
        tol = kv4_ref.many_row_tolerance(ref, A, big, Q[:, h], K, V, pos, D ** -0.5, 0)
        assert (np.abs(got[:, :, h] - ref) <= tol).all(), (h, float((np.abs(got[:, :, h] - ref) / tol).max()))


def test_a_wait_that_runs_out_leaves_the_workspace_fit(wq):  # noqa: F811
    """Items shared by CTAs, a CTA's range ending inside one it has not reached when it gives up; the same workspace
    afterwards, for this kernel and for the few-row one."""
    st = Step(wq, [16, 16, 16], [20000, 20000, 1000], D=128, group=128, page=256, Hkv=4, seed=40)
    one = wq.kv4_batch(st.batch.page_table, torch.arange(4, dtype=torch.int32, device=dev()), st.batch.kv_len, 3, max_q=1)
    ws = wq.kv4_workspace(16, st.cache)
    bits = kv4_ref.bf16(np.random.default_rng(41).normal(size=(st.T, 16, 128)))
    Q = bf16_to_dev(bits).view(st.T, 16, 128)

    def both():
        return (wq.kv4_attention(Q, st.cache, st.batch, workspace=ws),
                wq.kv4_attention(Q[:3], st.cache, one, workspace=ws))

    want = both()
    try:
        wq.wq_debug_set_wait_limit_ns(20_000_000)
        wq.wq_debug_force_timeout(2)
        both()
        torch.cuda.synchronize()
        assert wq.wq_last_device_error() == wq.WQ_ERR_DEVICE_TIMEOUT
    finally:
        wq.wq_debug_force_timeout(0)
        wq.wq_debug_set_wait_limit_ns(0)
        wq.wq_clear_device_error()
    counters = ws[:2048]  # of 608 CTAs
    assert not counters.any()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(want, both()))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("largest", [2.0 ** -7, 1.0, 2.0 ** 14, 2.0 ** 15])
@pytest.mark.parametrize("tokens,kv", [(20, 150), (40, 400)])
def test_queries_with_one_large_dimension(wq, D, largest, tokens, kv):  # noqa: F811
    """A dimension that no key has, 2^8 of the others' size, and scores from those others alone: they count with all
    their bits whatever the size of the largest (a bf16 query is exact, so only the products' sums round)."""
    st = Step(wq, [tokens], [kv], D=D, group=D, page=32, Hkv=1, seed=70)
    for p in range(st.pool.shape[0]):  # key codes of dimension 0: none
        n = st.page * D // 2
        words = st.pool[p, 0][:n].view("<u4").reshape(st.page, D // 8)
        w, nib = kv4_ref.key_place(D, 0)
        words[:, w] = (words[:, w] & ~np.uint32(15 << (4 * nib))) | np.uint32(8 << (4 * nib))
    st.upload(wq)
    Q = np.random.default_rng(71).normal(size=(tokens, 4, D)) * largest * 2.0 ** -8
    Q[:, :, 0] = largest
    bits = kv4_ref.bf16(Q)
    scale = 30 / (largest * 2.0 ** -8 * D ** 0.5 * 1.5)  # scores of some tens
    O = wq.kv4_attention(bf16_to_dev(bits).view(tokens, 4, D), st.cache, st.batch, scale=scale)
    st.check(bits, O, 4, float(np.float32(scale)), many_rows=True)
