"""The many-row attention over the 4-bit cache (more than 32 rows of a head of 128
and sequence, or 64 of a head of 64) where its own paths can go wrong."""
import numpy as np
import pytest
import torch

from tests import kv4_ref
from tests.gpu_util import bf16_to_dev, dev
from tests.test_kv4_gpu import Step, _attend, _i32, _no_error, _queries, wq  # noqa: F401  (fixtures)

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


MANY = [(64, 96), (128, 20)]  # heads of, and tokens with four grouped heads that take this kernel


@pytest.mark.parametrize("D,n", MANY)
@pytest.mark.parametrize("at", [0, 3, -1])   # the first page, one in the middle of a block, the last
def test_pages_outside_are_reported_and_not_followed(wq, D, n, at):  # noqa: F811
    """The other sequence's rows are what they are without the bad page."""
    st = Step(wq, [n, n], [300, 400], D=D, group=D // 2, page=16, Hkv=1, seed=80)
    bits, O = _attend(wq, st, Hq=4)
    last = -(-st.kv[0] // 16) - 1
    for bad in (-1, st.pool.shape[0], 2 ** 31 - 1, -2 ** 31):
        st.table[0, at if at >= 0 else last] = bad
        st.upload(wq)
        before = st.cache.pool.clone()
        _, O2 = _attend(wq, st, Hq=4)
        torch.cuda.synchronize()
        assert wq.wq_last_device_error() == wq.WQ_ERR_DEVICE_BOUNDS
        wq.wq_clear_device_error()
        assert torch.equal(O[n:], O2[n:]) and torch.equal(before, st.cache.pool)


@pytest.mark.parametrize("D,n", MANY)
def test_lengths_outside_are_clamped_and_reported(wq, D, n):  # noqa: F811
    st = Step(wq, [n, n], [300, 400], D=D, group=D, page=16, Hkv=1, seed=81)
    bits, O = _attend(wq, st, Hq=4)
    Q = bf16_to_dev(bits).view(2 * n, 4, D)
    for cu, kv, untouched in (([0, n, 5 * n], [300, 400], 0), ([0, n, 2 * n], [300, 2 ** 31 - 1], 0),
                              ([0, n, 2 * n], [-5, 400], 1), ([-9, n, 2 * n], [300, 400], 1),
                              ([0, n, 2 * n], [300, 400 + 16 * 16], 0)):
        batch = wq.kv4_batch(st.batch.page_table, _i32(cu), _i32(kv), 2 * n, max_q=n)
        O2 = wq.kv4_attention(Q, st.cache, batch)
        torch.cuda.synchronize()
        assert wq.wq_last_device_error() == wq.WQ_ERR_DEVICE_BOUNDS
        wq.wq_clear_device_error()
        rows = slice(untouched * n, untouched * n + n)
        assert torch.equal(O[rows], O2[rows])


@pytest.mark.parametrize("D,n", MANY)
def test_offsets_past_32_bits(wq, D, n):  # noqa: F811
    """A pool of over 4 GiB whose last pages hold the sequence."""
    block = kv4_ref.block_bytes(256, D, D)
    P = (1 << 32) // (2 * block) + 40
    st = Step(wq, [n], [600], D=D, group=D, page=256, Hkv=2, seed=82, spare=0)
    bits, want = _attend(wq, st, Hq=8)
    pool = torch.zeros((P, 2, block), dtype=torch.uint8, device=dev())
    pool[-3:] = st.cache.pool[torch.tensor(st.table[0], device=dev())]
    st.cache = wq.kv4_cache(P, 2, D, 256, D, pool=pool)
    st.batch = wq.kv4_batch(_i32([[P - 3, P - 2, P - 1]]), _i32([0, n]), _i32([600]), n, max_q=n)
    _, O = _attend(wq, st, Hq=8)
    assert torch.equal(O, want)
    st.check(bits, O, 8, D ** -0.5, many_rows=True)


@pytest.mark.parametrize("D,n", MANY)
def test_strided_rows_and_tokens_of_no_sequence(wq, D, n):  # noqa: F811
    st = Step(wq, [n, n - 3], [150, 160], D=D, group=D, page=16, Hkv=2, seed=83)
    T = st.T + 4
    bits = _queries(st.rng, T, 8, D)
    wide = torch.full((T, 11, 2 * D), 3.0, dtype=torch.bfloat16, device=dev())
    wide[:, 2:10, D:] = bf16_to_dev(bits).view(T, 8, D)
    out = torch.full((8, T, D), 7.0, dtype=torch.bfloat16, device=dev())
    batch = wq.kv4_batch(st.batch.page_table, st.batch.cu_q, st.batch.kv_len, T, max_q=n)
    O = wq.kv4_attention(wide[:, 2:10, D:], st.cache, batch, O=out.transpose(0, 1))
    st.check(bits[:st.T], O[:st.T].contiguous(), 8, D ** -0.5, many_rows=True)
    assert (O[st.T:] == 7).all()


@pytest.mark.parametrize("D,n", MANY)
def test_side_stream_and_graph_with_growing_lengths(wq, D, n):  # noqa: F811
    """Blocks of the same size after ever longer sequences, from one captured graph; the lengths pass a page and a
    block of 128 keys."""
    st = Step(wq, [n, n], [n + 7, 230], D=D, group=D, page=16, Hkv=2, seed=84, spare=40)
    free = sorted(set(range(st.pool.shape[0])) - {int(x) for x in st.table.flatten() if x >= 0})
    table = np.full((2, 40), -1)
    for b in range(2):
        used = -(-st.kv[b] // 16)
        table[b, :used] = st.table[b, :used]
        table[b, used:used + 18] = free[18 * b:18 * b + 18]
    st.table = table
    st.upload(wq)
    rope, ws = wq.rope_table(1000, D), wq.kv4_workspace(8, st.cache)
    qkv = torch.empty((2 * n, 12, D), dtype=torch.bfloat16, device=dev())
    side = torch.cuda.Stream()

    def step(stream=None):
        q = wq.kv4_append(st.cache, st.batch, qkv[:, 8:10], qkv[:, 10:], Q=qkv[:, :8], rope=rope, stream=stream)
        return q, wq.kv4_attention(q, st.cache, st.batch, workspace=ws, stream=stream)

    def new_tokens(seed):
        x = kv4_ref.bf16(np.random.default_rng(seed).normal(size=(2 * n, 12, D)))
        qkv.copy_(bf16_to_dev(x).view_as(qkv))
        torch.cuda.synchronize()

    def verify(q, O):
        torch.cuda.synchronize()
        st.pool = st.cache.pool.cpu().numpy()
        st.check(kv4_ref.bf16(q.float().cpu().numpy()), O, 8, D ** -0.5, many_rows=True)

    new_tokens(1)
    verify(*step(side))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, O = step()
    for i in range(2):
        st.kv = [m + n for m in st.kv]
        st.batch.kv_len.copy_(_i32(st.kv))
        new_tokens(2 + i)
        graph.replay()
        verify(q, O)


@pytest.mark.parametrize("D,n", MANY)
def test_more_sequences_than_threads(wq, D, n):  # noqa: F811
    """700 ragged sequences, some without new tokens, the longest with the block that picks this kernel."""
    rng = np.random.default_rng(85)
    q = rng.integers(0, 3, size=700).tolist()
    kv = [max(int(rng.integers(1, 40)), m) for m in q]
    q[411], kv[411] = n, 2000
    q[699], kv[699] = n // 2, 130
    st = Step(wq, q, kv, D=D, group=32, page=16, Hkv=1, seed=86)
    bits, O = _attend(wq, st, Hq=4)
    st.check(bits, O, 4, D ** -0.5, many_rows=True)
