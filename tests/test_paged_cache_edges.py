"""Paged KV cache: calls at the edges of what is promised, each against the plain
64-bit implementation of test_paged_cache.py or the documented status."""
import copy
import ctypes
import math

import numpy as np
import pytest
import torch

from block_quantized_weight_row_gb300.binding import _CacheStruct
from test_paged_cache import BF16, F16, F32, MANY, Q4, Q8, Batch, bq, gpu  # noqa: F401  (bq: a fixture)


def many_rows(bq, cache, elem, n_seqs, n_q, max_q, max_kv, heads, causal=True, window=0):  # noqa: F811
    """bq_paged_attn_many_rows of a call's arguments."""
    c = _CacheStruct(cache.k_pages.data_ptr(), cache.v_pages.data_ptr(), cache.k_pages.shape[0], cache.page_size,
                     cache.k_pages.shape[1], cache.head_dim, cache.k_type, cache.v_type, cache.k_basis)
    return bq.lib().bq_paged_attn_many_rows(c, elem, n_seqs, n_q, max_q, max_kv, heads, causal, window)


@gpu
def test_many_rows_from_cold_pages_every_time(bq):  # noqa: F811
    """Operand warps that arrive late (pages out of L2 and of the address caches, scattered over gigabytes): the same bits each time."""
    kv = [900, 64, 700, 385, 513, 800, 260, 129]
    b = Batch(bq, [64] * 8, kv, 48, 12, 128, 16, Q4, Q8, BF16, seed=5)  # row tiles enough that no tokens are split
    n_pages = (1 << 32) // (12 * b.pools[0].shape[2])
    pools = [torch.empty(n_pages, 12, p.shape[2], dtype=torch.uint8, device="cuda") for p in b.pools]
    far = torch.arange(b.pools[0].shape[0]) * ((n_pages - 1) // b.pools[0].shape[0])
    for pool, page in zip(pools, b.pools):
        pool[far.cuda()] = torch.from_numpy(page).cuda()
    b.cache = bq.PagedCache(*pools, 16, 128, Q4, Q8, 0)
    table = b.pt.long().cpu()
    used = table < len(far)  # the rest is never to be read
    b.pt = torch.where(used, far[torch.where(used, table, 0)], table).int().cuda()
    b.check()
    first = b.run()
    q, flush = b.q.cuda(), torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for _ in range(50):
        flush.fill_(1)
        for x, y in zip(b.run(q=q), first):
            assert torch.equal(x, y)


@gpu
@pytest.mark.parametrize("scale,peaked", [(0.0, 1.0), (0.0, 1e-13), (-0.0, 1e-25), (1e-30, 1e-10)])
@pytest.mark.parametrize("n,elem,kt", [(1, F32, Q4), (3, F32, Q8), (1, BF16, Q4), (5, BF16, Q8), (90, BF16, Q4)])
def test_scores_of_zero_give_the_mean(bq, n, elem, kt, scale, peaked):  # noqa: F811
    """A scale of 0, and products of scale and q below binary32's range: every token seen weighs the same, masked ones nothing."""
    b = Batch(bq, [n, n], [n + 300, n + 13], 8, 4, 128, 16, kt, Q4, elem, peaked=peaked)
    b.scale = scale
    b.check()


@gpu
@pytest.mark.parametrize("n,D,elem,kt", [(1, 128, BF16, Q4), (3, 64, F32, Q4), (2, 96, F16, Q8), (1, 256, BF16, Q4), (130, 128, BF16, Q4)])
@pytest.mark.parametrize("window", [1, 85, 102])
def test_pages_before_the_window_are_not_needed(bq, n, D, elem, kt, window):  # noqa: F811
    """Pages that lie wholly before what a sequence's first query sees have been given back: entries of no page are no error."""
    kv = [777, 300, 1000, n, 4099, 110]
    b = Batch(bq, [n] * 6, kv, 8, 4, D, 16, kt, Q4, elem)
    for s, length in enumerate(kv):
        b.pt[s, :max(0, length - n - window + 1) // 16] = -1 if s % 2 else 12345678
    b.check(window=window)


@gpu
@pytest.mark.parametrize("bits", [18.0, 26.3, 30.0, 34.0])
def test_fp32_small_weights_beside_dominant_ones(bq, bits):  # noqa: F811
    """Many tokens whose weights are 2^-bits of the largest, in every warp beside one of those, are not lost from an fp32 call.

    16 tokens of V = 0 hold almost all weight; the others have V = 7, so that the output is their share. Each other
    token's weight is off by half a step of binary16's subnormals where the largest V scale (1 here) times the
    row's largest weight is at least 2^12: 2^-37 of that largest weight; by 2^-22 of itself; and by the scores' and sums'
    roundings as derived in test_paged_cache.py.
    """
    n, D, page, B = 2048, 64, 64, 304
    k = np.zeros((n // page, 1, page * 2 * 34), np.uint8)
    v = np.full((n // page, 1, page * 2 * 18), 0xFF, np.uint8)  # codes of 7
    for pool, codes in ((k, 64), (v, 32)):
        pool[:, :, page * codes::2], pool[:, :, page * codes + 1::2] = 0x00, 0x3C  # scales of 1
    for t in range(0, 256, 16):  # in each of the 16-token tiles that the warps start with
        p, i = divmod(t, page)
        k[p, :, i * 64:(i + 1) * 64] = 1
        v[p, :, i * 32:(i + 1) * 32] = 0x88  # codes of 0
    cache = bq.PagedCache(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), page, D, Q8, Q4)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    scale = float(np.float32(bits * math.log(2) / D))
    o = bq.paged_attn(cache, torch.ones(B, 1, D, device="cuda"), torch.arange(B + 1, dtype=torch.int32, device="cuda"), i32([n] * B),
                      i32([list(range(n // page))] * B), scale, max_q_len=1, max_kv_len=n).double().cpu().numpy()
    u16, u32, mag = 2.0**-11, 2.0**-24, scale * D
    w = (n - 16) * math.exp(-mag)
    want = 7 * w / (16 + w)
    ds = (34 + 2 + 4) * 2 * u32 * mag + 3 * u16**2 * mag + 2 * u32 * mag
    rel = 2 * ds + u16**2 + 6 * u32 + (n / 8 + 64) * 2 * u32
    tol = rel * want * 1.01 + 7 * (n - 16) * 2.0**-37 / 16 + u32 * want
    assert np.isfinite(o).all() and np.abs(o - want).max() <= tol, f"{np.abs(o - want).max() / want:.3g} of the output, {tol / want:.3g} allowed"


@pytest.mark.parametrize("name", ["k_type", "v_type", "k_basis"])
@pytest.mark.parametrize("value", [Q4 + (1 << 32), Q8 - (1 << 32), 1 << 31, 1 << 62])
def test_codes_beyond_32_bits_are_refused(bq, name, value):  # noqa: F811
    """No type or basis reaches the library cut to 32 bits, past the check of the pools' sizes (looked at before any tensor)."""
    pool = torch.zeros(2, 1, 16 * 36, dtype=torch.uint8)
    c = bq.PagedCache(pool, pool.clone(), 16, 64, **{name: value})
    x, i = torch.zeros(1, 1, 64), torch.zeros(1, dtype=torch.int32)
    for call in (lambda: bq.paged_kv_write(c, x, x, i.long()), lambda: bq.paged_kv_read(c, i.long()),
                 lambda: bq.paged_attn(c, x, i, i, i[None], 0.1, max_q_len=1, max_kv_len=1)):
        with pytest.raises(ValueError, match=f"{name} must fit 32 bits"):
            call()


@gpu
def test_a_biass_basis_is_taken_as_given(bq):  # noqa: F811
    """Only no basis at all means the cache's: -1 and a code beyond 32 bits are refused."""
    c = bq.PagedCache.empty(2, 16, 1, 64)
    x, slots, bias = torch.zeros(1, 1, 64, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda"), torch.zeros(1, 64, device="cuda")
    bq.paged_kv_write(c, x, x, slots, bias)
    bq.paged_kv_read(c, slots, bias=bias, bias_basis=0)
    for basis, error in ((-1, bq.BQError), (1, bq.BQError), (1 << 32, ValueError)):
        with pytest.raises(error):
            bq.paged_kv_write(c, x, x, slots, bias, basis)
        with pytest.raises(error):
            bq.paged_kv_read(c, slots, bias=bias, bias_basis=basis)


@gpu
def test_attention_leaves_the_callers_workspace_set(bq):  # noqa: F811
    """paged_attn takes a workspace of its own: one that the thread had set for C calls is still set after it, a failed call too."""
    b = Batch(bq, [1], [100], 4, 2, 64, 16, Q4, Q4, F32)
    L = bq.lib()
    mine, size = torch.empty(1 << 20, dtype=torch.uint8, device="cuda"), ctypes.c_size_t()
    try:
        assert L.bq_set_workspace(mine.data_ptr(), 1 << 20) == 0
        b.run()
        assert (L.bq_get_workspace(size), size.value) == (mine.data_ptr(), 1 << 20)
        with pytest.raises(bq.BQError):
            b.run(causal=False, window=3)
        assert (L.bq_get_workspace(None), size.value) == (mine.data_ptr(), 1 << 20)
        L.bq_set_workspace(None, 0)
        b.run()
        assert (L.bq_get_workspace(size), size.value) == (None, 0)
    finally:
        L.bq_set_workspace(None, 0)


def test_workspace_is_read_as_it_was_set(bq):  # noqa: F811
    L, size = bq.lib(), ctypes.c_size_t(7)
    L.bq_set_workspace(None, 0)
    assert (L.bq_get_workspace(size), size.value) == (None, 0)
    try:
        assert L.bq_set_workspace(1 << 40, 4096) == 0
        assert (L.bq_get_workspace(size), size.value) == (1 << 40, 4096) and L.bq_get_workspace(None) == 1 << 40
        assert L.bq_set_workspace((1 << 40) + 8, 4096) != 0  # refused: the one before stays
        assert L.bq_get_workspace(None) == 1 << 40
    finally:
        L.bq_set_workspace(None, 0)


@gpu
def test_device_status_reports_every_kind_of_error(bq):  # noqa: F811
    """A wait that ran out and a wrong page in one batch: both are reported, one call each."""
    b = Batch(bq, [150, 1], [400, 100], 4, 2, 128, 16, Q4, Q4, BF16)
    b.pt[1, 0] = -1
    L = bq.lib()
    try:
        assert L.bq_set_spin_limit(0) == 0
        b.run()
    finally:
        L.bq_set_spin_limit(-1)
    assert [bq.binding.device_status() for _ in range(3)] == [-6, -9, 0]


@gpu
def test_serving_example_runs_both_attention_kernels(bq, monkeypatch):  # noqa: F811
    """Its tolerance and smoke() count on it: some step has a sequence on the many-row kernel beside single tokens."""
    from examples import paged_serving
    attn, steps = paged_serving.bq.paged_attn, []

    def noted(cache, q, q_start, kv_len, page_table, scale, *, max_q_len, max_kv_len):
        many = many_rows(bq, cache, 2, kv_len.numel(), q.shape[0], max_q_len, max_kv_len, q.shape[1])
        rows = q_start.diff().cpu() * (q.shape[1] // cache.k_pages.shape[1])
        steps.append([many > 0 and int(r) > many for r in rows])
        return attn(cache, q, q_start, kv_len, page_table, scale, max_q_len=max_q_len, max_kv_len=max_kv_len)

    monkeypatch.setattr(paged_serving.bq, "paged_attn", noted)
    paged_serving.main(report=lambda line: None)
    assert [False, True] in steps and [False, False] in steps


@gpu
@pytest.mark.parametrize("elem,D,q_len,kv_len,H,NKV,bound,window", [
    (BF16, 128, [33, 8, 1], [200, 900, 777], 8, 8, 4096 * 8, 0),      # 33 rows, one above the limit of bf16
    (BF16, 128, [32, 8, 1], [200, 900, 777], 8, 8, 4096 * 8, 0),      # 32 rows
    (F16, 64, [65, 1], [300, 40], 4, 4, 1 << 15, 0),
    (F16, 64, [64, 1], [300, 40], 4, 4, 1 << 15, 0),
    (BF16, 128, [100], [100], 8, 2, 100, 0),                           # too little work
    (BF16, 128, [300, 260], [900, 300], 32, 8, 900, 130),
    (BF16, 64, [300, 260], [900, 300], 32, 8, 900, 130),
    (F16, 96, [300, 260], [900, 300], 32, 8, 900, 0),                  # no such kernel for 96 and 256 channels, or fp32
    (BF16, 256, [300, 260], [900, 300], 32, 8, 900, 0),
    (F32, 128, [300, 260], [900, 300], 32, 8, 900, 0),
])
def test_calls_take_the_kernel_they_are_said_to(bq, elem, D, q_len, kv_len, H, NKV, bound, window):  # noqa: F811
    """The rule of include/bq.h, what the query says, and what runs: with no polls left the many-row kernel alone reports a wait that ran out."""
    b = Batch(bq, q_len, kv_len, H, NKV, D, 16, Q4, Q4, elem, wide=False)
    b.bound = bound
    limit, seen = 32 if elem == BF16 else 64, min(bound, window + max(q_len)) if window else bound
    work = -(-max(q_len) * (H // NKV) // 16) * len(q_len) * NKV * (seen + 512)
    many = elem != F32 and D in (64, 128) and max(q_len) * (H // NKV) > limit and work >= 250000
    assert many_rows(bq, b.cache, elem, len(q_len), sum(q_len), max(q_len), bound, H, True, window) == (limit if many else 0)
    L = bq.lib()
    try:
        assert L.bq_set_spin_limit(0) == 0
        b.run(window=window)
        assert bq.binding.device_status() == (-6 if many else 0)
    finally:
        L.bq_set_spin_limit(-1)
    b.check(window=window)


def test_the_route_of_a_call_on_the_host(bq):  # noqa: F811
    """The query beside the refusals of the call itself: no kernel for those."""
    ask = bq.lib().bq_paged_attn_many_rows
    c = _CacheStruct(1 << 40, 2 << 40, 100, 16, 8, 128, Q4, Q4, 0)
    assert ask(c, BF16, 1, 2048, 2048, 8192, 32, 1, 0) == 32 and ask(c, F16, 1, 2048, 2048, 8192, 32, 1, 0) == 64
    assert ask(c, F32, 1, 2048, 2048, 8192, 32, 1, 0) == 0
    assert ask(c, BF16, 64, 64, 1, 8192, 32, 1, 0) == 0  # 4 rows each
    assert ask(c, BF16, 1, 2048, 9, 100, 32, 1, 0) == 0  # little work by the bounds
    for bad in ((c, 5, 1, 2048, 2048, 8192, 32, 1, 0), (c, BF16, 1, 2048, 2048, 8192, 33, 1, 0), (c, BF16, 1, -1, 2048, 8192, 32, 1, 0),
                (c, BF16, 1, 2048, 2048, 8192, 32, 0, 5), (None, BF16, 1, 2048, 2048, 8192, 32, 1, 0)):
        assert ask(*bad) == 0


def streaming_reference(b, causal, window):
    """Batch.reference with the streaming kernel's tolerances for any number of rows: a sequence's rows a few at a time, each time over
    the tokens up to the last of them, which leaves what every row sees as it is."""
    c, most = copy.copy(b), max(1, (32 if b.elem == BF16 else 64) * b.NKV // b.H)
    c.q_len, c.kv_len, c.slots = [], [], []
    for n, kv, slots in zip(b.q_len, b.kv_len, b.slots):
        for i in range(0, n, most):
            m = min(most, n - i)
            c.q_len.append(m)
            c.kv_len.append(max(0, kv - n + i + m) if causal else kv)
            c.slots.append(slots[:c.kv_len[-1]])
    return c.reference(causal, window)


@gpu
@pytest.mark.parametrize("case", MANY, ids=str)
def test_many_rows_with_little_work_keep_the_streaming_kernels_accuracy(bq, case):  # noqa: F811
    """k^ and q exact, fp32 sums: calls below the many-row kernel's work are not held to that one's roundings only."""
    *args, causal, window = case
    b = Batch(bq, *args, wide=False)
    if many_rows(bq, b.cache, b.elem, len(b.q_len), b.q.shape[0], max(b.q_len), b.bound, b.H, causal, window):
        b.check(causal, window)  # enough work even so
        return
    o, lse = b.run(causal, window)
    assert bq.binding.device_status() == 0
    b.compare(o, lse, streaming_reference(b, causal, window))
