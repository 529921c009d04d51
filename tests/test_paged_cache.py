"""Paged KV cache: the quantizing write and the read, bit for bit against the
CPU oracle's blocks; attention against a plain 64-bit implementation; refusals
on the host. The plain implementations here share no code with the kernels:
pages are taken apart byte by byte from the layout in include/bq.h.

Attention tolerances, per output element, from the roundings that the operator
states. With u32 = 2^-24 and half a binary16 step u16 = 2^-11 (relative):
  scores: q enters in two binary16 terms (fp32 calls: u16^2 of its own and of
    the row's largest value) or exactly; a block's products are summed in fp32,
    34 terms of |q| u d with u <= 16 (4-bit codes carry their offset of 8) or
    |q c| d, then the blocks: ds = (34 + blocks + 4) * 2 u32 * max_j mag_j (2:
    an adder that truncates), mag_j = scale * sum_c |q_c| * (16 d or |k^|),
    plus the terms' part and 2 u32 of the score itself;
  weights: one term u16 (16-bit calls) or two (fp32: u16^2), the exponential
    and the scales' products 6 u32;
  weights below 2^-24 of their warp's common power of two, which is at least
    2^-6 of the largest V scale, round to a multiple of it or to nothing: sum_j
    min(w_j d_j, 2^-30 max d) |c_j| (binary32 weights vanish too, at 2^-149);
  sums: a warp's chain of products, then warps and pieces: (keys / 8 + 64) * 2 u32;
so |o - o_ref| <= (2 ds + all of those) * sum_j w_j |v^_j| + the output type's
half step of |o_ref|. The many-row kernel (16-bit calls with 64 or 128 channels,
sequences of more than 64 query rows per kv head, in bf16 32, and work enough) rounds k^, v^ and q to binary16 too:
u16 * mag in the scores for each (|k^| for 16 d), u16 in the sum, operands
below 2^-25 of their unit 2^-30 max d; its products chain over all channels
(D + 8 for 34 + blocks + 4) and its sums over all keys (keys for keys / 8).
"""
import ctypes
import itertools
import math

import numpy as np
import pytest
import torch

Q4, Q8 = 2, 8
OK, INVALID, SHAPE, UNSUPPORTED, ALIGN, WORKSPACE, BASIS, INDEX = 0, -1, -2, -3, -4, -7, -8, -9
F32, F16, BF16 = 0, 1, 2
FAKE = 0x7f0000000000
CODES = {Q4: 16, Q8: 32}
BLOCK = {Q4: 18, Q8: 34}
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def bq():
    import os
    from block_quantized_weight_row_gb300 import binding
    if not os.path.exists(binding.library_path()):
        import __graft_entry__
        __graft_entry__.build()
    import block_quantized_weight_row_gb300 as bq
    bq.lib()
    return bq


# ------------------------------------------------------ the layout, plainly --


def planes_of_blocks(blocks, kind, units):
    """Blocks as bytes (tokens, heads, nb * block bytes) -> code rows and scale rows (bytes) of the paged layout."""
    T, H = blocks.shape[:2]
    b = np.ascontiguousarray(blocks).reshape(T, H, -1, BLOCK[kind])
    nb, ub = b.shape[2], CODES[kind] // units
    row = np.zeros((T, H, nb * CODES[kind]), np.uint8)
    for unit in range(units):
        for k in range(nb):
            at = (unit * nb + k) * ub
            row[:, :, at:at + ub] = b[:, :, k, 2 + unit * ub:2 + (unit + 1) * ub]
    return row, np.ascontiguousarray(b[..., :2]).reshape(T, H, nb * 2)


def put_rows(pool, page, kind, dim, units, slots, blocks):
    """Writes token rows into a numpy pool (pages, heads, bytes) at slots (< 0: skipped)."""
    nb = dim // 32
    row, scale = planes_of_blocks(blocks, kind, units)
    for t, s in enumerate(slots):
        if s < 0 or s >= pool.shape[0] * page:
            continue
        p, i = divmod(int(s), page)
        rb = nb * CODES[kind]
        pool[p, :, i * rb:(i + 1) * rb] = row[t]
        at = page * rb + i * nb * 2
        pool[p, :, at:at + nb * 2] = scale[t]


def get_rows(pool, page, kind, dim, units, slots):
    """fp32 codes (tokens, heads, dim) and binary16 scales (tokens, heads, nb) at slots."""
    nb, ub, rb = dim // 32, CODES[kind] // units, dim // 32 * CODES[kind]
    H = pool.shape[1]
    codes = np.zeros((len(slots), H, dim), np.float32)
    scales = np.zeros((len(slots), H, nb), np.float16)
    p, i = np.divmod(np.asarray(slots, np.int64), page)
    for k in range(nb):
        at = page * rb + (i * nb + k) * 2
        scales[:, :, k] = (pool[p, :, at].astype(np.uint16) | pool[p, :, at + 1].astype(np.uint16) << 8).view(np.float16)
        for byte in range(CODES[kind]):
            unit, off = divmod(byte, ub)
            v = pool[p, :, i * rb + (unit * nb + k) * ub + off]
            if kind == Q8:
                codes[:, :, 32 * k + byte] = v.view(np.int8)
            else:
                codes[:, :, 32 * k + byte] = (v & 15).astype(np.float32) - 8
                codes[:, :, 32 * k + 16 + byte] = (v >> 4).astype(np.float32) - 8
    return codes, scales


def butterflies(x):
    """The rotation in fp32: spans 1 .. 32 of every 64 channels, then 1/8."""
    x = np.array(x, np.float32)
    v = x.reshape(-1, 64)
    for span in (1, 2, 4, 8, 16, 32):
        for j in range(64):
            if not j & span:
                a, b = v[:, j].copy(), v[:, j + span].copy()
                v[:, j], v[:, j + span] = a + b, a - b
    return (v * np.float32(0.125)).reshape(x.shape)


def hadamard(dim):
    i = np.arange(64)
    h = np.array([[(-1.0) ** bin(a & b).count("1") for b in i] for a in i]) / 8
    return np.kron(np.eye(dim // 64), h)


# ---------------------------------------------------------------- refusals --


def _struct(bq, **kw):
    from block_quantized_weight_row_gb300 import binding
    a = dict(k_pages=FAKE, v_pages=FAKE + (1 << 32), n_pages=10, page_size=16, n_kv_heads=2, head_dim=64, k_type=Q4,
             v_type=Q4, k_basis=0)
    a.update(kw)
    return binding._CacheStruct(*a.values())


IN1, IN2, OUT1, OUT2, IDX, WS = (FAKE + (k << 33) for k in range(1, 7))


def _write(bq, s, elem=F32, K=IN1, ks=(128, 64), V=IN2, vs=(128, 64), bias=None, basis=0, slots=IDX, n=3):
    return bq.lib().bq_paged_kv_write(s, elem, K, *ks, V, *vs, bias, basis, slots, n)


def _read(bq, s, elem=F32, K=OUT1, V=OUT2, bias=None, basis=0, slots=IDX, n=3):
    return bq.lib().bq_paged_kv_read(s, elem, K, V, bias, basis, slots, n)


def _attn(bq, s, elem=F32, q=IN1, qs=(256, 64), o=OUT1, os=(256, 64), lse=None, qst=IDX, kvl=IDX + 4096, pt=IDX + 8192,
          max_pages=4, B=3, n_q=5, max_q=2, max_kv=60, H=4, scale=0.1, causal=1, window=0):
    return bq.lib().bq_paged_attn(s, elem, q, *qs, o, *os, lse, qst, kvl, pt, max_pages, B, n_q, max_q, max_kv, H,
                                  scale, causal, window)


CACHE_FAULTS = [
    (dict(k_type=3), UNSUPPORTED), (dict(v_type=12), UNSUPPORTED), (dict(k_type=0), UNSUPPORTED),
    (dict(k_basis=2), UNSUPPORTED), (dict(n_pages=-1), INVALID), (dict(n_kv_heads=0), INVALID),
    (dict(head_dim=0), INVALID), (dict(page_size=0), INVALID), (dict(page_size=24), SHAPE), (dict(page_size=8), SHAPE),
    (dict(page_size=1 << 21), SHAPE), (dict(head_dim=48), SHAPE), (dict(head_dim=96, k_basis=1), SHAPE),
    (dict(n_pages=1 << 28), SHAPE), (dict(n_kv_heads=1 << 20), SHAPE), (dict(k_pages=None), INVALID),
    (dict(v_pages=None), INVALID), (dict(k_pages=FAKE + 8), ALIGN), (dict(v_pages=FAKE + 16), INVALID),
]


@pytest.mark.parametrize("kw,status", CACHE_FAULTS)
def test_bad_caches_are_refused(bq, kw, status):
    s = _struct(bq, **kw)
    for call in (_write, _read, _attn):
        assert call(bq, s) == status, (call.__name__, kw, bq.lib().bq_last_error())


def test_write_refusals(bq):
    s = _struct(bq)
    assert bq.lib().bq_paged_kv_write(None, F32, IN1, 1, 1, IN2, 1, 1, None, 0, IDX, 1) == INVALID
    assert _write(bq, s, elem=3) == UNSUPPORTED
    assert _write(bq, s, n=-1) == INVALID
    assert _write(bq, s, n=0, K=None, V=None, slots=None) == OK
    for kw in (dict(K=None), dict(V=None), dict(slots=None), dict(ks=(-64, 64)), dict(vs=(64, 1 << 41))):
        assert _write(bq, s, **kw) == INVALID, kw
    for kw in (dict(K=IN1 + 4), dict(ks=(130, 64)), dict(vs=(128, 66)), dict(slots=IDX + 4), dict(elem=BF16, ks=(132, 64)),
               dict(bias=IN1 + 4)):
        assert _write(bq, s, **kw) == ALIGN, kw
    assert _write(bq, _struct(bq, k_type=Q8), bias=FAKE + (40 << 33)) == UNSUPPORTED
    assert _write(bq, s, bias=FAKE + (40 << 33), basis=1) == BASIS
    assert _write(bq, s, K=FAKE) == INVALID and "overlap" in bq.lib().bq_last_error().decode()
    assert _write(bq, s, slots=FAKE + (1 << 32)) == INVALID


def test_read_refusals(bq):
    s = _struct(bq)
    assert _read(bq, s, elem=-1) == UNSUPPORTED
    assert _read(bq, s, n=-1) == INVALID
    assert _read(bq, s, n=0, K=None, V=None, slots=None) == OK
    for kw in (dict(K=None), dict(V=None), dict(slots=None), dict(V=OUT1 + 16), dict(K=FAKE), dict(V=IDX)):
        assert _read(bq, s, **kw) == INVALID, kw
    for kw in (dict(K=OUT1 + 8), dict(V=OUT2 + 4), dict(slots=IDX + 2)):
        assert _read(bq, s, **kw) == ALIGN, kw
    assert _read(bq, _struct(bq, n_pages=0)) == INVALID
    assert _read(bq, s, bias=FAKE + (40 << 33), basis=1) == BASIS
    assert _read(bq, _struct(bq, k_type=Q8), bias=FAKE + (40 << 33)) == UNSUPPORTED


def test_attention_refusals(bq):
    s, L = _struct(bq), bq.lib()
    L.bq_set_workspace(None, 0)
    assert _attn(bq, s) == WORKSPACE
    need = L.bq_paged_attn_workspace_size(s, F32, 3, 5, 2, 60, 4, 1, 0)
    assert need > 0
    assert _attn(bq, s, B=0) == OK and _attn(bq, s, n_q=0, q=None, o=None) == OK
    for kw in (dict(B=-1), dict(n_q=-1), dict(max_q=-1), dict(max_kv=-1), dict(max_pages=-1), dict(window=-1), dict(q=None),
               dict(o=None), dict(qst=None), dict(kvl=None), dict(pt=None), dict(scale=math.inf), dict(scale=math.nan),
               dict(os=(0, 64)), dict(os=(256, 0)), dict(os=(200, 64)), dict(o=IN1), dict(o=FAKE), dict(lse=OUT1), dict(lse=IDX)):
        assert _attn(bq, s, **kw) == INVALID, kw
    for kw in (dict(H=5), dict(H=0), dict(B=1 << 21), dict(max_kv=2**31 - 1)):
        assert _attn(bq, s, **kw) == SHAPE, kw
    assert _attn(bq, _struct(bq, n_pages=0)) == INVALID
    assert _attn(bq, _struct(bq, head_dim=32)) == SHAPE and _attn(bq, _struct(bq, head_dim=160)) == SHAPE
    assert _attn(bq, s, elem=7) == UNSUPPORTED and _attn(bq, s, causal=0, window=3) == UNSUPPORTED
    for kw in (dict(q=IN1 + 8), dict(qs=(258, 64)), dict(os=(256, 66)), dict(o=OUT1 + 4), dict(qst=IDX + 2), dict(lse=OUT2 + 2)):
        assert _attn(bq, s, **kw) == ALIGN, kw
    try:  # a workspace that overlaps an argument, and one too small
        assert L.bq_set_workspace(IN1, need) == OK
        assert _attn(bq, s) == INVALID
        assert L.bq_set_workspace(OUT1, need) == OK
        assert _attn(bq, s) == INVALID
        assert L.bq_set_workspace(WS, need - 1) == OK
        assert _attn(bq, s) == WORKSPACE
    finally:
        L.bq_set_workspace(None, 0)


def test_page_bytes(bq):
    f = bq.lib().bq_paged_page_bytes
    assert f(Q4, 16, 8, 128) == 16 * 8 * 4 * 18 and f(Q8, 32, 1, 96) == 32 * 3 * 34
    assert f(Q4, 8, 8, 128) == f(3, 16, 8, 128) == f(Q4, 16, 0, 128) == f(Q4, 16, 8, 100) == f(Q4, 16, 8, 0) == 0


@pytest.mark.parametrize("page", [16, 48, 64, 1008])
def test_slots_are_checked_before_they_become_addresses(bq, page):
    """The kernels' own slot code on the host: first, last, skipped and wrong slots."""
    s = _struct(bq, page_size=page, n_pages=7)
    p, i = ctypes.c_int64(), ctypes.c_int64()
    f = lambda slot: (bq.lib().bq_paged_slot_check(s, slot, p, i), p.value, i.value)  # noqa: E731
    for slot in (0, 1, page - 1, page, 5 * page + 3, 7 * page - 1):
        assert f(slot) == (OK, *divmod(slot, page))
    assert f(-1) == (OK, -1, -1)
    for slot in (7 * page, -2, 1 << 31, (1 << 32) + 1, 1 << 62, -(1 << 63)):
        assert f(slot) == (INDEX, -1, -1)
    assert bq.lib().bq_paged_slot_check(_struct(bq, n_pages=0), 0, p, i) == INDEX


def test_binding_refuses_cpu_tensors(bq):
    c = bq.PagedCache(torch.zeros(2, 1, 16 * 36, dtype=torch.uint8), torch.zeros(2, 1, 16 * 36, dtype=torch.uint8), 16, 64)
    x = torch.zeros(1, 1, 64)
    with pytest.raises(TypeError):
        bq.paged_kv_write(c, x, x, torch.zeros(1, dtype=torch.int64))
    with pytest.raises(TypeError):
        bq.paged_kv_read(c, torch.zeros(1, dtype=torch.int64))


# ------------------------------------------------------------ write and read --

DT = {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16}


def _rows(seed, T, H, D, dtype):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, D, generator=g) * torch.exp(torch.randn(T, H, 1, generator=g))
    if T > 2:
        x[1] = 0.0  # a zero row
        x[2, 0, :32] = torch.arange(32) * 0.5 - 7.5  # ties
    return x.to(dtype)


WRITE_CASES = [
    # T, H, D, page, kt, vt, elem, basis, bias, strided
    (1, 1, 64, 16, Q4, Q4, F32, 0, False, False),
    (1, 8, 128, 16, Q4, Q4, BF16, 1, True, True),
    (37, 3, 96, 16, Q4, Q8, F16, 0, True, False),
    (33, 5, 32, 48, Q8, Q4, F32, 0, False, True),
    (70, 2, 160, 32, Q4, Q4, BF16, 0, False, False),
    (130, 2, 256, 64, Q8, Q8, F16, 1, False, True),
    (257, 4, 64, 16, Q4, Q8, F32, 1, True, False),
    (1000, 8, 128, 16, Q4, Q8, F32, 0, True, True),
    (65, 1, 192, 128, Q4, Q4, F32, 1, True, False),
    (19, 7, 64, 16, Q8, Q8, BF16, 0, False, False),
]


def _case(bq, orc, T, H, D, page, kt, vt, elem, basis, with_bias, strided, seed=7):
    """A written cache, and what its pools and rows have to be."""
    rng = np.random.default_rng(seed)
    pages = -(-T // page) + 3
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    if T > 5:
        slots[3] = -1
    k, v = _rows(seed + 1, T, H, D, DT[elem]), _rows(seed + 2, T, H, D, DT[elem])
    bias = rng.standard_normal((H, D)).astype(np.float32) if with_bias else None
    dev = torch.device("cuda:0")
    if strided:  # token-major slices of one buffer, and heads in front of tokens
        kv = torch.zeros(T, 2 * H + 1, D, dtype=DT[elem], device=dev)
        kd = kv[:, 1:1 + H]
        vd = torch.zeros(H, T, D, dtype=DT[elem], device=dev).transpose(0, 1)
        kd.copy_(k)
        vd.copy_(v)
    else:
        kd, vd = k.to(dev), v.to(dev)
    cache = bq.PagedCache.empty(pages, page, H, D, kt, vt, basis, device=dev)
    for p in (cache.k_pages, cache.v_pages):
        p.fill_(0xA5)
    bd = None if bias is None else torch.from_numpy(bias).to(dev)
    bq.paged_kv_write(cache, kd, vd, torch.from_numpy(slots).to(dev), bias=bd)
    kw = orc.kv_quantize(kt, k.float().numpy(), bias, T, H, D, basis=basis)
    vw = orc.kv_quantize(vt, v.float().numpy(), None, T, H, D)
    want = []
    for kind, units, blocks in ((kt, 4, kw), (vt, 8, vw)):
        pool = np.full((pages, H, page * (D // 32) * BLOCK[kind]), 0xA5, np.uint8)
        put_rows(pool, page, kind, D, units, slots, np.asarray(blocks).reshape(T, H, -1))
        want.append(pool)
    return cache, slots, bias, bd, want


@gpu
@pytest.mark.parametrize("case", WRITE_CASES, ids=str)
def test_write_and_read_bits(bq, orc, case):
    T, H, D, page, kt, vt, elem, basis, with_bias, strided = case
    cache, slots, bias, bd, want = _case(bq, orc, *case)
    assert np.array_equal(cache.k_pages.cpu().numpy(), want[0])
    assert np.array_equal(cache.v_pages.cpu().numpy(), want[1])
    live = slots >= 0
    ck, sk = get_rows(want[0], page, kt, D, 4, slots[live])
    cv, sv = get_rows(want[1], page, vt, D, 8, slots[live])
    rk = np.zeros((T, H, D), np.float32)
    rv = np.zeros((T, H, D), np.float32)
    rk[live] = ck * np.repeat(sk.astype(np.float32), 32, axis=-1)
    rv[live] = cv * np.repeat(sv.astype(np.float32), 32, axis=-1)
    if bias is not None:
        rk[live] += bias
    if basis:
        rk = butterflies(rk)
    rk[~live] = 0
    for out in (F32, F16, BF16):
        k, v = bq.paged_kv_read(cache, torch.from_numpy(slots).cuda(), DT[out], bias=bd)
        assert torch.equal(v.cpu(), torch.from_numpy(rv).to(DT[out]))
        assert torch.equal(k.cpu(), torch.from_numpy(rk).to(DT[out]))
    assert bq.binding.device_status() == OK


@gpu
def test_write_equals_the_contiguous_write(bq):
    """One page that holds a run of tokens: the same codes and scales as kv_write's blocks."""
    T, H, D = 64, 2, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = torch.randn(T, H, D, generator=g, device="cuda"), torch.randn(T, H, D, generator=g, device="cuda")
    cache = bq.PagedCache.empty(1, T, H, D, Q4, Q8, 1)
    bq.paged_kv_write(cache, k, v, torch.arange(T, device="cuda"))
    kb, vb = bq.kv_write(Q4, k, None, Q8, v, basis=1)
    for pool, blocks, kind, units in ((cache.k_pages, kb, Q4, 4), (cache.v_pages, vb, Q8, 8)):
        want = np.zeros((1, H, T * D // 32 * BLOCK[kind]), np.uint8)
        put_rows(want, T, kind, D, units, range(T), blocks.cpu().numpy())
        assert np.array_equal(pool.cpu().numpy(), want)


@gpu
def test_wrong_slots_are_skipped_and_reported(bq):
    T, H, D, page = 20, 2, 64, 16
    k = torch.randn(T, H, D, device="cuda")
    cache = bq.PagedCache.empty(3, page, H, D)
    for p in (cache.k_pages, cache.v_pages):
        p.fill_(0x5A)
    slots = torch.arange(T, device="cuda")
    slots[4], slots[7], slots[9] = 3 * page, -2, 1 << 40
    bq.paged_kv_write(cache, k, k, slots)
    assert bq.binding.device_status() == INDEX
    assert bq.binding.device_status() == OK
    rk, rv = bq.paged_kv_read(cache, slots)
    assert bq.binding.device_status() == INDEX
    for t in (4, 7, 9):
        assert not rk[t].any() and not rv[t].any()
    untouched = [4, 7, 9] + list(range(T, 3 * page))  # their places kept what they held
    kept = np.full(tuple(cache.k_pages.shape), 0x5A, np.uint8)
    for a, b in zip(get_rows(cache.k_pages.cpu().numpy(), page, Q4, D, 4, untouched), get_rows(kept, page, Q4, D, 4, untouched)):
        assert (a == b).all()


@gpu
def test_pool_beyond_32_bit_offsets(bq):
    """Rows past 4 GiB in both pools: written, read back and attended."""
    H, D, page = 8, 128, 128
    n = 70_000  # pages of 73,728 bytes: 5.2 GB a pool
    cache = bq.PagedCache.empty(n, page, H, D)
    assert cache.k_pages.numel() > 1 << 32
    T = 300
    k, v = torch.randn(T, H, D, device="cuda"), torch.randn(T, H, D, device="cuda")
    table = torch.tensor([[n - 1, 3, n - 2]], dtype=torch.int32, device="cuda")
    j = torch.arange(T, device="cuda")
    slots = table[0].long()[j // page] * page + j % page
    bq.paged_kv_write(cache, k, v, slots)
    small = bq.PagedCache.empty(3, page, H, D)
    bq.paged_kv_write(small, k, v, j)
    for a, b in zip(bq.paged_kv_read(cache, slots), bq.paged_kv_read(small, j)):
        assert torch.equal(a, b)
    q = torch.randn(1, 16, D, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    kw = dict(max_q_len=1, max_kv_len=T)
    a = bq.paged_attn(cache, q, i32([0, 1]), i32([T]), table, 0.1, **kw)
    b = bq.paged_attn(small, q, i32([0, 1]), i32([T]), i32([[0, 1, 2]]), 0.1, **kw)
    assert torch.equal(a, b)
    del cache
    torch.cuda.empty_cache()


# --------------------------------------------------------------- attention --


class Batch:
    """A batch over a cache of random codes, with everything unused set to garbage (NaN scales)."""

    def __init__(self, bq, q_len, kv_len, H, NKV, D, page, kt, vt, elem, basis=0, seed=0, peaked=1.0, vscale=1.0, wide=True):
        rng = np.random.default_rng(seed)
        self.bq, self.q_len, self.kv_len, self.H, self.NKV, self.D, self.page = bq, q_len, kv_len, H, NKV, D, page
        self.kt, self.vt, self.elem, self.basis = kt, vt, elem, basis
        per = [-(-n // page) for n in kv_len]
        total = sum(per) + 2
        order = rng.permutation(total)[:sum(per)]
        self.table = np.full((len(kv_len), max(per + [1]) + 1), 12345678, np.int32)  # never to be read past a sequence's pages
        at = 0
        self.slots = []
        for b, n in enumerate(per):
            self.table[b, :n] = order[at:at + n]
            j = np.arange(kv_len[b])
            self.slots.append(order[at:at + n][j // page].astype(np.int64) * page + j % page if n else j)
            at += n
        nb = D // 32
        self.pools = []
        for kind, units, mul in ((kt, 4, 1.0), (vt, 8, vscale)):
            pool = np.full((total, NKV, page * nb * BLOCK[kind]), 0xFF, np.uint8)  # scales 0xFFFF: NaN
            used = np.concatenate(self.slots).astype(np.int64) if at else np.zeros(0, np.int64)
            blocks = rng.integers(0, 256, (len(used), NKV, nb, BLOCK[kind]), dtype=np.uint8)
            if kind == Q8:
                blocks[..., 2:] = np.where(blocks[..., 2:] == 128, 127, blocks[..., 2:])
            d = (np.exp(0.5 * rng.standard_normal((len(used), NKV, nb))) * (0.4 if kind == Q4 else 0.02) * mul).astype(np.float16)
            blocks[..., :2] = d[..., None].view(np.uint8)
            put_rows(pool, page, kind, D, units, used, blocks.reshape(len(used), NKV, -1))
            self.pools.append(pool)
        n_q = sum(q_len)
        self.q = torch.from_numpy(rng.standard_normal((n_q, H, D)).astype(np.float32) * peaked).to(DT[elem])
        self.cache = bq.PagedCache(torch.from_numpy(self.pools[0]).cuda(), torch.from_numpy(self.pools[1]).cuda(), page, D, kt, vt, basis)
        self.q_start = torch.tensor([0] + list(np.cumsum(q_len)), dtype=torch.int32, device="cuda")
        self.kvl = torch.tensor(kv_len, dtype=torch.int32, device="cuda")
        self.pt = torch.from_numpy(self.table).cuda()
        self.scale = 1.0 / math.sqrt(D)
        # wide: a bound of kv_len that gives a call of many rows the work by which the many-row kernel is taken
        self.bound = max(list(kv_len) + [0])
        rows = max(list(q_len) + [0]) * H // NKV
        if wide and rows > 32:
            self.bound = max(self.bound, 250000 // (-(-rows // 16) * len(q_len) * NKV))

    def run(self, causal=True, window=0, **kw):
        q = kw.pop("q", None)
        lse = torch.full((self.q.shape[0], self.H), 7.0, device="cuda")
        o = self.bq.paged_attn(self.cache, self.q.cuda() if q is None else q, self.q_start, self.kvl, self.pt, self.scale,
                               max_q_len=max(self.q_len + [0]), max_kv_len=self.bound, causal=causal,
                               window=window, lse=lse, **kw)
        return o, lse

    def reference(self, causal=True, window=0):
        """o, lse and their tolerances, in 64 bits."""
        u16, u32 = 2.0**-11, 2.0**-24
        G, D = self.H // self.NKV, self.D
        n_q = self.q.shape[0]
        o, tol = np.zeros((n_q, self.H, D)), np.zeros((n_q, self.H, D))
        lse, ltol = np.full((n_q, self.H), -np.inf), np.zeros((n_q, self.H))
        half_step = {F32: 2.0**-24, F16: 2.0**-11, BF16: 2.0**-8}[self.elem]
        t0 = 0
        for b, (n, kv) in enumerate(zip(self.q_len, self.kv_len)):
            if n == 0:
                continue
            ck, sk = get_rows(self.pools[0], self.page, self.kt, D, 4, self.slots[b])
            cv, sv = get_rows(self.pools[1], self.page, self.vt, D, 8, self.slots[b])
            dk = np.repeat(sk.astype(np.float64), 32, axis=-1)
            k, v = ck * dk, cv * np.repeat(sv.astype(np.float64), 32, axis=-1)
            many = self.elem != F32 and D in (64, 128) and n * G > (32 if self.elem == BF16 else 64)
            wide = np.abs(k) if many or self.kt == Q8 else 16 * dk
            q = self.q[t0:t0 + n].double().numpy()
            if self.basis:
                q = q @ hadamard(D)
            pos = kv - n + np.arange(n)[:, None]
            j = np.arange(kv)[None]
            see = np.ones((n, kv), bool)
            if causal:
                see = j <= pos
                if window:
                    see &= j > pos - window
            any_ = see.any(-1)
            for h in range(self.H):
                kh, vh = k[:, h // G], v[:, h // G]
                if kv == 0:
                    continue
                s = np.where(see, q[:, h] @ kh.T * self.scale, -np.inf)
                mag = np.where(see, np.abs(q[:, h]) @ wide[:, h // G].T * self.scale, 0).max(-1)
                # q's roundings reach every channel of its row as a share of the largest value
                peak = np.where(see, np.abs(q[:, h]).max(-1, keepdims=True) * np.abs(kh).sum(-1)[None] * self.scale, 0).max(-1)
                two = self.elem == F32
                qerr = 3 * u16**2 * peak if two else u16 * mag if self.basis or many else 0.0 * mag
                if self.basis:
                    qerr = qerr + 8 * u32 * peak  # the butterflies
                ds = (D + 8 if many else 34 + D // 32 + 4) * 2 * u32 * mag + qerr + 2 * u32 * np.abs(np.where(see, s, 0)).max(-1)
                if many:
                    ds = ds + u16 * mag + 2.0**-35 * peak + 2.0**-30 * dk[:, h // G].max() * np.abs(q[:, h]).sum(-1) * self.scale
                top = np.where(any_, s.max(-1, initial=-np.inf), 0.0)
                w = np.exp(s - top[:, None])
                tot = w.sum(-1)
                w = w / np.where(tot > 0, tot, 1)[:, None]
                rel = 2 * ds + (u16**2 if two else u16) + (u16 if many else 0.0) + 6 * u32 + ((kv if many else kv / 8) + 64) * 2 * u32
                o[t0:t0 + n, h] = w @ vh
                dv, cvh = sv[:, h // G].astype(np.float64), np.abs(cv[:, h // G]).astype(np.float64)
                gone = np.concatenate([np.minimum(w * dv[None, :, x], 2.0**-30 * dv.max()) @ cvh[:, 32 * x:32 * x + 32]
                                       for x in range(D // 32)], axis=-1)
                if many:
                    gone = gone + 2.0**-30 * dv.max()
                tol[t0:t0 + n, h] = rel[:, None] * (w @ np.abs(vh)) * 1.01 + half_step * np.abs(o[t0:t0 + n, h]) + gone
                lse[t0:t0 + n, h] = np.where(any_, top + np.log(np.where(tot > 0, tot, 1)), -np.inf)
                ltol[t0:t0 + n, h] = ds + (kv / 8 + 64) * 2 * u32 + 8 * u32 * (1 + np.abs(np.where(any_, lse[t0:t0 + n, h], 0)))
            t0 += n
        return o, tol, lse, ltol

    def compare(self, o, lse, reference, rows=slice(None)):
        ref, tol, rl, lt = (x[rows] for x in reference)
        o, lse = o.double().cpu().numpy()[rows], lse.double().cpu().numpy()[rows]
        assert np.isfinite(o).all()
        err = np.abs(o - ref)
        tol = tol + (2.0**-24 if self.elem == F16 else 0.0)  # binary16 subnormal outputs
        assert (err <= tol).all(), f"worst {np.max(err / np.maximum(tol, 1e-300)):.3g} of the tolerance at {np.unravel_index(np.argmax(err - tol), err.shape)}"
        dead = np.isneginf(rl)
        assert np.array_equal(np.isneginf(lse), dead)
        assert (o[dead] == 0).all()
        assert (np.abs(lse[~dead] - rl[~dead]) <= lt[~dead]).all(), f"lse off by {np.max(np.abs(lse[~dead] - rl[~dead]) - lt[~dead])}"

    def check(self, causal=True, window=0, **kw):
        o, lse = self.run(causal, window, **kw)
        assert self.bq.binding.device_status() == OK
        self.compare(o, lse, self.reference(causal, window))


DECODE = [
    # q_len, kv_len, H, NKV, D, page, kt, vt, elem, basis
    ([1], [1], 1, 1, 64, 16, Q4, Q4, F32, 0),
    ([1], [15], 8, 8, 128, 16, Q4, Q4, F32, 0),
    ([1], [16], 8, 4, 128, 16, Q4, Q8, BF16, 0),
    ([1], [17], 8, 2, 96, 16, Q8, Q4, F16, 0),
    ([1], [777], 16, 8, 128, 16, Q4, Q4, F32, 1),
    ([1, 1, 1], [33, 1000, 31], 12, 4, 64, 32, Q4, Q4, BF16, 1),
    ([1, 1], [2050, 4099], 16, 2, 128, 64, Q4, Q8, F16, 0),
    ([1] * 40, [(37 * i) % 701 for i in range(40)], 8, 2, 128, 16, Q4, Q4, BF16, 0),
    ([1], [5000], 7, 1, 256, 48, Q8, Q8, F32, 0),
    ([1, 1], [640, 70], 4, 4, 256, 16, Q4, Q4, F16, 1),
    ([1], [300], 10, 1, 96, 16, Q4, Q8, F32, 0),
    ([1], [129], 24, 1, 128, 16, Q8, Q8, BF16, 0),
]


@gpu
@pytest.mark.parametrize("case", DECODE, ids=str)
def test_attention_of_single_tokens(bq, case):
    Batch(bq, *case).check()


FEW = [
    # q_len, kv_len, H, NKV, D, page, kt, vt, elem, basis, causal, window
    ([5, 1, 0, 3], [40, 700, 90, 3], 8, 4, 128, 16, Q4, Q4, BF16, 0, True, 0),
    ([4, 2], [64, 33], 6, 2, 64, 16, Q4, Q8, F32, 1, False, 0),
    ([3, 8, 2], [1000, 500, 9], 12, 4, 96, 32, Q8, Q4, F16, 0, True, 100),
    ([7], [7], 4, 4, 128, 16, Q4, Q4, F32, 0, True, 1),
    ([6, 3], [2, 0], 4, 2, 128, 16, Q4, Q4, BF16, 0, True, 0),      # more queries than tokens: empty rows
    ([2, 2], [0, 5], 4, 2, 64, 16, Q4, Q4, F32, 0, False, 0),        # an empty cache
    ([9], [800], 4, 2, 256, 64, Q4, Q8, BF16, 1, True, 37),
    ([33], [33], 4, 1, 128, 16, Q8, Q8, F32, 0, True, 0),
    ([17, 1, 2], [300, 2000, 2], 8, 2, 128, 32, Q4, Q4, F16, 0, True, 16),
    ([5] * 6, [900, 17, 5, 64, 333, 1], 24, 8, 64, 32, Q4, Q4, F16, 0, True, 128),
]


@gpu
@pytest.mark.parametrize("case", FEW, ids=str)
def test_attention_of_a_few_tokens(bq, case):
    *args, causal, window = case
    Batch(bq, *args).check(causal, window)


MANY = [
    # q_len, kv_len, H, NKV, D, page, kt, vt, elem, basis, causal, window
    ([65], [65], 1, 1, 128, 16, Q4, Q4, BF16, 0, True, 0),
    ([200], [200], 4, 4, 64, 16, Q4, Q4, BF16, 0, True, 0),
    ([70, 1, 0, 300], [500, 900, 10, 300], 8, 4, 128, 16, Q4, Q8, F16, 1, True, 0),
    ([129, 40], [1000, 41], 6, 2, 128, 48, Q8, Q8, BF16, 0, False, 0),
    ([513], [700], 4, 2, 64, 32, Q8, Q4, F16, 1, True, 0),
    ([150, 90], [100, 0], 4, 2, 128, 16, Q4, Q4, BF16, 0, True, 0),     # rows before the first token, an empty cache
    ([260], [2000], 3, 1, 128, 64, Q4, Q4, F16, 0, True, 130),           # a window that ends inside tiles
    ([300], [5000], 4, 1, 64, 16, Q4, Q8, BF16, 0, True, 1),
    ([100], [3500], 8, 8, 128, 128, Q4, Q4, BF16, 1, True, 0),           # tokens split over CTAs
    ([700, 5, 333], [900, 800, 333], 16, 8, 128, 16, Q4, Q4, BF16, 0, True, 0),  # more CTAs than a split
    ([96], [2300], 8, 1, 64, 32, Q8, Q8, F16, 0, False, 0),
    # 33 to 64 rows per kv head, with sequences enough to fill SMs, beside shorter ones
    ([12, 9, 8, 1] * 3, [(61 * i) % 700 + 12 for i in range(12)], 16, 4, 128, 16, Q4, Q8, BF16, 1, True, 0),
    ([33, 64, 32] * 13, [(83 * i) % 900 for i in range(39)], 1, 1, 64, 16, Q4, Q4, BF16, 0, True, 200),
    ([5, 4] * 4, [300 + 150 * i for i in range(8)], 40, 5, 128, 48, Q8, Q4, F16, 0, False, 0),
    # row tiles enough that no tokens are split
    ([640, 700], [640, 900], 16, 8, 128, 16, Q4, Q4, F16, 0, True, 0),
    ([500], [520], 40, 20, 64, 32, Q8, Q8, BF16, 1, True, 0),
]


@gpu
@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("case", MANY, ids=str)
def test_attention_of_many_tokens(bq, case, wide):
    *args, causal, window = case
    Batch(bq, *args, wide=wide).check(causal, window)


@gpu
@pytest.mark.parametrize("vscale,peaked", [(1e-4, 1.0), (3000.0, 1.0), (1.0, 30.0), (1.0, 1e-3)])
def test_attention_of_many_tokens_scales(bq, vscale, peaked):
    Batch(bq, [150], [400], 4, 2, 128, 16, Q4, Q4, F16, vscale=vscale, peaked=peaked).check()


@gpu
@pytest.mark.parametrize("elem", [F32, BF16])
@pytest.mark.parametrize("vscale,peaked", [(1e-4, 1.0), (3000.0, 1.0), (1.0, 30.0), (1.0, 1e-3)])
def test_attention_scales_of_v_and_q(bq, elem, vscale, peaked):
    """V scales over the range of binary16 and scores from flat to one-hot."""
    Batch(bq, [1, 3], [500, 333], 8, 4, 128, 16, Q4, Q4, elem, vscale=vscale, peaked=peaked).check()


@gpu
@pytest.mark.parametrize("n,elem", [(1, F32), (90, BF16)])
def test_attention_v_scales_that_grow_along_the_cache(bq, n, elem):
    """The weights' common power of two has to follow: scales from 2^-14 to 2^12 in order, and back."""
    for flip in (False, True):
        b = Batch(bq, [n], [1024], 8, 4, 128, 16, Q4, Q4, elem, seed=3)
        nb, page = 4, 16
        d = np.exp2(np.linspace(-14, 12, 1024)).astype(np.float16)
        for j, slot in enumerate(b.slots[0]):
            p, i = divmod(int(slot), page)
            at = page * nb * 16 + i * nb * 2
            b.pools[1][p, :, at:at + nb * 2] = np.repeat(d[-1 - j if flip else j], nb).view(np.uint8)
        b.cache.v_pages.copy_(torch.from_numpy(b.pools[1]))
        b.check()


@gpu
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("n,elem", [(1, F32), (3, F16), (90, BF16)])
def test_attention_of_zero_scales(bq, n, elem, which):
    """Blocks of zeros: every weight alike (K), or outputs of exactly zero (V)."""
    b = Batch(bq, [n], [n + 300], 4, 2, 128, 16, Q4, Q4, elem)
    i = "kv".index(which)
    b.pools[i][:, :, 16 * 4 * 16:] = 0
    pools = [torch.from_numpy(p).cuda() for p in b.pools]
    b.cache = bq.PagedCache(*pools, 16, 128, Q4, Q4, 0)
    b.check()
    if which == "v":
        assert (b.run()[0] == 0).all()


@gpu
def test_attention_strides_and_given_outputs(bq):
    """q and o as slices with heads and tokens in either order."""
    b = Batch(bq, [2, 3], [50, 60], 8, 4, 64, 16, Q4, Q4, BF16)
    n, H, D = b.q.shape
    plain = b.run()[0]
    wide = torch.zeros(n, H + 3, D, dtype=torch.bfloat16, device="cuda")
    wide[:, 2:2 + H] = b.q.cuda()
    o = torch.full((H, n + 1, 2 * D), 5.0, dtype=torch.bfloat16, device="cuda")
    out = o[:, :n, D:].transpose(0, 1)
    got = b.run(q=wide[:, 2:2 + H], out=out)[0]
    assert got.data_ptr() == out.data_ptr() and torch.equal(got, plain)
    assert (o[:, n:] == 5).all() and (o[:, :, :D] == 5).all()


@gpu
@pytest.mark.parametrize("many", [1, 80])
def test_attention_is_the_same_every_time_and_on_any_stream(bq, many):
    b = Batch(bq, [1] * 8 + [many], [3000, 20, 1, 700, 2222, 64, 65, 1500, 4097], 16, 4, 128, 16, Q4, Q4, BF16)
    first = b.run()
    q = b.q.cuda()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(b.run(q=q))
    torch.cuda.synchronize()
    for o, lse in outs:
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


@gpu
def test_captured_step_follows_lengths_and_pages(bq):
    """One captured graph of write and attention, replayed as the sequences grow."""
    H, NKV, D, page, B, n = 8, 2, 128, 16, 3, 5
    cache = bq.PagedCache.empty(B * 4, page, NKV, D, Q4, Q8)
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(n, B, NKV, D, generator=g, device="cuda") for _ in range(2))
    q = torch.randn(n, B, H, D, generator=g, device="cuda")
    table = torch.arange(B * 4, dtype=torch.int32, device="cuda").reshape(B, 4)
    start = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    base = torch.tensor([14, 0, 30], device="cuda")
    pre = torch.randn(30, NKV, D, generator=g, device="cuda")
    for b in range(B):
        m = int(base[b])
        if m:
            j = torch.arange(m, device="cuda")
            bq.paged_kv_write(cache, pre[:m], pre[:m], table[b].long()[j // page] * page + j % page)
    ks, vs, qs = (torch.zeros_like(x[0]) for x in (k, v, q))
    slots = torch.full((B,), -1, dtype=torch.int64, device="cuda")
    kvl = torch.zeros(B, dtype=torch.int32, device="cuda")

    def step():
        bq.paged_kv_write(cache, ks, vs, slots)
        return bq.paged_attn(cache, qs, start, kvl, table, 0.1, max_q_len=1, max_kv_len=64)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    eager_cache = bq.PagedCache(cache.k_pages.clone(), cache.v_pages.clone(), page, D, Q4, Q8)
    for t in range(n):
        at = base + t
        now = table.long()[torch.arange(B, device="cuda"), at // page] * page + at % page
        for dst, src in ((ks, k[t]), (vs, v[t]), (qs, q[t]), (slots, now), (kvl, (at + 1).int())):
            dst.copy_(src)
        graph.replay()
        got = out.clone()
        bq.paged_kv_write(eager_cache, k[t], v[t], now)
        want = bq.paged_attn(eager_cache, q[t], start, (at + 1).int(), table, 0.1, max_q_len=1, max_kv_len=64)
        assert torch.equal(got, want)
    assert bq.binding.device_status() == OK


@gpu
def test_attention_reports_wrong_pages_and_lengths(bq):
    """Wrong device-side indices never become addresses: the call is finished, the rest of the batch right."""
    b = Batch(bq, [1, 1, 1], [100, 90, 80], 4, 2, 64, 16, Q4, Q4, F32)
    ref = b.reference()
    others = [0, 2]

    def with_(name, make):
        keep = getattr(b, name)
        setattr(b, name, make(keep.clone()))
        try:
            o, lse = b.run()
        finally:
            setattr(b, name, keep)
        assert bq.binding.device_status() == INDEX
        return o, lse

    def put(at, value):
        def f(t):
            t[at] = value
            return t
        return f

    for bad in (10**6, -1, -2**31):
        b.compare(*with_("pt", put((1, 2), bad)), ref, others)
    for bad in (-5, 10**9):
        b.compare(*with_("kvl", put(1, bad)), ref, others)
    b.compare(*with_("q_start", put(2, 1000)), ref, [0])  # both its neighbours' ranges are wrong then
    b.check()


@gpu
def test_nan_and_infinite_queries_stay_in_their_rows(bq):
    b = Batch(bq, [1, 2], [70, 300], 4, 2, 128, 16, Q4, Q4, F32)
    good = b.run()[0]
    q = b.q.cuda()
    q[1, 2, 5] = math.nan
    q[0, 1, 0] = math.inf
    o = b.run(q=q)[0]
    assert o[1, 2].isnan().all() and o[0, 1].isnan().all()
    for t, h in itertools.product(range(3), range(4)):
        if (t, h) not in ((1, 2), (0, 1)):
            assert torch.equal(o[t, h], good[t, h])


@gpu
def test_many_row_timeout_path_returns_error(bq):
    """A bounded wait that runs out ends the launch with a status, and the next call is right."""
    b = Batch(bq, [150], [400], 4, 2, 128, 16, Q4, Q4, BF16)
    L = bq.lib()
    q = b.q.cuda()
    try:
        assert L.bq_set_spin_limit(0) == OK
        b.run(q=q)
        assert bq.binding.device_status() == -6
    finally:
        L.bq_set_spin_limit(-1)
    b.check()


@gpu
@pytest.mark.parametrize("seed", [1, 2])
def test_serving_example(bq, seed):
    from examples import paged_serving
    lines = []
    assert paged_serving.main(seed, lines.append) <= paged_serving.TOLERANCE
    assert "2: 130" in lines[5]
