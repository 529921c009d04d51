"""The calls around the projections and the paged cache of a served layer:
extending paged sequences, the add and RMS norm with a Q8_0 output, projections
of Q8_0 activations, rotary positions on several axes, adapters of many requests.
Each against a plain implementation in 64 bits (whole numbers and 8-bit codes:
equal), refusals on the host. The plain implementations share no code with the
kernels.

Adapter tolerances, per output element, with u = 2^-24: a chain of n matrix
instructions adds at most 4 u of the sum of magnitudes each (an adder that
truncates 16 products and the sum so far); the first product chains 2 * terms * K
/ 32 of them (terms: 3 for fp32 rows beside bf16 adapters; 4 of the half size
beside fp16 ones) and adds at most 35 partial sums and the scale; fp32 rows beside
fp16 adapters keep 22 bits (2^-22); H enters the second product in 2^-22 (fp32
out, fp16 adapters; and 2^-25 of the row's largest) or 2^-18 (bf16 out), which
chains 2 * terms * rank / 32 instructions, rounded up; the sum with y is rounded
once, and the output to its type.
"""
import math

import numpy as np
import pytest
import torch

OK, INVALID, SHAPE, UNSUPPORTED, ALIGN, WORKSPACE, INDEX = 0, -1, -2, -3, -4, -7, -9
F32, F16, BF16 = 0, 1, 2
DT = {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16}
Q4, Q8 = 2, 8
FAKE = 0x7f0000000000
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


def at(i):
    """Made-up device addresses, far apart."""
    return FAKE + (i << 36)


def quiet(bq):
    from block_quantized_weight_row_gb300 import binding
    return binding.device_status()


# ---------------------------------------------------------------- refusals --


def _extend(bq, page=16, pages=10, kv=at(1), new=at(2), seqs=3, free=at(3), n_free=5, table=at(4), max_pages=4, start=at(5), out=at(6),
            slots=at(7), pos=at(8), n_slots=9, taken=at(9)):
    return bq.lib().bq_paged_extend(page, pages, kv, new, seqs, free, n_free, table, max_pages, start, out, slots, pos, n_slots, taken)


@pytest.mark.parametrize("kw,want", [
    (dict(page=0), INVALID), (dict(page=24), SHAPE), (dict(page=1 << 21), SHAPE), (dict(pages=-1), INVALID), (dict(pages=1 << 28), SHAPE),
    (dict(seqs=-1), INVALID), (dict(seqs=(1 << 20) + 1), SHAPE), (dict(n_free=-1), INVALID), (dict(n_slots=-1), INVALID),
    (dict(n_slots=1 << 31), SHAPE), (dict(n_free=1 << 31), SHAPE), (dict(max_pages=-1), INVALID), (dict(kv=None), INVALID), (dict(new=None), INVALID),
    (dict(free=None), INVALID), (dict(table=None), INVALID), (dict(start=None), INVALID), (dict(out=None), INVALID), (dict(slots=None), INVALID),
    (dict(taken=None), INVALID), (dict(kv=at(1) + 2), ALIGN), (dict(slots=at(7) + 4), ALIGN), (dict(pos=at(8) + 1), ALIGN),
    (dict(out=at(1)), INVALID), (dict(start=at(2) + 8), INVALID), (dict(slots=at(3) + 16), INVALID), (dict(pos=at(7) + 64), INVALID),
    (dict(taken=at(4) + 40), INVALID), (dict(table=at(3) - 40), INVALID)])
def test_extend_refusals(bq, kw, want):
    assert _extend(bq, **kw) == want


def _norm(bq, elem=F32, x=at(1), xs=64, res=at(2), rs=64, w=at(3), eps=1e-6, sum=at(4), ss=64, out=at(5), os=64, q8=at(6), rows=3, cols=64):
    return bq.lib().bq_add_rms_norm(elem, x, xs, res, rs, w, eps, sum, ss, out, os, q8, rows, cols)


@pytest.mark.parametrize("kw,want", [
    (dict(elem=3), UNSUPPORTED), (dict(cols=48), SHAPE), (dict(cols=65536 + 32, xs=1 << 20), SHAPE), (dict(rows=-1), INVALID), (dict(rows=1 << 31), SHAPE),
    (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID), (dict(res=None), INVALID),
    (dict(sum=None, out=None, q8=None), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(x=at(1) + 4), ALIGN),
    (dict(xs=66), ALIGN), (dict(elem=BF16, rs=68), ALIGN), (dict(q8=at(6) + 8), ALIGN), (dict(w=at(3) + 4), ALIGN), (dict(xs=-64), INVALID),
    (dict(os=32), INVALID), (dict(ss=0), INVALID), (dict(out=at(1)), INVALID), (dict(sum=at(1) + 256), INVALID), (dict(sum=at(1), xs=128), INVALID),
    (dict(q8=at(5)), INVALID), (dict(out=at(4) + 512), INVALID), (dict(q8=at(3) + 16), INVALID), (dict(out=at(2) + 16), INVALID)])
def test_norm_refusals(bq, kw, want):
    assert _norm(bq, **kw) == want


@pytest.mark.parametrize("eps,want", [(1e-31, INVALID), (1e-40, INVALID), (1e-50, INVALID), (1.1e30, INVALID), (1e39, INVALID), (1e300, INVALID)])
def test_norm_refuses_eps_beyond_its_arithmetic(bq, eps, want):
    """In fp32 these are zero, subnormal or infinite, or their reciprocal is: a row of zeros would become NaN."""
    assert _norm(bq, eps=eps) == want
    assert _norm(bq, eps=1e-30, rows=0) == OK and _norm(bq, eps=1e30, rows=0) == OK


def test_norm_without_rows_is_a_no_op(bq):
    assert _norm(bq, rows=0, x=None, w=None) == OK


def _rotary(bq, elem=BF16, q=at(1), qs=(256, 64), qh=4, k=at(2), ks=(128, 64), kh=2, eo=BF16, qo=at(3), qos=(256, 64), ko=at(4), kos=(128, 64), pos=at(5),
            pst=9, axes=2, freq=at(6), axis=at(7), rot=64, dim=64, n=9):
    return bq.lib().bq_rotary(elem, q, *qs, qh, k, *ks, kh, eo, qo, *qos, ko, *kos, pos, pst, axes, freq, axis, rot, dim, n, 0, 0)


@pytest.mark.parametrize("kw,want", [
    (dict(elem=5), UNSUPPORTED), (dict(eo=F16), UNSUPPORTED), (dict(elem=F16, eo=F32), UNSUPPORTED), (dict(dim=48), SHAPE), (dict(dim=0), SHAPE),
    (dict(rot=63), SHAPE), (dict(rot=66), SHAPE), (dict(axes=0), SHAPE), (dict(axes=17), SHAPE), (dict(qh=-1), INVALID), (dict(qh=70000), SHAPE), (dict(dim=65536, rot=64, qh=254, kh=3), SHAPE),
    (dict(n=-1), INVALID), (dict(n=1 << 31), SHAPE), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(ko=None), INVALID), (dict(pos=None), INVALID),
    (dict(freq=None), INVALID), (dict(q=at(1) + 8), ALIGN), (dict(qs=(260, 64)), ALIGN), (dict(kos=(128, 68)), ALIGN), (dict(pos=at(5) + 2), ALIGN),
    (dict(freq=at(6) + 4), ALIGN), (dict(qs=(-256, 64)), INVALID), (dict(qos=(64, 64)), INVALID), (dict(pst=-1), INVALID),
    (dict(qo=at(1) + 128), INVALID), (dict(qo=at(1), qos=(512, 64)), INVALID), (dict(ko=at(3) + 256), INVALID), (dict(qo=at(2)), INVALID),
    (dict(qo=at(5)), INVALID), (dict(ko=at(6) - 64), INVALID),
    # q and k in one buffer of rows of 384: q's outputs over k's rows
    (dict(q=at(1), qs=(384, 64), k=at(1) + 512, ks=(384, 64), qo=at(1) + 256, qos=(384, 64)), INVALID),
    (dict(qo=at(3), qos=(384, 64), ko=at(3) + 384, kos=(384, 64)), INVALID)])
def test_rotary_refusals(bq, kw, want):
    assert _rotary(bq, **kw) == want


def _lora(bq, xe=F32, x=at(1), xs=64, we=BF16, a=at(2), b=at(3), scale=at(4), n=3, rank=16, ids=at(5), ye=F32, y=at(6), ys=40, out=at(7), os=40, T=5, M=40, K=64):
    return bq.lib().bq_lora(xe, x, xs, we, a, b, scale, n, rank, ids, ye, y, ys, out, os, T, M, K)


@pytest.mark.parametrize("kw,want", [
    (dict(we=F32), UNSUPPORTED), (dict(xe=F16), UNSUPPORTED), (dict(ye=F16), UNSUPPORTED), (dict(xe=7), UNSUPPORTED), (dict(rank=0), SHAPE),
    (dict(rank=12), SHAPE), (dict(rank=136), SHAPE), (dict(K=48), SHAPE), (dict(K=0), SHAPE), (dict(K=1 << 24), SHAPE), (dict(M=1 << 24), SHAPE),
    (dict(T=(1 << 20) + 1), SHAPE), (dict(n=4097), SHAPE), (dict(T=-1), INVALID), (dict(M=-1), INVALID), (dict(x=None), INVALID), (dict(a=None), INVALID),
    (dict(b=None), INVALID), (dict(ids=None), INVALID), (dict(out=None), INVALID), (dict(x=at(1) + 8), ALIGN), (dict(xs=66), ALIGN),
    (dict(a=at(2) + 8), ALIGN), (dict(out=at(7) + 2), ALIGN), (dict(ids=at(5) + 2), ALIGN), (dict(os=39), INVALID), (dict(xs=-64), INVALID),
    (dict(out=at(1)), INVALID), (dict(out=at(6) + 160), INVALID), (dict(out=at(6), ys=48), INVALID), (dict(out=at(3)), INVALID), (dict(out=at(5)), INVALID),
    (dict(), WORKSPACE)])
def test_lora_refusals(bq, kw, want):
    bq.lib().bq_set_workspace(None, 0)
    assert _lora(bq, **kw) == want


def test_lora_refuses_a_workspace_in_its_arguments(bq):
    L = bq.lib()
    need = L.bq_lora_workspace_size(5, 3, 16, 64, 40)
    assert need >= 5 * 16 * 4 and L.bq_lora_workspace_size(5, 3, 12, 64, 40) == 0
    for base in (at(1), at(2), at(3) + 256, at(5), at(6), at(7)):
        L.bq_set_workspace(base, need)
        assert _lora(bq) == INVALID
    L.bq_set_workspace(None, 0)


def test_lora_of_nothing_is_a_no_op(bq):
    assert _lora(bq, T=0, x=None, out=None) == OK and _lora(bq, M=0, out=None, os=0, ys=0) == OK


@pytest.mark.parametrize("kw,want", [(dict(t=4), UNSUPPORTED), (dict(K=48), SHAPE), (dict(K=65536 + 32), SHAPE), (dict(M=-1), INVALID), (dict(x=None), INVALID),
                                     (dict(x=at(2) + 8), ALIGN), (dict(y=at(2)), INVALID), (dict(y=at(1) + 4), INVALID), (dict(), WORKSPACE)])
def test_q8_gemv_refusals(bq, kw, want):
    a = dict(t=Q8, w=at(1), x=at(2), y=at(3), M=5, K=64)
    a.update(kw)
    bq.lib().bq_set_workspace(None, 0)
    assert bq.lib().bq_gemv_q8(*a.values()) == want


@pytest.mark.parametrize("kw,want", [(dict(t=Q4), UNSUPPORTED), (dict(t=4), UNSUPPORTED), (dict(K=48), SHAPE), (dict(M=1 << 31), SHAPE), (dict(N=-1), INVALID),
                                     (dict(x=None), INVALID), (dict(x=at(2) + 8), ALIGN), (dict(y=at(2)), INVALID), (dict(K=256), WORKSPACE)])
def test_q8_gemm_refusals(bq, kw, want):
    a = dict(t=Q8, w=at(1), x=at(2), y=at(3), M=5, N=3, K=64)
    a.update(kw)
    bq.lib().bq_set_workspace(None, 0)
    assert bq.lib().bq_gemm_q8(*a.values()) == want


def test_wrong_tensors_raise(bq):
    """Tensors of the host are refused before anything else."""
    i = torch.zeros(3, dtype=torch.int32)
    f = torch.zeros(3, 64)
    with pytest.raises(TypeError):
        bq.paged_extend(16, 4, i, i, torch.zeros(3, 2, dtype=torch.int32), i, 4)
    with pytest.raises(TypeError):
        bq.add_rms_norm(f, f[0], 1e-6)
    with pytest.raises(TypeError):
        bq.rotary(f.view(3, 1, 64), None, i, torch.zeros(32, dtype=torch.float64))
    with pytest.raises(TypeError):
        bq.lora(f, f.half().view(1, 3, 64), f.half().view(1, 64, 3), i)


# ------------------------------------------------------------------ extend --


def extend_ref(page, n_pages, kv, new, table, free, n_slots):
    """One sequence and one token at a time."""
    kv, new, free = kv.tolist(), new.tolist(), free.tolist()
    table, wide = table.clone(), table.shape[1]
    starts, out, slots, pos, taken, needed, bad = [0], [], [-1] * n_slots, [0] * n_slots, 0, 0, False
    for b, (have, n) in enumerate(zip(kv, new)):
        start = starts[-1]
        starts.append(start + max(n, 0))
        fits = have >= 0 and n >= 0 and have + n <= wide * page
        need = -(-(have + n) // page) - -(-have // page) if fits else 0
        ok = fits and (n == 0 or start + n <= n_slots) and (need == 0 or needed + need <= len(free))
        if ok:
            for i in range(need):
                if 0 <= free[needed + i] < n_pages:
                    table[b, -(-have // page) + i] = free[needed + i]
            if need:
                taken = needed + need
        needed += need
        bad |= not ok
        out.append(have + n if ok else have)
        for i in range(max(n, 0)):
            if start + i < n_slots:
                p = max(have, 0) + i
                pos[start + i] = p
                if ok:
                    col = p // page
                    first = -(-have // page)
                    entry = free[needed - need + col - first] if col >= first else int(table[b, col])
                    if 0 <= entry < n_pages:
                        slots[start + i] = entry * page + p % page
                    else:
                        bad = True
    return table, starts, out, slots, pos, [taken, needed], bad


def check_extend(bq, page, kv, new, n_slots, n_free=None, wide=None, n_pages=None, seed=0, spoil=None):
    g = torch.Generator().manual_seed(seed)
    kv, new = torch.tensor(kv, dtype=torch.int32), torch.tensor(new, dtype=torch.int32)
    grown = [-(-(max(int(a), 0) + max(int(b), 0)) // page) for a, b in zip(kv, new)]
    owned = [-(-max(int(a), 0) // page) for a in kv]
    wide = wide if wide is not None else max(grown + [1])
    total = sum(grown) + 3
    order = torch.randperm(total, generator=g).int()
    table = torch.full((len(kv), wide), -7, dtype=torch.int32)
    k = 0
    for b, n in enumerate(owned):
        table[b, : min(n, wide)] = order[k: k + min(n, wide)]
        k += n
    free = order[k:]
    if n_free is not None:
        free = free[:n_free]
    if spoil is not None:
        free = free.clone()
        free[spoil] = total + 5
    n_pages = total if n_pages is None else n_pages
    want = extend_ref(page, n_pages, kv, new, table, free, n_slots)
    assert quiet(bq) == OK
    t = table.cuda()
    got = bq.paged_extend(page, n_pages, kv.cuda(), new.cuda(), t, free.cuda(), n_slots)
    assert quiet(bq) == (INDEX if want[-1] else OK)
    assert torch.equal(t.cpu(), want[0])
    for name, w in zip(("q_start", "kv_len", "slots", "positions", "taken"), want[1:]):
        assert getattr(got, name).tolist() == w, name
    return got


@gpu
@pytest.mark.parametrize("page", [16, 48, 1 << 20])
@pytest.mark.parametrize("kv,new,spare", [
    ([0], [1], 0), ([0], [0], 0), ([16], [1], 3), ([15], [1], 0), ([15], [2], 1), ([47, 48, 49], [1, 1, 1], 0),
    ([0, 0, 0], [100, 0, 33], 5), ([5, 0, 200, 31, 32], [0, 0, 7, 1, 0], 0), ([1000], [5000], 100), ([0, 4095, 4096], [1, 1, 1], 2)])
def test_extend(bq, page, kv, new, spare):
    check_extend(bq, page, kv, new, sum(new) + spare)


@gpu
@pytest.mark.parametrize("B,seed", [(1, 1), (33, 2), (511, 3), (512, 4), (513, 5), (5000, 6)])
def test_extend_many_sequences(bq, B, seed):
    r = np.random.default_rng(seed)
    new = r.integers(0, 40, B) * (r.random(B) < 0.7)
    check_extend(bq, 16, r.integers(0, 300, B).tolist(), new.tolist(), int(new.sum()) + int(r.integers(0, 9)), seed=seed)


@gpu
def test_extend_without_sequences(bq):
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    for n_slots in (0, 5):
        got = bq.paged_extend(16, 3, e, e, e.view(0, 4), e, n_slots)
        assert got.q_start.tolist() == [0] and got.slots.tolist() == [-1] * n_slots and got.taken.tolist() == [0, 0]
    assert quiet(bq) == OK


@gpu
@pytest.mark.parametrize("kw", [
    dict(kv=[10, 20, 30], new=[1, -4, 2], n_slots=5),              # a negative length
    dict(kv=[10, -1, 30], new=[1, 4, 2], n_slots=8),
    dict(kv=[10, 100, 30], new=[1, 40, 2], n_slots=50, wide=8),    # longer than the table
    dict(kv=[10, 300, 30], new=[1, 0, 2], n_slots=50, wide=8),
    dict(kv=[16, 16, 5, 32], new=[1, 100, 1, 1], n_slots=103, n_free=4),   # the second needs 7 pages of 4: the last gets none
    dict(kv=[16, 16, 5, 32], new=[1, 1, 1, 1], n_slots=4, n_free=0),
    dict(kv=[16, 16, 5, 32], new=[3, 9, 0, 6], n_slots=11),        # no room for the second's and the last's tokens
    dict(kv=[16, 16], new=[3, 9], n_slots=0),
    dict(kv=[16, 16, 5, 32], new=[1, 40, 1, 1], n_slots=50, spoil=2),      # a free page outside the pool
    dict(kv=[17, 16], new=[20, 1], n_slots=50, n_pages=2),
    dict(kv=[2**31 - 1, 3, 5], new=[1, 2**31 - 1, 1], n_slots=20, wide=4, page=1 << 20)])
def test_extend_that_cannot_grow(bq, kw):
    kw = dict(page=16) | kw
    if kw["page"] == 1 << 20:  # lengths beyond 31 bits: q_start saturates, which the plain form does not
        page = kw["page"]
        t = torch.zeros(3, 4, dtype=torch.int32, device="cuda")
        got = bq.paged_extend(page, 9, torch.tensor(kw["kv"], dtype=torch.int32, device="cuda"), torch.tensor(kw["new"], dtype=torch.int32, device="cuda"),
                              t, torch.arange(1, 9, dtype=torch.int32, device="cuda"), 20)
        assert got.q_start.tolist() == [0, 1, 2**31 - 1, 2**31 - 1] and got.kv_len.tolist() == kw["kv"]
        assert got.slots.tolist() == [-1] * 20 and got.taken.tolist() == [0, 0] and quiet(bq) == INDEX
        return
    check_extend(bq, **kw)


@gpu
def test_extend_on_another_stream_and_captured(bq):
    """A graph of one step, replayed as the lengths are moved on, on a side stream."""
    page, B, wide = 16, 5, 6
    kv = torch.tensor([0, 15, 16, 31, 40], dtype=torch.int32, device="cuda")
    new = torch.tensor([3, 1, 0, 2, 9], dtype=torch.int32, device="cuda")
    order = torch.randperm(30, generator=torch.Generator().manual_seed(1)).int()
    table = torch.full((B, wide), -7, dtype=torch.int32)
    used = 0
    for b, n in enumerate([0, 1, 1, 2, 3]):
        table[b, :n] = order[used: used + n]
        used += n
    free = torch.zeros(30, dtype=torch.int32)
    free[: 30 - used] = order[used:]
    host = [kv.cpu(), table.clone(), order[used:].tolist()]
    table, free = table.cuda(), free.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        bq.paged_extend(page, 30, kv, new, table.clone(), free, 20)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = bq.paged_extend(page, 30, kv, new, table, free, 20)
        for _ in range(3):
            graph.replay()
            left = torch.tensor(host[2], dtype=torch.int32)
            want = extend_ref(page, 30, host[0], new.cpu(), host[1], left, 20)
            side.synchronize()
            assert torch.equal(table.cpu(), want[0]) and got.slots.tolist() == want[3] and got.kv_len.tolist() == want[2]
            host = [torch.tensor(want[2], dtype=torch.int32), want[0], host[2][want[5][0]:]]
            kv.copy_(got.kv_len)
            new.fill_(1)
            free.zero_()
            free[: len(host[2])] = torch.tensor(host[2], dtype=torch.int32, device="cuda")
    torch.cuda.current_stream().wait_stream(side)


# -------------------------------------------------------------------- norm --


def norm_ref(x, res, w, eps):
    """h, y in fp32 from a 64-bit sum, and y's Q8_0 blocks as bytes (numpy)."""
    h = x if res is None else (x.float() + res.float()).to(x.dtype)
    v = h.float().numpy()
    f = (1.0 / np.sqrt((v.astype(np.float64) ** 2).mean(-1, keepdims=True) + eps)).astype(np.float32)
    y = (v * f) * w.numpy()
    b = y.reshape(y.shape[0], -1, 32)
    amax = np.abs(b).max(-1, keepdims=True)
    d = (amax / np.float32(127)).astype(np.float16)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(d > 0, np.rint(b / d.astype(np.float32)), 0)
    q = np.clip(q, -127, 127).astype(np.int8)
    blocks = np.concatenate([d.view(np.uint8).reshape(*d.shape[:2], 2), q.view(np.uint8)], -1)
    return h, torch.from_numpy(y), torch.from_numpy(blocks.reshape(y.shape[0], -1))


def norm_rows(rows, cols, dtype, seed, kind="plain"):
    g = torch.Generator().manual_seed(seed)
    x, r = torch.randn(rows, cols, generator=g), torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(1, cols, generator=g))
    w = 1 + 0.3 * torch.randn(cols, generator=g)
    if kind == "zero":
        x, r = x * 0, r * 0
    elif kind == "tiny":
        x, r = x * 1e-6, r * 1e-6
    elif kind == "large":
        x, r = x * 500, r * 100
    elif kind == "spike":
        x[:, cols // 2] = 3e4
    return x.to(dtype), r.to(dtype), w


@gpu
@pytest.mark.parametrize("elem", [F32, F16, BF16])
@pytest.mark.parametrize("rows,cols", [(1, 32), (5, 64), (3, 256), (7, 288), (2, 1024), (9, 1056), (4, 4096), (3, 4128), (2, 11008), (1, 16384), (2, 32800), (1, 65536)])
@pytest.mark.parametrize("residual", [True, False])
def test_norm(bq, elem, rows, cols, residual):
    x, r, w = norm_rows(rows, cols, DT[elem], rows + cols)
    r = r if residual else None
    h, y, blocks = norm_ref(x, r, w, 1e-6)
    got = bq.add_rms_norm(x.cuda(), w.cuda(), 1e-6, None if r is None else r.cuda(), q8=True)
    assert torch.equal(got.out.cpu(), y.to(x.dtype))
    assert torch.equal(got.q8.cpu(), blocks)
    assert got.sum is None if r is None else torch.equal(got.sum.cpu(), h)


@gpu
@pytest.mark.parametrize("elem", [F32, F16, BF16])
@pytest.mark.parametrize("kind", ["zero", "tiny", "large", "spike"])
@pytest.mark.parametrize("eps", [1e-6, 1e-30, 0.25])
def test_norm_of_odd_values(bq, elem, kind, eps):
    x, r, w = norm_rows(4, 544, DT[elem], 3, kind)
    h, y, blocks = norm_ref(x, r, w, eps)
    got = bq.add_rms_norm(x.cuda(), w.cuda(), eps, r.cuda(), q8=True)
    assert torch.equal(got.sum.cpu(), h) and torch.equal(got.out.cpu(), y.to(x.dtype)) and torch.equal(got.q8.cpu(), blocks)


@gpu
@pytest.mark.parametrize("elem", [F32, BF16])
@pytest.mark.parametrize("power,eps", [(47, 1e-6), (47, 1e30), (-60, 1e-30), (-20, 1e-30)])
@pytest.mark.parametrize("cols", [64, 4096, 65536])
def test_norm_at_the_ends_of_its_range(bq, elem, power, eps, cols):
    """|h| near 2^50 and far below the smallest eps."""
    x, _, w = norm_rows(3, cols, torch.float32, cols)
    x = (x.clamp(-7.9, 7.9) * 2.0**power).to(DT[elem])
    h, y, blocks = norm_ref(x, None, w, eps)
    got = bq.add_rms_norm(x.cuda(), w.cuda(), eps, q8=True)
    assert torch.equal(got.out.cpu(), y.to(x.dtype)) and torch.equal(got.q8.cpu(), blocks)


@gpu
@pytest.mark.parametrize("elem", [F32, BF16])
def test_norm_strides_in_place_and_given_outputs(bq, elem):
    x, r, w = norm_rows(6, 320, DT[elem], 4)
    h, y, blocks = norm_ref(x, r, w, 1e-5)
    wide = torch.full((6, 352), 7.0, dtype=x.dtype, device="cuda")
    xs, out = wide[:, 16:336], torch.full((6, 640), 9.0, dtype=x.dtype, device="cuda")
    xs.copy_(x)
    stream, q8 = r.cuda(), torch.zeros_like(blocks, device="cuda")
    got = bq.add_rms_norm(xs, w.cuda(), 1e-5, stream, out=out[:, :320], q8=q8, sum=stream)
    assert torch.equal(stream.cpu(), h) and torch.equal(out[:, :320].cpu(), y.to(x.dtype)) and torch.equal(q8.cpu(), blocks)
    assert (out[:, 320:] == 9).all() and got.sum.data_ptr() == stream.data_ptr()
    got = bq.add_rms_norm(xs, w.cuda(), 1e-5, r.cuda(), out=False, q8=False, sum=xs)  # onto x
    assert got.out is None and got.q8 is None and torch.equal(xs.cpu(), h)
    assert (wide[:, :16] == 7).all() and (wide[:, 336:] == 7).all()


@gpu
@pytest.mark.parametrize("kind", [2, 3, 6, 7, 8, 12, 14])
@pytest.mark.parametrize("M,K", [(37, 256), (64, 4096), (19, 2048), (33, 96), (8, 65536)])
def test_gemv_of_q8_activations(bq, kind, M, K):
    """Bit for bit what the quantizer inside the call leads to."""
    if K % bq.block_values(kind):
        pytest.skip("k-quants hold whole super-blocks")
    g = torch.Generator(device="cuda").manual_seed(M + K)
    w = bq.quantize_rows(kind, torch.randn(M, K, generator=g, device="cuda"))
    x = torch.randn(K, generator=g, device="cuda")
    xq = bq.quantize_rows(Q8, x[None])
    assert torch.equal(bq.gemv(kind, w, xq, M, K), bq.gemv(kind, w, x, M, K))
    from block_quantized_weight_row_gb300 import binding
    binding.set_weight_prefetch(True)
    try:
        assert torch.equal(bq.gemv(kind, w, xq, M, K), bq.gemv(kind, w, x, M, K))
    finally:
        binding.set_weight_prefetch(False)


@gpu
@pytest.mark.parametrize("M,N,K", [(64, 8, 256), (130, 1, 512), (300, 129, 1024), (70, 257, 96), (33, 3, 32)])
def test_gemm_of_q8_activations(bq, M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    w = bq.quantize_rows(Q8, torch.randn(M, K, generator=g, device="cuda"))
    x = torch.randn(N, K, generator=g, device="cuda")
    xq = bq.quantize_rows(Q8, x)
    assert torch.equal(bq.gemm(Q8, w, xq, M, N, K), bq.gemm(Q8, w, x, M, N, K))
    with pytest.raises(ValueError):
        bq.gemm(Q8, w, xq[:, :-1].contiguous(), M, N, K)


# ------------------------------------------------------------------ rotary --


def rotary_ref(x, pos, freq, axis, interleaved, sign=1.0):
    """64-bit rotation of (tokens, heads, dim)."""
    x, n = x.double().clone(), len(freq)
    theta = pos.double()[axis.long()].T * freq
    c, s = theta.cos()[:, None], sign * theta.sin()[:, None]
    i = torch.arange(n)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    a, b = x[..., ia].clone(), x[..., ib].clone()
    x[..., ia], x[..., ib] = a * c - b * s, a * s + b * c
    mag = torch.zeros_like(x)
    mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    return x, mag


def check_rotary(got, x, pos, freq, axis, interleaved, sign=1.0):
    """sin and cos 2 ulp and the angle 2^-31 of a turn (2 pi 2^-31 < 2^-28), 2^-22 together; products and sum 3 roundings; then the type's."""
    ref, mag = rotary_ref(x, pos, freq, axis, interleaved, sign)
    tol = (2**-22 + 3 * 2**-24) * mag + torch.finfo(got.dtype).eps / 2 * ref.abs() + 1e-7 * (got.dtype == torch.float16)
    assert ((got.cpu().double() - ref).abs() <= tol).all(), float(((got.cpu().double() - ref).abs() - tol).max())


@gpu
@pytest.mark.parametrize("types", [(F32, F32), (F32, F16), (F32, BF16), (F16, F16), (BF16, BF16)])
@pytest.mark.parametrize("dim,rot", [(128, 128), (64, 64), (96, 72), (256, 64), (128, 74), (32, 2), (96, 48), (64, 0), (160, 160), (128, 96)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary(bq, types, dim, rot, interleaved):
    g = torch.Generator().manual_seed(dim + rot)
    T, H, KH, A = 7, 3, 2, 3
    q, k = torch.randn(T, H, dim, generator=g).to(DT[types[0]]), torch.randn(T, KH, dim, generator=g).to(DT[types[0]])
    pos = torch.randint(-(2**31), 2**31, (A, T), generator=g).int()
    pos[:, :3] = torch.tensor([[0, 1, 5], [2, 3, 4], [-1, 7, 100]], dtype=torch.int32)
    freq = 10000.0 ** -(torch.arange(rot // 2).double() / max(rot // 2, 1))
    axis = torch.randint(0, A, (rot // 2,), generator=g).int()
    # positions of 31 bits: a 64-bit angle is off by 2^31 2^-53 itself, 2^-22, so the reference's is taken from whole numbers
    near = pos.long() % 1000003
    a, b = bq.rotary(q.cuda(), k.cuda(), near.int().cuda(), freq.cuda(), axis.cuda(), interleaved=interleaved, dtype=DT[types[1]])
    check_rotary(a, q, near, freq, axis, interleaved)
    check_rotary(b, k, near, freq, axis, interleaved)
    a, _ = bq.rotary(q.cuda(), None, near.int().cuda(), freq.cuda(), axis.cuda(), interleaved=interleaved, inverse=True, dtype=DT[types[1]])
    check_rotary(a, q, near, freq, axis, interleaved, -1.0)


@gpu
def test_rotary_of_far_positions(bq):
    """Frequencies that are whole fractions of a turn: the angle of any position is known exactly."""
    T, n = 64, 16
    g = torch.Generator().manual_seed(2)
    turns = torch.randint(1, 2**20, (n,), generator=g)  # of 2^-20 turns per position
    freq = turns.double() * 2**-20 * (2 * math.pi)
    pos = torch.randint(-(2**31), 2**31, (1, T), generator=g)
    q = torch.randn(T, 2, 32, generator=g)
    got, _ = bq.rotary(q.cuda(), None, pos.int().cuda(), freq.cuda())
    angle = (pos.T * turns % 2**20).double() * (2 * math.pi / 2**20)  # 51 bits: exact before the product
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    x = q.double()
    ref = torch.cat((x[..., :n] * c - x[..., n:] * s, x[..., :n] * s + x[..., n:] * c), -1)
    # freq has 53 bits, and so has its quotient by 2 pi: 2^31 * 2^-52 of a turn, 2^-18 in radians
    assert ((got.cpu().double() - ref).abs() <= 2 * math.pi * 2**-20 * 4).all()


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [128, 96, 74])
def test_rotary_in_place_strides_and_back(bq, interleaved, rot):
    """q and k as slices of one projection, turned in place and back."""
    g = torch.Generator(device="cuda").manual_seed(3)
    T, H, KH, D = 9, 4, 2, 128
    qkv = torch.randn(T, H + 2 * KH, D, generator=g, device="cuda").bfloat16()
    was = qkv.clone()
    q, k = qkv[:, :H], qkv[:, H:H + KH]
    pos = torch.randint(0, 5000, (2, T), generator=g, device="cuda", dtype=torch.int32)
    freq = (10000.0 ** -(torch.arange(rot // 2).double() / (rot // 2))).cuda()
    axis = (torch.arange(rot // 2, device="cuda") % 2).int()
    a, b = bq.rotary(q, k, pos, freq, axis, interleaved=interleaved)
    c, d = bq.rotary(q, k, pos, freq, axis, interleaved=interleaved, out_q=q, out_k=k)
    assert c.data_ptr() == q.data_ptr() and torch.equal(q, a) and torch.equal(k, b) and torch.equal(qkv[:, H + KH:], was[:, H + KH:])
    check_rotary(a, was[:, :H].cpu(), pos.cpu(), freq.cpu(), axis.cpu(), interleaved)
    check_rotary(b, was[:, H:H + KH].cpu(), pos.cpu(), freq.cpu(), axis.cpu(), interleaved)
    bq.rotary(q, k, pos, freq, axis, interleaved=interleaved, inverse=True, out_q=q, out_k=k)
    # two roundings to bf16, of values up to sqrt(2) the pair's larger one
    assert ((qkv.float() - was.float()).abs() <= 4 * 2**-8 * was.float().abs().amax(-1, keepdim=True)).all()
    # heads before tokens, the outputs of both in one buffer
    both = torch.zeros(H + KH, T + 1, D, dtype=torch.bfloat16, device="cuda")
    oq, ok = both[:H, :T].transpose(0, 1), both[H:, :T].transpose(0, 1)
    bq.rotary(was[:, :H], was[:, H:H + KH], pos, freq, axis, interleaved=interleaved, out_q=oq, out_k=ok)
    assert torch.equal(oq, a) and torch.equal(ok, b) and (both[:, T] == 0).all()


@gpu
@pytest.mark.parametrize("elem", [F32, BF16])
@pytest.mark.parametrize("dim,rot", [(96, 74), (256, 74), (128, 10), (32, 6), (160, 154)])
def test_rotary_of_odd_halves(bq, elem, dim, rot):
    """Halves on no 16-byte boundary, heads of any number of units: apart, on q alone and on both, the same bits."""
    g = torch.Generator(device="cuda").manual_seed(dim + rot)
    T, H, KH = 13, 3, 2
    q, k = (torch.randn(T, n, dim, generator=g, device="cuda").to(DT[elem]) for n in (H, KH))
    pos = torch.randint(0, 9000, (T,), generator=g, device="cuda", dtype=torch.int32)
    freq = (10000.0 ** -(torch.arange(rot // 2).double() / (rot // 2))).cuda()
    a, b = bq.rotary(q, k, pos, freq)
    axis = torch.zeros(rot // 2, dtype=torch.int32)
    check_rotary(a, q.cpu(), pos[None].cpu(), freq.cpu(), axis, False)
    check_rotary(b, k.cpu(), pos[None].cpu(), freq.cpu(), axis, False)
    c, d = bq.rotary(q, k, pos, freq, out_k=k.clone())
    q2, k2 = q.clone(), k.clone()
    _, f = bq.rotary(q2, k, pos, freq, out_q=q2)
    assert torch.equal(c, a) and torch.equal(d, b) and torch.equal(q2, a) and torch.equal(f, b)
    bq.rotary(q, k2, pos, freq, out_q=q, out_k=k2)
    assert torch.equal(q, a) and torch.equal(k2, b)


@gpu
@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16), (F16, F16), (F32, BF16)])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("rot", [2, 6, 10, 74, 126])
def test_rotary_leaves_the_other_channels(bq, types, interleaved, rot):
    """Channels behind `rot` are copies, whatever stands beside them: infinities, zeros of either sign."""
    T, H, dim = 7, 2, 128
    g = torch.Generator().manual_seed(rot)
    q = torch.randn(T, H, dim, generator=g)
    odd = torch.tensor([math.inf, -1.5, -0.0, -2.0, 0.0, -math.inf, 3.0])
    q[..., rot:] = odd[torch.randint(0, 7, (T, H, dim - rot), generator=g)]
    q = q.to(DT[types[0]])
    pos = torch.randint(-50, 9000, (T,), generator=g, dtype=torch.int32).cuda()
    freq = (10000.0 ** -(torch.arange(rot // 2).double() / (rot // 2))).cuda()
    rest = q[..., rot:].to(DT[types[1]])
    want = rest.view(torch.int32 if types[1] == F32 else torch.int16)
    out, _ = bq.rotary(q.cuda(), None, pos, freq, interleaved=interleaved, dtype=DT[types[1]])
    assert torch.equal(out[..., rot:].contiguous().cpu().view(want.dtype), want)
    assert bool(out[..., :rot].isfinite().all())
    if types[0] == types[1]:
        own = q.cuda()
        bq.rotary(own, None, pos, freq, interleaved=interleaved, out_q=own)
        assert torch.equal(own.cpu().view(want.dtype), out.cpu().view(want.dtype))


@gpu
def test_rotary_bad_axis_and_one_axis(bq):
    assert quiet(bq) == OK
    q = torch.randn(3, 1, 64, device="cuda")
    pos = torch.tensor([[1, 2, 3], [4, 5, 6]], dtype=torch.int32, device="cuda")
    freq = torch.full((32,), 0.1, dtype=torch.float64, device="cuda")
    first, _ = bq.rotary(q, None, pos, freq)
    assert torch.equal(first, bq.rotary(q, None, pos[0], freq)[0]) and quiet(bq) == OK
    axis = torch.zeros(32, dtype=torch.int32, device="cuda")
    axis[3], axis[4] = 2, -1
    assert torch.equal(first, bq.rotary(q, None, pos, freq, axis)[0]) and quiet(bq) == INDEX


# ---------------------------------------------------------------- adapters --


def lora_case(T, n, rank, K, M, x, w, y, ids, seed=0):
    g = torch.Generator().manual_seed(seed)
    X = torch.randn(T, K, generator=g).to(DT[x])
    A = (torch.randn(n, rank, K, generator=g) / math.sqrt(K)).to(DT[w])
    B = (0.3 * torch.randn(n, M, rank, generator=g)).to(DT[w])
    s = torch.rand(n, generator=g) + 0.5
    Y = torch.randn(T, M, generator=g).to(DT[y])
    if ids == "random":
        ids = torch.randint(-1, n, (T,), generator=g).int()
    elif ids == "runs":
        ids = torch.randint(-1, n, (T,), generator=g).int().sort().values
    elif ids == "same":
        ids = torch.full((T,), n - 1, dtype=torch.int32)
    elif ids == "none":
        ids = torch.full((T,), -1, dtype=torch.int32)
    return X, A, B, s, Y, ids


def check_lora(got, X, A, B, s, Y, ids):
    ids = torch.where((ids >= 0) & (ids < len(A)), ids, -1)
    u, K, rank = 2.0**-24, X.shape[1], A.shape[1]
    half = A.dtype == torch.float16
    terms = 1 if X.dtype != torch.float32 else 4 if half else 3
    y32 = got.dtype == torch.float32
    terms2 = 2 if half or not y32 else 3
    ref = Y.double().clone() if Y is not None else torch.zeros(got.shape, dtype=torch.float64)
    tol = torch.zeros_like(ref)
    for a in ids.unique().tolist():
        if a < 0:
            continue
        i = ids == a
        x, A64, B64, f = X[i].double(), A[a].double(), B[a].double(), float(s[a]) if s is not None else 1.0
        h, hm = f * (x @ A64.T), f * (x.abs() @ A64.abs().T)
        ref[i] += h @ B64.T
        eh = hm * ((4 * 2 * terms * -(-K // 32) + 37) * u + (2**-22 if terms == 4 else 0))
        kept = 2**-22 if half or y32 else 2**-18
        eh = eh + kept * h.abs() + (2**-24 * h.abs().amax(-1, keepdim=True) if half else 0)
        tol[i] = eh @ B64.abs().T + 4 * 2 * terms2 * -(-rank // 32) * u * (h.abs() @ B64.abs().T)
    tol += 2 * u * ref.abs() + torch.finfo(got.dtype).eps / 2 * ref.abs() + (2**-25 if got.dtype == torch.float16 else 0)
    err = (got.cpu().double() - ref).abs()
    assert (err <= tol).all(), (float((err - tol).max()), int((err > tol).sum()))
    none = ids < 0
    if Y is not None and none.any():
        assert torch.equal(got.cpu()[none], Y[none])


def run_lora(bq, X, A, B, s, Y, ids, **kw):
    c = [None if t is None else t.cuda() for t in (X, A, B, ids, Y, s)]
    return bq.lora(*c, **kw)


TYPES = [(F32, BF16, F32), (BF16, BF16, BF16), (BF16, BF16, F32), (F32, BF16, BF16), (F16, F16, F16), (F32, F16, F32), (F16, F16, F32), (F32, F16, F16)]


@gpu
@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("T,n,rank,K,M,ids", [(1, 1, 8, 32, 32, "same"), (1, 3, 16, 128, 40, "same"), (5, 2, 24, 96, 1, "random"), (17, 4, 16, 256, 33, "random"),
                                              (48, 16, 16, 1024, 300, "random"), (256, 3, 64, 512, 129, "same"), (200, 64, 32, 64, 65, "random"),
                                              (33, 1, 128, 160, 96, "same"), (16, 5, 40, 4096, 257, "random")])
def test_lora_few_tokens(bq, types, T, n, rank, K, M, ids):
    c = lora_case(T, n, rank, K, M, *types, ids)
    check_lora(run_lora(bq, *c), *c)


@gpu
@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("T,n,rank,K,M,ids", [(257, 1, 16, 64, 40, "same"), (300, 64, 24, 256, 131, "random"), (1000, 3, 64, 512, 200, "runs"),
                                              (1025, 7, 128, 96, 264, "random"), (2500, 2000, 8, 32, 33, "random"), (700, 4, 40, 2048, 77, "runs"),
                                              (4100, 5, 32, 288, 520, "random")])
def test_lora_many_tokens(bq, types, T, n, rank, K, M, ids):
    c = lora_case(T, n, rank, K, M, *types, ids, seed=T)
    check_lora(run_lora(bq, *c), *c)


@gpu
@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("T,n,rank,K,M,ids", [(2100, 2, 24, 32, 50, "runs"), (1100, 1, 128, 32, 257, "same"), (1300, 3, 72, 160, 66, "random"),
                                              (900, 2, 104, 416, 130, "random"), (1500, 2, 48, 1376, 64, "runs"), (800, 1, 64, 4096, 40, "same")])
def test_lora_large_tiles(bq, types, T, n, rank, K, M, ids):
    """Tiles of 64 tokens: one stage of 32 k and many, ranks on both sides of 64, K split over a cluster."""
    c = lora_case(T, n, rank, K, M, *types, ids, seed=T)
    check_lora(run_lora(bq, *c), *c)


@gpu
@pytest.mark.parametrize("T", [20, 600])
def test_lora_without_base_scale_or_adapter(bq, T):
    X, A, B, s, Y, ids = lora_case(T, 3, 16, 128, 70, F32, BF16, F32, "random")
    check_lora(run_lora(bq, X, A, B, None, Y, ids), X, A, B, None, Y, ids)
    got = run_lora(bq, X, A, B, s, None, ids)
    check_lora(got, X, A, B, s, None, ids)
    assert (got.cpu()[ids < 0] == 0).all()
    assert run_lora(bq, X, A, B, s, None, ids, dtype=torch.bfloat16).dtype == torch.bfloat16
    none = torch.full((T,), -1, dtype=torch.int32)
    assert torch.equal(run_lora(bq, X, A, B, s, Y, none).cpu(), Y)
    assert torch.equal(run_lora(bq, X, A[:0], B[:0], s[:0], Y, none).cpu(), Y)


@gpu
@pytest.mark.parametrize("T", [40, 500])
def test_lora_in_place_strides_and_odd_rows(bq, T):
    """y's rows in a wider buffer, on no boundary of 16 bytes; out onto y."""
    for y, off, extra in ((F32, 1, 3), (BF16, 3, 5), (BF16, 8, 8), (F32, 4, 0)):
        X, A, B, s, Y, ids = lora_case(T, 3, 32, 128, 99, F32, BF16, y, "random")
        wide = torch.full((T, off + 99 + extra), 5.0, dtype=DT[y], device="cuda")
        view = wide[:, off:off + 99]
        view.copy_(Y)
        xw = torch.zeros(T, 136, device="cuda")
        xw[:, :128] = X.cuda()
        got = bq.lora(xw[:, :128], A.cuda(), B.cuda(), ids.cuda(), view, s.cuda(), out=view)
        assert got.data_ptr() == view.data_ptr()
        check_lora(got, X, A, B, s, Y, ids)
        assert (wide[:, :off] == 5).all() and (wide[:, off + 99:] == 5).all()


@gpu
@pytest.mark.parametrize("T", [40, 500])
def test_lora_adapters_out_of_range(bq, T):
    assert quiet(bq) == OK
    X, A, B, s, Y, ids = lora_case(T, 3, 16, 64, 40, F32, BF16, F32, "random")
    ids[3], ids[T - 1], ids[7] = 3, -2, 2**31 - 1
    got = run_lora(bq, X, A, B, s, Y, ids)
    assert quiet(bq) == INDEX
    check_lora(got, X, A, B, s, Y, ids)


@gpu
@pytest.mark.parametrize("T", [48, 900])
def test_lora_rows_do_not_see_each_other(bq, T):
    """The same bits in any order of the tokens, every time, with NaN and infinities in other rows."""
    X, A, B, s, Y, ids = lora_case(T, 4, 16, 256, 70, BF16, BF16, F32, "random")
    first = run_lora(bq, X, A, B, s, Y, ids).cpu()
    p = torch.randperm(T, generator=torch.Generator().manual_seed(5))
    assert torch.equal(run_lora(bq, X[p], A, B, s, Y[p], ids[p]).cpu(), first[p])
    X[5], X[11] = math.inf, math.nan
    got = run_lora(bq, X, A, B, s, Y, ids).cpu()
    keep = torch.ones(T, dtype=torch.bool)
    keep[5] = keep[11] = False
    assert torch.equal(got[keep], first[keep])


@gpu
@pytest.mark.parametrize("xe,we,ye,rank", [(BF16, BF16, F32, 64), (BF16, BF16, BF16, 40), (BF16, BF16, BF16, 128), (F32, BF16, F32, 48), (F32, BF16, BF16, 120),
                                           (F32, F16, F32, 64), (F16, F16, F16, 104)])
def test_lora_large_tiles_do_not_see_each_other(bq, xe, we, ye, rank):
    """As above, in tiles of 64 tokens of every type."""
    T = 1100
    X, A, B, s, Y, ids = lora_case(T, 3, rank, 288, 130, xe, we, ye, "random")
    first = run_lora(bq, X, A, B, s, Y, ids).cpu()
    p = torch.randperm(T, generator=torch.Generator().manual_seed(6))
    assert torch.equal(run_lora(bq, X[p], A, B, s, Y[p], ids[p]).cpu(), first[p])
    X[5, 3], X[11], X[700, 100] = math.inf, math.nan, -math.inf
    got = run_lora(bq, X, A, B, s, Y, ids).cpu()
    keep = torch.ones(T, dtype=torch.bool)
    keep[5] = keep[11] = keep[700] = False
    assert torch.equal(got[keep], first[keep])


@gpu
@pytest.mark.parametrize("T", [1, 40, 256, 300, 1200])
@pytest.mark.parametrize("rank", [8, 64])
def test_lora_without_any_adapter(bq, T, rank):
    """Nobody has one: y as it is, in place and apart, zeros without y; the next call on the stream sees them."""
    X, A, B, s, Y, _ = (t.cuda() for t in lora_case(T, 3, rank, 288, 130, BF16, BF16, F32, "random"))
    ids = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    want = Y.clone()
    for _ in range(3):
        assert bq.lora(X, A, B, ids, Y, s, out=Y) is not None
        X.zero_()
    assert torch.equal(Y, want) and torch.equal(bq.lora(X, A, B, ids, Y, s), want)
    assert not bool(bq.lora(X, A, B, ids, None, s, dtype=torch.float32).any())


@gpu
@pytest.mark.parametrize("T", [30, 700])
def test_lora_captured_and_on_many_streams(bq, T):
    X, A, B, s, Y, ids = (t.cuda() for t in lora_case(T, 4, 16, 256, 70, F32, BF16, F32, "random"))
    first = bq.lora(X, A, B, ids, Y, s)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(3)], []
    for _ in range(3):
        for st in streams:
            with torch.cuda.stream(st):
                outs.append(bq.lora(X, A, B, ids, Y, s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = bq.lora(X, A, B, ids, Y, s)
        graphs.append((g, out))
    other = torch.randint(-1, 4, (T,), generator=torch.Generator(device="cuda").manual_seed(9), device="cuda", dtype=torch.int32)
    want = bq.lora(X, A, B, other, Y, s)
    ids.copy_(other)
    torch.cuda.synchronize()
    for st, (g, _) in zip(streams, graphs):  # two graphs at once
        with torch.cuda.stream(st):
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for _, out in graphs)
