"""The calls around a served layer at the sizes whose kernels and branches small batches
do not reach, each against its formula: rows beyond a resident grid, thousands of
sequences, several tokens per CTA, several turns per tile, tiles of 64 tokens in every form."""
import math

import numpy as np
import pytest
import torch

from test_layer_ops import BF16, DT, F16, F32, INDEX, OK, TYPES, bq, check_lora, lora_case, quiet, run_lora  # noqa: F401

pytestmark = pytest.mark.gpu


# -------------------------------------------------------------------- norm --


def norm_formula(x, res, w, eps):
    """The sum, the norm's fp32 values and their Q8_0 blocks as bytes; and which rows' factor lies so far from a border of rounding that
    the kernel's sum, exact to 2^-44, cannot be on the other side of it."""
    h = x if res is None else (x.float() + res.float()).to(x.dtype)
    f = 1.0 / torch.sqrt(h.double().square().mean(-1, keepdim=True) + eps)
    certain = ((f * (1 - 2.0**-42)).float() == (f * (1 + 2.0**-42)).float()).flatten()
    y = (h.float() * f.float()) * w
    b = y.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    d = (amax / torch.full_like(amax, 127.0)).half()  # a tensor divisor: one division, rounded once
    q = torch.where(d > 0, (b / d.float()).round(), torch.zeros_like(b)).clamp(-127, 127).to(torch.int8)
    blocks = torch.cat((d.view(torch.uint8), q.view(torch.uint8)), -1).flatten(1)
    return h, y, blocks, certain


@pytest.mark.parametrize("elem", [F32, F16, BF16])
@pytest.mark.parametrize("rows,cols", [(20000, 64), (20011, 256), (9000, 288), (9001, 512), (9001, 544), (9003, 1024), (5000, 1376), (5001, 2048),
                                       (3001, 2080), (6001, 4096), (3000, 4128), (3001, 8192), (1500, 8224), (1501, 16384), (800, 16416), (400, 65536)])
def test_norm_of_many_rows(bq, elem, rows, cols):  # noqa: F811
    """Every kernel of the norm, each CTA with several rows: with a residual, onto x, onto the residual and without one."""
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=g, device="cuda").to(DT[elem])
    r = (torch.randn(rows, cols, generator=g, device="cuda") * torch.exp(torch.randn(1, cols, generator=g, device="cuda"))).to(DT[elem])
    w = 1 + 0.3 * torch.randn(cols, generator=g, device="cuda")
    h, y, blocks, certain = norm_formula(x, r, w, 1e-6)
    assert int((~certain).sum()) <= 3 + (rows >> 14)
    out = y.to(x.dtype)
    for onto in (None, "x", "residual"):
        a, b = x.clone(), r.clone()
        got = bq.add_rms_norm(a, w, 1e-6, b, q8=True, sum={"x": a, "residual": b}.get(onto))
        assert torch.equal(got.sum, h) and torch.equal(got.out[certain], out[certain]) and torch.equal(got.q8[certain], blocks[certain])
    assert torch.equal(bq.add_rms_norm(x, w, 1e-6, r, q8=False).out, got.out)
    assert torch.equal(bq.add_rms_norm(x, w, 1e-6, r, out=False, q8=True).q8, got.q8)
    _, y, blocks, certain = norm_formula(x, None, w, 1e-6)
    got = bq.add_rms_norm(x, w, 1e-6, q8=True)
    assert got.sum is None and torch.equal(got.out[certain], y.to(x.dtype)[certain]) and torch.equal(got.q8[certain], blocks[certain])


# ------------------------------------------------------------------ extend --


def extend_formula(page, n_pages, kv, new, table, free, n_slots):
    """All sequences and tokens at once, in whole numbers of 64 bits."""
    def ceil(v):
        return (v + page - 1) // page

    wide = table.shape[1]
    have, n = np.maximum(kv, 0), np.maximum(new, 0)
    ok = (kv >= 0) & (new >= 0) & (kv + new <= wide * page)
    owned = ceil(have)
    need = np.where(ok, ceil(have + n) - owned, 0)
    ends, base = np.cumsum(n), np.cumsum(need) - need
    gets = ok & ((n == 0) | (ends <= n_slots)) & ((need == 0) | (base + need <= len(free)))
    taken = int((base + need)[gets & (need > 0)].max(initial=0))
    seq = np.repeat(np.arange(len(kv)), n)[:n_slots]
    at = have[seq] + np.arange(len(seq)) - (ends - n)[seq]
    col = at // page
    fresh = col >= owned[seq]
    live = gets[seq]
    entry = np.where(fresh, free[np.where(live & fresh, base[seq] + col - owned[seq], 0)], table[seq, np.where(live, col, 0)])
    good = (entry >= 0) & (entry < n_pages)
    slots, pos = np.full(n_slots, -1, np.int64), np.zeros(n_slots, np.int64)
    slots[: len(seq)] = np.where(live & good, entry * page + at % page, -1)
    pos[: len(seq)] = at
    table = table.copy()
    put = live & fresh & good
    table[seq[put], col[put]] = entry[put]
    bad = not gets.all() or bool((live & ~good).any())
    return {"q_start": np.concatenate(([0], ends)), "kv_len": np.where(gets, kv + new, kv), "slots": slots, "positions": pos,
            "taken": np.array([taken, need.sum()])}, table, bad


@pytest.mark.parametrize("B,max_kv,max_new,page,short", [
    (40000, 60, 9, 16, None),              # several groups of 32 sequences to a chunk
    (1 << 20, 40, 2, 16, None),            # the most sequences
    (33000, 100, 3, 48, "pages"),
    (70000, 50, 5, 16, "slots"),
    (900, 3000, 900, 16, None),            # above 311 000 rows: tiles of 4096
    (300, 5000, 5000, 64, None),           # 750 000: a CTA's second tile
    (8192, 2048, 300, 16, None),           # 1 200 000
    (8192, 2048, 300, 16, "pages"), (8192, 2048, 300, 48, "slots"), (8192, 2048, 300, 32, "lengths"),
    (1, 100000, 1500000, 128, None),       # one sequence over all tiles
    (2000, 10, 1, 16, None)])              # tiles of 2048
def test_extend_of_large_batches(bq, B, max_kv, max_new, page, short):  # noqa: F811
    r = np.random.default_rng(B + page)
    kv, new = r.integers(0, max_kv + 1, B), r.integers(0, max_new + 1, B) * (r.random(B) < 0.9)
    new[0] = max_new
    wide = int(-(-(kv + new).max() // page))
    owned, total = -(-kv // page), -(-(kv + new) // page)
    if short == "lengths":
        kv[r.integers(0, B, 9)] = -1
        new[r.integers(0, B, 9)] = wide * page + 1
    n_pages = int(total.sum()) + 5
    order = r.permutation(n_pages).astype(np.int64)
    table = np.full((B, wide), -7, np.int64)
    table[np.arange(wide) < owned[:, None]] = order[: owned.sum()]
    free = order[owned.sum():]
    n_slots = int(np.maximum(new, 0).sum()) + 77
    if short == "pages":
        free = free[: len(free) * 2 // 3]
    if short == "slots":
        n_slots = n_slots * 2 // 3
    want, grown, bad = extend_formula(page, n_pages, kv, new, table, free, n_slots)
    assert bad == (short is not None)
    assert quiet(bq) == OK
    t = torch.from_numpy(table).int().cuda()
    got = bq.paged_extend(page, n_pages, torch.from_numpy(kv).int().cuda(), torch.from_numpy(new).int().cuda(), t, torch.from_numpy(free).int().cuda(), n_slots)
    assert quiet(bq) == (INDEX if bad else OK)
    for name, right in want.items():
        assert np.array_equal(getattr(got, name).cpu().numpy(), right), name
    assert np.array_equal(t.cpu().numpy(), grown)


# ------------------------------------------------------------------ rotary --


def rotary_formula(x, pos, freq, axis, interleaved):
    """64-bit rotation, and the magnitude its roundings are relative to."""
    x, n = x.double().clone(), len(freq)
    theta = pos.double()[axis.long()].T * freq
    c, s = theta.cos()[:, None], theta.sin()[:, None]
    i = torch.arange(n, device=x.device)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    a, b = x[..., ia], x[..., ib]
    mag = torch.zeros_like(x)
    mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    x[..., ia], x[..., ib] = a * c - b * s, a * s + b * c
    return x, mag


def check_rotary(got, x, pos, freq, axis, interleaved):
    """sin and cos 2 ulp, the angle 2^-32 of a turn and (position times 2^-51) the double's: 2^-22; products and sum 3 roundings; the type's."""
    right, mag = rotary_formula(x, pos, freq, axis, interleaved)
    tol = (2**-22 + 3 * 2**-24) * mag + torch.finfo(got.dtype).eps / 2 * right.abs() + 1e-7 * (got.dtype == torch.float16)
    beyond = float(((got.double() - right).abs() - tol).max())
    assert beyond <= 0, beyond


@pytest.mark.parametrize("types", [(F32, F32), (F32, F16), (F32, BF16), (F16, F16), (BF16, BF16)])
@pytest.mark.parametrize("dim,rot,interleaved", [
    (128, 128, False), (128, 96, False), (96, 96, False), (256, 64, False),  # halves on 16-byte boundaries
    (128, 74, False), (96, 74, False), (160, 154, False), (32, 6, False),    # on none
    (128, 128, True), (96, 72, True), (128, 74, True), (64, 2, True)])       # adjacent pairs
def test_rotary_of_many_tokens(bq, types, dim, rot, interleaved):  # noqa: F811
    """A CTA has several tokens, the last one fewer; apart, and where the types allow onto q and k, onto q alone."""
    T, H, KH, A = 5003, 5, 3, 3
    g = torch.Generator(device="cuda").manual_seed(dim + rot)
    qkv = torch.randn(T, H + KH + 1, dim, generator=g, device="cuda").to(DT[types[0]])
    q, k = qkv[:, :H], qkv[:, H:H + KH]
    pos = torch.randint(-1000, 1000000, (A, T), generator=g, device="cuda", dtype=torch.int32)
    freq = 10000.0 ** -(torch.arange(rot // 2, device="cuda", dtype=torch.float64) / (rot // 2))
    axis = torch.randint(0, A, (rot // 2,), generator=g, device="cuda", dtype=torch.int32)
    a, b = bq.rotary(q, k, pos, freq, axis, interleaved=interleaved, dtype=DT[types[1]])
    check_rotary(a, q, pos, freq, axis, interleaved)
    check_rotary(b, k, pos, freq, axis, interleaved)
    if types[0] == types[1]:
        was = qkv.clone()
        _, d = bq.rotary(q, k, pos, freq, axis, interleaved=interleaved, out_q=q)
        assert torch.equal(q, a) and torch.equal(d, b) and torch.equal(qkv[:, H:], was[:, H:])
        qkv.copy_(was)
        bq.rotary(q, k, pos, freq, axis, interleaved=interleaved, out_q=q, out_k=k)
        assert torch.equal(q, a) and torch.equal(k, b) and torch.equal(qkv[:, -1], was[:, -1])


@pytest.mark.parametrize("types", [(F32, F32), (F32, BF16), (BF16, BF16)])
@pytest.mark.parametrize("T,dim,rot,interleaved", [(3, 16384, 16384, False), (1300, 16384, 16384, True), (1300, 4096, 4094, False), (700, 6144, 6144, False),
                                                   (5, 65536, 16382, False), (5, 65536, 16384, True)])
def test_rotary_of_large_heads(bq, types, T, dim, rot, interleaved):  # noqa: F811
    """Tables of up to 128 KB: fewer tokens per CTA than there are, down to one."""
    g = torch.Generator(device="cuda").manual_seed(T)
    q, k = (torch.randn(T, h, dim, generator=g, device="cuda").to(DT[types[0]]) for h in (2, 1))
    pos = torch.randint(0, 100000, (1, T), generator=g, device="cuda", dtype=torch.int32)
    freq = 10000.0 ** -(torch.arange(rot // 2, device="cuda", dtype=torch.float64) / (rot // 2))
    axis = torch.zeros(rot // 2, dtype=torch.int32, device="cuda")
    a, b = bq.rotary(q, k, pos, freq, interleaved=interleaved, dtype=DT[types[1]])
    check_rotary(a, q, pos, freq, axis, interleaved)
    check_rotary(b, k, pos, freq, axis, interleaved)
    if types[0] == types[1]:
        bq.rotary(q, k, pos, freq, interleaved=interleaved, out_q=q, out_k=k)
        assert torch.equal(q, a) and torch.equal(k, b)


# ---------------------------------------------------------------- adapters --


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("T,n,rank,M,ids", [(200, 16, 16, 4096, "random"), (256, 64, 40, 4099, "random"), (256, 3, 16, 11008, "random"), (130, 2, 104, 11011, "runs"),
                                            (400, 90, 24, 8200, "random")])
def test_lora_of_wide_outputs(bq, types, T, n, rank, M, ids):  # noqa: F811
    """Tiles of 16 tokens, a CTA with several turns of 256 columns."""
    c = lora_case(T, n, rank, 96, M, *types, ids, seed=T)
    check_lora(run_lora(bq, *c), *c)
    X, A, B, s, Y, i = (t.cuda() for t in c)
    want = bq.lora(X, A, B, i, Y, s)
    assert torch.equal(bq.lora(X, A, B, i, Y, s, out=Y), want)


LARGE = [(1100, 3, 64), (1030, 2, 40), (600, 1, 128)]  # tokens, adapters, rank: tiles of 64


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("T,n,rank", LARGE)
@pytest.mark.parametrize("M", [99, 260])
def test_lora_large_tiles_in_place_and_strided(bq, types, T, n, rank, M):  # noqa: F811
    """y's rows in a wider buffer, on 16-byte boundaries and on none, out onto y and into another such buffer; x's rows apart."""
    X, A, B, s, Y, ids = lora_case(T, n, rank, 160, M, *types, "random")
    xw = torch.zeros(T, 160 + 8, dtype=X.dtype, device="cuda")
    xw[:, :160] = X.cuda()
    for off, extra in ((1, 3), (8, 8 - M % 8), (2, 2 - M % 2)):
        wide = torch.full((T, off + M + extra), 5.0, dtype=Y.dtype, device="cuda")
        view = wide[:, off:off + M]
        view.copy_(Y)
        other = torch.full((T, M + 8), 3.0, dtype=Y.dtype, device="cuda")
        apart = bq.lora(xw[:, :160], A.cuda(), B.cuda(), ids.cuda(), view, s.cuda(), out=other[:, :M])
        check_lora(apart, X, A, B, s, Y, ids)
        got = bq.lora(xw[:, :160], A.cuda(), B.cuda(), ids.cuda(), view, s.cuda(), out=view)
        assert got.data_ptr() == view.data_ptr() and torch.equal(got, apart)
        assert (wide[:, :off] == 5).all() and (wide[:, off + M:] == 5).all() and (other[:, M:] == 3).all()


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("T,n,rank", LARGE)
def test_lora_large_tiles_without_base_scale_or_adapter(bq, types, T, n, rank):  # noqa: F811
    X, A, B, s, Y, ids = lora_case(T, n, rank, 96, 130, *types, "random")
    check_lora(run_lora(bq, X, A, B, None, Y, ids), X, A, B, None, Y, ids)
    got = run_lora(bq, X, A, B, s, None, ids, dtype=Y.dtype)
    check_lora(got, X, A, B, s, None, ids)
    assert (got.cpu()[ids < 0] == 0).all()
    ids[5], ids[T - 1], ids[70] = n, -2, 2**31 - 1
    assert quiet(bq) == OK
    got = run_lora(bq, X, A, B, s, Y, ids)
    assert quiet(bq) == INDEX
    check_lora(got, X, A, B, s, Y, ids)


@pytest.mark.parametrize("types", TYPES)
def test_lora_large_tiles_captured_and_on_many_streams(bq, types):  # noqa: F811
    T, n, rank = LARGE[0]
    host = lora_case(T, n, rank, 160, 130, *types, "random")
    X, A, B, s, Y, ids = (t.cuda() for t in host)
    first = bq.lora(X, A, B, ids, Y, s)
    check_lora(first, *host)
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
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = bq.lora(X, A, B, ids, Y, s)
        graphs.append((graph, out))
    other = torch.randint(-1, n, (T,), generator=torch.Generator().manual_seed(9), dtype=torch.int32)
    ids.copy_(other)
    want = bq.lora(X, A, B, ids, Y, s)
    check_lora(want, *host[:5], other)
    torch.cuda.synchronize()
    for _ in range(10):
        for st, (graph, _) in zip(streams, graphs):  # two graphs at once
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for _, out in graphs)
