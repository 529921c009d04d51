"""The calls around a served layer's projections and paged cache, run together as a
program runs them, and captured as one step; rows beyond 2^32 bytes; waits that run
out."""
import pytest
import torch

gpu = pytest.mark.gpu
OK, TIMEOUT = 0, -6
Q4, Q8 = 2, 8


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


def status():
    from block_quantized_weight_row_gb300 import binding
    return binding.device_status()


@gpu
@pytest.mark.parametrize("seed", [1, 2])
def test_example_layer(bq, seed):
    from examples import serving_layer
    off = serving_layer.main(seed, report=lambda line: None)
    assert off.keys() == serving_layer.TOLERANCES.keys()
    for name, most in serving_layer.TOLERANCES.items():
        assert off[name] <= most, (name, off[name], most)
    assert status() == OK


@gpu
def test_captured_decode_step(bq):
    """One token each of a batch: the whole step captured once and replayed as the sequences grow, against the same calls made eagerly."""
    from examples import serving_layer
    g = torch.Generator(device="cuda").manual_seed(3)
    layers = [serving_layer.Layer(torch.Generator(device="cuda").manual_seed(4)) for _ in range(2)]
    T, hidden, steps = 4, layers[0].hidden, 20  # 20 tokens: every sequence moves on to new pages
    x, r = torch.zeros(T, hidden, device="cuda"), torch.zeros(T, hidden, device="cuda")
    n_new = torch.ones(T, dtype=torch.int32, device="cuda")
    adapter = torch.tensor([0, 2, -1, 1], dtype=torch.int32, device="cuda")

    def step(layer):
        at = bq.paged_extend(layer.page, layer.n_pages, layer.kv_len, n_new, layer.page_table, layer.free_pages, T)
        rows = bq.add_rms_norm(x, layer.norm, 1e-6, r, out=True, q8=True)
        qkv = bq.gemm(Q8, layer.w_qkv, rows.q8, layer.rows_qkv, T, hidden)
        heads = bq.lora(rows.out, layer.a, layer.b, adapter, qkv, layer.scale, out=qkv).view(T, -1, layer.dim)
        q, k, v = heads[:, :layer.n_heads], heads[:, layer.n_heads:-layer.n_kv], heads[:, -layer.n_kv:]
        q, k = bq.rotary(q, k, at.positions.expand(3, -1), layer.inv_freq, layer.axis, out_q=q, out_k=k)
        bq.paged_kv_write(layer.cache, k, v, at.slots)
        out = bq.paged_attn(layer.cache, q, at.q_start, at.kv_len, layer.page_table, 0.1, max_q_len=1, max_kv_len=64)
        return out, at

    def move_on(layer, at):
        layer.kv_len.copy_(at.kv_len)
        layer.free_pages.copy_(torch.roll(layer.free_pages, -int(at.taken[0])))

    for layer in layers:  # the captured layer's first calls are made outside the capture
        keep = [t.clone() for t in (layer.page_table, layer.kv_len)]
        step(layer)
        layer.page_table.copy_(keep[0])
        layer.kv_len.copy_(keep[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(layers[0])
    for _ in range(steps):
        x.normal_(generator=g)
        r.normal_(generator=g)
        graph.replay()
        out, at = step(layers[1])
        assert torch.equal(captured[0], out) and torch.equal(captured[1].slots, at.slots)
        move_on(layers[0], captured[1])
        move_on(layers[1], at)
    assert torch.equal(layers[0].page_table, layers[1].page_table) and layers[0].kv_len.tolist() == [steps] * T
    assert status() == OK


@gpu
def test_norm_beyond_4_gigabytes(bq):
    rows, cols = 68000, 16384
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(rows, cols, device="cuda").normal_(generator=g)
    assert x.numel() * 4 > 2**32
    w = torch.ones(cols, device="cuda")
    got = bq.add_rms_norm(x, w, 1e-6, q8=True)
    for i in (0, 65535, 65536, rows - 1):
        one = bq.add_rms_norm(x[i:i + 1].clone(), w, 1e-6, q8=True)
        assert torch.equal(got.out[i], one.out[0]) and torch.equal(got.q8[i], one.q8[0])


@gpu
def test_rotary_beyond_4_gigabytes(bq):
    T, H, D = 300000, 32, 256
    q = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda").normal_()
    assert q.numel() * 2 > 2**32
    freq = 10000.0 ** -(torch.arange(D // 2, dtype=torch.float64, device="cuda") / (D // 2))
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    got, _ = bq.rotary(q, None, pos, freq)
    for i in (0, 262143, 262144, T - 1):
        assert torch.equal(got[i:i + 1], bq.rotary(q[i:i + 1].clone(), None, pos[i:i + 1], freq)[0])


@gpu
@pytest.mark.parametrize("y", [torch.bfloat16, torch.float32])
def test_lora_beyond_4_gigabytes(bq, y):
    T, K, M, n, rank = (1 << 20, 32, 2056, 3, 8) if y == torch.bfloat16 else (530000, 32, 2056, 3, 8)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    a, b = torch.randn(n, rank, K, generator=g, device="cuda").bfloat16(), torch.randn(n, M, rank, generator=g, device="cuda").bfloat16()
    ids = torch.randint(-1, n, (T,), generator=g, device="cuda", dtype=torch.int32)
    base = torch.empty(T, M, dtype=y, device="cuda").normal_(generator=g)
    assert base.numel() * base.element_size() > 2**32
    got = bq.lora(x, a, b, ids, base)
    pick = torch.tensor([0, 1, 500000, 522240, 522241, T - 1], device="cuda")
    # few tokens take other kernels: sums of 32 products in another order, then the output's rounding
    want = bq.lora(x[pick], a, b, ids[pick], base[pick])
    h = x[pick].double().abs() @ a.double().abs().amax(0).T
    most = base[pick].double().abs() + h @ b.double().abs().amax(0).T
    assert ((got[pick].double() - want.double()).abs() <= (2 * 2**-17 + torch.finfo(y).eps) * most).all()
    none = (ids == -1).nonzero().flatten()[-5:]
    assert torch.equal(got[none], base[none])


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_lora_timeout_path_returns_error(bq, dtype):
    """Every bounded wait gives up at once: the call ends, the status says so, and the next call is right."""
    from block_quantized_weight_row_gb300 import binding
    g = torch.Generator(device="cuda").manual_seed(1)
    T, K, M, n, rank = 4096, 128, 700, 2, 64  # tiles of 64 tokens, on the tensor-memory kernel
    x = torch.randn(T, K, generator=g, device="cuda").to(dtype)
    a, b = torch.randn(n, rank, K, generator=g, device="cuda").bfloat16(), torch.randn(n, M, rank, generator=g, device="cuda").bfloat16()
    ids = torch.randint(0, n, (T,), generator=g, device="cuda", dtype=torch.int32)
    first = bq.lora(x, a, b, ids)
    assert status() == OK
    try:
        binding.lib().bq_set_spin_limit(0)
        bq.lora(x, a, b, ids)
        assert status() == TIMEOUT
    finally:
        binding.lib().bq_set_spin_limit(-1)
    assert torch.equal(bq.lora(x, a, b, ids), first) and status() == OK
