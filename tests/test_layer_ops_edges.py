"""What the calls around a served layer, and those that their outputs go into, do at
their edges: wrong element types and sizes, workspaces, kernels of large batches."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

Q4, Q8 = 2, 8
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


# ------------------------------------------------------- types and sizes --


def refused(call, tensors, error):
    """`call` with tensors of the device that have no memory: (shape, type) or None each."""
    with FakeTensorMode():
        t = [None if s is None else torch.empty(s[0], dtype=s[1], device="cuda") for s in tensors]
        with pytest.raises(error):
            call(*t)


U8, BF16, F16, F32 = torch.uint8, torch.bfloat16, torch.float16, torch.float32
W4, W8 = ((5 * 2 * 18,), U8), ((5 * 2 * 34,), U8)  # 5 rows of 64


@pytest.mark.parametrize("x,out,error", [
    ((64, BF16), None, TypeError), ((64, F16), None, TypeError), ((64, torch.float64), None, TypeError), ((64, torch.int8), None, TypeError),
    ((63, F32), None, ValueError), ((2 * 34 - 1, U8), None, ValueError), ((2 * 34 + 1, U8), None, ValueError),
    ((64, F32), (5, BF16), TypeError), ((64, F32), (4, F32), ValueError), ((2 * 34, U8), (4, F32), ValueError)])
def test_gemv_refuses_other_types_and_sizes(bq, x, out, error):
    refused(lambda w, x, y: bq.gemv(Q4, w, x, 5, 64, out=y), [W4, x and ((x[0],), x[1]), out and ((out[0],), out[1])], error)


@pytest.mark.parametrize("x,out,error", [
    ((3, 64, BF16), None, TypeError), ((3, 64, F16), None, TypeError), ((2, 64, F32), None, ValueError), ((3, 67, U8), None, ValueError),
    ((3, 64, F32), (3, 5, BF16), TypeError), ((3, 64, F32), (2, 5, F32), ValueError), ((3, 68, U8), (2, 5, F32), ValueError)])
def test_gemm_refuses_other_types_and_sizes(bq, x, out, error):
    refused(lambda w, x, y: bq.gemm(Q8, w, x, 5, 3, 64, out=y), [W8, (x[:-1], x[-1]), out and (out[:-1], out[-1])], error)


@pytest.mark.parametrize("x,error", [((64, BF16), TypeError), ((68, U8), TypeError), ((63, F32), ValueError)])
def test_gemv_batches_refuse_other_types_and_sizes(bq, x, error):
    refused(lambda w, x: bq.gemv_multi(Q4, [w], x, [5], 64), [W4, ((x[0],), x[1])], error)
    refused(lambda w, x: bq.gemv_sequence(Q4, [([w], x, [5], 64, None)]), [W4, ((x[0],), x[1])], error)


@pytest.mark.parametrize("outs,error", [([((5,), BF16)], TypeError), ([((4,), F32)], ValueError)])
def test_gemv_batches_refuse_other_outputs(bq, outs, error):
    refused(lambda w, x, *y: bq.gemv_multi(Q4, [w], x, [5], 64, outs=list(y)), [W4, ((64,), F32), *outs], error)
    refused(lambda w, x, *y: bq.gemv_sequence(Q4, [([w], x, [5], 64, list(y))]), [W4, ((64,), F32), *outs], error)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_rows_of_another_type_are_refused(bq, dtype):
    """What rotary gives in the rows' type, taken on by the calls of an unpaged cache."""
    rows, f32 = ((7, 2, 64), dtype), ((7, 2, 64), F32)
    refused(lambda q, k, v: bq.attn_decode(Q4, Q8, q, k, v, 2, 0.1), [((4, 64), dtype), ((7, 2, 36), U8), ((7, 2, 68), U8)], TypeError)
    refused(lambda r: bq.kv_quantize(Q8, r, None), [rows], TypeError)
    refused(lambda r, b: bq.kv_quantize(Q8, r, b), [f32, ((2, 64), dtype)], TypeError)
    refused(lambda k, v: bq.kv_write(Q4, k, None, Q8, v), [rows, f32], TypeError)
    refused(lambda k, v: bq.kv_write(Q4, k, None, Q8, v), [f32, rows], TypeError)
    refused(lambda k, b, v: bq.kv_write(Q4, k, b, Q8, v), [f32, ((2, 64), dtype), f32], TypeError)
    refused(bq.kv_bias, [rows], TypeError)


@pytest.mark.parametrize("blocks,out,error", [
    (((3, 68), F32), None, TypeError), (((3, 68), torch.int16), None, TypeError), (((3, 68), U8), ((3, 64), BF16), TypeError),
    (((3, 68), U8), ((3, 64), torch.float64), TypeError), (((3, 68), U8), ((2, 64), F32), ValueError), (((3, 68), U8), ((3, 63), F32), ValueError)])
def test_dequantize_refuses_other_types_and_sizes(bq, blocks, out, error):
    refused(lambda b, y: bq.dequantize_rows(Q8, b, 64, out=y), [blocks, out], error)


def test_dequantize_refuses_strided_outputs_and_those_of_the_host(bq):
    with FakeTensorMode():
        blocks = torch.empty(3, 68, dtype=U8, device="cuda")
        with pytest.raises(ValueError):
            bq.dequantize_rows(Q8, blocks, 64, out=torch.empty(3, 128, device="cuda")[:, :64])
        with pytest.raises(TypeError):
            bq.dequantize_rows(Q8, blocks, 64, out=torch.empty(3, 64))
        if torch.cuda.device_count() != 1:  # with one device there is no name for another
            with pytest.raises(ValueError):
                bq.dequantize_rows(Q8, blocks, 64, out=torch.empty(3, 64, device="cuda:1"))


@pytest.fixture
def library_alone(bq, monkeypatch):
    """libbq.so without the extension beside it, as a build without g++ or torch's headers leaves them."""
    import sys
    from block_quantized_weight_row_gb300 import binding
    monkeypatch.setattr(binding, "_ext", None)
    monkeypatch.delattr(bq, "_paged", raising=False)
    monkeypatch.setitem(sys.modules, bq.__name__ + "._paged", None)
    with pytest.raises(ImportError):
        binding._paged()
    return bq


@pytest.mark.parametrize("blocks,out,error", [
    (((3, 68), F32), None, TypeError), (((3, 68), U8), ((3, 64), BF16), TypeError), (((3, 68), U8), ((2, 64), F32), ValueError)])
def test_dequantize_refuses_the_same_without_the_extension(library_alone, blocks, out, error):
    refused(lambda b, y: library_alone.dequantize_rows(Q8, b, 64, out=y), [blocks, out], error)


@gpu
def test_dequantize_needs_no_extension(bq, library_alone):
    g = torch.Generator(device="cuda").manual_seed(1)
    blocks = bq.quantize_rows(Q8, torch.randn(5, 96, generator=g, device="cuda"))
    got = bq.dequantize_rows(Q8, blocks, 96)
    scales = blocks.view(5, 3, 34)[..., :2].contiguous().view(torch.float16).float()
    want = (blocks.view(5, 3, 34)[..., 2:].contiguous().view(torch.int8).float() * scales).view(5, 96)  # 11 + 7 bits: exact
    assert torch.equal(got, want)
    out = torch.zeros(5, 96, device="cuda")
    assert bq.dequantize_rows(Q8, blocks, 96, out=out) is out and torch.equal(out, want)
    with pytest.raises(bq.BQError):
        bq.dequantize_rows(Q8, blocks, 48)


# ------------------------------------------------------------ workspaces --


def test_workspaces_are_not_shared(bq, monkeypatch):
    """Streams, threads and captured calls have their own; a captured one is given to nobody else."""
    import threading
    from block_quantized_weight_row_gb300 import binding
    given, now = [], {"stream": 1, "capturing": False}

    class Library:
        def bq_set_workspace(self, p, n):
            given.append((p, n))
            return 0

        def bq_set_stream(self, s):
            return 0

    monkeypatch.setattr(binding, "lib", Library)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now["capturing"])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: type("Stream", (), {"cuda_stream": now["stream"]}))
    made = []

    def empty(n, dtype, device):  # of the host, whatever the device, and never freed
        made.append(torch.zeros(n, dtype=dtype))
        return made[-1]

    monkeypatch.setattr(binding.torch, "empty", empty)

    def of(n, stream=1, capturing=False):
        now.update(stream=stream, capturing=capturing)
        device = torch.device("cuda:5")
        binding._prep(device)
        ws = binding._workspace(device, n)
        assert given[-1] == (ws.data_ptr(), ws.numel()) and ws.numel() >= n
        return ws.data_ptr()

    first = of(1000)
    assert of(2000) == first and of(0) == first  # a stream's calls follow one another
    second = of(1000, stream=2)
    captured = [of(1000, capturing=True), of(1000, capturing=True), of(5 << 20, capturing=True)]
    assert of(1000) == first and of(1000, stream=2) == second
    larger = of(5 << 20)
    assert of(5 << 20, stream=2) != second and of(1000) == larger
    elsewhere = []
    other = threading.Thread(target=lambda: elsewhere.append(of(1000)))
    other.start()
    other.join()
    assert len({first, second, larger, *captured, *elsewhere}) == 7


@gpu
def test_captured_projections_keep_their_workspace(bq):
    """Graphs of calls with a workspace, replayed after larger calls and other tensors had their turn, and two at once."""
    g = torch.Generator(device="cuda").manual_seed(2)
    M, N, K = 96, 40, 1024

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    w8, w4 = bq.quantize_rows(Q8, normal(M, K)), bq.quantize_rows(Q4, normal(M, K))
    x = [normal(N, K) for _ in range(3)]
    xq = [bq.quantize_rows(Q8, t) for t in x]
    kq, vq = bq.quantize_rows(Q4, normal(300 * 2, 64)).view(300, 2, -1), bq.quantize_rows(Q8, normal(300 * 2, 64)).view(300, 2, -1)

    def step(rows, q8):
        return (bq.gemm(Q8, w8, q8, M, N, K), bq.gemv(Q4, w4, q8[0], M, K), bq.gemm(Q8, w8, rows, M, N, K), bq.gemv(Q4, w4, rows[0], M, K),
                bq.gemv_multi(Q4, [w4, w4], rows[1], [M, M], K)[1], bq.gemv_sequence(Q4, [([w4], rows[2], [M], K, None)])[0][0],
                bq.attn_decode(Q4, Q8, rows[0, :256].view(4, 64), kq, vq, 2, 0.125))

    want = [[t.clone() for t in step(x[i], xq[i])] for i in range(3)]
    cases = []
    for i in range(2):
        own = x[i].clone(), xq[i].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step(*own)
        cases.append((own, graph, outs))
    big = normal(2048, 4096)
    bq.gemm(Q8, bq.quantize_rows(Q8, normal(128, 4096)), big, 128, 2048, 4096)  # a much larger workspace
    others = [torch.full((1 << 20,), 7.0, device="cuda") for _ in range(64)]
    for (own, graph, outs), rows, q8, right in zip(cases, x[1:], xq[1:], want[1:]):
        own[0].copy_(rows)
        own[1].copy_(q8)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(outs, right))
    assert all(bool((t == 7).all()) for t in others)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(50):
        for st, (_, graph, _) in zip(streams, cases):
            with torch.cuda.stream(st):
                graph.replay()
        with torch.cuda.stream(streams[2]):
            eager = step(x[0], xq[0])
    torch.cuda.synchronize()
    for got, right in ((cases[0][2], want[1]), (cases[1][2], want[2]), (eager, want[0])):
        assert all(torch.equal(a, b) for a, b in zip(got, right))


# ---------------------------------------------------------------- rotary --


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotary_angles_to_the_32nd_bit_of_a_turn(bq, interleaved, inverse):
    """Angles of 32 bits, at half a turn above all, where the sine is small and shows what the angle lost: the turn of (1, 0) is cosine
    and sine. Off by the angle's 2^-32 of a turn, 2 ulp of sincospif and the rounding of what its argument's last bits add."""
    import math
    import random
    rng = random.Random(3)
    near = [0, 1 << 30, 1 << 31, 3 << 30, 1 << 29]
    units = [c + s * d for c in near for s in (1, -1) for d in (1, 77, 128, 255, 4097, rng.randrange(1 << 20), rng.randrange(1 << 26))]
    units += [rng.getrandbits(32) for _ in range(128 - len(units))]  # of 2^-32 turns per position
    n, where = len(units), [1, -1, 3, -5, 0]
    # in -1/2 .. 1/2 turns, so that the double holds them to 2^-54
    signed = [(u + 2**31) % 2**32 - 2**31 for u in units]
    freq = torch.tensor(signed, dtype=torch.float64) * 2**-32 * (2 * math.pi)
    q = torch.zeros(len(where), 1, 2 * n)
    first, second = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, n), slice(n, None))
    q[..., first] = 1
    got, _ = bq.rotary(q.cuda(), None, torch.tensor(where, dtype=torch.int32).cuda(), freq.cuda(), interleaved=interleaved, inverse=inverse)
    got = got.cpu().double()[:, 0]
    turned = torch.tensor([[(p * s + 2**31) % 2**32 - 2**31 for s in signed] for p in where], dtype=torch.float64)
    quarter = (turned / 2**30).round()  # whole quarters are exact; the rest is small enough for the library's sine
    rest = (turned - quarter * 2**30) * (2 * math.pi * 2**-32)
    c, s = rest.cos(), rest.sin()
    k = (quarter % 4).long()
    cos, sin = (torch.stack(v).gather(0, k[None])[0] for v in ((c, -s, -c, s), (s, c, -s, -c)))
    if inverse:
        sin = -sin
    for value, right in ((got[:, first], cos), (got[:, second], sin)):
        tol = 1.01 * 2 * math.pi * 2**-32 + 2.5 * 2**-23 * right.abs()
        beyond = float(((value - right).abs() - tol).max())
        assert beyond <= 0, beyond


# -------------------------------------------------------------- adapters --


@gpu
@pytest.mark.parametrize("x,y", [(F32, F32), (F16, F32), (F32, F16)])
@pytest.mark.parametrize("T,rank", [(20, 16), (300, 64), (1100, 64), (1100, 128)])
def test_lora_small_ranks_beside_dominant_ones(bq, x, y, T, rank):
    """fp16 adapters whose ranks differ by 2^15 in A x and as much, the other way, in B: all matter alike. Chains of matrix instructions
    add 4 u of the magnitudes each, A x enters the second product in 22 bits, or 2^-40 of its row's largest; outputs are rounded."""
    g = torch.Generator().manual_seed(T + rank)
    n, K, M, u = 2, 64, 70, 2.0**-24
    power = torch.pow(2.0, 6 - torch.arange(rank) * 15 // (rank - 1))
    X = torch.randn(T, K, generator=g).to(x)
    A = (torch.randn(n, rank, K, generator=g) / 8 * power[:, None]).half()
    B = (torch.randn(n, M, rank, generator=g) / power).half()
    Y = torch.randn(T, M, generator=g).to(y)
    ids = torch.randint(0, n, (T,), generator=g).int()
    got = bq.lora(X.cuda(), A.cuda(), B.cuda(), ids.cuda(), Y.cuda()).cpu().double()
    a, b = A.double()[ids.long()], B.double()[ids.long()]
    h = torch.einsum("trk,tk->tr", a, X.double())
    hm = torch.einsum("trk,tk->tr", a.abs(), X.double().abs())
    right = Y.double() + torch.einsum("tmr,tr->tm", b, h)
    terms = 4 if x == F32 else 1
    eh = hm * ((4 * 2 * terms * K // 32 + 37) * u + (2**-22 if x == F32 else 0)) + 2**-22 * h.abs() + 2**-40 * h.abs().amax(-1, keepdim=True)
    tol = torch.einsum("tmr,tr->tm", b.abs(), eh + 4 * 2 * 2 * -(-rank // 32) * u * h.abs())
    tol += 2 * u * right.abs() + torch.finfo(y).eps / 2 * right.abs()
    beyond = float(((got - right).abs() - tol).max())
    assert beyond <= 0, beyond


@gpu
@pytest.mark.parametrize("w", [BF16, F16])
@pytest.mark.parametrize("rank,seed", [(16, 1), (16, 2), (64, 3)])
def test_lora_of_fp32_rows_is_as_exact_as_fp32_sums(bq, w, rank, seed):
    """A decode batch, against the same formula in 64 bits: no further off, in the output's norm, than fp32 products and sums are."""
    as_exact(bq, w, 48, 16, rank, 4096, 1024, seed)


@gpu
@pytest.mark.parametrize("w,rank,K", [(F16, 64, 1024), (BF16, 128, 8192)])
def test_lora_prompts_of_fp32_rows_are_as_exact_as_fp32_sums(bq, w, rank, K):
    """The same in tiles of 64 tokens: long chains of instructions."""
    as_exact(bq, w, 4096, 4, rank, K, 2048, 1)


def as_exact(bq, w, T, n, rank, K, M, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    X = torch.randn(T, K, generator=g, device="cuda")
    A = (torch.randn(n, rank, K, generator=g, device="cuda") / K**0.5).to(w)
    B = (torch.randn(n, M, rank, generator=g, device="cuda") * 0.2).to(w)
    Y = torch.randn(T, M, generator=g, device="cuda")
    ids = torch.randint(0, n, (T,), generator=g, device="cuda", dtype=torch.int32)

    def formula(t):
        h = (X.to(t) @ A.to(t).flatten(0, 1).T).view(T, n, rank)
        h = torch.where(ids[:, None, None] == torch.arange(n, device="cuda")[:, None], h, torch.zeros((), dtype=t, device="cuda"))
        return Y.to(t) + h.flatten(1) @ B.to(t).permute(0, 2, 1).flatten(0, 1)

    right = formula(torch.float64)
    off = float((bq.lora(X, A, B, ids, Y).double() - right).norm())
    plain = float((formula(F32).double() - right).norm())
    assert off <= plain, (off, plain)
