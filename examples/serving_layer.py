"""One decoder layer served to several requests: quantized projections with the
requests' own adapters, rotary positions, the paged cache, and the norms between.

Every step is the same calls, whether a request brings a chunk of its prompt or one
token, and all lengths stay on the device; the host reads one number, the pages
taken, to move the front of the free list on:

    paged_extend    page tables, slots and positions of the step's tokens
    add_rms_norm    the residual stream's sum and norm, in fp32 for the adapters and
                    in Q8_0 for the projections
    gemm            W in Q8_0 times the Q8_0 rows
    lora            + each request's low-rank adapter
    rotary          q and k, in place of their angles; here on three axes, as text
                    with images has them (equal on all three for text)
    paged_kv_write, paged_attn

    python examples/serving_layer.py            # on one GB300

main() checks each of these against its formula in 64 bits, on the inputs it had.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_quantized_weight_row_gb300 as bq  # noqa: E402

EPS = 1e-6

# Largest difference of a call from its formula in 64 bits, relative to the largest value of the formula's result (the
# whole numbers and 8-bit codes are equal). Products of fp32 sums: 2^-24 for each of the up to 600 terms of a sum of 1024
# values. The norm's rows: three roundings. Rotary and attention: half a bf16 step, 2^-8; attention's weights and rotated q
# in binary16 as in paged_serving.py.
TOLERANCES = {"norm": 4 * 2**-24, "projection": 600 * 2**-24, "adapters": 600 * 2**-24, "rotary": 2**-8, "attention": 2**-8 + 2 * 2 * 2**-11 * 21 + 2 * 2**-11}


class Layer:
    """Weights (random), adapters, the cache and the lengths of one layer's batch."""

    def __init__(self, gen, hidden=1024, n_heads=8, n_kv=2, dim=128, n_adapters=3, rank=16, n_pages=48, page=16, max_seqs=4, max_pages=12):
        def normal(*shape, scale=1.0):
            return torch.randn(shape, generator=gen, device="cuda") * scale

        self.hidden, self.n_heads, self.n_kv, self.dim, self.page, self.n_pages = hidden, n_heads, n_kv, dim, page, n_pages
        self.rows_qkv, self.rows_o = (n_heads + 2 * n_kv) * dim, hidden
        self.w_qkv = bq.quantize_rows(bq.Q8_0, normal(self.rows_qkv, hidden, scale=hidden**-0.5))
        self.w_o = bq.quantize_rows(bq.Q8_0, normal(hidden, n_heads * dim, scale=(n_heads * dim)**-0.5))
        self.norm = 1 + 0.1 * normal(hidden)
        self.a = normal(n_adapters, rank, hidden, scale=hidden**-0.5).bfloat16()
        self.b = normal(n_adapters, self.rows_qkv, rank, scale=0.2).bfloat16()
        self.scale = torch.rand(n_adapters, generator=gen, device="cuda") + 0.5
        pairs = dim // 2
        self.inv_freq = 1e6 ** -(torch.arange(pairs, dtype=torch.float64, device="cuda") / pairs)
        self.axis = (torch.arange(pairs, device="cuda") * 3 // pairs).int()
        self.cache = bq.PagedCache.empty(n_pages, page, n_kv, dim, bq.Q4_0, bq.Q8_0, bq.BASIS_HADAMARD64)
        self.page_table = torch.full((max_seqs, max_pages), -1, dtype=torch.int32, device="cuda")
        self.free_pages = torch.randperm(n_pages, generator=gen, device="cuda").int()
        self.kv_len = torch.zeros(max_seqs, dtype=torch.int32, device="cuda")

    def step(self, x, residual, n_new, adapter, grid, max_q_len, max_kv_len):
        """One pass over the batch: x and residual (tokens, hidden) fp32, the last
        layer's output and the stream; n_new (sequences) int32, tokens per sequence;
        adapter (tokens) int32; grid (2, tokens) int32 or None: rows and columns of
        image tokens. Returns the layer's attention output, the stream, and what lay
        between (for the checks)."""
        at = bq.paged_extend(self.page, self.n_pages, self.kv_len, n_new, self.page_table, self.free_pages, x.shape[0])
        rows = bq.add_rms_norm(x, self.norm, EPS, residual, out=True, q8=True)
        qkv = bq.gemm(bq.Q8_0, self.w_qkv, rows.q8, self.rows_qkv, x.shape[0], self.hidden)
        adapted = bq.lora(rows.out, self.a, self.b, adapter, qkv, self.scale)
        heads = adapted.view(x.shape[0], -1, self.dim)
        q, k, v = heads[:, :self.n_heads], heads[:, self.n_heads:-self.n_kv], heads[:, -self.n_kv:]
        positions = torch.stack((at.positions, *(at.positions if grid is None else grid).expand(2, -1)))
        q_turned, k_turned = bq.rotary(q, k, positions, self.inv_freq, self.axis, dtype=torch.bfloat16)
        bq.paged_kv_write(self.cache, k_turned, v.to(torch.bfloat16), at.slots)
        out = bq.paged_attn(self.cache, q_turned, at.q_start, at.kv_len, self.page_table, self.dim**-0.5, max_q_len=max_q_len, max_kv_len=max_kv_len)
        y = bq.gemm(bq.Q8_0, self.w_o, out.float().view(x.shape[0], -1), self.hidden, x.shape[0], self.n_heads * self.dim)
        seen = dict(at=at, before=self.kv_len, rows=rows, qkv=qkv, adapted=adapted, q=q, k=k, positions=positions, q_turned=q_turned, k_turned=k_turned, out=out)
        # the pages taken leave the front of the free list, and the lengths grow
        self.free_pages = torch.roll(self.free_pages, -int(at.taken[0]))  # a scheduler that keeps the list on the host reads this number too
        self.kv_len = at.kv_len
        return y, rows.sum, seen


def _off(got, ref):
    return float((got.double() - ref).abs().max() / ref.abs().max().clamp_min(1e-30))


def check(layer, x, residual, adapter, seen):
    """The largest differences of a step's calls from their formulas."""
    s = (x.double() + residual.double()).float().double()
    norm = s / (s.square().mean(-1, keepdim=True) + EPS).sqrt() * layer.norm.double()
    w = bq.dequantize_rows(bq.Q8_0, layer.w_qkv, layer.hidden).double()
    codes = bq.dequantize_rows(bq.Q8_0, seen["rows"].q8, layer.hidden).double()
    assert torch.equal(bq.quantize_rows(bq.Q8_0, seen["rows"].out), seen["rows"].q8)
    off = {"norm": _off(seen["rows"].out, norm), "projection": _off(seen["qkv"], codes @ w.T)}
    delta = torch.zeros_like(seen["qkv"], dtype=torch.float64)
    for i in range(len(layer.a)):
        mine = adapter == i
        delta[mine] = (seen["rows"].out[mine].double() @ layer.a[i].double().T) @ layer.b[i].double().T * layer.scale[i].double()
    off["adapters"] = _off(seen["adapted"], seen["qkv"].double() + delta)
    theta = seen["positions"].double()[layer.axis.long()].T * layer.inv_freq
    c, sn, half = theta.cos()[:, None], theta.sin()[:, None], layer.dim // 2
    turn = lambda t: torch.cat((t[..., :half] * c - t[..., half:] * sn, t[..., :half] * sn + t[..., half:] * c), -1)  # noqa: E731
    off["rotary"] = max(_off(seen["q_turned"], turn(seen["q"].double())), _off(seen["k_turned"], turn(seen["k"].double())))
    # attention over the rows read back, sequence by sequence, by tables that are looked up here
    at, off["attention"] = seen["at"], 0.0
    for b, (first, end, length, before) in enumerate(zip(at.q_start[:-1].tolist(), at.q_start[1:].tolist(), at.kv_len.tolist(), seen["before"].tolist())):
        if first == end:
            continue
        assert length == before + end - first and at.positions[first:end].tolist() == list(range(before, length))
        t = torch.arange(length, device="cuda")
        slots = layer.page_table[b].long()[t // layer.page] * layer.page + t % layer.page
        assert torch.equal(slots[before:], at.slots[first:end])
        k, v = (r.double().repeat_interleave(layer.n_heads // layer.n_kv, 1) for r in bq.paged_kv_read(layer.cache, slots))
        score = torch.einsum("ihd,jhd->hij", seen["q_turned"][first:end].double(), k) * layer.dim**-0.5
        score = score.masked_fill(t[None, :] > t[before:, None], float("-inf"))
        ref = torch.einsum("hij,jhd->ihd", torch.softmax(score, -1), v)
        off["attention"] = max(off["attention"], float((seen["out"][first:end].double() - ref).abs().max() / v.abs().max()))
    return off


def main(seed: int = 1, report=print) -> dict[str, float]:
    """Serve four requests; returns the largest difference of each call from its formula."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    layer = Layer(gen)
    worst = dict.fromkeys(TOLERANCES, 0.0)
    of_request = [0, 2, -1, 1]  # their adapters
    length = [0] * 4
    # prompts enter in chunks beside others' single tokens; the last request has an image of 4 x 8 patches
    for counts in ([100, 0, 17, 0], [1, 37, 1, 32], [1, 1, 1, 1], [1, 5, 0, 1], [1, 1, 1, 1]):
        n = sum(counts)
        x, residual = (torch.randn(n, layer.hidden, generator=gen, device="cuda") for _ in range(2))
        adapter = torch.tensor([a for a, c in zip(of_request, counts) for _ in range(c)], dtype=torch.int32, device="cuda")
        grid = None
        if counts[3] == 32:
            t = torch.arange(n, device="cuda") - (n - 32)
            grid = torch.stack((torch.where(t < 0, t, t // 8), torch.where(t < 0, t, t % 8))).int()
        length = [a + c for a, c in zip(length, counts)]
        _, _, seen = layer.step(x, residual, torch.tensor(counts, dtype=torch.int32, device="cuda"), adapter, grid, max(counts), max(length))
        off = check(layer, x, residual, adapter, seen)
        worst = {k: max(worst[k], off[k]) for k in worst}
        report(f"step {counts}: lengths {length}, pages taken {int(seen['at'].taken[0])}")
    report("largest differences from the formulas: " + ", ".join(f"{k} {v:.1e}" for k, v in worst.items()))
    return worst


if __name__ == "__main__":
    main()
