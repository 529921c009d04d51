"""Serving a few sequences from a paged, quantized KV cache: one attention layer.

Sequences of different lengths share a pool of pages. Their prompts enter in
chunks, batched with the other sequences' single tokens (`step`); every step
quantizes its new K and V rows into the pages (`paged_kv_write`) and attends over
all that is cached (`paged_attn`). A finished sequence's pages go back to the
pool and serve the next one. At the end the rows of a sequence are read back
(`paged_kv_read`) as they would be to move it to another cache.

    python examples/paged_serving.py            # on one GB300

K is held in Q4_0 after a mean-centering bias and the Hadamard rotation, V in
Q8_0. The bias adds the same number to every score of a query row, so attention
needs nothing of it; reading K back adds it again.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_quantized_weight_row_gb300 as bq  # noqa: E402

# The largest difference between a step and plain attention over the rows read back, relative to max |v|: half a bf16
# step of the output, 2^-8; a chunk's rotated q, k and v and its weights each rounded to binary16, 2^-11, which moves a
# score by 2 * 2^-11 * scale |q| |k| (below 21 for these rows) and the output by twice that and by 2 * 2^-11.
TOLERANCE = 2**-8 + 2 * 2 * 2**-11 * 21 + 2 * 2**-11


class Layer:
    """One attention layer's cache, its free pages and the sequences in it."""

    def __init__(self, n_pages=64, page_size=16, n_heads=8, n_kv_heads=2, head_dim=128, max_seqs=4, dtype=torch.bfloat16,
                 calibration=None):
        self.cache = bq.PagedCache.empty(n_pages, page_size, n_kv_heads, head_dim, bq.Q4_0, bq.Q8_0,
                                         bq.BASIS_HADAMARD64)
        self.bias = None
        if calibration is not None:  # fp32 K rows (tokens, n_kv_heads, head_dim) of typical text
            self.bias = bq.kv_bias(calibration, bq.BASIS_HADAMARD64)
        self.n_heads, self.scale, self.dtype = n_heads, head_dim**-0.5, dtype
        self.free = list(range(n_pages))
        self.max_pages = n_pages // max_seqs
        self.pages: dict[int, list[int]] = {}
        self.length: dict[int, int] = {}

    def add(self, seq: int) -> None:
        self.pages[seq], self.length[seq] = [], 0

    def drop(self, seq: int) -> None:
        self.free += self.pages.pop(seq)
        del self.length[seq]

    def slots(self, seq: int, first: int, count: int) -> list[int]:
        size = self.cache.page_size
        return [self.pages[seq][t // size] * size + t % size for t in range(first, first + count)]

    def step(self, new: dict[int, tuple[torch.Tensor, torch.Tensor, torch.Tensor]]) -> dict[int, torch.Tensor]:
        """One forward pass: new[seq] = (q, k, v) of the sequence's next tokens,
        one of them (decode) or many (a chunk of its prompt), all (tokens, heads,
        head_dim). Returns each sequence's attention output."""
        slots, starts, lens, table = [], [0], [], []
        for seq, (q, _, _) in new.items():
            first, count = self.length[seq], q.shape[0]
            while len(self.pages[seq]) * self.cache.page_size < first + count:
                if len(self.pages[seq]) == self.max_pages or not self.free:
                    raise RuntimeError(f"no page left for sequence {seq}")
                self.pages[seq].append(self.free.pop())
            slots += self.slots(seq, first, count)
            self.length[seq] = first + count
            starts.append(starts[-1] + count)
            lens.append(first + count)
            table.append(self.pages[seq] + [-1] * (self.max_pages - len(self.pages[seq])))
        q, k, v = (torch.cat([rows[i] for rows in new.values()]) for i in range(3))
        dev = q.device
        bq.paged_kv_write(self.cache, k, v, torch.tensor(slots, dtype=torch.int64, device=dev), self.bias)
        out = bq.paged_attn(self.cache, q, torch.tensor(starts, dtype=torch.int32, device=dev),
                            torch.tensor(lens, dtype=torch.int32, device=dev),
                            torch.tensor(table, dtype=torch.int32, device=dev), self.scale,
                            max_q_len=max(b - a for a, b in zip(starts, starts[1:])), max_kv_len=max(lens))
        return {seq: out[a:b] for seq, a, b in zip(new, starts, starts[1:])}

    def rows(self, seq: int) -> tuple[torch.Tensor, torch.Tensor]:
        """A sequence's K and V as the cache holds them, in the model's basis."""
        slots = torch.tensor(self.slots(seq, 0, self.length[seq]), dtype=torch.int64, device=self.cache.k_pages.device)
        return bq.paged_kv_read(self.cache, slots, torch.float32, self.bias)


def attend(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: float) -> torch.Tensor:
    """Plain causal attention of the last q.shape[0] tokens over rows k, v, in 64 bits."""
    n, T, group = q.shape[0], k.shape[0], q.shape[1] // k.shape[1]
    k, v = (x.double().repeat_interleave(group, 1) for x in (k, v))
    s = torch.einsum("ihd,jhd->hij", q.double(), k) * scale
    last = torch.arange(T - n, T, device=q.device)
    s = s.masked_fill(torch.arange(T, device=q.device)[None, :] > last[:, None], float("-inf"))
    return torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), v)


def main(seed: int = 1, report=print) -> float:
    """Serve three sequences; returns the largest difference between a step's
    output and plain attention over the rows read back, relative to the largest
    value of V."""
    gen = torch.Generator().manual_seed(seed)
    n_heads, n_kv, dim = 32, 8, 128  # heads enough that the chunk of 129 tokens runs on the tensor-memory kernel
    mean = torch.randn((1, n_kv, dim), generator=gen) * 2  # what the bias is there for

    def rows(n):
        q = torch.randn((n, n_heads, dim), generator=gen)
        k = torch.randn((n, n_kv, dim), generator=gen) + mean
        v = torch.randn((n, n_kv, dim), generator=gen)
        return tuple(x.to("cuda", torch.bfloat16) for x in (q, k, v))

    calibration = (torch.randn((512, n_kv, dim), generator=gen) + mean).cuda()
    layer = Layer(n_heads=n_heads, n_kv_heads=n_kv, head_dim=dim, calibration=calibration)
    worst = 0.0

    def step(**counts):
        nonlocal worst
        new = {int(name[1:]): rows(n) for name, n in counts.items()}
        for seq, out in layer.step(new).items():
            k, v = layer.rows(seq)
            ref = attend(new[seq][0], k, v, layer.scale)
            worst = max(worst, float((out.double() - ref).abs().max() / v.abs().max()))
        report(f"step {counts}: lengths {layer.length}, {len(layer.free)} pages free")

    for seq in (0, 1):
        layer.add(seq)
    step(s0=100)            # the first prompt, in one chunk
    step(s0=1, s1=37)       # it decodes while the second prompt enters
    step(s0=1, s1=1)        # both decode
    step(s0=5, s1=1)        # five tokens of a draft are checked at once
    layer.drop(0)           # its pages serve the next sequence
    layer.add(2)
    step(s1=1, s2=129)
    step(s1=1, s2=1)
    report(f"largest difference from plain attention over the rows read back: {worst:.2e} of max |v|")
    return worst


if __name__ == "__main__":
    main()
