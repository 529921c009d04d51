"""Cases and plain forms of the paged KV-cache operators: the quantizing cache
write, reading the cache back, and attention over the cache.

A cache is a pool of pages that the sequences of a batch share. A page holds
`page_size` tokens of every kv head; token row `place` of page `p` is slot
p * page_size + place. Per page and kv head the bytes are the codes of the
page's tokens, then their binary16 scales [place][head_dim / 32]. A block of 32
channels has the 16 code bytes of Q4_0 (byte j: channel j in the low nibble,
channel j + 16 in the high one, each as q + 8) or the 32 int8 codes of Q8_0.
These bytes are cut into 4 units (K) or 8 units (V), and a token's row of codes
is unit 0 of every block, unit 1 of every block, and so on.

`own` chooses between the plain form (elementary torch operations in 32 bits)
and the package's operators.
"""
import math
import random

import torch

own = False

Q4_0, Q8_0 = 2, 8
PLAIN, HADAMARD64 = 0, 1
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
BLOCK_BYTES = {Q4_0: 18, Q8_0: 34}
CODE_BYTES = {Q4_0: 16, Q8_0: 32}
QMAX = {Q4_0: 7, Q8_0: 127}
DEV = "cuda"


def listed():
    return [
        # one decode step of a batch of 32 sequences: a new token's K and V each
        {"name": "write_step", "op": "write", "tokens": 32, "heads": 8, "dim": 128, "page": 16, "k_type": Q4_0, "v_type": Q4_0,
         "dtype": "bf16", "basis": HADAMARD64, "bias": True},
        # a prompt chunk with an odd length, from a fused projection in binary16
        {"name": "write_odd", "op": "write", "tokens": 5003, "heads": 5, "dim": 64, "page": 32, "k_type": Q8_0, "v_type": Q8_0,
         "dtype": "fp16", "basis": PLAIN, "bias": False},
        # a whole layer of a long prompt: mean-centred 4-bit K, 8-bit V, fp32 rows
        {"name": "write_layer", "op": "write", "tokens": 32768, "heads": 8, "dim": 128, "page": 16, "k_type": Q4_0, "v_type": Q8_0,
         "dtype": "fp32", "basis": PLAIN, "bias": True},
        # a short prefix handed to another program, 96 channels per head
        {"name": "read_prefix", "op": "read", "tokens": 1037, "heads": 4, "dim": 96, "page": 16, "k_type": Q4_0, "v_type": Q8_0,
         "dtype": "fp32", "basis": PLAIN, "bias": True},
        # a layer's cache back to bf16 rows, out of the rotated basis
        {"name": "read_layer", "op": "read", "tokens": 65536, "heads": 8, "dim": 128, "page": 64, "k_type": Q4_0, "v_type": Q4_0,
         "dtype": "bf16", "basis": HADAMARD64, "bias": True},
        # one sequence, one token: the latency of a single user's decode step
        {"name": "decode_one", "op": "attn", "seqs": 1, "max_kv": 777, "max_q": 1, "q_heads": 16, "heads": 8, "dim": 128, "page": 16,
         "k_type": Q4_0, "v_type": Q4_0, "dtype": "fp32", "basis": PLAIN, "causal": True, "window": 0},
        # a serving batch of ragged contexts, one token each
        {"name": "decode_batch", "op": "attn", "seqs": 64, "max_kv": 8192, "max_q": 1, "q_heads": 32, "heads": 8, "dim": 128, "page": 16,
         "k_type": Q4_0, "v_type": Q4_0, "dtype": "bf16", "basis": HADAMARD64, "causal": True, "window": 0},
        # a few very long contexts, 8-bit V
        {"name": "decode_long", "op": "attn", "seqs": 4, "max_kv": 131071, "max_q": 1, "q_heads": 16, "heads": 8, "dim": 128, "page": 64,
         "k_type": Q4_0, "v_type": Q8_0, "dtype": "bf16", "basis": PLAIN, "causal": True, "window": 0},
        # drafted tokens checked five at a time, sliding window, odd head grouping
        {"name": "verify_window", "op": "attn", "seqs": 24, "max_kv": 5000, "max_q": 5, "q_heads": 24, "heads": 8, "dim": 64, "page": 32,
         "k_type": Q4_0, "v_type": Q4_0, "dtype": "fp16", "basis": PLAIN, "causal": True, "window": 1024},
        # a prompt chunk against its own and earlier tokens
        {"name": "prefill_chunk", "op": "attn", "seqs": 1, "max_kv": 8192, "max_q": 2048, "q_heads": 32, "heads": 8, "dim": 128, "page": 64,
         "k_type": Q4_0, "v_type": Q4_0, "dtype": "bf16", "basis": PLAIN, "causal": True, "window": 0},
        # prompts and decode steps in one batch, ragged
        {"name": "mixed_batch", "op": "attn", "seqs": 9, "max_kv": 6001, "max_q": 1500, "q_heads": 16, "heads": 4, "dim": 128, "page": 16,
         "k_type": Q4_0, "v_type": Q8_0, "dtype": "bf16", "basis": HADAMARD64, "causal": True, "window": 0},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng: random.Random):
    op = rng.choice(["write", "read", "attn", "attn", "attn"])
    case = {"op": op, "page": rng.choice([16, 32, 64, 128]), "k_type": rng.choice([Q4_0, Q4_0, Q8_0]), "v_type": rng.choice([Q4_0, Q8_0]),
            "dtype": rng.choice(["fp32", "fp16", "bf16", "bf16"]), "dim": rng.choice([64, 96, 128, 128, 128, 256]), "heads": rng.choice([1, 2, 4, 5, 8])}
    case["basis"] = rng.choice([PLAIN, HADAMARD64]) if case["dim"] % 64 == 0 else PLAIN
    if op != "attn":
        case["tokens"] = _spread(rng, 1, 32768 * 1024 // (case["heads"] * case["dim"]) if case["heads"] * case["dim"] > 1024 else 32768)
        case["bias"] = case["k_type"] == Q4_0 and rng.random() < 0.5
        return case
    case["q_heads"] = case["heads"] * rng.choice([1, 2, 3, 4, 8])
    kind = rng.choice(["decode", "decode", "verify", "prefill"])
    case["max_q"] = 1 if kind == "decode" else rng.randint(2, 8) if kind == "verify" else _spread(rng, 16, 1024)
    case["seqs"] = _spread(rng, 1, 64 if kind == "decode" else 32 if kind == "verify" else 4)
    rows = case["seqs"] * case["max_q"] * case["q_heads"]
    most = min(65536, 4 * 131071 // case["seqs"], (1 << 27) // rows, (1 << 29) // (case["seqs"] * case["heads"] * case["dim"]))
    case["max_kv"] = max(case["max_q"], _spread(rng, 1, most))
    case["causal"] = rng.random() < 0.8
    case["window"] = _spread(rng, 1, case["max_kv"]) if case["causal"] and rng.random() < 0.3 else 0
    return case


def _lengths(case):
    """Query and cache lengths of the batch: the longest, then lengths spread over the range, as a scheduler would have them."""
    n, q, kv = case["seqs"], [], []
    for i in range(n):
        f = 1.0 if i == 0 else ((i * 40503 + 12345) % 65536) / 65536.0
        kv.append(max(1, int(round(case["max_kv"] * f))))
        g = 1.0 if i == 0 else ((i * 26125 + 4321) % 65536) / 65536.0
        q.append(min(kv[-1], max(1, int(round(case["max_q"] * g)))))
    return q, kv


# ------------------------------------------------------------ plain form --


def _hadamard64(x):
    """H64 x / 8 on every 64 channels: butterflies of span 1, 2, ..., 32, then the scaling."""
    shape = x.shape
    for span in (1, 2, 4, 8, 16, 32):
        v = x.reshape(*shape[:-1], shape[-1] // (2 * span), 2, span)
        a, b = v[..., 0, :], v[..., 1, :]
        x = torch.stack((a + b, a - b), dim=-2).reshape(shape)
    return x * 0.125


def _quantize(x, kind):
    """Codes (int32, blocks of 32) and binary16 scales of fp32 rows."""
    v = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    amax = v.abs().amax(dim=-1)
    scale = (amax / torch.full_like(amax, float(QMAX[kind]))).half()  # a tensor divisor: one IEEE division
    d = scale.float().unsqueeze(-1)
    q = torch.where(d > 0, v / d, torch.zeros_like(v)).round()
    return q.clamp(-8 if kind == Q4_0 else -127, QMAX[kind]).to(torch.int32), scale


def _planes(pages, page, kind, dim):
    """Views of a page pool: codes (page, head, place, bytes) and scales (page, head, place, block)."""
    n, heads = pages.shape[0], pages.shape[1]
    row = dim // 32 * CODE_BYTES[kind]
    codes = pages[:, :, : page * row].unflatten(2, (page, row))
    scales = pages[:, :, page * row:].view(torch.float16).unflatten(2, (page, dim // 32))
    assert codes.shape[:2] == (n, heads)
    return codes, scales


def _store(pages, page, kind, dim, units, slots, q, scale):
    """Writes codes and scales of token rows into the pool."""
    u = torch.where(q < 0, q + 256, q) if kind == Q8_0 else q + 8
    u = u if kind == Q8_0 else u[..., :16] + 16 * u[..., 16:]
    u = u.to(torch.uint8).unflatten(-1, (units, CODE_BYTES[kind] // units))  # (token, head, block, unit, byte)
    row = u.transpose(-3, -2).reshape(*u.shape[:2], -1)
    codes, scales = _planes(pages, page, kind, dim)
    at, place = slots // page, slots % page
    codes[at, :, place] = row
    scales[at, :, place] = scale


def _values(pages, page, kind, dim, units, slots):
    """The fp32 values (..., head, dim) of the token rows at slots (...)."""
    codes, scales = _planes(pages, page, kind, dim)
    flat = slots.reshape(-1)
    at, place = flat // page, flat % page
    row = codes[at, :, place]
    heads, nb = row.shape[1], dim // 32
    b = row.unflatten(-1, (units, nb, CODE_BYTES[kind] // units)).transpose(-3, -2).reshape(-1, heads, nb, CODE_BYTES[kind])
    q = b.view(torch.int8).float() if kind == Q8_0 else torch.cat((b & 15, b >> 4), dim=-1).float() - 8.0
    v = q * scales[at, :, place].float().unsqueeze(-1)
    return v.reshape(*slots.shape, heads, dim)


def _plain_read(s):
    c = s["case"]
    k = _values(s["k_pages"], c["page"], c["k_type"], c["dim"], 4, s["slots"])
    v = _values(s["v_pages"], c["page"], c["v_type"], c["dim"], 8, s["slots"])
    if s["bias"] is not None:
        k = k + s["bias"]
    if c["basis"] == HADAMARD64:
        k = _hadamard64(k)
    t = DTYPES[c["dtype"]]
    return k.to(t), v.to(t)


def _plain_write(s):
    c = s["case"]
    k, v = s["k"].float(), s["v"].float()
    if c["basis"] == HADAMARD64:
        k = _hadamard64(k)
    if s["bias"] is not None:
        k = k - s["bias"]
    _store(s["k_pages"], c["page"], c["k_type"], c["dim"], 4, s["slots"], *_quantize(k, c["k_type"]))
    _store(s["v_pages"], c["page"], c["v_type"], c["dim"], 8, s["slots"], *_quantize(v, c["v_type"]))


def _plain_attn(s):
    c = s["case"]
    page, n, heads, dim, group = c["page"], c["seqs"], c["heads"], c["dim"], c["q_heads"] // c["heads"]
    # the batch padded to its longest context and query
    j = torch.arange(c["max_kv"], device=DEV)
    slots = s["page_table"].long()[:, j // page] * page + j % page
    live = j < s["kv_len"].long()[:, None]
    slots = torch.where(live, slots, torch.zeros_like(slots))
    k = _values(s["k_pages"], page, c["k_type"], dim, 4, slots).permute(0, 2, 1, 3)  # (seq, head, key, dim)
    v = _values(s["v_pages"], page, c["v_type"], dim, 8, slots).permute(0, 2, 1, 3)
    i = torch.arange(c["max_q"], device=DEV)
    q_len = (s["q_start"][1:] - s["q_start"][:-1]).long()
    token = torch.where(i < q_len[:, None], s["q_start"][:-1].long()[:, None] + i, torch.zeros_like(i))
    q = s["q"].float()
    q = _hadamard64(q) if c["basis"] == HADAMARD64 else q
    q = q[token].reshape(n, c["max_q"], heads, group, dim).permute(0, 2, 3, 1, 4).reshape(n, heads, -1, dim)
    score = (q @ k.transpose(-1, -2)) * s["scale"]
    at = (s["kv_len"].long() - q_len)[:, None] + i  # position of each query
    seen = live[:, None, :].expand(n, c["max_q"], -1)
    if c["causal"]:
        seen = seen & (j <= at[..., None])
        if c["window"]:
            seen = seen & (j > at[..., None] - c["window"])
    seen = seen[:, None, None].expand(n, 1, group, c["max_q"], -1).reshape(n, 1, -1, c["max_kv"])
    score = torch.where(seen, score, torch.full_like(score, -math.inf))
    top = score.amax(dim=-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    total = p.sum(dim=-1, keepdim=True)
    o = (p @ v) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.reshape(n, heads, group, c["max_q"], dim).permute(0, 3, 1, 2, 4).reshape(n * c["max_q"], c["q_heads"], dim)
    return o[s["rows"]].to(DTYPES[c["dtype"]])


# ----------------------------------------------------------------- cases --


def _pool(n_tokens, case, gen):
    """An empty page pool of a few more pages than the tokens need, and a random order of its pages."""
    pages = -(-n_tokens // case["page"])
    n = pages + 3
    nb = case["dim"] // 32
    pools = [torch.zeros(n, case["heads"], case["page"] * nb * BLOCK_BYTES[case[t]], dtype=torch.uint8, device=DEV) for t in ("k_type", "v_type")]
    return pools, torch.randperm(n, generator=gen, device=DEV)[:pages]


def _rows(shape, mean, gen):
    return torch.randn(shape, generator=gen, device=DEV) + mean


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    heads, dim, page = case["heads"], case["dim"], case["page"]
    mean = torch.rand(heads, dim, generator=gen, device=DEV) * 4 - 2  # K has channels with an offset
    centred = _hadamard64(mean) if case["basis"] == HADAMARD64 else mean
    s = {"case": case}
    if case["op"] != "attn":
        t, n = DTYPES[case["dtype"]], case["tokens"]
        (s["k_pages"], s["v_pages"]), order = _pool(n, case, gen)
        at = torch.arange(n, device=DEV)
        s["slots"] = order[at // page] * page + at % page
        s["bias"] = centred if case["bias"] else None
        k, v = _rows((n, heads, dim), mean, gen), _rows((n, heads, dim), 0.0, gen)
        if case["op"] == "read":
            s["k"], s["v"] = k, v
            _plain_write(s)
            del s["k"], s["v"]
        else:  # K and V as slices of one projection's output
            kv = torch.stack((k, v), dim=1).to(t)
            s["k"], s["v"] = kv[:, 0], kv[:, 1]
        return s
    q_len, kv_len = _lengths(case)
    per = [-(-n // page) for n in kv_len]
    (s["k_pages"], s["v_pages"]), order = _pool(sum(per) * page, case, gen)
    table = torch.zeros(len(per), max(per), dtype=torch.int32)
    first = [sum(per[:b]) for b in range(len(per))]
    order = order.to(torch.int32).cpu()
    for b, n in enumerate(per):
        table[b, :n] = order[first[b]: first[b] + n]
    # the caches as the write leaves them: every place of the pages used, the last page's rest too
    for name, kind, units, m in (("k_pages", "k_type", 4, 0.0 if case["k_type"] == Q4_0 else centred), ("v_pages", "v_type", 8, 0.0)):
        n_slots = s[name].shape[0] * page
        step = max(1, (1 << 26) // (heads * dim))
        for a in range(0, n_slots, step):
            slots = torch.arange(a, min(n_slots, a + step), device=DEV)
            _store(s[name], page, case[kind], dim, units, slots, *_quantize(_rows((len(slots), heads, dim), m, gen), case[kind]))
    s["page_table"] = table.to(DEV)
    s["kv_len"] = torch.tensor(kv_len, dtype=torch.int32, device=DEV)
    starts = [0]
    for n in q_len:
        starts.append(starts[-1] + n)
    s["q_start"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
    s["q"] = (1.5 * torch.randn(starts[-1], case["q_heads"], dim, generator=gen, device=DEV)).to(DTYPES[case["dtype"]])
    s["scale"] = 1.0 / math.sqrt(dim)
    s["rows"] = torch.tensor([b * case["max_q"] + i for b, n in enumerate(q_len) for i in range(n)], device=DEV)
    return s


def run(state):
    c = state["case"]
    if own:
        import block_quantized_weight_row_gb300 as bq

        cache = bq.PagedCache(state["k_pages"], state["v_pages"], c["page"], c["dim"], c["k_type"], c["v_type"], c["basis"])
        if c["op"] == "attn":
            return bq.paged_attn(cache, state["q"], state["q_start"], state["kv_len"], state["page_table"], state["scale"],
                                 max_q_len=c["max_q"], max_kv_len=c["max_kv"], causal=c["causal"], window=c["window"])
        if c["op"] == "write":
            bq.paged_kv_write(cache, state["k"], state["v"], state["slots"], bias=state["bias"])
        return bq.paged_kv_read(cache, state["slots"], DTYPES[c["dtype"]], bias=state["bias"])
    if c["op"] == "attn":
        return _plain_attn(state)
    if c["op"] == "write":
        _plain_write(state)
    return _plain_read(state)  # what the written bytes stand for


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    nb, dim, heads = case["dim"] // 32, case["dim"], case["heads"]
    token = heads * nb * (BLOCK_BYTES[case["k_type"]] + BLOCK_BYTES[case["v_type"]])  # a token's cache bytes
    if case["op"] != "attn":
        n = case["tokens"]
        rows = 2 * n * heads * dim * size
        extra = n * 8 + (heads * dim * 4 if case["bias"] else 0)
        # read: the cache and the slots in, the rows out. write: the rows in, the cache out, and the rows read back from it
        return {"bytes": rows + n * token + extra if case["op"] == "read" else 2 * rows + 2 * n * token + 2 * extra, "flops": 8.0 * n * heads * dim}
    q_len, kv_len = _lengths(case)
    pairs = keys = 0
    for n, kv in zip(q_len, kv_len):
        first = kv
        for i in range(n):
            hi = min(kv, kv - n + i + 1) if case["causal"] else kv
            lo = max(0, kv - n + i + 1 - case["window"]) if case["window"] else 0
            pairs += max(0, hi - lo)
            first = min(first, lo)
        keys += kv - first
    rows = sum(q_len) * case["q_heads"] * dim * size
    return {"bytes": keys * token + 2 * rows + 4 * (keys // case["page"] + 3 * len(q_len)), "flops": 4.0 * dim * case["q_heads"] * pairs}


# ----------------------------------------------------------------- exact --


def _f32(x):
    return x.float().double()


def _fwht64(x):
    """The butterflies with every sum rounded to 32 bits, as the basis is defined."""
    y = x.unflatten(-1, (-1, 64))
    order = torch.arange(64, device=x.device)
    for bit in range(6):
        other = y[..., order ^ (1 << bit)]
        y = _f32(torch.where((order >> bit & 1).bool(), other - y, y + other))
    return (y / 8).flatten(-2)


def _decode(pages, case, kind, units, slots):
    """64-bit values of one pool at slots, byte by byte from the layout."""
    page, nb = case["page"], case["dim"] // 32
    cb = CODE_BYTES[kind]
    ub = cb // units
    channel = torch.arange(case["dim"], device=DEV)
    block, e = channel // 32, channel % 32
    byte = e if kind == Q8_0 else e % 16
    col = (byte // ub) * nb * ub + block * ub + byte % ub
    at, place = slots // page, slots % page
    got = []
    for h in range(case["heads"]):
        raw = pages[at, h]
        c = raw.gather(1, place[:, None] * nb * cb + col).long()
        q = torch.where(c > 127, c - 256, c) if kind == Q8_0 else torch.where(e < 16, c % 16, c // 16) - 8
        two = page * nb * cb + 2 * (place[:, None] * nb + block)
        bits = (raw.gather(1, two).long() + 256 * raw.gather(1, two + 1).long()).to(torch.int32)
        d = torch.where(bits > 32767, bits - 65536, bits).to(torch.int16).view(torch.float16).double()
        got.append(q * d)
    return torch.stack(got, dim=1)


def _round_trip(x, kind):
    """Values that the block rule gives for rows x: its division and its scale are defined in 32 and 16 bits."""
    v = x.unflatten(-1, (-1, 32))
    d = _f32(v.abs().amax(-1, keepdim=True) / QMAX[kind]).half().double()
    q = torch.where(d > 0, torch.round(_f32(v / torch.where(d > 0, d, 1.0))), 0.0)
    return (q.clamp(-8 if kind == Q4_0 else -127, QMAX[kind]) * d).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] != "attn":
        if case["op"] == "write":
            k = s["k"].double()
            k = _fwht64(k) if case["basis"] == HADAMARD64 else k
            k = _f32(k - s["bias"].double()) if s["bias"] is not None else k
            k, v = _round_trip(k, case["k_type"]), _round_trip(s["v"].double(), case["v_type"])
        else:
            k, v = _decode(s["k_pages"], case, case["k_type"], 4, s["slots"]), _decode(s["v_pages"], case, case["v_type"], 8, s["slots"])
        k = k + s["bias"].double() if s["bias"] is not None else k
        if case["basis"] == HADAMARD64:
            i = torch.arange(64, device=DEV)
            sign = i[:, None] & i
            sign = sum(sign >> b & 1 for b in range(6)) % 2
            k = (k.unflatten(-1, (-1, 64)) @ (1.0 - 2.0 * sign.double()) / 8).flatten(-2)
        return k, v
    q_len, kv_len = _lengths(case)
    group, page = case["q_heads"] // case["heads"], case["page"]
    out = torch.zeros(sum(q_len), case["q_heads"], case["dim"], dtype=torch.float64, device=DEV)
    i64 = torch.arange(64, device=DEV)
    bits = i64[:, None] & i64
    H = (1.0 - 2.0 * (sum(bits >> b & 1 for b in range(6)) % 2).double()) / 8
    t0 = 0
    for b, (n, kv) in enumerate(zip(q_len, kv_len)):
        j = torch.arange(kv, device=DEV)
        slots = s["page_table"][b].long()[j // page] * page + j % page
        k, v = _decode(s["k_pages"], case, case["k_type"], 4, slots), _decode(s["v_pages"], case, case["v_type"], 8, slots)
        q = s["q"][t0: t0 + n].double()
        if case["basis"] == HADAMARD64:
            q = (q.unflatten(-1, (-1, 64)) @ H).flatten(-2)
        pos = kv - n + torch.arange(n, device=DEV)[:, None]
        off = torch.zeros(n, kv, dtype=torch.bool, device=DEV)
        if case["causal"]:
            off = j > pos
            if case["window"]:
                off = off | (j <= pos - case["window"])
        for h in range(case["q_heads"]):
            w = (q[:, h] @ k[:, h // group].T * s["scale"]).masked_fill(off, -math.inf)
            w = torch.softmax(w, dim=-1).masked_fill(off.all(-1, keepdim=True), 0.0)
            out[t0: t0 + n, h] = w @ v[:, h // group]
        t0 += n
    return out
