"""Cases and plain forms of the operators around the projections and the paged
cache of a served layer: extending the sequences of a paged cache (page tables,
slots and positions from lengths), the root-mean-square norm with the residual's
addition and a Q8_0 output, rotary positions on several axes, and low-rank
adapters of many requests beside a shared projection.

`own` chooses between the plain form (elementary torch operations in 32 bits;
in 64 the angles of far positions, and the mean square, on whose last bit the
8-bit codes of values next to a border hang) and the package's operators.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"fp32": 4, "fp16": 2, "bf16": 2}
Q4_0, Q8_0 = 2, 8
EPS = 1e-6


def listed():
    return [
        # a decode step of a serving batch: a token each, every sixteenth sequence onto a new page
        {"name": "extend_step", "op": "extend", "seqs": 64, "max_kv": 8192, "max_new": 1, "page": 16, "spare": 0},
        # prompts of all lengths entering beside sequences that decode or wait; a page size that is no power of two
        {"name": "extend_mixed", "op": "extend", "seqs": 300, "max_kv": 6001, "max_new": 1500, "page": 48, "spare": 77},
        # a large batch of prompt chunks, as an offline job has them
        {"name": "extend_large", "op": "extend", "seqs": 8192, "max_kv": 2048, "max_new": 257, "page": 16, "spare": 1000},
        # the norm before a projection in a decode step of 16 sequences; only the 8-bit rows are wanted
        {"name": "norm_step", "op": "norm", "rows": 16, "cols": 4096, "dtype": "fp32", "residual": True, "out": False},
        # rows of an odd number of blocks, no residual, both outputs
        {"name": "norm_odd", "op": "norm", "rows": 999, "cols": 1376, "dtype": "fp16", "residual": False, "out": True},
        # a long prompt in bf16: 8-bit rows for the projection, bf16 rows for its adapters
        {"name": "norm_prompt", "op": "norm", "rows": 16384, "cols": 4096, "dtype": "bf16", "residual": True, "out": True},
        # q and k of a decode step of 32 sequences, text, image rows and columns
        {"name": "rotary_step", "op": "rotary", "tokens": 32, "q_heads": 32, "k_heads": 8, "dim": 128, "rot": 128, "axes": 3,
         "interleaved": False, "dtype": "bf16", "far": 1 << 20},
        # patches of an image: two axes, adjacent pairs, part of the channels
        {"name": "rotary_patches", "op": "rotary", "tokens": 4999, "q_heads": 12, "k_heads": 12, "dim": 96, "rot": 72, "axes": 2,
         "interleaved": True, "dtype": "fp16", "far": 100},
        # a long prompt of text with video
        {"name": "rotary_prompt", "op": "rotary", "tokens": 32768, "q_heads": 32, "k_heads": 8, "dim": 128, "rot": 128, "axes": 3,
         "interleaved": False, "dtype": "bf16", "far": 32768},
        # a decode step: 48 requests with 16 adapters between them, beside an fp32 projection
        {"name": "lora_step", "op": "lora", "tokens": 48, "adapters": 16, "rank": 16, "cols": 4096, "out": 4096, "x": "fp32", "w": "bf16",
         "y": "fp32", "runs": False},
        # short prompts, odd sizes, all in binary16
        {"name": "lora_odd", "op": "lora", "tokens": 777, "adapters": 5, "rank": 24, "cols": 1376, "out": 1027, "x": "fp16", "w": "fp16",
         "y": "fp16", "runs": True},
        # prompts of eight requests, bf16 rows beside the fp32 output of the widest projection
        {"name": "lora_prompt", "op": "lora", "tokens": 8192, "adapters": 8, "rank": 64, "cols": 4096, "out": 11008, "x": "bf16", "w": "bf16",
         "y": "fp32", "runs": True},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng: random.Random):
    op = rng.choice(["extend", "norm", "rotary", "lora", "lora"])
    if op == "extend":
        seqs = _spread(rng, 1, 8192)
        new = 1 if rng.random() < 0.4 else _spread(rng, 1, min(65536, 257 * 8192 // seqs))
        return {"op": op, "seqs": seqs, "max_kv": _spread(rng, 1, min(131072, 2048 * 8192 // seqs)), "max_new": new,
                "page": rng.choice([16, 16, 32, 48, 64, 128]), "spare": rng.choice([0, 0, 1, 333])}
    if op == "norm":
        cols = 32 * _spread(rng, 1, 512)
        return {"op": op, "rows": _spread(rng, 1, min(65536, 50_000_000 // cols)), "cols": cols, "dtype": rng.choice(["fp32", "fp16", "bf16"]),
                "residual": rng.random() < 0.7, "out": rng.random() < 0.5}
    if op == "rotary":
        dim, kh = rng.choice([64, 96, 128, 128, 256]), rng.choice([1, 2, 4, 5, 8])
        qh = kh * rng.choice([1, 2, 3, 4, 8])
        return {"op": op, "tokens": _spread(rng, 1, min(131072, (1 << 27) // ((qh + kh) * dim))), "q_heads": qh, "k_heads": kh, "dim": dim,
                "rot": rng.choice([dim, dim, dim // 2, 2 * rng.randint(1, dim // 2)]), "axes": rng.randint(1, 4),
                "interleaved": rng.random() < 0.4, "dtype": rng.choice(["fp32", "fp16", "bf16", "bf16"]), "far": _spread(rng, 10, 1 << 24)}
    w = rng.choice(["fp16", "bf16", "bf16"])
    case = {"op": op, "tokens": _spread(rng, 1, 8192), "adapters": _spread(rng, 1, 64), "rank": rng.choice([8, 8, 16, 16, 24, 32, 64, 128]),
            "cols": 32 * _spread(rng, 4, 256), "out": _spread(rng, 100, 8192), "x": rng.choice(["fp32", w]), "w": w, "y": rng.choice(["fp32", w]),
            "runs": rng.random() < 0.6}
    case["tokens"] = min(case["tokens"], (1 << 22) // (case["adapters"] * case["rank"]))  # bounds the plain form's products
    return case


def _unit(i, a, b):
    """An even spread over [0, 1) without a generator: lengths belong to the case."""
    return ((i * a + b) % 65536) / 65536.0


def _lengths(case):
    """Cached and new tokens of the batch: the longest first, then lengths spread over the range; every ninth sequence waits."""
    kv, new = [], []
    for i in range(case["seqs"]):
        kv.append(case["max_kv"] if i == 0 else int(case["max_kv"] * _unit(i, 40503, 12345)))
        new.append(case["max_new"] if i == 0 else 0 if i % 9 == 5 else max(1, int(round(case["max_new"] * _unit(i, 26125, 4321)))))
    return kv, new


# ------------------------------------------------------------ plain form --


def _plain_extend(s):
    c, page = s["case"], s["case"]["page"]
    kv, new = s["kv_len"].long(), s["n_new"].long()
    owned = (kv + page - 1) // page
    length = kv + new
    need = (length + page - 1) // page - owned
    ends = torch.cumsum(new, 0)
    base = torch.cumsum(need, 0) - need
    t = torch.arange(s["n_slots"], device=DEV)
    seq = torch.searchsorted(ends, t, right=True)
    live = seq < c["seqs"]
    seq = torch.where(live, seq, torch.zeros_like(seq))
    at = torch.where(live, kv[seq] + t - (ends - new)[seq], torch.zeros_like(t))
    column = at // page
    fresh = column - owned[seq]
    listed_page = s["free_pages"].long()[torch.where(live & (fresh >= 0), base[seq] + fresh, torch.zeros_like(t))]
    pages = torch.where(fresh >= 0, listed_page, s["page_table"].long()[seq, column])
    slots = torch.where(live, pages * page + at % page, torch.full_like(t, -1))
    n = s["tokens"]
    s["page_table"][seq[:n], column[:n]] = pages[:n].int()
    q_start = torch.cat((torch.zeros(1, dtype=torch.int64, device=DEV), ends)).int()
    taken = need.sum()
    return {"page_table": s["page_table"], "q_start": q_start, "kv_len": length.int(), "slots": slots, "positions": at.int(),
            "taken": torch.stack((taken, taken)).int()}


def _plain_norm(s):
    c, t = s["case"], DTYPES[s["case"]["dtype"]]
    h = s["x"].float()
    if c["residual"]:
        h = (h + s["residual"].float()).to(t).float()
    mean = (h.double() * h.double()).mean(dim=-1, keepdim=True)
    y = (h * (1.0 / torch.sqrt(mean + EPS)).float()) * s["weight"]
    v = y.unflatten(-1, (-1, 32))
    amax = v.abs().amax(dim=-1, keepdim=True)
    d = (amax / torch.full_like(amax, 127.0)).half().float()  # a tensor divisor: one IEEE division
    q = torch.where(d > 0, v / d, torch.zeros_like(v)).round().clamp(-127, 127)
    got = {"values": (q * d).flatten(-2)}
    if c["residual"]:
        got["sum"] = h.to(t)
    if c["out"]:
        got["out"] = y.to(t)
    return got


def _plain_rotate(x, cos, sin, rot, interleaved):
    v = x.float()
    turned, rest = v[..., :rot], v[..., rot:]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if interleaved else (turned[..., : rot // 2], turned[..., rot // 2:])
    a, b = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((a, b), dim=-1).flatten(-2) if interleaved else torch.cat((a, b), dim=-1)
    return torch.cat((turned, rest), dim=-1).to(x.dtype)


def _plain_rotary(s):
    c = s["case"]
    angle = s["positions"].double()[s["axis"].long()].T * s["inv_freq"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    return tuple(_plain_rotate(s[name], cos, sin, c["rot"], c["interleaved"]) for name in ("q", "k"))


def _plain_lora(s):
    """All adapters' products for every token, of which the token's own are kept."""
    c = s["case"]
    n, r = c["adapters"], c["rank"]
    h = (s["x"].float() @ s["a"].float().flatten(0, 1).T).unflatten(-1, (n, r))
    mine = s["adapter"].long()[:, None] == torch.arange(n, device=DEV)
    h = torch.where(mine[..., None], h * s["scale"][:, None], torch.zeros_like(h)).flatten(-2)
    delta = h @ s["b"].float().permute(0, 2, 1).flatten(0, 1)
    return (s["y"].float() + delta).to(s["y"].dtype)


# ----------------------------------------------------------------- cases --


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": case}

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    if case["op"] == "extend":
        kv, new = _lengths(case)
        page = case["page"]
        owned = torch.tensor([-(-a // page) for a in kv])
        total = torch.tensor([-(-(a + b) // page) for a, b in zip(kv, new)])
        n_owned, wide = int(owned.sum()), int(total.max())
        n_pages = int(total.sum()) + 5
        order = torch.randperm(n_pages, generator=gen, device=DEV).int()
        table = torch.full((case["seqs"], wide), -1, dtype=torch.int32, device=DEV)
        table[torch.arange(wide, device=DEV) < owned.to(DEV)[:, None]] = order[:n_owned]
        s["page_table"], s["free_pages"] = table, order[n_owned:].clone()
        s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=DEV)
        s["n_new"] = torch.tensor(new, dtype=torch.int32, device=DEV)
        s["tokens"], s["n_slots"], s["n_pages"] = sum(new), sum(new) + case["spare"], n_pages
    elif case["op"] == "norm":
        t, shape = DTYPES[case["dtype"]], (case["rows"], case["cols"])
        spread = torch.exp(normal(1, case["cols"]))  # a few channels carry much of a row
        s["x"] = normal(*shape).mul_(0.3).to(t)
        s["residual"] = (normal(*shape) * spread).to(t) if case["residual"] else None
        s["weight"] = 1.0 + 0.3 * normal(case["cols"])
    elif case["op"] == "rotary":
        t, n, pairs = DTYPES[case["dtype"]], case["tokens"], case["rot"] // 2
        heads = case["q_heads"] + 2 * case["k_heads"]
        qkv = normal(n, heads, case["dim"]).to(t)  # q, k and v of one projection
        s["q"], s["k"] = qkv[:, : case["q_heads"]], qkv[:, case["q_heads"]: case["q_heads"] + case["k_heads"]]
        s["positions"] = torch.randint(0, case["far"], (case["axes"], n), generator=gen, device=DEV, dtype=torch.int32)
        s["inv_freq"] = torch.pow(torch.full((pairs,), 1e6, dtype=torch.float64, device=DEV), -torch.arange(pairs, device=DEV, dtype=torch.float64) / pairs)
        s["axis"] = (torch.arange(pairs, device=DEV) * case["axes"] // pairs).int()  # sections in a row
    else:
        n, a, r = case["tokens"], case["adapters"], case["rank"]
        w = DTYPES[case["w"]]
        s["x"] = normal(n, case["cols"]).to(DTYPES[case["x"]])
        s["a"] = (normal(a, r, case["cols"]) / math.sqrt(case["cols"])).to(w)
        s["b"] = (normal(a, case["out"], r) * 0.2).to(w)
        s["scale"] = 0.5 + torch.rand(a, generator=gen, device=DEV)
        s["y"] = normal(n, case["out"]).to(DTYPES[case["y"]])
        ids = torch.randint(-1, a, (n,), generator=gen, device=DEV, dtype=torch.int32)  # some requests have none
        s["adapter"] = torch.sort(ids).values if case["runs"] else ids
    return s


def run(state):
    c = state["case"]
    if own:
        import block_quantized_weight_row_gb300 as bq

        if c["op"] == "extend":
            step = bq.paged_extend(c["page"], state["n_pages"], state["kv_len"], state["n_new"], state["page_table"], state["free_pages"],
                                   state["n_slots"])
            return {"page_table": state["page_table"], "q_start": step.q_start, "kv_len": step.kv_len, "slots": step.slots,
                    "positions": step.positions, "taken": step.taken}
        if c["op"] == "norm":
            n = bq.add_rms_norm(state["x"], state["weight"], EPS, residual=state["residual"], out=c["out"], q8=True)
            got = {"values": bq.dequantize_rows(Q8_0, n.q8, c["cols"])}
            if c["residual"]:
                got["sum"] = n.sum
            if c["out"]:
                got["out"] = n.out
            return got
        if c["op"] == "rotary":
            return bq.rotary(state["q"], state["k"], state["positions"], state["inv_freq"], state["axis"], interleaved=c["interleaved"])
        return bq.lora(state["x"], state["a"], state["b"], state["adapter"], state["y"], state["scale"])
    return {"extend": _plain_extend, "norm": _plain_norm, "rotary": _plain_rotary, "lora": _plain_lora}[c["op"]](state)


def work(case):
    if case["op"] == "extend":
        kv, new = _lengths(case)
        page = case["page"]
        pages = sum(-(-(a + b) // page) - -(-a // page) for a, b in zip(kv, new))
        return {"bytes": 16.0 * case["seqs"] + 8 * pages + 12 * (sum(new) + case["spare"]), "flops": 8.0 * sum(new)}
    if case["op"] == "norm":
        n, size = case["rows"] * case["cols"], SIZE[case["dtype"]]
        q8 = n * 34 / 32
        rows = 1 + 2 * case["residual"] + case["out"]  # x; the residual and the sum; the norm's rows
        return {"bytes": rows * n * size + 2 * q8 + 4 * n + 4 * case["cols"], "flops": 12.0 * n}  # the 8-bit rows written, read and given as values
    if case["op"] == "rotary":
        n = case["tokens"] * (case["q_heads"] + case["k_heads"]) * case["dim"]
        return {"bytes": 2.0 * n * SIZE[case["dtype"]] + 4 * case["tokens"] * case["axes"] + 6 * case["rot"], "flops": 3.0 * n}
    n, k, m, r = case["tokens"], case["cols"], case["out"], case["rank"]
    used = min(case["adapters"], n)
    return {"bytes": n * (k * SIZE[case["x"]] + 2 * m * SIZE[case["y"]] + 4) + 2.0 * used * r * (k + m), "flops": 2.0 * n * r * (k + m)}


# ----------------------------------------------------------------- exact --


def _f32(x):
    return x.float().double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "extend":
        return None  # whole numbers
    if case["op"] == "norm":
        t = DTYPES[case["dtype"]]
        h = s["x"].double()
        if case["residual"]:
            h = _f32(h + s["residual"].double()).to(t).double()
        # the norm is defined with a 32-bit factor and 32-bit products, so that its 8-bit codes are the same everywhere
        factor = _f32(torch.rsqrt(h.square().sum(-1) / case["cols"] + EPS))
        y = _f32(_f32(h * factor[:, None]) * s["weight"].double())
        v = y.unflatten(-1, (-1, 32))
        d = _f32(v.abs().amax(-1, keepdim=True) / 127).half().double()
        q = torch.where(d > 0, torch.round(_f32(v / torch.where(d > 0, d, 1.0))), 0.0).clamp(-127, 127)
        got = {"values": (q * d).flatten(-2)}
        if case["residual"]:
            got["sum"] = h
        if case["out"]:
            got["out"] = y
        return got
    if case["op"] == "rotary":
        pair = torch.arange(case["rot"], device=DEV)
        half = case["rot"] // 2
        pair, second = (pair // 2, pair % 2 == 1) if case["interleaved"] else (pair % half, pair >= half)
        other = torch.arange(case["rot"], device=DEV)
        other = torch.where(second, other - 1, other + 1) if case["interleaved"] else torch.where(second, other - half, other + half)
        theta = s["positions"].double().index_select(0, s["axis"].long()[pair]).T * s["inv_freq"][pair]
        sign = torch.where(second, 1.0, -1.0).double()
        got = []
        for name in ("q", "k"):
            x = s[name].double()
            x[..., : case["rot"]] = x[..., : case["rot"]] * theta.cos()[:, None] + sign * x[..., other] * theta.sin()[:, None]
            got.append(x)
        return tuple(got)
    out = s["y"].double()
    for a in range(case["adapters"]):
        rows = torch.nonzero(s["adapter"] == a).flatten()
        h = s["x"][rows].double() @ s["a"][a].double().T
        out[rows] += (h @ s["b"][a].double().T) * s["scale"][a].double()
    return out
