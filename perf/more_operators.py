"""Workloads of the operators at both ends of a decoding step: kv_rotate, kv_append_rotated, sample_rows.

What a projection gives becomes queries and keys by a norm of each head and the position rotation (kv_rotate), on the
way into the pages of a bounded cache where there is one (kv_append_rotated).  What the last projection gives becomes a
token (sample_rows): from the distribution with temperature, cut off by top-k, top-p and min-p, by one given uniform
number per row.

An angle is position times frequency, and a far position's is not known to a 32-bit product: angles are 64-bit here.
A token is the first of the descending order (ties: the lower column) whose running sum passes u times the kept sum:
next to a border 32 bits would name its neighbour, so sums are 64-bit too.
"""
import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # A decoding step's queries and keys of 64 sequences at far positions: latency.
        {"name": "rotate_step", "op": "rotate", "dtype": "bf16", "tokens": 64, "q_heads": 64, "heads": 8, "dim": 128,
         "rot": 128, "pairing": "halves", "norm": "shared", "fused": False, "far": 131072},
        # A prompt of odd length, views of one fused projection, half of each narrow head rotated, pairs side by side.
        {"name": "rotate_partial", "op": "rotate", "dtype": "f16", "tokens": 4093, "q_heads": 16, "heads": 16,
         "dim": 80, "rot": 40, "pairing": "neighbours", "norm": "none", "fused": True, "far": 0},
        # Long prompts, every head with a norm weight of its own: the largest.
        {"name": "rotate_prompts", "op": "rotate", "dtype": "bf16", "tokens": 20011, "q_heads": 64, "heads": 8,
         "dim": 128, "rot": 128, "pairing": "halves", "norm": "own", "fused": True, "far": 0},
        # A decoding step of 64 sequences, queries with it; positions run ahead of the slots, as after an eviction.
        {"name": "append_step", "op": "append", "dtype": "bf16", "seqs": 64, "len": 1, "held": 2047, "even": True,
         "q_heads": 32, "heads": 8, "dim": 128, "rot": 128, "pairing": "halves", "norm": "shared", "page": 16,
         "layout": "head", "ahead": 30000},
        # Prompts of unequal lengths behind what is held, keys and values only, a quarter of each head rotated.
        {"name": "append_keys", "op": "append", "dtype": "f16", "seqs": 16, "len": 1021, "held": 77, "even": False,
         "q_heads": 0, "heads": 8, "dim": 128, "rot": 32, "pairing": "halves", "norm": "none", "page": 64,
         "layout": "token", "ahead": 0},
        # The same with queries and norms, and longer: the largest.
        {"name": "append_prompts", "op": "append", "dtype": "bf16", "seqs": 16, "len": 4093, "held": 77, "even": False,
         "q_heads": 32, "heads": 8, "dim": 128, "rot": 128, "pairing": "halves", "norm": "shared", "page": 64,
         "layout": "head", "ahead": 0},
        # One user's next token: the smallest call, latency.
        {"name": "sample_one", "op": "sample", "dtype": "bf16", "rows": 1, "cols": 131072, "spread": 2.5,
         "temperature": 0.7, "top_k": 50, "top_p": 0.95, "min_p": 0.0, "mixed": False, "masked": 0.0},
        # A batch from the whole distribution, nothing cut off, flat rows of a small vocabulary in 16 bits: many ties.
        {"name": "sample_flat", "op": "sample", "dtype": "f16", "rows": 128, "cols": 32768, "spread": 1.0,
         "temperature": 1.0, "top_k": 0, "top_p": 1.0, "min_p": 0.0, "mixed": False, "masked": 0.0},
        # An ordinary batch cut by top-p alone, an odd number of columns.
        {"name": "sample_top_p", "op": "sample", "dtype": "f32", "rows": 64, "cols": 131001, "spread": 2.5,
         "temperature": 1.0, "top_k": 0, "top_p": 0.95, "min_p": 0.0, "mixed": False, "masked": 0.0},
        # A large batch with top-k and top-p, as most requests have them.
        {"name": "sample_top_k", "op": "sample", "dtype": "bf16", "rows": 256, "cols": 160000, "spread": 2.5,
         "temperature": 0.8, "top_k": 50, "top_p": 0.95, "min_p": 0.0, "mixed": False, "masked": 0.0},
        # Every request with parameters of its own (some greedy), half of the columns forbidden by a grammar.
        {"name": "sample_mixed", "op": "sample", "dtype": "bf16", "rows": 200, "cols": 131072, "spread": 3.0,
         "temperature": 1.0, "top_k": 0, "top_p": 1.0, "min_p": 0.0, "mixed": True, "masked": 0.5},
        # The largest: many rows of a large vocabulary in 32 bits, cut by min-p.
        {"name": "sample_full", "op": "sample", "dtype": "f32", "rows": 512, "cols": 262144, "spread": 2.5,
         "temperature": 1.0, "top_k": 0, "top_p": 1.0, "min_p": 0.02, "mixed": False, "masked": 0.0},
    ]


def _log(rng, low, high):
    return int(round(low * (high / low) ** rng.random()))


def draw(rng):
    op = rng.choice(["rotate", "append", "sample", "sample"])
    if op == "sample":
        rows = _log(rng, 1, 512)
        cols = _log(rng, 1000, 262144)
        return {"op": op, "dtype": rng.choice(["bf16", "f16", "f32"]), "rows": rows, "cols": cols,
                "spread": rng.choice([0.5, 1.0, 2.0, 2.5, 3.0, 4.0]),
                "temperature": rng.choice([0.3, 0.7, 0.8, 1.0, 1.0, 1.4]),
                "top_k": rng.choice([0, 0, 1, 20, 50, 200, 3000]), "top_p": rng.choice([1.0, 1.0, 0.99, 0.95, 0.9, 0.6]),
                "min_p": rng.choice([0.0, 0.0, 0.01, 0.05, 0.2]), "mixed": rng.random() < 0.25,
                "masked": rng.choice([0.0, 0.0, 0.3, 0.9])}
    case = {"op": op, "dtype": rng.choice(["bf16", "f16"]), "heads": rng.choice([1, 2, 4, 5, 8, 16]),
            "dim": rng.choice([64, 80, 96, 128, 128, 256]), "pairing": rng.choice(["halves", "halves", "neighbours"]),
            "norm": rng.choice(["none", "shared", "shared", "own"])}
    case["rot"] = case["dim"] // rng.choice([1, 1, 1, 2, 4]) // 2 * 2
    case["q_heads"] = case["heads"] * rng.choice([1, 2, 4, 7, 8])
    row = (case["q_heads"] + 2 * case["heads"]) * case["dim"]  # values per token
    if op == "rotate":
        case["tokens"] = _log(rng, 1, min(32768, (1 << 27) // row))
        case["fused"] = rng.random() < 0.5
        case["far"] = rng.choice([0, 0, 131072, 1000000])
        return case
    case["seqs"] = _log(rng, 1, 64)
    case["len"] = _log(rng, 1, max(1, min(8192, (1 << 27) // (row * case["seqs"]))))
    case["held"] = _log(rng, 1, 2048) - 1
    case["even"] = rng.random() < 0.3
    case["page"] = rng.choice([8, 16, 32, 48, 64, 128, 256])
    case["layout"] = rng.choice(["head", "token"])
    case["ahead"] = rng.choice([0, 0, 30000, 1000000])
    if rng.random() < 0.3:
        case["q_heads"] = 0
    return case


def _lens(case):
    """New tokens of each sequence: all alike, or spread from about a quarter of `len` to `len` in a shuffled order."""
    n, top = case["seqs"], case["len"]
    if case["even"] or n == 1:
        return [top] * n
    return [max(1, top - (top * 3 // 4) * ((i * 7) % n) // max(1, n - 1)) for i in range(n)]


def _randn(gen, *shape, dtype):
    return torch.randn(*shape, dtype=dtype, device="cuda", generator=gen)


def _heads(gen, case, tokens, parts, fused):
    """Tensors [tokens, heads, dim] of one projection: views of one array, or an array each."""
    dim, dtype = case["dim"], DTYPES[case["dtype"]]
    if not fused:
        return [_randn(gen, tokens, h, dim, dtype=dtype) for h in parts]
    return list(_randn(gen, tokens, sum(parts), dim, dtype=dtype).split(parts, 1))


def _norm(gen, case, heads):
    if case["norm"] == "none":
        return None
    shape = (case["dim"],) if case["norm"] == "shared" else (heads, case["dim"])
    return (1 + 0.2 * torch.randn(*shape, device="cuda", generator=gen)).to(DTYPES[case["dtype"]])


def _freq(case):
    half = case["rot"] // 2
    return (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).to(torch.float32).cuda()


def _prepare_sample(case, gen):
    rows, cols = case["rows"], case["cols"]
    # A projection's logits: some rows are sure of their token, some are not.
    sure = 0.6 + 0.8 * torch.rand(rows, 1, device="cuda", generator=gen)
    x = torch.randn(rows, cols, device="cuda", generator=gen).mul_(case["spread"] * sure)
    if case["masked"]:
        x.masked_fill_(torch.rand(rows, cols, device="cuda", generator=gen) < case["masked"], -torch.inf)
        x[:, cols // 2] = 0.0  # never everything
    state = {"op": "sample", "logits": x.to(DTYPES[case["dtype"]]),
             "u": torch.rand(rows, device="cuda", generator=gen)}
    names = {"temperature": [0.0, 0.3, 0.7, 1.0, 1.0, 1.3], "top_k": [0, 0, 1, 20, 50, 1000],
             "top_p": [1.0, 1.0, 0.99, 0.95, 0.8, 0.5], "min_p": [0.0, 0.0, 0.0, 0.02, 0.1]}
    for name, choices in names.items():
        state[name] = case[name]
        if case["mixed"]:
            choices = torch.tensor(choices, dtype=torch.int32 if name == "top_k" else torch.float32, device="cuda")
            state[name] = choices[torch.randint(0, len(choices), (rows,), device="cuda", generator=gen)]
    return state


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if case["op"] == "sample":
        return _prepare_sample(case, gen)
    dtype, heads, q_heads, dim = DTYPES[case["dtype"]], case["heads"], case["q_heads"], case["dim"]
    state = {"op": case["op"], "freq": _freq(case), "pairing": case["pairing"], "eps": 1e-6,
             "q_norm": _norm(gen, case, q_heads) if q_heads else None, "k_norm": _norm(gen, case, heads)}
    if case["op"] == "rotate":
        n = case["tokens"]
        state["q"], state["k"] = _heads(gen, case, n, [q_heads, heads, heads], case["fused"])[:2]
        state["pos"] = torch.arange(n, dtype=torch.int32, device="cuda")
        if case["far"]:  # tokens of many sequences, each somewhere in its own
            state["pos"] = torch.randint(0, case["far"], (n,), dtype=torch.int32, device="cuda", generator=gen)
        state["q_out"], state["k_out"] = (torch.empty(n, h, dim, dtype=dtype, device="cuda") for h in (q_heads, heads))
        return state
    lens, held, page, seqs = _lens(case), case["held"], case["page"], case["seqs"]
    width = -(-(max(lens) + held) // page)
    pages = seqs * width
    # The pages that a sequence got over time, in no order.
    state["table"] = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32).reshape(seqs, width)
    shape = (pages, heads, page, dim) if case["layout"] == "head" else (pages, page, heads, dim)
    k, v = (_randn(gen, *shape, dtype=dtype) for _ in range(2))
    if case["layout"] == "head":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    state["k"], state["v"] = k, v
    starts = np.concatenate([[0], np.cumsum(lens)])
    n = int(starts[-1])
    state["lens"] = torch.full((seqs,), held, dtype=torch.int32, device="cuda")
    state["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    new = _heads(gen, case, n, [q_heads, heads, heads] if q_heads else [heads, heads], True)
    state["k_new"], state["v_new"] = new[-2:]
    state["q"] = new[0] if q_heads else None
    state["q_out"] = torch.empty(n, q_heads, dim, dtype=dtype, device="cuda") if q_heads else None
    cap = width * page
    state["weight"] = torch.exp(2 * torch.randn(seqs, heads, cap, device="cuda", generator=gen))
    state["pos"] = torch.full((seqs, heads, cap), -1, dtype=torch.int32, device="cuda")
    state["next_pos"] = state["lens"] + torch.randint(0, case["ahead"] + 1, (seqs,), dtype=torch.int32, device="cuda",
                                                      generator=gen)
    return state


def _plain_rotate(x, pos, norm, s):
    """Norm and rotation of [tokens, heads, dim] at positions [tokens]."""
    y = x.float()
    if norm is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + s["eps"]) * norm.float()
    angle = pos.double()[:, None, None] * s["freq"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    half = cos.shape[-1]
    y = y.clone() if y is x else y
    if s["pairing"] == "halves":
        a, b = y[..., :half], y[..., half:2 * half]
    else:
        a, b = y[..., :2 * half:2], y[..., 1:2 * half:2]
    new_a, new_b = a * cos - b * sin, b * cos + a * sin
    a.copy_(new_a)
    b.copy_(new_b)
    return y.to(x.dtype)


def _plain_append(s):
    k, v, table, page = s["k"], s["v"], s["table"].long(), s["k"].shape[1]
    starts = s["starts"].long()
    tokens = torch.arange(s["k_new"].shape[0], device="cuda")
    seq = (tokens[:, None] >= starts[None, 1:]).sum(1)
    at = tokens - starts[seq]
    slot, pos = s["lens"].long()[seq] + at, s["next_pos"].long()[seq] + at
    where = table[seq, slot // page], slot % page
    k[where] = _plain_rotate(s["k_new"], pos, s["k_norm"], s)
    v[where] = s["v_new"]
    s["weight"][seq, :, slot] = 0
    s["pos"][seq, :, slot] = pos.to(torch.int32)[:, None]
    out = {"k": k, "v": v, "weight": s["weight"], "pos": s["pos"]}
    if s["q"] is not None:
        out["q"] = _plain_rotate(s["q"], pos, s["q_norm"], s)
    return out


def _column(value, like, dtype):
    """A parameter as a column: its own number for each row, or one for all."""
    if isinstance(value, torch.Tensor):
        return value.to(dtype)[:, None]
    return torch.full((like.shape[0], 1), value, dtype=torch.float32, device=like.device).to(dtype)


def _plain_sample(s):
    x = s["logits"]
    rows, cols = x.shape
    temperature, top_p, min_p = (_column(s[n], x, torch.float64) for n in ("temperature", "top_p", "min_p"))
    top_k = _column(s["top_k"], x, torch.int64)
    value, order = torch.sort(x, dim=-1, descending=True, stable=True)
    greedy = temperature == 0
    value = value.double()
    value = (value - value[:, :1]) / torch.where(greedy, 1.0, temperature)
    mass = torch.cumsum(torch.exp(value), -1)
    rank = torch.arange(cols, device="cuda")
    count = torch.where((top_k > 0) & (top_k < cols), top_k, cols)
    whole = mass.gather(1, count - 1)
    # The entries before which less than top_p of the mass lies; all of them, but of the sum's last place, where it is 1.
    before = torch.cat([torch.zeros_like(mass[:, :1]), mass[:, :-1]], 1)
    kept = (rank < count) & ((before < top_p * whole) | (top_p >= 1)) & (value >= torch.log(min_p))
    kept[:, 0] = True
    kept &= (rank == 0) | ~greedy
    total = mass.gather(1, kept.sum(1, keepdim=True) - 1)
    at = (mass <= s["u"].double()[:, None] * total).sum(1, keepdim=True)
    at = torch.minimum(at, kept.sum(1, keepdim=True) - 1)
    logp = value.gather(1, at) - torch.log(total)
    return {"token": order.gather(1, at)[:, 0].to(torch.int32), "logp": logp[:, 0].float()}


def run(s):
    if not own:
        if s["op"] == "sample":
            return _plain_sample(s)
        if s["op"] == "append":
            return _plain_append(s)
        return {"q": _plain_rotate(s["q"], s["pos"], s["q_norm"], s),
                "k": _plain_rotate(s["k"], s["pos"], s["k_norm"], s)}
    import topk_selection_gb300 as tk

    if s["op"] == "sample":
        token, logp = tk.sample_rows(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
                                     top_p=s["top_p"], min_p=s["min_p"])
        return {"token": token, "logp": logp}
    if s["op"] == "rotate":
        q, k = tk.kv_rotate(s["q"], s["k"], s["pos"], s["freq"], q_norm=s["q_norm"], k_norm=s["k_norm"],
                            eps=s["eps"], pairing=s["pairing"], q_out=s["q_out"], k_out=s["k_out"])
        return {"q": q, "k": k}
    q = tk.kv_append_rotated(s["k"], s["v"], s["table"], s["lens"], s["k_new"], s["v_new"], s["freq"],
                             starts=s["starts"], weight=s["weight"], pos=s["pos"], next_pos=s["next_pos"],
                             k_norm=s["k_norm"], eps=s["eps"], pairing=s["pairing"], q=s["q"], q_norm=s["q_norm"],
                             q_out=s["q_out"])
    out = {"k": s["k"], "v": s["v"], "weight": s["weight"], "pos": s["pos"]}
    if q is not None:
        out["q"] = q
    return out


def work(case):
    if case["op"] == "sample":
        values = case["rows"] * case["cols"]
        # The logits once; a uniform number and the parameters in, a token and its logarithm out.  A scaling, an
        # exponential and a sum each.
        return {"bytes": values * SIZES[case["dtype"]] + case["rows"] * (28 if case["mixed"] else 12),
                "flops": 3 * values}
    dim, heads, q_heads = case["dim"], case["heads"], case["q_heads"]
    tokens = case["tokens"] if case["op"] == "rotate" else sum(_lens(case))
    turned = tokens * (q_heads + heads) * dim
    # Three operations a turned element, four for the norm of any.
    flops = (3 * case["rot"] + (4 * dim if case["norm"] != "none" else 0)) * (turned // dim)
    if case["op"] == "rotate":
        return {"bytes": 4 * turned + 4 * tokens, "flops": flops}
    return {"bytes": 4 * (turned + tokens * heads * dim) + 8 * tokens * heads + 12 * case["seqs"], "flops": flops}


def _exact_rotate(x, pos, norm, case):
    y = x.double()
    if norm is not None:
        y = y / (torch.linalg.vector_norm(y, dim=-1, keepdim=True) ** 2 / case["dim"] + 1e-6).sqrt() * norm.double()
    half = case["rot"] // 2
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"),
                       torch.outer(pos.double(), _freq(case).double()))[:, None, :]
    if case["pairing"] == "halves":
        z = torch.complex(y[..., :half], y[..., half:2 * half]) * turn
        return torch.cat([z.real, z.imag, y[..., 2 * half:]], -1)
    z = torch.view_as_complex(y[..., :2 * half].reshape(*y.shape[:-1], half, 2).contiguous()) * turn
    return torch.cat([torch.view_as_real(z).flatten(-2), y[..., 2 * half:]], -1)


def _exact_sample(case, s):
    rows, cols = s["logits"].shape
    given = {}
    for n in ("temperature", "top_k", "top_p", "min_p"):
        v = s[n] if isinstance(s[n], torch.Tensor) else torch.full((rows,), s[n], dtype=torch.float32)
        given[n] = v.cpu().numpy().astype(np.float64)
    u = s["u"].cpu().numpy().astype(np.float64)
    token, logp = np.zeros(rows, np.int32), np.zeros(rows)
    for r in range(rows):
        x = s["logits"][r].double()
        # Descending, the lower column first: ascending in the negated value, which keeps the order of equals.
        neg, order = torch.sort(-x, stable=True)
        if given["temperature"][r] == 0:
            token[r] = int(order[0])
            continue
        z = (neg[0] - neg) / given["temperature"][r]
        running = torch.exp(z).cumsum(0).cpu().numpy()
        n = cols
        if 0 < given["top_k"][r] < cols:
            n = int(given["top_k"][r])
        keep = n
        if given["top_p"][r] < 1:
            keep = min(keep, int(np.searchsorted(running[:n], given["top_p"][r] * running[n - 1], "left")) + 1)
        if given["min_p"][r] > 0:
            keep = min(keep, max(1, int((z >= np.log(given["min_p"][r])).sum())))
        at = min(keep - 1, int(np.searchsorted(running[:keep], u[r] * running[keep - 1], "right")))
        token[r] = int(order[at])
        logp[r] = float(z[at]) - np.log(running[keep - 1])
    return {"token": token, "logp": logp}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sample":
        return _exact_sample(case, s)
    if case["op"] == "rotate":
        return {n: _exact_rotate(s[n], s["pos"], s[n + "_norm"], case) for n in ("q", "k")}
    lens, page, held = _lens(case), case["page"], case["held"]
    table = s["table"].cpu().numpy()
    next_pos = s["next_pos"].cpu().numpy().astype(np.int64)
    pos = torch.tensor(np.concatenate([next_pos[b] + np.arange(n) for b, n in enumerate(lens)]), device="cuda")
    keys = _exact_rotate(s["k_new"], pos, s["k_norm"], case)
    k, v, first = s["k"].double(), s["v"], 0
    for b, n in enumerate(lens):
        at = held
        while at < held + n:  # a run of slots inside one page
            count = min(held + n - at, page - at % page)
            new = slice(first + at - held, first + at - held + count)
            k[table[b, at // page], at % page:at % page + count] = keys[new]
            v[table[b, at // page], at % page:at % page + count] = s["v_new"][new]
            at += count
        s["weight"][b, :, held:held + n] = 0
        s["pos"][b, :, held:held + n] = pos[first:first + n].to(torch.int32)
        first += n
    out = {"k": k, "v": v, "weight": s["weight"], "pos": s["pos"]}
    if s["q"] is not None:
        out["q"] = _exact_rotate(s["q"], pos, s["q_norm"], case)
    return out
