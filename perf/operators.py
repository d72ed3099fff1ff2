"""Workloads of the key-value cache operators: append, attend, evict.

A decoder's cache is a pool of pages; a table names the pages of each sequence.  One decoding step appends the new
token's keys and values (kv_append), attends to everything held while accumulating how much attention each slot got
(kv_attend), and now and then keeps the slots with the most accumulated attention (kv_evict).

Pools are indexed [page, slot in page, head, dim]; `layout` says how they lie in memory: "head" keeps a head's slots of
a page together, "token" keeps a token's heads together.
"""
import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # A decoding step's new token of each of 64 sequences: latency.
        {"name": "append_step", "op": "append", "dtype": "bf16", "seqs": 64, "len": 1, "held": 2047, "even": True,
         "heads": 8, "dim": 128, "page": 16, "layout": "head"},
        # Prompts of unequal lengths, behind what the sequences already hold.
        {"name": "append_prompts", "op": "append", "dtype": "f16", "seqs": 16, "len": 4093, "held": 77, "even": False,
         "heads": 8, "dim": 128, "page": 64, "layout": "token"},
        # One short sequence, a small model: the smallest call.
        {"name": "attend_one_short", "op": "attend", "dtype": "f16", "seqs": 1, "len": 300, "even": True, "empty": 0,
         "q_heads": 8, "heads": 2, "dim": 64, "page": 16, "layout": "head", "weights": True},
        # An ordinary batch of unequal lengths with grouped heads; one sequence holds nothing yet.
        {"name": "attend_batch", "op": "attend", "dtype": "bf16", "seqs": 32, "len": 4096, "even": False, "empty": 1,
         "q_heads": 32, "heads": 8, "dim": 128, "page": 16, "layout": "head", "weights": True},
        # A head of its own for every query head, narrow heads, pages laid out token by token.
        {"name": "attend_own_heads", "op": "attend", "dtype": "f16", "seqs": 24, "len": 2001, "even": False, "empty": 0,
         "q_heads": 16, "heads": 16, "dim": 64, "page": 32, "layout": "token", "weights": False},
        # One very long sequence: the length has to be split over the whole GPU.
        {"name": "attend_long", "op": "attend", "dtype": "bf16", "seqs": 1, "len": 131071, "even": True, "empty": 0,
         "q_heads": 64, "heads": 8, "dim": 128, "page": 128, "layout": "head", "weights": True},
        # All query heads on one key-value head, an odd number of them, a dim that is no power of two.
        {"name": "attend_shared_head", "op": "attend", "dtype": "bf16", "seqs": 40, "len": 9001, "even": False,
         "empty": 0, "q_heads": 12, "heads": 1, "dim": 96, "page": 64, "layout": "token", "weights": True},
        # A full batch of long sequences: the largest.
        {"name": "attend_full", "op": "attend", "dtype": "bf16", "seqs": 64, "len": 16384, "even": False, "empty": 0,
         "q_heads": 64, "heads": 8, "dim": 128, "page": 64, "layout": "head", "weights": False},
        # A small batch a little over its budget.
        {"name": "evict_small", "op": "evict", "dtype": "f16", "seqs": 4, "len": 1101, "even": False, "heads": 8,
         "dim": 64, "page": 16, "layout": "head", "budget": 1024, "sink": 4, "recent": 64},
        # An ordinary batch; some sequences are still below the budget.
        {"name": "evict_batch", "op": "evict", "dtype": "bf16", "seqs": 32, "len": 4500, "even": False, "heads": 8,
         "dim": 128, "page": 16, "layout": "head", "budget": 2048, "sink": 4, "recent": 256},
        # One long prompt cut to an eighth: few rows, each long.
        {"name": "evict_long", "op": "evict", "dtype": "bf16", "seqs": 1, "len": 131072, "even": True, "heads": 8,
         "dim": 128, "page": 128, "layout": "token", "budget": 16384, "sink": 16, "recent": 1024},
        # A full batch cut to half.
        {"name": "evict_full", "op": "evict", "dtype": "bf16", "seqs": 64, "len": 8192, "even": True, "heads": 8,
         "dim": 128, "page": 64, "layout": "head", "budget": 4096, "sink": 4, "recent": 512},
    ]


def _log(rng, low, high):
    return int(round(low * (high / low) ** rng.random()))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "evict"])
    case = {"op": op, "dtype": rng.choice(["bf16", "f16"]), "seqs": _log(rng, 1, 64), "even": rng.random() < 0.3,
            "heads": rng.choice([1, 2, 4, 5, 8, 16]), "dim": rng.choice([64, 80, 96, 128, 128, 256]),
            "page": rng.choice([8, 16, 32, 48, 64, 128, 256]), "layout": rng.choice(["head", "token"])}
    row = case["seqs"] * case["heads"] * case["dim"]  # values per token of every sequence
    if op == "append":
        case["len"] = _log(rng, 1, max(1, min(8192, (1 << 26) // row)))
        case["held"] = _log(rng, 1, 2048) - 1
    elif op == "attend":
        case["len"] = _log(rng, 1, max(1, min(131072, (1 << 29) // row)))
        case["q_heads"] = case["heads"] * rng.choice([1, 1, 2, 3, 4, 7, 8, 12, 16])
        case["empty"] = rng.choice([0, 0, 1]) if case["seqs"] > 1 else 0
        case["weights"] = rng.random() < 0.6
    else:
        case["len"] = _log(rng, 40, max(80, min(131072, (1 << 28) // row)))
        case["budget"] = max(16, int(case["len"] * rng.choice([0.1, 0.25, 0.5, 0.9])))
        case["sink"] = rng.choice([0, 1, 4])
        case["recent"] = rng.choice([0, case["budget"] // 8, case["budget"] // 2])
    return case


def _lens(case):
    """The sequences' lengths: all alike, or spread from about a quarter of `len` to `len` in a shuffled order."""
    n, top = case["seqs"], case["len"]
    if case["even"] or n == 1:
        lens = [top] * n
    else:
        lens = [max(1, top - (top * 3 // 4) * ((i * 7) % n) // max(1, n - 1)) for i in range(n)]
    for i in range(case.get("empty", 0)):
        lens[-1 - i] = 0
    return lens


def _randn(gen, *shape, dtype):
    return torch.randn(*shape, dtype=dtype, device="cuda", generator=gen)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    seqs, heads, dim, page = case["seqs"], case["heads"], case["dim"], case["page"]
    lens = _lens(case)
    held = case.get("held", 0)
    width = -(-(max(lens) + held) // page)  # pages a sequence's row of the table has room for
    pages = seqs * width
    # The pages that a sequence got over time, in no order.
    table = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32).reshape(seqs, width)
    shape = (pages, heads, page, dim) if case["layout"] == "head" else (pages, page, heads, dim)
    k, v = (_randn(gen, *shape, dtype=dtype) for _ in range(2))
    if case["layout"] == "head":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    state = {"op": case["op"], "k": k, "v": v, "table": table}
    cap = width * page
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    # Accumulated attention is heavy-tailed, and slots that nothing has looked at hold 0.
    weight = torch.exp(2 * torch.randn(seqs, heads, cap, device="cuda", generator=gen))
    weight *= torch.rand(seqs, heads, cap, device="cuda", generator=gen) > 0.05
    if case["op"] == "append":
        starts = np.concatenate([[0], np.cumsum(lens)])
        state["lens"] = torch.full((seqs,), held, dtype=torch.int32, device="cuda")
        state["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        state["k_new"], state["v_new"] = (_randn(gen, int(starts[-1]), heads, dim, dtype=dtype) for _ in range(2))
        state["weight"] = weight
        state["pos"] = torch.full((seqs, heads, cap), -1, dtype=torch.int32, device="cuda")
        state["next_pos"] = state["lens"] + torch.randint(0, 1000, (seqs,), dtype=torch.int32, device="cuda",
                                                          generator=gen)
    elif case["op"] == "attend":
        state["lens"] = lens_t
        # Sharper than unit scores: a few slots carry most of a head's attention.
        state["q"] = 2 * _randn(gen, seqs, case["q_heads"], dim, dtype=dtype)
        state["scale"] = dim ** -0.5
        if case["weights"]:
            state["weight"] = weight
            state["weight_out"] = torch.zeros_like(weight)
    else:
        state["lens"] = lens_t
        state["weight"] = weight
        # Slots do not lie in the order of time once a cache has been evicted from; the newest tokens come last.
        old = max(1, case["len"] // 2)
        pos = torch.arange(cap, dtype=torch.int32, device="cuda").repeat(seqs, heads, 1)
        pos[:, :, :old] = torch.argsort(torch.rand(seqs, heads, old, device="cuda", generator=gen), -1).to(torch.int32)
        state["pos"] = pos
        state["next_pos"] = lens_t.clone()
        keep = min(case["budget"], cap)
        state["weight_out"] = torch.zeros(seqs, heads, keep, device="cuda")
        state["pos_out"] = torch.zeros(seqs, heads, keep, dtype=torch.int32, device="cuda")
        state["lens_out"] = torch.zeros_like(lens_t)
        state.update({n: case[n] for n in ("budget", "sink", "recent")})
    return state


def _plain_append(s):
    k, v, table, page = s["k"], s["v"], s["table"].long(), s["k"].shape[1]
    starts = s["starts"].long()
    tokens = torch.arange(s["k_new"].shape[0], device="cuda")
    seq = (tokens[:, None] >= starts[None, 1:]).sum(1)
    at = tokens - starts[seq]
    slot = s["lens"].long()[seq] + at
    where = table[seq, slot // page], slot % page
    k[where] = s["k_new"]
    v[where] = s["v_new"]
    s["weight"][seq, :, slot] = 0
    s["pos"][seq, :, slot] = (s["next_pos"].long()[seq] + at).to(torch.int32)[:, None]
    return {"k": k, "v": v, "weight": s["weight"], "pos": s["pos"]}


def _plain_attend(s):
    q, table, page = s["q"], s["table"].long(), s["k"].shape[1]
    seqs, heads, dim = q.shape[0], s["k"].shape[2], q.shape[2]
    cap = table.shape[1] * page
    k, v = (p[table].reshape(seqs, cap, heads, dim).permute(0, 2, 1, 3).float() for p in (s["k"], s["v"]))
    held = torch.arange(cap, device="cuda")[None, :] < s["lens"][:, None]
    held = held[:, None, None, :]
    # One product per key-value head, with its group of query heads as rows.
    score = q.float().reshape(seqs, heads, -1, dim) @ k.transpose(2, 3) * s["scale"]
    top = torch.where(held, score, -torch.inf).amax(-1, keepdim=True)
    top = torch.where(top == -torch.inf, 0.0, top)
    e = torch.where(held, torch.exp(score - top), 0.0)
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total > 0, total, 1.0)
    out = (p @ v).reshape(seqs, -1, dim).to(q.dtype)
    lse = (top + torch.log(total)).reshape(seqs, -1)
    if "weight" not in s:
        return {"out": out, "lse": lse}
    weight = torch.where(held[:, 0], s["weight"] + p.sum(2), s["weight_out"])
    return {"out": out, "lse": lse, "weight": weight}


def _plain_evict(s):
    k, v, table, page = s["k"], s["v"], s["table"].long(), s["k"].shape[1]
    weight, pos, lens = s["weight"], s["pos"], s["lens"][:, None, None]
    slot = torch.arange(weight.shape[2], device="cuda")
    held = (slot < lens).expand_as(weight)
    safe = (pos < s["sink"]) | (pos >= s["next_pos"][:, None, None] - s["recent"])
    key = torch.where(held, torch.where(safe, torch.inf, weight), -torch.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, slot.expand_as(order).contiguous())
    kept = held & (rank < s["budget"])
    low = slot < s["budget"]
    # Per row there are as many kept slots above the budget as holes below it, and both come in order.
    src, dst = torch.nonzero(kept & ~low).unbind(1), torch.nonzero(held & ~kept & low).unbind(1)
    stay = torch.nonzero(kept & low).unbind(1)
    for name in ("weight", "pos"):
        s[name + "_out"][stay] = s[name][stay]
        s[name + "_out"][dst] = s[name][src]
    (b, h, at), to = src, dst[2]
    for p in (k, v):
        p[table[b, to // page], to % page, h] = p[table[b, at // page], at % page, h]
    s["lens_out"].copy_(torch.clamp(s["lens"], max=s["budget"]))
    return {"k": k, "v": v, "weight": s["weight_out"], "pos": s["pos_out"], "lens": s["lens_out"]}


def run(s):
    if not own:
        return {"append": _plain_append, "attend": _plain_attend, "evict": _plain_evict}[s["op"]](s)
    import topk_selection_gb300 as tk

    if s["op"] == "append":
        tk.kv_append(s["k"], s["v"], s["table"], s["lens"], s["k_new"], s["v_new"], starts=s["starts"],
                     weight=s["weight"], pos=s["pos"], next_pos=s["next_pos"])
        return {"k": s["k"], "v": s["v"], "weight": s["weight"], "pos": s["pos"]}
    if s["op"] == "attend":
        weights = "weight" in s
        out, lse = tk.kv_attend(s["q"], s["k"], s["v"], s["table"], s["lens"], scale=s["scale"],
                                weight=s["weight"] if weights else None,
                                weight_out=s["weight_out"] if weights else None)
        return {"out": out, "lse": lse, "weight": s["weight_out"]} if weights else {"out": out, "lse": lse}
    weight, pos, lens = tk.kv_evict(s["k"], s["v"], s["table"], s["lens"], s["weight"], s["pos"], s["next_pos"],
                                    s["budget"], sink=s["sink"], recent=s["recent"], weight_out=s["weight_out"],
                                    pos_out=s["pos_out"], lens_out=s["lens_out"])
    return {"k": s["k"], "v": s["v"], "weight": weight, "pos": pos, "lens": lens}


def work(case):
    lens, heads, dim = _lens(case), case["heads"], case["dim"]
    tokens = sum(lens)
    pair = 2 * dim * 2  # a key and a value, 2 bytes each
    if case["op"] == "append":
        return {"bytes": tokens * heads * (2 * pair + 8) + 12 * case["seqs"], "flops": 0}
    if case["op"] == "attend":
        rows = case["seqs"] * case["q_heads"]
        side = 8 * tokens * heads if case["weights"] else 0
        return {"bytes": tokens * heads * pair + side + rows * (4 * dim + 4) + 4 * case["seqs"],
                "flops": 4 * tokens * case["q_heads"] * dim}
    moves, kept = 0.0, 0
    for n in lens:
        kept += min(n, case["budget"])
        if n > case["budget"]:
            # The newest tokens lie above the budget as far as they can; of the others, the share that is kept.
            above, newest = n - case["budget"], case["recent"]
            moves += min(newest, above) + max(0, above - newest) * (case["budget"] - newest) / (n - newest)
    return {"bytes": heads * (8 * (tokens + kept) + 2 * pair * moves), "flops": 0}


def exact(case, seed):
    s = prepare(case, seed)
    page, table = s["k"].shape[1], s["table"].cpu().numpy()
    if case["op"] == "append":
        k, v, weight, pos = s["k"], s["v"], s["weight"], s["pos"]
        first = 0
        for b, n in enumerate(_lens(case)):
            for i in range(0, n):
                if i and (case["held"] + i) % page:
                    continue
                at = case["held"] + i  # a run of slots inside one page
                count = min(n - i, page - at % page)
                for new, pool in ((s["k_new"], k), (s["v_new"], v)):
                    pool[table[b, at // page], at % page:at % page + count] = new[first + i:first + i + count]
            weight[b, :, case["held"]:case["held"] + n] = 0
            pos[b, :, case["held"]:case["held"] + n] = int(s["next_pos"][b]) + torch.arange(n, dtype=torch.int32,
                                                                                            device="cuda")
            first += n
        return {"k": k, "v": v, "weight": weight, "pos": pos}
    if case["op"] == "attend":
        group = case["q_heads"] // case["heads"]
        out = torch.zeros(*s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(out.shape[:2], -torch.inf, dtype=torch.float64, device="cuda")
        weight = s["weight_out"].double() if case["weights"] else None
        for b, n in enumerate(_lens(case)):
            if n == 0:
                continue
            pages = s["table"][b, :-(-n // page)].long()
            k, v = (p[pages].reshape(-1, case["heads"], case["dim"])[:n].double() for p in (s["k"], s["v"]))
            for h in range(case["heads"]):
                mine = slice(h * group, (h + 1) * group)
                score = s["scale"] * (k[:, h] @ s["q"][b, mine].double().T)
                lse[b, mine] = torch.logsumexp(score, 0)
                p = torch.exp(score - lse[b, mine])
                out[b, mine] = p.T @ v[:, h]
                if weight is not None:
                    weight[b, h, :n] = s["weight"][b, h, :n].double() + p.sum(1)
        return {"out": out, "lse": lse, "weight": weight} if weight is not None else {"out": out, "lse": lse}
    weight, pos, lens = s["weight"].cpu().numpy(), s["pos"].cpu().numpy(), _lens(case)
    w_out, p_out = s["weight_out"].cpu().numpy().astype(np.float64), s["pos_out"].cpu().numpy()
    budget = case["budget"]
    moved = []
    for b, n in enumerate(lens):
        for h in range(case["heads"]):
            source = np.arange(min(n, budget))
            if n > budget:
                safe = (pos[b, h, :n] < case["sink"]) | (pos[b, h, :n] >= n - case["recent"])
                kept = np.lexsort((np.arange(n), -weight[b, h, :n].astype(np.float64), ~safe))[:budget]
                holes = np.setdiff1d(source, kept)
                source[holes] = np.sort(kept[kept >= budget])
                moved += [(table[b, o // page], o % page, table[b, i // page], i % page, h)
                          for i, o in zip(holes.tolist(), source[holes].tolist())]
            w_out[b, h, :source.size] = weight[b, h, source]
            p_out[b, h, :source.size] = pos[b, h, source]
    if moved:
        sp, so, dp, do, h = torch.tensor(np.array(moved), device="cuda").long().unbind(1)
        for p in (s["k"], s["v"]):
            p[dp, do, h] = p[sp, so, h]
    return {"k": s["k"], "v": s["v"], "weight": w_out, "pos": p_out,
            "lens": torch.tensor([min(n, budget) for n in lens], dtype=torch.int32)}
