"""The key-value cache operators against their definitions in 64 bits.

Copies (append, evict) have to be exact; attention is held to bounds that
tests/_kv.py derives from float32 arithmetic.  Slots that no sequence holds
are NaN throughout, and table entries past a sequence's slots name no page."""
import numpy as np
import pytest
import torch

import _kv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tk():
    import topk_selection_gb300

    yield topk_selection_gb300
    topk_selection_gb300.check_stream()


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


def run_attend(tk, cache, q, scale=None, weight=None, **kw):
    k, v, table, lens = cache.dev()
    w = None if weight is None else weight.cuda()
    w_out = None if weight is None else torch.full_like(w, -1.0)
    out, lse = tk.kv_attend(q.cuda(), k, v, table, lens, scale=scale, weight=w, weight_out=w_out, **kw)
    return out, lse, w_out


def check_attend(tk, lens, heads, group, dim, page, dtype, layout, weights=True, room=0, seed=1, q_scale=2.0):
    cache = _kv.Cache(lens, heads, dim, page, dtype, layout, room=room, seed=seed)
    g = torch.Generator().manual_seed(seed + 100)
    q = (q_scale * torch.randn(len(lens), heads * group, dim, generator=g)).to(dtype)
    weight = torch.rand(len(lens), heads, cache.capacity, generator=g) if weights else None
    out, lse, w = run_attend(tk, cache, q, weight=weight)
    eo, el, ew, to, tl, tw = _kv.attend(cache, q, dim ** -0.5, weight)
    _kv.close(out, eo, to)
    _kv.close(lse, el, tl)
    if weights:
        for b, n in enumerate(lens):
            _kv.close(w[b, :, :n], ew[b, :, :n], tw[b, :, :n])
            assert torch.all(w[b, :, n:] == -1.0)  # nothing is written past the slots


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("layout", ["head", "token"])
@pytest.mark.parametrize("lens", [[1], [0], [2, 0, 1], [127, 128, 129], [300, 7, 0, 256, 1000], [15, 16, 17]])
def test_attend_lengths(tk, lens, layout, dtype):
    check_attend(tk, lens, 2, 4, 128, 16, dtype, layout)


@pytest.mark.parametrize("dim", [8, 16, 40, 64, 72, 80, 96, 128, 136, 192, 200, 256])
@pytest.mark.parametrize("weights", [False, True])
def test_attend_dims(tk, dim, weights):
    check_attend(tk, [259, 33, 1], 2, 2, dim, 32, torch.bfloat16, "token", weights)
    check_attend(tk, [130, 600], 1, 3, dim, 8, torch.float16, "head", weights)


@pytest.mark.parametrize("heads,group", [(1, 1), (5, 1), (2, 7), (3, 8), (1, 9), (2, 16), (1, 17), (1, 33), (2, 48)])
def test_attend_head_groups(tk, heads, group):
    check_attend(tk, [140, 511], heads, group, 64, 16, torch.float16, "head")
    check_attend(tk, [200, 3], heads, group, 128, 64, torch.bfloat16, "token")


@pytest.mark.parametrize("page", [8, 16, 24, 32, 48, 64, 128, 136, 256, 1024])
def test_attend_page_sizes(tk, page):
    check_attend(tk, [1023, 129, 5], 2, 4, 64, page, torch.bfloat16, "head", room=page)
    check_attend(tk, [700, 0, 256], 2, 2, 128, page, torch.float16, "token", weights=False)


def test_attend_long_sequence(tk):
    check_attend(tk, [70001], 1, 8, 128, 64, torch.bfloat16, "head")
    check_attend(tk, [40003, 1, 0, 20000], 2, 2, 64, 16, torch.float16, "token")


def test_attend_many_short_sequences(tk):
    lens = [(i * 37) % 91 for i in range(700)]
    check_attend(tk, lens, 2, 2, 64, 16, torch.float16, "head")


def test_attend_rising_and_falling_scores(tk):
    """A maximum that keeps growing (the running reference has to move), and one that never does."""
    for sign in (1.0, -1.0):
        cache = _kv.Cache([3000], 1, 64, 16, torch.float16, "head", seed=3)
        k = torch.zeros(3000, 64)
        k[:, 0] = sign * torch.linspace(-60, 60, 3000)
        k[:, 1] = torch.randn(3000, generator=torch.Generator().manual_seed(5))
        for i in range(0, 3000, 16):
            cache.k[cache.table[0, i // 16], :min(16, 3000 - i), 0] = k[i:i + 16].half()
        q = torch.zeros(1, 4, 64, dtype=torch.float16)
        q[:, :, 0] = torch.tensor([1.0, 4.0, 8.0, 0.125])
        q[:, :, 1] = 1.0
        weight = torch.zeros(1, 1, cache.capacity)
        out, lse, w = run_attend(tk, cache, q, scale=1.0, weight=weight)
        eo, el, ew, to, tl, tw = _kv.attend(cache, q, 1.0, weight)
        _kv.close(out, eo, to)
        _kv.close(lse, el, tl)
        _kv.close(w[:, :, :3000], ew[:, :, :3000], tw[:, :, :3000])


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_attend_values_that_are_not_finite(tk, value):
    """In slots that are held they count as the formula says; the head beside them is untouched."""
    cache = _kv.Cache([300], 2, 64, 16, torch.bfloat16, "head", seed=4)
    q = torch.ones(1, 2, 64, dtype=torch.bfloat16)
    cache.v[cache.table[0, 2], 3, 0, 5] = value
    out, lse, _ = run_attend(tk, cache, q)
    eo, el, _, to, tl, _ = _kv.attend(cache, q, 0.125)
    assert not torch.isfinite(out[0, 0, 5])  # inf or NaN
    eo[0, 0, 5] = out[0, 0, 5]
    _kv.close(out, eo, np.nan_to_num(to))
    _kv.close(lse, el, tl)
    cache = _kv.Cache([300], 2, 64, 16, torch.bfloat16, "head", seed=4)
    cache.k[cache.table[0, 2], 3, 0, 5] = value
    weight = torch.zeros(1, 2, cache.capacity)
    out, lse, w = run_attend(tk, cache, q, weight=weight)
    eo, el, ew, to, tl, tw = _kv.attend(cache, q, 0.125, weight)
    if value > 0:  # exp(inf - inf): a +inf score has no softmax
        assert np.isnan(eo[0, 0]).all()
    _kv.close(out, eo, np.nan_to_num(to))
    if value != float("inf"):
        _kv.close(lse, el, np.nan_to_num(tl))
        _kv.close(w[:, :, :300], ew[:, :, :300], np.nan_to_num(tw[:, :, :300]))
    else:
        assert torch.isnan(lse[0, 0]) and torch.isnan(w[0, 0, 35])
        _kv.close(lse[:, 1], el[:, 1], tl[:, 1])


def test_attend_scores_of_minus_infinity(tk):
    """A head whose every score is -inf is as empty as a sequence without slots."""
    cache = _kv.Cache([200], 2, 64, 16, torch.float16, "head", seed=6)
    for i in range(0, 200, 16):
        cache.k[cache.table[0, i // 16], :min(16, 200 - i), 0, 0] = float("-inf")
    q = torch.ones(1, 2, 64, dtype=torch.float16)
    weight = torch.rand(1, 2, cache.capacity, generator=torch.Generator().manual_seed(1))
    out, lse, w = run_attend(tk, cache, q, weight=weight)
    assert torch.all(out[0, 0] == 0) and lse[0, 0] == float("-inf")
    assert torch.equal(w[0, 0, :200].cpu(), weight[0, 0, :200])
    eo, el, ew, to, tl, tw = _kv.attend(cache, q, 0.125, weight)
    _kv.close(out[:, 1], eo[:, 1], to[:, 1])
    _kv.close(w[:, 1, :200], ew[:, 1, :200], tw[:, 1, :200])


def test_attend_in_place_weights_strides_and_stream(tk):
    """Weights in place inside a larger array, queries and pools as views, on a stream of their own, twice."""
    lens = [333, 90]
    cache = _kv.Cache(lens, 2, 64, 16, torch.bfloat16, "head", seed=7)
    k, v, table, lens_d = cache.dev()
    both = torch.stack([k.transpose(1, 2), v.transpose(1, 2)], 1)  # [pages, 2, heads, slots, dim]
    k, v = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
    wide = torch.randn(2, 4, 3 * 64, device="cuda").to(torch.bfloat16)
    q = wide[:, :, 64:128]
    table = torch.cat([table, torch.full_like(table, 7)], 1)[:, :table.shape[1]]
    big = torch.rand(2, 3, cache.capacity + 40, device="cuda")
    weight = big[:, :2, :cache.capacity]
    before, whole = weight.cpu().clone(), big.clone()
    eo, el, ew, to, tl, tw = _kv.attend(cache, q.cpu(), 0.125, before)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out, lse = tk.kv_attend(q, k, v, table, lens_d, weight=weight)
    s.synchronize()
    tk.check_stream(s)
    _kv.close(out, eo, to)
    _kv.close(lse, el, tl)
    for b, n in enumerate(lens):
        _kv.close(weight[b, :, :n], ew[b, :, :n], tw[b, :, :n])
    once = weight.clone()
    weight.copy_(whole[:, :2, :cache.capacity])
    out2, lse2 = tk.kv_attend(q, k, v, table, lens_d, weight=weight)
    assert torch.equal(bits(out), bits(out2)) and torch.equal(lse, lse2) and torch.equal(once, weight)
    assert torch.equal(big[:, 2], whole[:, 2]) and torch.equal(big[:, :, cache.capacity:], whole[:, :, cache.capacity:])


def test_attend_lengths_out_of_range_and_pages_of_none(tk):
    """Lengths are clamped to [0, capacity], and a page that the table does not name counts as zeros."""
    cache = _kv.Cache([64, 64], 1, 64, 16, torch.float16, "head", seed=8)
    k, v, table, _ = cache.dev()
    q = torch.randn(2, 2, 64, device="cuda").half()
    out, lse = tk.kv_attend(q, k, v, table, torch.tensor([1000, -5], dtype=torch.int32, device="cuda"))
    cache.lens = [64, 0]
    eo, el, _, to, tl, _ = _kv.attend(cache, q.cpu(), 0.125)
    _kv.close(out, eo, to)
    _kv.close(lse, el, tl)
    for bad in (-1, cache.k.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[0, 1] = bad
        out, lse = tk.kv_attend(q, k, v, t, torch.tensor([64, 0], dtype=torch.int32, device="cuda"))
        zero = _kv.Cache([64, 64], 1, 64, 16, torch.float16, "head", seed=8)
        zero.lens = [64, 0]
        zero.k[zero.table[0, 1]] = 0
        zero.v[zero.table[0, 1]] = 0
        eo, el, _, to, tl, _ = _kv.attend(zero, q.cpu(), 0.125)
        _kv.close(out, eo, to)
        _kv.close(lse, el, tl)


def test_offsets_beyond_32_bits(tk):
    """A pool of more than 2^31 elements, used at its end: attend, append and evict."""
    page, heads, dim = 64, 8, 128
    per = page * heads * dim
    pages = 2 ** 31 // per + 40
    k, v = (torch.empty(pages, heads, page, dim, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
            for _ in range(2))
    n = 500
    small = _kv.Cache([n], heads, dim, page, torch.bfloat16, "head", room=40, seed=9)
    base = pages - small.k.shape[0]
    k[base:].copy_(small.k)
    v[base:].copy_(small.v)
    table = torch.where(small.table < 2 ** 30, small.table + base, small.table).cuda()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    q = torch.randn(1, 16, dim, device="cuda").to(torch.bfloat16)
    out, lse = tk.kv_attend(q, k, v, table, lens)
    eo, el, _, to, tl, _ = _kv.attend(small, q.cpu(), dim ** -0.5)
    _kv.close(out, eo, to)
    _kv.close(lse, el, tl)
    new = torch.randn(40, heads, dim, device="cuda").to(torch.bfloat16)
    tk.kv_append(k, v, table, lens, new, -new, starts=torch.tensor([0, 40], dtype=torch.int32, device="cuda"))
    small.lens = [540]
    assert torch.equal(small.rows(0, k[base:].cpu())[n:], new.cpu())
    assert torch.equal(small.rows(0, v[base:].cpu())[n:], -new.cpu())
    before = small.rows(0, k[base:].cpu())
    weight = torch.rand(1, heads, 576, device="cuda")
    pos = torch.arange(576, dtype=torch.int32, device="cuda").repeat(1, heads, 1)
    lens.fill_(540)
    w0 = weight.cpu().numpy()
    tk.kv_evict(k, v, table, lens, weight, pos, lens.clone(), 300, recent=10)
    after = small.rows(0, k[base:].cpu())
    for h in range(heads):
        src = _kv.evict_sources(w0[0, h], np.arange(576), 540, 540, 300, 0, 10)
        assert torch.equal(after[:300, h], before[torch.from_numpy(src), h])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("layout", ["head", "token"])
@pytest.mark.parametrize("counts,dim,heads", [([1, 1, 1], 128, 8), ([5, 0, 33], 64, 2), ([0, 0, 4], 8, 1),
                                              ([200, 17, 1], 256, 3), ([3, 0, 0], 200, 5)])
def test_append(tk, counts, dim, heads, layout, dtype):
    held = [30, 0, 47]
    cache = _kv.Cache(held, heads, dim, 16, dtype, layout, room=max(counts), seed=11)
    k, v, table, lens = cache.dev()
    tokens = sum(counts)
    new = torch.randn(tokens, 2, heads, dim, device="cuda").to(dtype)  # views: strides of their own
    starts = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    weight = torch.full((3, heads, cache.capacity), 5.0, device="cuda")
    pos = torch.full((3, heads, cache.capacity), -7, dtype=torch.int32, device="cuda")
    next_pos = torch.tensor([100, 2 ** 30, 47], dtype=torch.int32, device="cuda")
    ek, ev, ew, ep = k.cpu().clone(), v.cpu().clone(), weight.cpu().clone(), pos.cpu().clone()
    at = 0
    for b in range(3):
        for i in range(counts[b]):
            slot = held[b] + i
            ek[cache.table[b, slot // 16], slot % 16] = new[at, 0].cpu()
            ev[cache.table[b, slot // 16], slot % 16] = new[at, 1].cpu()
            ew[b, :, slot] = 0
            ep[b, :, slot] = int(next_pos[b]) + i
            at += 1
    one = all(c == 1 for c in counts)
    tk.kv_append(k, v, table, lens, new[:, 0], new[:, 1], starts=None if one else starts, weight=weight, pos=pos,
                 next_pos=next_pos)
    assert torch.equal(bits(k.cpu()), bits(ek)) and torch.equal(bits(v.cpu()), bits(ev))
    assert torch.equal(weight.cpu(), ew) and torch.equal(pos.cpu(), ep)
    assert lens.tolist() == held


def test_append_drops_what_has_no_place(tk):
    """Tokens past the capacity, tokens past the last start, and tokens whose page the table does not name."""
    cache = _kv.Cache([20, 32], 2, 64, 16, torch.float16, "head", seed=12)  # capacity 32
    k, v, table, lens = cache.dev()
    table[0, 1] = -3
    before = k.clone()
    new = torch.randn(40, 2, 64, device="cuda").half()
    weight = torch.full((2, 2, 32), 5.0, device="cuda")
    starts = torch.tensor([0, 20, 30], dtype=torch.int32, device="cuda")
    tk.kv_append(k, v, table, lens, new, new, starts=starts, weight=weight)
    assert torch.equal(bits(k), bits(before))
    tk.kv_append(k, v, table, lens, new[:0], new[:0], starts=torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert torch.equal(bits(k), bits(before))
    assert torch.all(weight[1] == 5.0) and torch.all(weight[0, :, :20] == 5.0)
    torch.cuda.synchronize()


def check_evict(tk, lens, heads, dim, page, budget, sink, recent, weight, pos=None, next_pos=None, dtype=torch.float16,
                layout="head", in_place=False, room=0):
    cache = _kv.Cache(lens, heads, dim, page, dtype, layout, room=room, seed=13)
    k, v, table, lens_d = cache.dev()
    seqs, cap = len(lens), cache.capacity
    w = weight(seqs, heads, cap)
    if pos is None:
        pos = torch.arange(cap, dtype=torch.int32).repeat(seqs, heads, 1)
    if next_pos is None:
        next_pos = torch.tensor(lens, dtype=torch.int32)
    keep = min(budget, cap)
    wd, pd = w.cuda(), pos.cuda()
    if in_place:
        wo, po, lo = tk.kv_evict(k, v, table, lens_d, wd, pd, next_pos.cuda(), budget, sink, recent)
        assert wo is wd and po is pd and lo is lens_d
    else:
        wo = torch.full((seqs, heads, keep + 3), -5.0, device="cuda")[:, :, :keep]
        po = torch.full((seqs, heads, keep), -5, dtype=torch.int32, device="cuda")
        lo = torch.full((seqs,), -5, dtype=torch.int32, device="cuda")
        tk.kv_evict(k, v, table, lens_d, wd, pd, next_pos.cuda(), budget, sink, recent, wo, po, lo)
        assert torch.equal(bits(wd.cpu()), bits(w)) and torch.equal(pd.cpu(), pos) and lens_d.tolist() == list(lens)
    assert lo.tolist() == [min(n, budget) for n in lens]
    kc, vc = k.cpu(), v.cpu()
    for b, n in enumerate(lens):
        old_k, old_v, new_k, new_v = (cache.rows(b, p) for p in (cache.k, cache.v, kc, vc))
        for h in range(heads):
            src = _kv.evict_sources(w[b, h].numpy(), pos[b, h].numpy(), n, next_pos[b], budget, sink, recent)
            m = len(src)
            src = torch.from_numpy(src)
            assert torch.equal(bits(wo[b, h, :m].cpu()), bits(w[b, h][src]))
            assert torch.equal(po[b, h, :m].cpu(), pos[b, h][src])
            assert torch.equal(bits(new_k[:m, h]), bits(old_k[src, h]))
            assert torch.equal(bits(new_v[:m, h]), bits(old_v[src, h]))
            assert torch.equal(bits(new_k[m:, h]), bits(old_k[m:, h]))  # above the budget nothing changes
            if not in_place:
                assert torch.all(wo[b, h, m:] == -5.0) and torch.all(po[b, h, m:] == -5)


def rand_weight(seqs, heads, cap):
    return torch.exp(2 * torch.randn(seqs, heads, cap, generator=torch.Generator().manual_seed(14)))


def few_values(seqs, heads, cap):
    return torch.randint(0, 3, (seqs, heads, cap), generator=torch.Generator().manual_seed(15)).float() - 1.0


def specials(seqs, heads, cap):
    pool = torch.tensor([float("nan"), float("inf"), float("-inf"), 0.0, -0.0, 1.0, -1.0, 1e-45, 3.4e38,
                         torch.finfo(torch.float32).min])
    pool[0] = torch.tensor(-1, dtype=torch.int32).view(torch.float32)  # a negative NaN
    return pool[torch.randint(0, 10, (seqs, heads, cap), generator=torch.Generator().manual_seed(16))]


@pytest.mark.parametrize("weight", [rand_weight, few_values, specials])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,budget", [([100, 40, 0, 63], 40), ([513, 1025, 2049], 512), ([7], 1), ([1, 2, 3], 2),
                                         ([64, 64], 64), ([64, 63], 200), ([5000, 100], 300), ([3001], 2990)])
def test_evict(tk, lens, budget, in_place, weight):
    check_evict(tk, lens, 2, 64, 16, budget, 0, 0, weight, in_place=in_place)


@pytest.mark.parametrize("dim,page,layout,dtype", [(8, 8, "head", torch.float16), (128, 48, "token", torch.bfloat16),
                                                   (200, 128, "token", torch.float16), (256, 64, "head", torch.bfloat16)])
def test_evict_shapes(tk, dim, page, layout, dtype):
    check_evict(tk, [700, 1, 400], 3, dim, page, 250, 2, 20, rand_weight, dtype=dtype, layout=layout, room=page)


@pytest.mark.parametrize("sink,recent", [(4, 0), (0, 64), (4, 60), (16, 240), (256, 0), (0, 256)])
def test_evict_protected(tk, sink, recent):
    """Protected slots lie anywhere: positions are shuffled."""
    pos = torch.stack([torch.randperm(1008, generator=torch.Generator().manual_seed(i)) for i in range(4)])
    pos = pos.to(torch.int32).reshape(2, 2, 1008)
    check_evict(tk, [1008, 900], 2, 64, 16, 256, sink, recent, rand_weight, pos=pos,
                next_pos=torch.tensor([1008, 1008], dtype=torch.int32))


def test_evict_more_protected_than_fit_and_wide_positions(tk):
    """Repeated positions protect more slots than the budget: the lowest stay.  next_pos - recent does not wrap."""
    pos = torch.zeros(1, 2, 400, dtype=torch.int32)
    check_evict(tk, [390], 2, 64, 16, 100, 1, 0, rand_weight, pos=pos)
    pos = torch.full((1, 2, 400), -2 ** 31, dtype=torch.int32)
    check_evict(tk, [390], 2, 64, 16, 100, 0, 100, rand_weight, pos=pos,
                next_pos=torch.tensor([-2 ** 31], dtype=torch.int32))


def test_evict_long_rows(tk):
    check_evict(tk, [70000], 2, 8, 64, 9000, 4, 100, rand_weight)
    check_evict(tk, [70000], 2, 8, 64, 9000, 4, 100, few_values)
    check_evict(tk, [131072 + 7], 1, 8, 128, 120000, 0, 0, few_values, in_place=True)


def test_evict_rows_beyond_shared_memory(tk):
    check_evict(tk, [900001], 1, 8, 1024, 100000, 4, 1000, rand_weight)
    check_evict(tk, [400300], 1, 8, 1024, 400200, 4, 1000, few_values, in_place=True)  # few moves


@pytest.mark.parametrize("lens,budget,heads", [([1040, 1025, 1024], 1024, 8), ([2100] * 70, 2048, 4), ([33], 32, 1),
                                               ([5000, 4990, 4800], 4900, 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_a_few(tk, lens, budget, heads, in_place):
    """What a decoder evicts that stays at its budget: few slots of each row, moved by the launch that selects."""
    check_evict(tk, lens, heads, 64, 16, budget, 2, 20, rand_weight, in_place=in_place, dtype=torch.bfloat16)


def test_evict_pages_of_none(tk):
    """A move from or to a page that the table does not name is dropped; the other moves are made."""
    cache = _kv.Cache([64], 1, 64, 16, torch.float16, "head", seed=17)
    k, v, table, lens = cache.dev()
    w = torch.cat([torch.zeros(32), torch.ones(32)]).reshape(1, 1, 64).cuda()
    pos = torch.arange(64, dtype=torch.int32, device="cuda").reshape(1, 1, 64).contiguous()
    table[0, 1] = cache.k.shape[0]
    before = k.clone()
    tk.kv_evict(k, v, table, lens, w, pos, torch.tensor([64], dtype=torch.int32, device="cuda"), 32)
    t = cache.table[0]
    assert torch.equal(k[t[0]], before[t[2]]) and torch.equal(bits(k[t[1]]), bits(before[t[1]]))
    assert pos[0, 0, :32].tolist() == list(range(32, 64)) and lens.tolist() == [32]


def test_operators_together(tk):
    """A decoder's loop: prompts, steps with accumulated weights, evictions -- against the same loop on lists."""
    torch.manual_seed(0)
    seqs, heads, group, dim, page, budget, recent, sink = 3, 2, 4, 64, 16, 96, 16, 2
    width = 9  # room for 144 slots
    k, v = (torch.zeros(seqs * width, heads, page, dim, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
            for _ in range(2))
    table = torch.randperm(seqs * width, device="cuda").to(torch.int32).reshape(seqs, width)
    lens, seen = (torch.zeros(seqs, dtype=torch.int32, device="cuda") for _ in range(2))
    weight = torch.full((seqs, heads, width * page), float("nan"), device="cuda")
    pos = torch.full((seqs, heads, width * page), -1, dtype=torch.int32, device="cuda")
    mirror = [[[] for _ in range(heads)] for _ in range(seqs)]  # (key, value, weight, position) per slot
    counts = [100, 31, 1]
    for step in range(60):
        n = counts if step == 0 else [1] * seqs
        new = torch.randn(2, sum(n), heads, dim, device="cuda").to(torch.bfloat16)
        starts = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")
        tk.kv_append(k, v, table, lens, new[0], new[1], starts=starts if step % 2 == 0 else
                     (starts if step == 0 else None), weight=weight, pos=pos, next_pos=seen)
        host = new.double().cpu().numpy()
        for b in range(seqs):
            for i in range(n[b]):
                t = int(starts[b]) + i
                for h in range(heads):
                    mirror[b][h].append([host[0, t, h], host[1, t, h], 0.0, int(seen[b]) + i])
        add = torch.tensor(n, dtype=torch.int32, device="cuda")
        lens, seen = lens + add, seen + add
        q = torch.randn(seqs, heads * group, dim, device="cuda").to(torch.bfloat16)
        out, lse = tk.kv_attend(q, k, v, table, lens, weight=weight)
        qh = q.double().cpu().numpy()
        for b in range(seqs):
            for h in range(heads):
                row = mirror[b][h]
                s = np.array([r[0] for r in row]) @ qh[b, h * group:(h + 1) * group].T * dim ** -0.5
                p = np.exp(s - s.max(0))
                p /= p.sum(0)
                want = p.T @ np.array([r[1] for r in row])
                got = out[b, h * group:(h + 1) * group].double().cpu().numpy()
                assert np.abs(got - want).max() < 2.0 ** -8 * np.abs(want).max() + 2.0 ** -10
                for r, x in zip(row, p.sum(1)):
                    r[2] += x
        for b in range(seqs):
            for h in range(heads):
                m = len(mirror[b][h])
                got = weight[b, h, :m].double().cpu().numpy()
                assert np.abs(got - [r[2] for r in mirror[b][h]]).max() < 1e-4
                assert pos[b, h, :m].tolist() == [r[3] for r in mirror[b][h]]
        if step % 15 == 14:
            held = weight.cpu().numpy()
            before = lens.tolist()
            tk.kv_evict(k, v, table, lens, weight, pos, seen, budget, sink, recent)
            for b in range(seqs):
                for h in range(heads):
                    row = mirror[b][h]
                    src = _kv.evict_sources(held[b, h], np.array([r[3] for r in row]), before[b], int(seen[b]),
                                            budget, sink, recent)
                    mirror[b][h] = [row[i] for i in src]
            assert lens.tolist() == [len(mirror[b][0]) for b in range(seqs)]


@pytest.mark.parametrize("dim", [64, 80, 128, 256])
@pytest.mark.parametrize("group", [1, 2, 8, 16])
def test_attend_many_rows_of_a_block(tk, dim, group):
    """More tiles than there are SMs, in short rows of unequal lengths: a block goes through several rows."""
    lens = [(i * 61) % 700 + (i % 5 == 0) for i in range(60)]
    check_attend(tk, lens, 4, group, dim, 16, torch.bfloat16, "head", seed=21)


def test_allocation_failure_is_a_status(tk):
    """Scratch that cannot be had: nothing is written, and the same call works afterwards."""
    cache = _kv.Cache([200], 2, 64, 16, torch.float16, "head", seed=23)
    k, v, table, lens = cache.dev()
    q = torch.randn(1, 4, 64, device="cuda").half()
    out = torch.full((1, 4, 64), 7.0, dtype=torch.float16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    tk.set_option(tk.OPT_FAULT_ALLOC, 1)
    try:
        with torch.cuda.stream(s), pytest.raises(tk.TopKError) as err:
            tk.kv_attend(q, k, v, table, lens, out=out)
        assert err.value.status == 3  # TOPK_ERR_NO_MEMORY
    finally:
        tk.set_option(tk.OPT_FAULT_ALLOC, 0)
    torch.cuda.synchronize()
    assert torch.all(out == 7.0)
    with torch.cuda.stream(s):
        tk.kv_attend(q, k, v, table, lens, out=out)
    s.synchronize()
    eo, _, _, to, _, _ = _kv.attend(cache, q.cpu(), 0.125)
    _kv.close(out, eo, to)


def test_a_selection_after_them_waits(tk):
    """A TopK behind a cache operator on the stream must not start before it ends: it may read what that wrote."""
    lens = [1500]
    cache = _kv.Cache(lens, 1, 64, 16, torch.float16, "head", seed=24)
    k, v, table, lens_d = cache.dev()
    q = torch.randn(1, 1, 64, device="cuda").half()
    weight = torch.zeros(1, 1, cache.capacity, device="cuda")
    for _ in range(20):
        tk.topk_f32(weight.reshape(-1)[:1500], 8)
        tk.kv_attend(q, k, v, table, lens_d, weight=weight)
        best = tk.topk_f32(weight.reshape(-1)[:1500], 8)
        assert not tk.last_launch_early()
        assert torch.equal(best.cpu(), torch.sort(weight.cpu().reshape(-1)[:1500], descending=True).values[:8])


def test_captured_in_a_graph(tk):
    """The calls only enqueue, once a first one on the stream has made their scratch."""
    cache = _kv.Cache([700, 300], 2, 64, 16, torch.bfloat16, "token", room=8, seed=25)
    k, v, table, lens = cache.dev()
    q = torch.randn(2, 8, 64, device="cuda").to(torch.bfloat16)
    new = torch.randn(2, 2, 64, device="cuda").to(torch.bfloat16)
    weight = torch.zeros(2, 2, cache.capacity, device="cuda")
    pos = torch.arange(cache.capacity, dtype=torch.int32, device="cuda").repeat(2, 2, 1)
    w_out, p_out, l_out = torch.zeros_like(weight), torch.zeros_like(pos), torch.zeros_like(lens)

    def step():
        tk.kv_append(k, v, table, lens, new, new, weight=weight)
        out, _ = tk.kv_attend(q, k, v, table, lens, weight=weight, weight_out=w_out)
        tk.kv_evict(k, v, table, lens, w_out, pos, lens, 256, weight_out=weight, pos_out=p_out, lens_out=l_out)
        return out

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    k0, v0, w0 = k.clone(), v.clone(), weight.clone()
    with torch.cuda.stream(s):
        want = step().clone()
        kept = k.clone()
        for t, t0 in ((k, k0), (v, v0), (weight, w0)):
            t.copy_(t0)
        graph = torch.cuda.CUDAGraph()
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            out = step()
        for _ in range(3):
            for t, t0 in ((k, k0), (v, v0), (weight, w0)):
                t.copy_(t0)
            graph.replay()
    s.synchronize()
    assert torch.equal(bits(out), bits(want)) and torch.equal(bits(k), bits(kept))
    assert l_out.tolist() == [256, 256]


def test_example_runs():
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "kv_decode.py"), "--seqs", "3", "--prompt", "150",
                        "--steps", "120", "--limit", "200", "--budget", "96", "--recent", "16", "--dim", "64"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "of 273 tokens held" in r.stdout
