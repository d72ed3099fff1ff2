"""Where the key-value cache operators can go wrong without a large error:
shares of attention to the last bit, numbers that are not finite in slots
that hardly count, views, streams and state."""
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


@pytest.fixture(scope="module")
def side():
    """side(): a stream beside the current one, behind what that has been given; the same one throughout."""
    s = torch.cuda.Stream()

    def behind():
        s.wait_stream(torch.cuda.current_stream())
        return s

    yield behind
    s.synchronize()


def fill(cache, b, slot, pool, head, value):
    """pool's vector of a slot that sequence b holds."""
    pool[cache.table[b, slot // cache.page], slot % cache.page, head] = value


@pytest.mark.parametrize("dtype,group", [(torch.float16, 1), (torch.float16, 4), (torch.float16, 16),
                                         (torch.bfloat16, 8)])
@pytest.mark.parametrize("dim", [64, 256])
def test_a_long_rows_sum_does_not_drift(tk, dim, group, dtype):
    """As many rows as SMs, so that a block adds up a whole long one, and a few large values at its end that cancel what
    came before.  An addition of the product may leave 2^-23 of the sum that far, always in the same direction: 2^-17
    for the 64 of them before the sum is put aside, and 2^-24 for each of the 2^7 times that it is, another 2^-17.
    Shares are off by less than 2^-19 of themselves (scores are exact products, below 16).  In one piece it would be
    2^13 additions, and 2^-12 in the mean."""
    n, page = 2 ** 18, 1024
    seqs = torch.cuda.get_device_properties(0).multi_processor_count
    g = torch.Generator().manual_seed(44)
    key = (torch.rand(n, generator=g) * 2 - 1).to(dtype)
    key[-16:] = 8.0
    p = torch.softmax(key.double(), 0)
    v = torch.ones(n, dtype=torch.float64)
    rest = p[:-16].sum()
    for i in range(n - 16, n):  # a part of what is left each, and the last four all of it
        v[i] = (-rest / p[i] / max(1, n - 4 - i)).to(dtype).double()
        rest = rest + p[i] * v[i]
    k_pool, v_pool = (torch.zeros(n // page, page, 1, dim, dtype=dtype, device="cuda") for _ in range(2))
    k_pool.view(n, dim)[:, 0] = key.cuda()
    v_pool.view(n, dim)[:] = v.to(dtype).cuda()[:, None]
    table = torch.arange(n // page, dtype=torch.int32, device="cuda").repeat(seqs, 1)
    q = torch.zeros(seqs, group, dim, dtype=dtype, device="cuda")
    q[:, :, 0] = 1
    lens = torch.full((seqs,), n, dtype=torch.int32, device="cuda")
    out, lse = tk.kv_attend(q, k_pool, v_pool, table, lens, scale=1.0)
    want = (p * v).sum().item()
    tol = _kv.UNIT[dtype] * abs(want) + 2.0 ** -25 + (2.0 ** -16 + 2.0 ** -19) * (p @ v.abs()).item()
    assert (out.double() - want).abs().max().item() <= tol
    assert (lse.double() - torch.logsumexp(key.double(), 0).item()).abs().max().item() <= 2.0 ** -19


def scores_cache(scores, dim, dtype, heads=1, page=16, seed=30):
    """One sequence whose slots' scores are `scores` for a query of ones at
    element 0 and scale 1: keys hold them there, and zeros elsewhere."""
    cache = _kv.Cache([len(scores)], heads, dim, page, dtype, "head", seed=seed)
    for i, s in enumerate(scores):
        key = torch.zeros(dim, dtype=dtype)
        key[0] = s
        fill(cache, 0, i, cache.k, 0, key)
    q = torch.zeros(1, heads, dim, dtype=dtype)
    q[:, :, 0] = 1
    return cache, q


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("group", [1, 3, 8])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_shares_enter_the_product_with_float32s_bits(tk, dim, group, dtype):
    """Values chosen so that they cancel: what is left of the output is the
    shares' error.  Scores are exact products.  An exponent is off by its
    own rounding (2^-22 below 8) and the scale's (2^-23.5), so a share by
    2^-21.9 of itself, and by 2^-22 for the exponential; the sums of 15
    products of at most 128 in float32, by a total of 400, 2^-21.7.
    Altogether less than 2^-20 * sum p |v|; shares of 16 bits would be off by
    up to 2^-17 of themselves."""
    seqs, n = 48, 5
    g = torch.Generator().manual_seed(31)
    cache = _kv.Cache([n] * seqs, 1, dim, 8, dtype, "token", seed=32)
    q = torch.zeros(seqs, group, dim, dtype=dtype)
    q[:, :, 0] = 1
    for b in range(seqs):
        s = torch.tensor([0.0, -0.1, -0.2, -3.0, -3.1]) - torch.rand(n, generator=g) * 0.1
        s[0] = 0
        s = s.to(dtype).double()
        p = torch.softmax(s, 0)
        v = torch.zeros(n, dtype=torch.float64)
        v[1] = 1
        rest = p[1]
        for i in (2, 3, 4):
            v[i] = (-rest / p[i]).to(dtype).double()
            rest = rest + p[i] * v[i]
        for i in range(n):
            key = torch.zeros(dim, dtype=dtype)
            key[0] = s[i]
            fill(cache, b, i, cache.k, 0, key)
            fill(cache, b, i, cache.v, 0, torch.full((dim,), float(v[i]), dtype=dtype))
    k, v, table, lens = cache.dev()
    out, _ = tk.kv_attend(q.cuda(), k, v, table, lens, scale=1.0)
    want, _, _, _, _, _ = _kv.attend(cache, q, 1.0)
    tol = np.zeros_like(want)
    for b in range(seqs):
        kk, vv = (cache.rows(b, x).double().numpy()[:, 0] for x in (cache.k, cache.v))
        p = np.exp(kk[:, 0]) / np.exp(kk[:, 0]).sum()
        tol[b] = _kv.UNIT[dtype] * np.abs(want[b]) + 2.0 ** -25 + 2.0 ** -20 * (p @ np.abs(vv))
    _kv.close(out, want, tol)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_score_that_is_not_a_number_reaches_every_weight_of_its_head(tk, value):
    """Also those in tiles that hold only -inf besides."""
    scores = [0.0] * 128 + [float("-inf")] * 128 + [0.5] * 44
    scores[3] = value
    cache, q = scores_cache(scores, 64, torch.float16)
    k, v, table, lens = cache.dev()
    weight = torch.ones(1, 1, cache.capacity, device="cuda")
    out, lse = tk.kv_attend(q.cuda(), k, v, table, lens, scale=1.0, weight=weight)
    assert torch.isnan(out).all() and torch.isnan(lse).all()
    assert torch.isnan(weight[0, 0, :300]).all() and torch.all(weight[0, 0, 300:] == 1)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("low", [-200.0, float("-inf")])
@pytest.mark.parametrize("n,first,last,bad", [(300, 128, 256, 130), (40000, 5000, 20000, 12345)])
def test_a_value_that_is_not_finite_shows_however_small_its_share(tk, n, first, last, bad, low, value):
    """Its element of the output is not finite, the others are as they would be without it."""
    scores = torch.zeros(n)
    scores[first:last] = low
    cache, q = scores_cache(scores.tolist(), 64, torch.bfloat16)
    want, lse, _, tol, lse_tol, _ = _kv.attend(cache, q, 1.0)
    cache.v[cache.table[0, bad // 16], bad % 16, 0, 5] = value
    k, v, table, lens = cache.dev()
    out, got = tk.kv_attend(q.cuda(), k, v, table, lens, scale=1.0)
    assert not torch.isfinite(out[0, 0, 5])
    out[0, 0, 5] = want[0, 0, 5]
    if low > float("-inf"):  # else the bound of _kv.attend is not finite
        _kv.close(out, want, tol)
        _kv.close(got, lse, lse_tol)


@pytest.mark.parametrize("start", [-2 ** 31, -2 ** 31 + 1, -2 ** 31 + 5, -2 ** 30, -2 ** 30 - 7, -2 ** 31 + 2 ** 30])
def test_append_of_tokens_far_past_the_capacity(tk, start):
    """A token's number in its sequence and its slot may pass 2^31: it is dropped, not wrapped to a slot below 0.
    (Starts below 0 stand for that many tokens before the ones that k_new holds.)"""
    cache = _kv.Cache([20, 5], 2, 64, 16, torch.float16, "head", room=12, seed=43)
    k, v, table, lens = cache.dev()
    before = k.clone(), v.clone()
    new = torch.randn(40, 2, 64, device="cuda").half()
    starts = torch.tensor([start, 38, 40], dtype=torch.int32, device="cuda")
    weight = torch.full((2, 2, cache.capacity), 5.0, device="cuda")
    pos = torch.full((2, 2, cache.capacity), -7, dtype=torch.int32, device="cuda")
    tk.kv_append(k, v, table, lens, new, new, starts=starts, weight=weight, pos=pos, next_pos=lens)
    at = cache.table[1, 0]
    for pool, was in zip((k, v), before):
        assert torch.equal(pool[at, 5:7], new[38:])
        was[at, 5:7] = new[38:]
        assert torch.equal(pool.view(torch.int16), was.view(torch.int16))
    assert pos[1, 0].tolist() == [-7] * 5 + [5, 6] + [-7] * (cache.capacity - 7)
    assert torch.all(pos[0] == -7) and torch.all(weight[0] == 5.0)


@pytest.mark.parametrize("rising", [False, True])
def test_protected_slots_are_equal_whatever_they_weigh(tk, rising):
    """Positions at or past next_pos protect more slots than are kept: the lowest of them stay, the heaviest of the
    others do not; where fewer are protected, weights decide among the others alone."""
    n, budget = 300, 64
    c = decoder(1, n, 1, 1, 64)
    weight = torch.arange(1, n + 1, dtype=torch.float32, device="cuda") if rising else \
        torch.arange(n, 0, -1, dtype=torch.float32, device="cuda")
    weight[7] = float("nan")
    for protected in (range(100, 300, 2), range(200, 230)):
        pos = torch.zeros_like(c["pos"])
        pos[0, 0, list(protected)] = 1000
        w = torch.zeros_like(c["weight"])
        w[0, 0, :n] = weight
        p_out = torch.arange(pos.shape[2], dtype=torch.int32, device="cuda").reshape(1, 1, -1)
        p_in = pos.clone()
        p_in[0, 0, :n] += torch.arange(n, device="cuda", dtype=torch.int32)  # tells the slots apart
        kept = list(protected)[:budget]
        rest = sorted(set(range(n)) - set(protected), key=lambda i: (i != 7, -float(weight[i]), i))
        kept = sorted(kept + rest[:budget - len(kept)])
        tk.kv_evict(c["k"].clone(), c["v"].clone(), c["table"], c["lens"], w, p_in,
                    torch.tensor([1000], dtype=torch.int32, device="cuda"), budget, weight_out=torch.zeros_like(w),
                    pos_out=p_out, lens_out=torch.zeros_like(c["lens"]))
        assert sorted(p % 1000 for p in p_out[0, 0, :budget].tolist()) == kept


def decoder(seqs, n, heads, group, dim, dtype=torch.float16, seed=42):
    """A cache of `n` slots in each sequence, weights to attend with, and what to evict to."""
    g = torch.Generator("cuda").manual_seed(seed)
    page = 16
    width = n // page + 1
    k, v = (torch.randn(seqs * width, heads, page, dim, device="cuda", generator=g).to(dtype).transpose(1, 2)
            for _ in range(2))
    table = torch.randperm(seqs * width, device="cuda", generator=g).to(torch.int32).reshape(seqs, width)
    lens = torch.full((seqs,), n, dtype=torch.int32, device="cuda")
    q = torch.randn(seqs, heads * group, dim, device="cuda", generator=g).to(dtype)
    weight = torch.rand(seqs, heads, width * page, device="cuda", generator=g)
    pos = torch.arange(width * page, dtype=torch.int32, device="cuda").repeat(seqs, heads, 1)
    return dict(k=k, v=v, table=table, lens=lens, q=q, weight=weight, pos=pos)


def attend_and_evict(tk, c, k, v):
    """A step on copies of the pools: (out, lse, weights, evicted weights, positions)."""
    w_out = torch.full_like(c["weight"], -1.0)
    out, lse = tk.kv_attend(c["q"], k, v, c["table"], c["lens"], weight=c["weight"], weight_out=w_out)
    n = c["weight"].shape[2]
    w, p, _ = tk.kv_evict(k, v, c["table"], c["lens"], w_out, c["pos"], c["lens"], n // 2, sink=2, recent=8,
                          weight_out=torch.full_like(w_out, -1.0), pos_out=torch.full_like(c["pos"], -1),
                          lens_out=torch.zeros_like(c["lens"]))
    return out, lse, w_out, w, p


def test_graphs_outlive_larger_calls(tk, side):
    """One graph per batch size, captured on one stream from small to large: each goes on working, and no replay writes
    into what was allocated since."""
    s = side()
    graphs = []
    with torch.cuda.stream(s):
        for seqs, n in ((1, 700), (3, 2100), (8, 6000), (8, 6100), (24, 9000)):
            c = decoder(seqs, n, 2, 4, 64)
            k, v = c["k"].clone(), c["v"].clone()
            want = [t.clone() for t in attend_and_evict(tk, c, k, v)]
            k.copy_(c["k"])
            v.copy_(c["v"])
            s.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                got = attend_and_evict(tk, c, k, v)
            graphs.append((graph, c, k, v, want, got))
        big = decoder(40, 16000, 4, 8, 64)
        attend_and_evict(tk, big, big["k"].clone(), big["v"].clone())
        s.synchronize()
        del big
        torch.cuda.empty_cache()
        patterns = [torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda")
                    for size in [2 ** 20] * 8 + [2 ** 21] * 8 + [2 ** 23] * 4 + [2 ** 25] * 4 + [2 ** 28]]
        for _ in range(2):
            for graph, c, k, v, want, got in graphs:
                k.copy_(c["k"])
                v.copy_(c["v"])
                for t in got:
                    t.zero_()
                graph.replay()
                for a, b in zip(got, want):
                    assert torch.equal(a, b)
        assert all(bool((p == 0x5A).all()) for p in patterns)
    s.synchronize()


def test_a_capture_that_would_allocate_is_refused(tk, side):
    """The status comes back, the capture goes on, and the same call works on the stream afterwards."""
    torch.cuda.synchronize()
    tk.release_workspace()  # other tests' scratch would be large enough
    s = side()
    c = decoder(2, 300, 2, 2, 64)
    big = decoder(20, 3000, 4, 8, 64)
    x = torch.zeros(4, device="cuda")
    with torch.cuda.stream(s):
        attend_and_evict(tk, c, c["k"].clone(), c["v"].clone())
        s.synchronize()
        w_out = torch.zeros_like(big["weight"])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            with pytest.raises(tk.TopKError) as err:
                tk.kv_attend(big["q"], big["k"], big["v"], big["table"], big["lens"], weight=big["weight"],
                             weight_out=w_out)
            x += 1
        assert err.value.status == 3  # TOPK_ERR_NO_MEMORY
        graph.replay()
        assert x.tolist() == [1, 1, 1, 1]
        tk.kv_attend(big["q"], big["k"], big["v"], big["table"], big["lens"], weight=big["weight"], weight_out=w_out)
    s.synchronize()
    tk.check_stream(s)


def test_host_threads_on_one_stream(tk, side):
    """Two threads whose calls meet on one stream, one with small and growing caches: each gets its own results."""
    import threading

    cases = [[decoder(2, 500, 2, 4, 64, seed=50), decoder(3, 900, 2, 4, 64, seed=51), decoder(6, 4000, 2, 4, 64, seed=52)],
             [decoder(4, 1500, 4, 2, 128, seed=53)]]
    want = [[[t.clone() for t in attend_and_evict(tk, c, c["k"].clone(), c["v"].clone())] for c in cs] for cs in cases]
    s = side()
    failures = []

    def work(which):
        try:
            with torch.cuda.stream(s):
                for round_ in range(40):
                    at = round_ * len(cases[which]) // 40
                    c = cases[which][at]
                    got = attend_and_evict(tk, c, c["k"].clone(), c["v"].clone())
                    if not all(torch.equal(a, b) for a, b in zip(got, want[which][at])):
                        failures.append((which, round_))
        except Exception as e:  # noqa: BLE001 (reported by the main thread)
            failures.append((which, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    s.synchronize()
    tk.check_stream(s)
    assert failures == []


def test_outputs_belong_to_the_stream_of_the_call(tk, side):
    """What kv_attend allocates is its stream's memory, however the stream is given, so that the allocator hands it on
    only behind the call."""
    c = decoder(2, 300, 2, 2, 64)

    def owner(t):
        for segment in torch.cuda.memory_snapshot():
            if segment["address"] <= t.data_ptr() < segment["address"] + segment["total_size"]:
                return segment["stream"]
        raise AssertionError("not the allocator's")

    args = c["q"], c["k"], c["v"], c["table"], c["lens"]
    torch.cuda.synchronize()
    want, want_lse = tk.kv_attend(*args)
    assert owner(want) == torch.cuda.current_stream().cuda_stream
    s = side()
    for given in (s, s.cuda_stream):
        before = torch.cuda.current_stream()
        out, lse = tk.kv_attend(*args, stream=given)
        assert torch.cuda.current_stream() == before
        assert owner(out) == s.cuda_stream and owner(lse) == s.cuda_stream
        s.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    with torch.cuda.stream(s):
        out, _ = tk.kv_attend(*args, stream=0)
        assert owner(out) == 0
        other, _ = tk.kv_attend(*args, stream=1)  # the legacy stream's other handle
        assert owner(other) == 0
        assert torch.cuda.current_stream() == s
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(other, want)


@pytest.fixture
def withhold(tk):
    """Makes the first block of kv_attend keep something back, with short waits; cleared afterwards."""
    def put(what):
        tk.set_option(tk.OPT_KV_SPINS, 200 if what else 0)
        tk.set_option(tk.OPT_KV_WITHHOLD, what)

    yield put
    put(0)


SHORT, RAGGED, LONG = (1, 300, 2, 4, 64), (20, 700, 4, 8, 128), (2, 40000, 2, 12, 64)
WIDE = (3, 900, 2, 8, 256)


@pytest.mark.parametrize("what", [1, 2, 3])
@pytest.mark.parametrize("shape", [SHORT, RAGGED, LONG, WIDE])
def test_waits_of_attend_run_out(tk, side, withhold, shape, what):
    """Nothing hangs, the status says so, and nothing is written outside the outputs."""
    c = decoder(*shape)
    k0, v0 = c["k"].clone(), c["v"].clone()
    args = c["q"], c["k"], c["v"], c["table"], c["lens"]
    seqs, heads, cap = c["weight"].shape
    want = tk.kv_attend(*args, weight=c["weight"], weight_out=torch.zeros_like(c["weight"]))
    tk.check_stream()
    rows, dim = c["q"].shape[0] * c["q"].shape[1], c["q"].shape[2]
    out = torch.full((rows + 16, dim), 7.0, dtype=c["q"].dtype, device="cuda")
    lse = torch.full((rows + 16,), 7.0, device="cuda")
    w = torch.full((seqs, heads, cap + 64), 7.0, device="cuda")
    s = side()
    withhold(what)
    with torch.cuda.stream(s):
        tk.kv_attend(*args, weight=c["weight"], weight_out=w[:, :, :cap], out=out[:rows].view_as(c["q"]),
                     lse=lse[:rows].view(c["q"].shape[:2]))
    with pytest.raises(tk.TopKError) as err:
        tk.check_stream(s)
    assert err.value.status == 5  # TOPK_ERR_DEVICE_TIMEOUT
    tk.check_stream(s)  # told once
    withhold(0)
    assert torch.all(out[rows:] == 7.0) and torch.all(lse[rows:] == 7.0) and torch.all(w[:, :, cap:] == 7.0)
    assert torch.equal(c["k"], k0) and torch.equal(c["v"], v0)
    assert torch.equal(c["weight"], decoder(*shape)["weight"])
    got = tk.kv_attend(*args, weight=c["weight"], weight_out=torch.zeros_like(c["weight"]))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_options_of_the_waits(tk):
    for option, bad in ((tk.OPT_KV_SPINS, -1), (tk.OPT_KV_WITHHOLD, 4), (tk.OPT_KV_WITHHOLD, -1)):
        with pytest.raises(tk.TopKError):
            tk.set_option(option, bad)


def cut_short(tk, withhold, c, what=2):
    withhold(what)
    tk.kv_attend(c["q"], c["k"], c["v"], c["table"], c["lens"], weight=c["weight"],
                 weight_out=torch.zeros_like(c["weight"]))
    withhold(0)


@pytest.mark.parametrize("what", [1, 2, 3])
@pytest.mark.parametrize("checked", [False, True])
@pytest.mark.parametrize("order", ["l", "el", "sl", "ssl", "seel", "e", "se", "lel"])
def test_calls_after_one_cut_short(tk, side, withhold, order, checked, what):
    """Evictions (e), small attentions (s) and large ones (l) that come next on the stream are right, whether the
    status was asked for or not."""
    small, large = decoder(*SHORT, seed=60), decoder(*LONG, seed=61)
    args = {kind: (c["q"], c["k"], c["v"], c["table"], c["lens"]) for kind, c in (("s", small), ("l", large))}

    def run(kind):
        if kind != "e":
            return tk.kv_attend(*args[kind])
        return tk.kv_evict(small["k"].clone(), small["v"].clone(), small["table"], small["lens"], small["weight"],
                           small["pos"], small["lens"], 150, weight_out=torch.zeros_like(small["weight"]),
                           pos_out=torch.zeros_like(small["pos"]), lens_out=torch.zeros_like(small["lens"]))

    want = {kind: [t.clone() for t in run(kind)] for kind in "sle"}
    s = side()
    with torch.cuda.stream(s):
        cut_short(tk, withhold, large, what)
        if checked:
            with pytest.raises(tk.TopKError):
                tk.check_stream(s)
        for kind in order:
            assert all(torch.equal(a, b) for a, b in zip(run(kind), want[kind])), kind
    if not checked:
        with pytest.raises(tk.TopKError):
            tk.check_stream(s)
    tk.check_stream(s)


@pytest.mark.parametrize("before", [0, 1])
def test_graphs_after_a_call_cut_short(tk, side, withhold, before):
    """A graph's call always has the same counters: once the status was asked for, its replays are right."""
    c = decoder(*LONG)
    want = [t.clone() for t in tk.kv_attend(c["q"], c["k"], c["v"], c["table"], c["lens"])]
    s = side()
    with torch.cuda.stream(s):
        tk.kv_attend(c["q"], c["k"], c["v"], c["table"], c["lens"], weight=c["weight"].clone())
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = tk.kv_attend(c["q"], c["k"], c["v"], c["table"], c["lens"])
        for _ in range(before):
            tk.kv_attend(c["q"], c["k"], c["v"], c["table"], c["lens"])
        cut_short(tk, withhold, c)
        with pytest.raises(tk.TopKError):
            tk.check_stream(s)
        for _ in range(3):
            for t in got:
                t.zero_()
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    s.synchronize()
    tk.check_stream(s)


def test_side_arrays_that_lie_between_one_another(tk):
    """Rows of weight and weight_out alternate in one array: they do not overlap.  Dimensions of one element may have
    any stride."""
    cache = _kv.Cache([200, 90], 2, 64, 16, torch.float16, "head", seed=36)
    k, v, table, lens = cache.dev()
    q = torch.randn(2, 4, 64, device="cuda").half()
    weight = torch.rand(2, 2, cache.capacity, generator=torch.Generator().manual_seed(37))
    both = torch.zeros(2, 2, 2, cache.capacity, device="cuda")
    both[:, :, 0] = weight.cuda()
    tk.kv_attend(q, k, v, table, lens, weight=both[:, :, 0], weight_out=both[:, :, 1])
    plain = weight.cuda()
    tk.kv_attend(q, k, v, table, lens, weight=plain)
    for b, n in enumerate(cache.lens):
        assert torch.equal(both[b, :, 1, :n], plain[b, :, :n])
    assert torch.equal(both[:, :, 0].cpu(), weight)
    pos = torch.arange(cache.capacity, dtype=torch.int32, device="cuda").repeat(2, 2, 1)
    pair = torch.zeros(2, 2, 2, cache.capacity, dtype=torch.int32, device="cuda")
    pair[:, :, 0] = pos
    w_out, p_out, l_out = tk.kv_evict(k, v, table, lens, both[:, :, 1], pair[:, :, 0], lens, 64,
                                      weight_out=both[:, :, 0], pos_out=pair[:, :, 1], lens_out=lens.clone())
    assert l_out.tolist() == [64, 64] and torch.equal(lens.cpu(), torch.tensor([200, 90], dtype=torch.int32))
    for b in range(2):
        for h in range(2):
            src = _kv.evict_sources(plain[b, h].cpu().numpy(), np.arange(cache.capacity), cache.lens[b],
                                    cache.lens[b], 64, 0, 0)
            assert p_out[b, h, :64].tolist() == src.tolist()
    one = plain[:1]
    same = torch.as_strided(one, one.shape, (7 * one.stride(0), one.stride(1), 1), one.storage_offset())
    tk.kv_attend(q[:1], k, v, table[:1], lens[:1].clone(), weight=one, weight_out=same)


def test_what_is_written_says_so(tk):
    """Tensors that an operator writes count a change, as for torch's own."""
    cache = _kv.Cache([40, 30], 2, 64, 16, torch.float16, "head", room=4, seed=38)
    k, v, table, lens = cache.dev()
    q = torch.randn(2, 4, 64, device="cuda").half()
    new = torch.randn(2, 2, 64, device="cuda").half()
    weight = torch.zeros(2, 2, cache.capacity, device="cuda")
    pos = torch.arange(cache.capacity, dtype=torch.int32, device="cuda").repeat(2, 2, 1)

    def versions(*ts):
        return [t._version for t in ts]

    before = versions(k, v, weight, pos, lens, table, q, new)
    tk.kv_append(k, v, table, lens, new, new, weight=weight, pos=pos, next_pos=lens)
    after = versions(k, v, weight, pos, lens, table, q, new)
    assert all(a > b for a, b in zip(after[:4], before[:4])) and after[4:] == before[4:]
    out, lse = torch.empty_like(q), torch.empty(2, 4, device="cuda")
    before = versions(weight, out, lse, k, v, q)
    tk.kv_attend(q, k, v, table, lens, weight=weight, out=out, lse=lse)
    after = versions(weight, out, lse, k, v, q)
    assert all(a > b for a, b in zip(after[:3], before[:3])) and after[3:] == before[3:]
    before = versions(k, v, weight, pos, lens)
    tk.kv_evict(k, v, table, lens, weight, pos, lens.clone(), 16)
    assert all(a > b for a, b in zip(versions(k, v, weight, pos, lens), before))
    with torch.inference_mode():
        tk.kv_attend(q.clone(), k, v, table, lens, weight=torch.zeros_like(weight))


def test_gradients_that_there_are_not(tk):
    """Calls that autograd follows run, and say so: at the backward pass, by a warning, or at once where a tensor that
    requires grad would be written."""
    import warnings

    c = decoder(2, 40, 2, 2, 64)
    rest = c["k"], c["v"], c["table"], c["lens"]
    want, want_lse = tk.kv_attend(c["q"], *rest)
    assert not want.requires_grad
    q = c["q"].clone().requires_grad_()
    for of in (0, 1):
        got = tk.kv_attend(2 * q / 2, *rest, weight=c["weight"].clone())
        assert got[0].requires_grad and got[1].requires_grad and torch.equal(got[0], want)
        with pytest.raises(RuntimeError, match="kv_attend is not implemented"):
            got[of].float().sum().backward()
    k = c["k"].clone().requires_grad_()
    out, _ = tk.kv_attend(c["q"], k, *rest[1:])
    with pytest.raises(RuntimeError, match="kv_attend is not implemented"):
        out.float().sum().backward()
    with torch.no_grad():
        got, _ = tk.kv_attend(q, *rest, out=torch.empty_like(want))
    assert not got.requires_grad and torch.equal(got, want)
    for given in (dict(out=torch.empty_like(want)), dict(lse=torch.empty_like(want_lse))):
        with pytest.raises(RuntimeError, match="no gradient"):
            tk.kv_attend(q, *rest, **given)
    new = c["q"][:, :2].clone()
    lens = c["lens"] - 1
    with pytest.warns(UserWarning, match="no gradient"):
        tk.kv_append(rest[0], rest[1], c["table"], lens, new.clone().requires_grad_(), new)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        tk.kv_append(rest[0], rest[1], c["table"], lens, new, new)
        with torch.no_grad():
            tk.kv_append(rest[0], rest[1], c["table"], lens, new.clone().requires_grad_(), new)
        with pytest.raises(UserWarning):
            tk.kv_append(rest[0], rest[1], c["table"], lens, new, new.clone().requires_grad_())
    followed = c["weight"].clone().requires_grad_()
    with pytest.raises(RuntimeError, match="no gradient"):
        tk.kv_attend(c["q"], *rest, weight=followed)
    with pytest.raises(RuntimeError, match="no gradient"):
        tk.kv_append(k, rest[1], c["table"], lens, new, new)
    with pytest.raises(RuntimeError, match="no gradient"):
        tk.kv_evict(*rest, followed, c["pos"], c["lens"], 16)
    given = dict(weight_out=c["weight"].clone(), pos_out=c["pos"].clone(), lens_out=c["lens"].clone())
    tk.kv_evict(*rest, followed, c["pos"], c["lens"], 16, **given)  # only read


@pytest.mark.parametrize("name", ["weight", "weight_out", "out", "lse"])
def test_what_is_no_tensor_is_refused(tk, name):
    c = decoder(2, 40, 2, 2, 64)
    given = dict(weight=c["weight"], weight_out=torch.zeros_like(c["weight"]), out=torch.zeros_like(c["q"]),
                 lse=torch.zeros(2, 4, device="cuda"))
    for bad in (5, "x", [1.0], c["q"].cpu().numpy()):
        with pytest.raises(TypeError, match=name):
            tk.kv_attend(c["q"], c["k"], c["v"], c["table"], c["lens"], **dict(given, **{name: bad}))
    for i in range(4):
        args = [c["k"], c["v"], c["table"], c["lens"], c["weight"], c["pos"], c["lens"]]
        args[i] = 5
        with pytest.raises(TypeError):
            tk.kv_evict(*args, 16)
    for key in ("weight", "pos", "next_pos", "starts"):
        extra = dict(weight=c["weight"], pos=c["pos"], next_pos=c["lens"])
        extra[key] = 5
        with pytest.raises(TypeError, match=key):
            tk.kv_append(c["k"], c["v"], c["table"], c["lens"], c["q"][:, :2], c["q"][:, :2], **extra)


def test_an_empty_batch_is_nothing_to_do(tk):
    cache = _kv.Cache([40], 2, 64, 16, torch.float16, "head", seed=39)
    k, v, table, lens = cache.dev()
    table, lens = table[:0], lens[:0]
    weight, pos = torch.zeros(0, 2, 48, device="cuda"), torch.zeros(0, 2, 48, dtype=torch.int32, device="cuda")
    before = k.clone()
    new = torch.zeros(0, 2, 64, device="cuda").half()
    tk.kv_append(k, v, table, lens, new, new, weight=weight, pos=pos, next_pos=lens)
    out, lse = tk.kv_attend(torch.zeros(0, 4, 64, device="cuda").half(), k, v, table, lens, weight=weight)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    got = tk.kv_evict(k, v, table, lens, weight, pos, lens, 16)
    assert got[0] is weight and got[2] is lens
    assert torch.equal(k.view(torch.int16), before.view(torch.int16))


def bounds_of_finite(cache, q, scale, weight):
    """_kv.attend with the scores of -inf left out of the bounds: they are
    products of -inf, not sums that round, and their shares are exactly 0."""
    out, lse, w, _, _, _ = _kv.attend(cache, q, scale, weight)
    tol, lse_tol, w_tol = np.zeros_like(out), np.zeros_like(lse), np.zeros_like(w)
    group = q.shape[1] // cache.heads
    for b in range(q.shape[0]):
        n = cache.lens[b]
        k, v = (cache.rows(b, p).double().numpy() for p in (cache.k, cache.v))
        for j in range(q.shape[1]):
            h = j // group
            qq = q[b, j].double().numpy()
            with np.errstate(invalid="ignore"):
                s = scale * (k[:, h] @ qq)
            held = np.isfinite(s)
            if not held.any():
                continue
            d = 2 * cache.dim * 2.0 ** -24 * abs(scale) * (np.abs(k[held, h]) @ np.abs(qq)).max()
            p = np.where(held, np.exp(np.where(held, s, 0) - lse[b, j]), 0.0)
            rel = 2 * d + 2.0 ** -20 + n * 2.0 ** -24
            tol[b, j] = _kv.UNIT[cache.dtype] * np.abs(out[b, j]) + 2.0 ** -25 + \
                (rel + 2.0 ** -15 + n * 2.0 ** -30) * (p @ np.abs(v[:, h])) + n * 2.0 ** -30 * np.abs(v[:, h]).max(0)
            lse_tol[b, j] = rel + 2.0 ** -22 * abs(lse[b, j])
            w_tol[b, h, :n] += np.where(held, p * rel + 2.0 ** -23 * np.abs(w[b, h, :n]), 0.0)
    assert np.isfinite(tol).all() and np.isfinite(lse_tol).all() and np.isfinite(w_tol).all()
    return out, lse, w, tol, lse_tol, w_tol


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,masked", [(300, [35]), (300, range(0, 256)), (700, range(100, 600)), (700, range(0, 699)),
                                      (20001, range(0, 15000)), (20001, range(1, 20001, 2))])
def test_scores_of_minus_infinity_among_finite_ones(tk, n, masked, dtype):
    """Masked slots get a share of exactly nothing, whole tiles of them at the
    front, in the middle and over several blocks included."""
    cache = _kv.Cache([n, 40], 2, 64, 16, dtype, "token", seed=33)
    q = torch.randn(2, 6, 64, generator=torch.Generator().manual_seed(34)).to(dtype)
    q[:, :, 0] = q[:, :, 0].abs() + 0.5
    for i in masked:
        cache.k[cache.table[0, i // 16], i % 16, 0, 0] = float("-inf")
    weight = torch.rand(2, 2, cache.capacity, generator=torch.Generator().manual_seed(35))
    k, v, table, lens = cache.dev()
    w = torch.zeros_like(weight).cuda()
    out, lse = tk.kv_attend(q.cuda(), k, v, table, lens, weight=weight.cuda(), weight_out=w)
    eo, el, ew, to, tl, tw = bounds_of_finite(cache, q, 0.125, weight)
    _kv.close(out, eo, to)
    _kv.close(lse, el, tl)
    for b, m in enumerate(cache.lens):
        _kv.close(w[b, :, :m], ew[b, :, :m], tw[b, :, :m])
    at = list(masked)
    assert torch.equal(w[0, 0, at].cpu(), weight[0, 0, at])


def rand_weight(seqs, heads, cap):
    return torch.exp(2 * torch.randn(seqs, heads, cap, generator=torch.Generator().manual_seed(40)))


@pytest.mark.parametrize("lens,heads,budget,page,room", [
    ([2100 + 7 * i for i in range(20)], 16, 700, 16, 0),        # more than 304 rows, 256 threads each
    ([5000 + i for i in range(10)], 31, 4000, 16, 0),
    ([5200 + 3 * i for i in range(10)], 31, 4000, 16, 0),       # the same with 512
    ([1500] * 20, 16, 100, 16, 9000),                           # short rows in a wide table
    ([400300], 20, 100000, 1024, 0),                            # beyond shared memory, on more than 152 blocks
])
def test_evict_by_every_kind_of_block(tk, lens, heads, budget, page, room):
    seqs, dim = len(lens), 8
    width = -(-(max(lens) + room) // page)
    k = torch.randint(-30000, 30000, (seqs * width, heads, page, dim), dtype=torch.int16, device="cuda",
                      generator=torch.Generator("cuda").manual_seed(41)).view(torch.float16).transpose(1, 2)
    v = k.flip(0).contiguous()
    table = torch.randperm(seqs * width, device="cuda").to(torch.int32).reshape(seqs, width)
    cap = width * page
    weight = rand_weight(seqs, heads, cap)
    weight[:, :, 5::11] = 0
    pos = torch.arange(cap, dtype=torch.int32).repeat(seqs, heads, 1)
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def held(pool, b):
        return pool.view(torch.int16)[table[b].long()].reshape(cap, heads, dim)

    old = [(held(k, b).clone(), held(v, b).clone()) for b in range(seqs)]
    w_out = torch.full((seqs, heads, budget), -5.0, device="cuda")
    p_out = torch.full((seqs, heads, budget), -5, dtype=torch.int32, device="cuda")
    tk.kv_evict(k, v, table, lens_d, weight.cuda(), pos.cuda(), lens_d, budget, 2, 50, w_out, p_out, lens_d.clone())
    for b, n in enumerate(lens):
        now = held(k, b), held(v, b)
        for h in range(heads):
            src = torch.from_numpy(_kv.evict_sources(weight[b, h].numpy(), pos[b, h].numpy(), n, n, budget, 2, 50))
            assert torch.equal(p_out[b, h].cpu(), src.to(torch.int32))
            assert torch.equal(w_out[b, h].cpu(), weight[b, h][src])
            for was, is_ in zip(old[b], now):
                assert torch.equal(is_[:budget, h], was[src.cuda(), h]) and torch.equal(is_[budget:, h], was[budget:, h])
