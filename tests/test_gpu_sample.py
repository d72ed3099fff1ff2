"""sample_rows against its definition in 64 bits (tests/_rotate.py): the token
has to be the definition's wherever u is not within 2^-34 of a border."""
import numpy as np
import pytest
import torch

import _rotate

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def tk():
    import topk_selection_gb300

    yield topk_selection_gb300
    topk_selection_gb300.check_stream()


def each(value, rows):
    return value.tolist() if isinstance(value, torch.Tensor) else [value] * rows


def check(tk, x, u, **kw):
    """Compares every row; the parameters in kw are numbers or tensors.  Weights are right to 2^-23.4, so a logarithm of
    their quotient to 2^-18 with room, besides its own roundings."""
    rows = x.shape[0]
    there = {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in kw.items()}
    token, logp = tk.sample_rows(x.cuda(), u.cuda(), **there)
    token, logp = token.tolist(), logp.tolist()
    given = {n: each(v, rows) for n, v in kw.items()}
    for r in range(rows):
        want, lp, near = _rotate.sample(x[r], u[r].item(), **{n: v[r] for n, v in given.items()})
        what = {n: v[r] for n, v in given.items()}
        if near > 2.0 ** -34:
            assert token[r] == want, (r, token[r], want, u[r].item(), near, what)
        if token[r] == want:
            assert (np.isnan(lp) and np.isnan(logp[r])) or abs(lp - logp[r]) <= 2.0 ** -18 + 2.0 ** -22 * abs(lp), \
                (r, lp, logp[r], what)
    return token


def logits(rows, cols, dtype, spread=2.5, seed=0):
    return (spread * torch.randn(rows, cols, generator=torch.Generator().manual_seed(seed))).to(dtype)


def uniform(rows, seed=1):
    return torch.rand(rows, generator=torch.Generator().manual_seed(seed))


PARAMETERS = [dict(), dict(top_k=50), dict(top_p=0.95), dict(min_p=0.05), dict(temperature=0.0), dict(temperature=0.3),
              dict(top_k=50, top_p=0.9), dict(top_k=1), dict(top_p=0.0), dict(top_p=0.5, min_p=0.1, top_k=20),
              dict(temperature=3.0, top_p=0.8), dict(temperature=30.0, top_k=1500), dict(top_p=0.99, min_p=0.01),
              dict(top_k=2000, top_p=0.999, temperature=2.0), dict(min_p=1.0), dict(top_k=7, min_p=0.3)]


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("kw", PARAMETERS, ids=str)
@pytest.mark.parametrize("rows,cols", [(7, 1000), (3, 32768), (40, 5001)])
def test_parameters(tk, rows, cols, kw, dtype):
    check(tk, logits(rows, cols, dtype, seed=cols), uniform(rows, rows), **kw)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("cols", [1, 2, 3, 7, 8, 9, 31, 33, 255, 257, 1023, 1025, 4099, 8191, 16385, 65537, 100003, 262144])
def test_columns(tk, cols, dtype):
    x, u = logits(2, cols, dtype, seed=cols), uniform(2, cols)
    check(tk, x, u)
    check(tk, x, u, top_k=50, top_p=0.95, temperature=0.8)
    check(tk, x, u, top_p=0.9)
    check(tk, x, u, temperature=0.0)


@pytest.mark.parametrize("rows", [1, 2, 30, 152, 153, 305, 700])
@pytest.mark.parametrize("kw", [dict(), dict(top_k=40, top_p=0.9), dict(top_p=0.95), dict(min_p=0.1)], ids=str)
def test_rows(tk, rows, kw):
    check(tk, logits(rows, 3001, BF16, seed=rows), uniform(rows), **kw)


@pytest.mark.parametrize("spread", [0.0, 1e-3, 0.5, 1.0, 4.0, 30.0, 1000.0])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_flat_and_sharp_rows(tk, spread, dtype):
    """From rows that are one value, through rows of many ties, to rows that are one token."""
    x, u = logits(6, 20011, dtype, spread=spread, seed=3), uniform(6, 4)
    for kw in (dict(), dict(top_p=0.9), dict(top_k=3000), dict(top_k=9000, top_p=0.7), dict(top_k=40), dict(min_p=0.5),
               dict(top_p=0.7, min_p=0.9)):
        check(tk, x, u, **kw)


@pytest.mark.parametrize("cols", [1000, 1024, 4096, 50000, 131072])
@pytest.mark.parametrize("dtype", [F16, F32])
def test_uniform_rows_give_every_column_its_turn(tk, cols, dtype):
    """All logits equal: the token is floor(u * n) exactly, on borders too."""
    at = torch.tensor([0, 1, 2, cols // 2, cols - 1, cols // 3])
    u = torch.cat([at.double() / cols, torch.tensor([0.0, 0.5, 0.25, 0.75, 1 - 2.0 ** -24])]).float()
    x = torch.full((len(u), cols), 1.7).to(dtype)
    token, logp = tk.sample_rows(x.cuda(), u.cuda())
    want = torch.floor(u.double() * cols).int()
    assert token.tolist() == want.tolist()
    assert torch.allclose(logp.cpu().double(), torch.full((len(u),), -np.log(cols), dtype=torch.float64), atol=1e-5)
    half, _ = tk.sample_rows(x.cuda(), u.cuda(), top_p=0.5)  # the least prefix with half of the weight
    assert half.tolist() == torch.floor(u.double() * ((cols + 1) // 2)).int().tolist()
    few, _ = tk.sample_rows(x.cuda(), u.cuda(), top_k=300)
    assert few.tolist() == torch.floor(u.double() * 300).int().tolist()


def test_two_values(tk):
    """Ties on both sides of a border that is known exactly: weights 1 and 2^-k."""
    cols, k = 70000, 3
    for high in (1, 5, 2000, 40000):
        x = torch.zeros(1, cols)
        where = torch.randperm(cols, generator=torch.Generator().manual_seed(high))[:high]
        x[0, where] = k
        order = torch.cat([where.sort().values, torch.ones(cols, dtype=torch.bool).index_fill_(0, where, False).nonzero()[:, 0]])
        temperature = 1 / np.log(2)
        w = np.exp2(-k * np.float64(np.log2(np.e)) / np.float64(np.float32(temperature)))
        total = high + (cols - high) * w
        for rank in (0, high - 1, high, high + 1, cols - 1, (cols + high) // 2):
            mid = (rank + 0.5 if rank < high else high + (rank - high + 0.5) * w) / total
            u = torch.tensor([mid], dtype=torch.float32)
            rank_of = u.double().item() * total
            rank_of = int(rank_of) if rank_of < high else high + int((rank_of - high) / w)
            token, _ = tk.sample_rows(x.cuda(), u.cuda(), temperature=temperature)
            assert token.item() == order[rank_of].item(), (high, rank)


def test_zeros_of_both_signs_are_equal(tk):
    x = torch.full((4, 3000), -1.0)
    x[:, 5], x[:, 900], x[:, 2000] = -0.0, 0.0, -0.0
    for dtype in (F16, BF16, F32):
        token, _ = tk.sample_rows(x.to(dtype).cuda(), torch.tensor([0.0, 0.4, 0.9, 0.99]).cuda(), top_k=3)
        assert token.tolist() == [5, 900, 2000, 2000]
    y = torch.zeros(3, 9000)
    y[:, ::2] = -0.0
    token, _ = tk.sample_rows(y.cuda(), torch.tensor([0.0, 0.5, 1 - 2.0 ** -24]).cuda())
    assert token.tolist() == [0, 4500, 8999]


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_masked_columns_are_never_taken(tk, dtype):
    x = logits(50, 9001, dtype, seed=8)
    for share, value in ((0.5, -float("inf")), (0.99, -float("inf")), (0.5, torch.finfo(dtype).min)):
        y = x.clone()
        y[torch.rand(x.shape, generator=torch.Generator().manual_seed(9)) < share] = value
        y[:, 4000] = 1.0
        u = uniform(50, 10)
        u[:5] = 1 - 2.0 ** -24
        for kw in (dict(), dict(top_k=100), dict(top_k=5000), dict(top_p=0.95), dict(min_p=0.01), dict(temperature=0.0)):
            token = check(tk, y, u, **kw)
            assert all(y[r, t] > value for r, t in enumerate(token))


def test_rows_without_a_distribution(tk):
    x = logits(9, 5000, F32, seed=11)
    x[0] = -float("inf")
    x[1, 77] = float("nan")
    x[2, 78] = float("inf")
    x[3, 4999] = float("nan")
    temperature, top_p, min_p, u = torch.ones(9), torch.ones(9), torch.zeros(9), torch.full((9,), 0.5)
    temperature[4], temperature[5], top_p[6], min_p[7], u[8] = -1.0, float("nan"), float("nan"), float("nan"), float("nan")
    token, logp = tk.sample_rows(x.cuda(), u.cuda(), temperature=temperature.cuda(), top_p=top_p.cuda(), min_p=min_p.cuda())
    assert token.tolist() == [-1] * 9 and torch.isnan(logp).all()
    lowest = torch.full((2, 700), torch.finfo(F32).min)  # nothing left but the type's lowest value: all are equal
    token, _ = tk.sample_rows(lowest.cuda(), torch.tensor([0.0, 0.5]).cuda())
    assert token.tolist() == [0, 350]


def test_parameters_of_each_row(tk):
    rows = 300
    g = torch.Generator().manual_seed(12)
    pick = lambda values: torch.tensor(values)[torch.randint(0, len(values), (rows,), generator=g)]
    kw = dict(temperature=pick([0.0, 0.3, 0.7, 1.0, 1.3, 20.0, 1e-30, 1e30, float("inf")]),
              top_k=pick([-5, 0, 1, 20, 50, 1500, 2 ** 31 - 1]).int(), top_p=pick([1.0, 0.99, 0.9, 0.5, 0.0, 7.0, -1.0]),
              min_p=pick([0.0, -1.0, 0.02, 0.5, 1.0, 3.0]))
    u = uniform(rows, 13)
    u[:20], u[20:40] = 0.0, 1.0
    u[40:50], u[50:60] = -3.0, 5.0
    for dtype in (BF16, F32):
        check(tk, logits(rows, 6007, dtype, seed=14), u, **kw)


def test_far_from_zero(tk):
    """Large logits of either sign, and temperatures at which they still differ."""
    for shift, t in ((1000.0, 1.0), (-1000.0, 1.0), (1e4, 0.01), (1e30, 1e28), (-3e38, 1e30)):
        x = logits(4, 3000, F32, seed=15) * max(1.0, abs(shift) * 1e-3) + shift
        check(tk, x, uniform(4, 16), temperature=t)
        check(tk, x, uniform(4, 17), temperature=t, top_k=30, top_p=0.9)


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("first,stride", [(0, 1001), (1, 1003), (3, 1024), (5, 1000), (7, 4096)])
def test_strides_and_alignment(tk, first, stride, dtype):
    """Rows that begin anywhere: what lies beside them is not looked at."""
    rows, cols = 9, 1000
    flat = torch.full((first + rows * stride + 8,), float("inf"), dtype=dtype)
    x = flat[first:first + rows * stride].view(rows, stride)[:, :cols]
    x.copy_(logits(rows, cols, dtype, seed=stride))
    there = flat.cuda()[first:first + rows * stride].view(rows, stride)[:, :cols]
    u = uniform(rows, 18)
    for kw in (dict(), dict(top_k=30, top_p=0.9), dict(top_p=0.9)):
        token, _ = tk.sample_rows(there, u.cuda(), **kw)
        assert token.tolist() == check(tk, x.contiguous(), u, **kw)


def test_close_to_borders(tk):
    """u just beside the borders, nearer than weights of 24 bits can tell."""
    cols = 20000
    x = logits(1, cols, F32, spread=1.0, seed=19)
    best = _rotate.order(x[0])
    w = np.exp(x[0].double().numpy()[best] - x[0].double().numpy().max())
    run = np.cumsum(w) / w.sum()
    g = np.random.default_rng(20)
    u = []
    for i in g.integers(0, cols - 1, 400):
        near = np.float32(run[i])
        u += [near, np.nextafter(near, np.float32(0)), np.nextafter(near, np.float32(1))]
    u = torch.tensor(np.array(u))
    check(tk, x.expand(len(u), cols).contiguous(), u)
    top_p = torch.tensor(np.float32(run[g.integers(0, cols - 1, 200)]))
    check(tk, x.expand(200, cols).contiguous(), uniform(200, 21), top_p=top_p)


def test_outputs_streams_and_graphs(tk):
    x, u = logits(20, 9000, BF16, seed=22), uniform(20, 23)
    want = check(tk, x, u, top_p=0.9)
    xd, ud = x.cuda(), u.cuda()
    token, logp = torch.zeros(20, dtype=torch.int32).cuda(), torch.zeros(20).cuda()
    got = tk.sample_rows(xd, ud, top_p=0.9, token=token, logp=logp)
    assert got[0] is token and got[1] is logp and token.tolist() == want
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    t2, l2 = tk.sample_rows(xd, ud, top_p=0.9, stream=side)
    side.synchronize()
    assert t2.tolist() == want and torch.equal(l2, logp)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tk.sample_rows(xd, ud, top_p=0.9, token=token, logp=logp)
    u3 = uniform(20, 24)
    ud.copy_(u3.cuda())
    token.zero_()
    graph.replay()
    assert token.tolist() == check(tk, x, u3, top_p=0.9)
    empty = tk.sample_rows(xd[:0], ud[:0])
    assert empty[0].shape == (0,) and empty[1].shape == (0,)


def test_refusals(tk):
    x, u = logits(4, 100, F32).cuda(), uniform(4).cuda()
    with pytest.raises(TypeError):
        tk.sample_rows(x.double(), u)
    with pytest.raises(TypeError):
        tk.sample_rows(x, u.double())
    with pytest.raises(TypeError):
        tk.sample_rows(x, u, top_k=torch.ones(4, dtype=torch.int64).cuda())
    with pytest.raises(TypeError):
        tk.sample_rows(x, u, temperature="1")
    for kw in (dict(temperature=-0.5), dict(temperature=float("nan")), dict(temperature=torch.ones(3).cuda()),
               dict(token=torch.zeros(5, dtype=torch.int32).cuda()), dict(logp=torch.zeros(4, 2).cuda()[:, 0])):
        with pytest.raises(ValueError):
            tk.sample_rows(x, u, **kw)
    for kw in (dict(top_p=float("nan")), dict(min_p=float("nan"))):
        with pytest.raises(tk.TopKError):
            tk.sample_rows(x, u, **kw)
    with pytest.raises(ValueError):
        tk.sample_rows(x[0], u)
    with pytest.raises(ValueError):
        tk.sample_rows(x.t(), u)
    with pytest.raises(ValueError):
        tk.sample_rows(x, u.cpu())
    with pytest.raises(ValueError):
        tk.sample_rows(x[:, :0], u)
    with pytest.raises(tk.TopKError):
        tk.sample_rows(torch.zeros(1, 2 ** 21 + 1, dtype=F16).cuda(), u[:1])
    with pytest.raises(tk.TopKError):  # rows over one another
        tk.sample_rows(x[:1].expand(4, 100), u)
    y = x.clone().requires_grad_()
    _, logp = tk.sample_rows(y, u)
    with pytest.raises(RuntimeError, match="not implemented"):
        logp.sum().backward()
    with pytest.raises(RuntimeError, match="no gradient"):
        tk.sample_rows(y, u, logp=torch.zeros(4).cuda())


@pytest.mark.parametrize("dtype,cols", [(F16, 2 ** 21), (F32, 2 ** 21), (BF16, 1300003)])
def test_the_widest_rows(tk, dtype, cols):
    x, u = logits(2, cols, dtype, spread=2.0, seed=30), uniform(2, 31)
    for kw in (dict(), dict(top_p=0.95), dict(top_k=50), dict(top_k=100000, top_p=0.9)):
        check(tk, x, u, **kw)
    flat = torch.full((1, cols), -3.0).to(dtype)
    token, _ = tk.sample_rows(flat.cuda(), torch.tensor([0.75]).cuda())
    assert token.item() == int(0.75 * cols)


def test_two_streams_at_once(tk):
    """Calls on two streams share nothing."""
    x, u = logits(60, 50000, BF16, seed=32), uniform(60, 33)
    xd, ud = x.cuda(), u.cuda()
    want = check(tk, x, u, top_p=0.9)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [tk.sample_rows(xd, ud, top_p=0.9, stream=streams[i % 2])[0] for i in range(10)]
    torch.cuda.synchronize()
    assert all(t.tolist() == want for t in got)


def test_a_decoders_steps(tk):
    """Rotated append, attention, eviction and sampling together, as a decoder makes them, against torch in 64 bits: one
    layer whose hidden state picks the next token's embedding; a captured step is the same as an eager one."""
    seqs, heads, group, dim, page, vocabulary, budget = 3, 2, 2, 64, 16, 2000, 24
    g = torch.Generator().manual_seed(34)
    q_heads, width = heads * group, 4
    embed = torch.randn(vocabulary, (q_heads + 2 * heads) * dim, generator=g).to(BF16)
    head = (torch.randn(q_heads * dim, vocabulary, generator=g) * 0.3).to(BF16)
    norm = (1 + 0.1 * torch.randn(dim, generator=g)).to(BF16)
    freq = (1000.0 ** (-torch.arange(32) / 32)).float()
    steps = 40
    u = torch.rand(steps, seqs, generator=g)
    dev = dict(device="cuda")

    def run(captured):
        k, v = (torch.zeros(seqs * width, heads, page, dim, dtype=BF16, **dev).transpose(1, 2) for _ in range(2))
        table = torch.arange(seqs * width, dtype=torch.int32, **dev).reshape(seqs, width)
        lens, seen = (torch.zeros(seqs, dtype=torch.int32, **dev) for _ in range(2))
        weight = torch.zeros(seqs, heads, width * page, **dev)
        pos = torch.zeros(seqs, heads, width * page, dtype=torch.int32, **dev)
        token, logp = torch.arange(seqs, dtype=torch.int32, **dev), torch.zeros(seqs, **dev)
        e, w, n, f, now = embed.cuda(), head.cuda(), norm.cuda(), freq.cuda(), torch.zeros(seqs, **dev)
        rows = []

        def step():
            x = e[token.long()].view(seqs, -1, dim)
            q, kn, vn = x.split([q_heads, heads, heads], 1)
            q = tk.kv_append_rotated(k, v, table, lens, kn, vn, f, weight=weight, pos=pos, next_pos=seen, k_norm=n, q=q,
                                     q_norm=n)
            lens.add_(1)
            seen.add_(1)
            out, _ = tk.kv_attend(q, k, v, table, lens, weight=weight)
            tk.kv_evict(k, v, table, lens, weight, pos, seen, budget, sink=2, recent=8)
            tk.sample_rows(out.reshape(seqs, -1) @ w, now, temperature=0.8, top_k=40, top_p=0.9, token=token, logp=logp)

        step_of = step
        if captured:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step()  # allocates what a capture may not
                for t in (lens, seen, weight, pos, k, v):
                    t.zero_()
                token.copy_(torch.arange(seqs))
                graph = torch.cuda.CUDAGraph()
                torch.cuda.synchronize()
                with torch.cuda.graph(graph, stream=side):
                    step()
            torch.cuda.synchronize()
            step_of = graph.replay
        for i in range(steps):
            now.copy_(u[i])
            step_of()
            rows.append((token.tolist(), logp.clone(), lens.tolist(), seen.tolist()))
        torch.cuda.synchronize()
        return rows, [t.cpu() for t in (k, v, weight, pos)]

    eager, state = run(False)
    replayed, state2 = run(True)
    assert [r[0] for r in eager] == [r[0] for r in replayed]
    assert all(torch.equal(a, b) for a, b in zip(state, state2))
    assert eager[-1][2] == [budget] * seqs and eager[-1][3] == [steps] * seqs
    # Until the first eviction, one sequence's first steps by the definitions.
    b, keys, values, token = 1, [], [], 1
    for i in range(budget - 1):
        x = embed[token].view(-1, dim)
        at = np.array([i])
        q = torch.from_numpy(_rotate.rotate(x[None, :q_heads], at, freq, norm)[0][0]).to(BF16).double()
        keys.append(torch.from_numpy(_rotate.rotate(x[None, q_heads:q_heads + heads], at, freq, norm)[0][0]).to(BF16).double())
        values.append(x[q_heads + heads:].double())
        kk, vv = (torch.stack(s).repeat_interleave(group, 1) for s in (keys, values))
        p = torch.softmax(torch.einsum("hd,thd->ht", q, kk) * dim ** -0.5, -1)
        logits_ = (torch.einsum("ht,thd->hd", p, vv).to(BF16).double().reshape(-1) @ head.double()).to(BF16)
        ranked = torch.softmax(logits_.double() / 0.8, 0)
        token = eager[i][0][b]
        # The projection's and the attention's roundings may move a border: the token is one that is kept, or nearly.
        assert ranked[token] >= torch.sort(ranked, descending=True).values[44]


@pytest.mark.parametrize("ties", [511, 512, 513, 1500])
def test_limits_of_the_list(tk, ties):
    """As many equal best entries as a list has room for, and one more or less; top_k around the same number."""
    x = logits(4, 9000, F32, spread=1.0, seed=35)
    x[:, torch.randperm(9000, generator=torch.Generator().manual_seed(36))[:ties]] = 6.0
    u = torch.tensor([0.0, 0.3, 0.77, 1 - 2.0 ** -24])
    for kw in (dict(temperature=0.0), dict(top_k=ties), dict(top_k=ties - 1), dict(top_k=ties + 1), dict(min_p=0.9),
               dict(top_k=512), dict(top_k=513), dict(top_p=0.3), dict()):
        check(tk, x, u, **kw)


def test_temperatures_below_the_types_range(tk):
    """A number that 32 bits round to 0 is above 0 all the same: equal best entries take turns, with 1e-30 as with 1e-60."""
    x = torch.full((4, 1000), -1.0)
    x[:, [5, 70, 900]] = 2.0
    u = torch.tensor([0.0, 0.4, 0.9, 0.99])
    for t in (1e-30, 1e-45, 1e-50, 1e-300):
        token, logp = tk.sample_rows(x.cuda(), u.cuda(), temperature=t)
        assert token.tolist() == [5, 70, 900, 900]
        assert torch.allclose(logp.cpu(), torch.full((4,), -np.log(3.0), dtype=F32), atol=2.0 ** -18)
    token, logp = tk.sample_rows(x.cuda(), u.cuda(), temperature=0.0)
    assert token.tolist() == [5] * 4 and logp.tolist() == [0.0] * 4
    with pytest.raises(ValueError):
        tk.sample_rows(x.cuda(), u.cuda(), temperature=-1e-50)
