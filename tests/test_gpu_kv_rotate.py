"""kv_rotate and kv_append_rotated against their definition in 64 bits
(tests/_rotate.py derives the bounds)."""
import numpy as np
import pytest
import torch

import _kv
import _rotate

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def tk():
    import topk_selection_gb300

    yield topk_selection_gb300
    topk_selection_gb300.check_stream()


def gen(seed=0):
    return torch.Generator().manual_seed(seed)


def freqs(pairs, base=10000.0):
    return (base ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float()


def norm_of(kind, heads, dim, dtype, seed):
    if kind is None:
        return None
    shape = (dim,) if kind == "shared" else (heads, dim)
    return (1 + 0.3 * torch.randn(*shape, generator=gen(seed))).to(dtype)


def cuda(t):
    return None if t is None else t.cuda()


def check(tk, tokens, q_heads, heads, dim, pairs, dtype, pairing, kind, far=0, seed=1, fused=True, eps=1e-6):
    q, k, _ = torch.randn(tokens, q_heads + 2 * heads, dim, generator=gen(seed)).to(dtype).split(
        [q_heads, heads, heads], 1)
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    pos = torch.randint(0, far, (tokens,), generator=gen(2)) if far else torch.arange(tokens)
    freq = freqs(pairs)
    qn, kn = norm_of(kind, q_heads, dim, dtype, 3), norm_of(kind, heads, dim, dtype, 4)
    qd, kd = q.cuda(), k.cuda()
    qo, ko = tk.kv_rotate(qd, kd, pos.int().cuda(), freq.cuda(), q_norm=cuda(qn), k_norm=cuda(kn), eps=eps,
                          pairing=pairing)
    for got, x, n in ((qo, q, qn), (ko, k, kn)):
        want, tol = _rotate.rotate(x, pos.numpy(), freq, n, eps, pairing)
        _rotate.close(got, want, tol)
    assert torch.equal(qd.cpu(), q) and torch.equal(kd.cpu(), k)


@pytest.mark.parametrize("pairing", ["halves", "neighbours"])
@pytest.mark.parametrize("kind", [None, "shared", "own"])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("dim,pairs", [(128, 64), (128, 16), (128, 24), (80, 40), (80, 10), (64, 32), (96, 48), (256, 128),
                                       (256, 32), (8, 4), (8, 1), (16, 8), (40, 20), (72, 36), (72, 8), (136, 3),
                                       (248, 124), (200, 96), (112, 56)])
def test_dims(tk, dim, pairs, dtype, kind, pairing):
    check(tk, 5, 4, 2, dim, pairs, dtype, pairing, kind)


@pytest.mark.parametrize("tokens", [1, 2, 31, 64, 257, 3001])
@pytest.mark.parametrize("q_heads,heads", [(1, 1), (32, 8), (7, 1), (64, 8), (5, 5), (40, 10)])
def test_tokens_and_heads(tk, tokens, q_heads, heads):
    check(tk, tokens, q_heads, heads, 128, 64, BF16, "halves", "shared")


@pytest.mark.parametrize("dim,pairs", [(128, 64), (72, 36)])
@pytest.mark.parametrize("far", [4096, 10 ** 6, 2 ** 31 - 1])
def test_far_positions(tk, far, dim, pairs):
    """Where a 32-bit product of position and frequency is off by whole radians."""
    check(tk, 100, 2, 2, dim, pairs, F16, "halves", None, far=far)


def test_angles_to_the_last_bits(tk):
    """Unit vectors: the results are the cosines and sines themselves, of
    negative positions and frequencies, of zeros and of large ones.  64 bits of
    a frequency's turns leave 2^-64 * 2^31 of them per unit of its mantissa's
    scale; float16 shows 2^-12."""
    freq = torch.tensor([1.0, -1.0, 0.0, 1e-8, 3.14159274, 1e-30, 1e-42, 6000.5, -0.3, 0.5, 2.0 ** -31, 1.5], dtype=torch.float32)
    pos = torch.tensor([0, 1, -1, 2, 1000, -99999, 2 ** 31 - 1, -2 ** 31, 12345678], dtype=torch.int64)
    x = torch.zeros(len(pos), 1, 24, dtype=F16)
    x[..., :12] = 1
    got, none = tk.kv_rotate(x.cuda(), None, pos.int().cuda(), freq.cuda())
    assert none is None
    f = freq.double().numpy()
    # The exact product: 2^31 times 24 bits fit 64.
    angle = pos.numpy().astype(np.longdouble)[:, None] * f.astype(np.longdouble)
    want = np.concatenate([np.cos(angle), np.sin(angle)], -1).astype(np.float64)[:, None]
    tol = 2.0 ** -22 + 2.0 ** -11 * np.abs(want) + 2.0 ** -25
    _rotate.close(got, want, np.where(np.abs(np.concatenate([f, f])) > 1000, tol + 2.0 ** -20, tol))


def test_frequencies_that_are_no_numbers(tk):
    freq = torch.tensor([float("inf"), float("nan"), 1.0, 0.5])
    x = torch.ones(1, 1, 16, dtype=F16).cuda()
    got = tk.kv_rotate(x, None, torch.tensor([3], dtype=torch.int32).cuda(), freq.cuda())[0][0, 0].cpu()
    assert torch.isnan(got[[0, 1, 4, 5]]).all() and torch.isfinite(got[[2, 3, 6, 7, *range(8, 16)]]).all()


@pytest.mark.parametrize("dim,pairs", [(64, 8), (40, 3)])
def test_what_is_not_finite_stays_in_its_head(tk, dim, pairs):
    x = torch.randn(3, 4, dim, generator=gen(5)).to(BF16)
    x[1, 2, 0] = float("nan")   # a turned element
    x[2, 1, dim - 1] = float("inf")  # one that is not
    args = torch.arange(3, dtype=torch.int32).cuda(), freqs(pairs).cuda()
    plain = tk.kv_rotate(x.cuda(), None, *args)[0].cpu()
    want = torch.zeros_like(plain, dtype=torch.bool)
    want[1, 2, [0, pairs]] = True
    assert torch.equal(torch.isnan(plain), want)
    assert plain[2, 1, dim - 1] == float("inf") and torch.isfinite(plain[2, 1, :dim - 1].float()).all()
    w = torch.ones(dim, dtype=BF16).cuda()
    normed = tk.kv_rotate(x.cuda(), None, *args, q_norm=w)[0].cpu()
    bad = ~torch.isfinite(normed.float())
    assert bad[1, 2].all() and bad[2, 1, dim - 1] and not bad[0].any() and not bad[1, 3].any() and not bad[2, 0].any()


def test_zeros_and_eps(tk):
    x = torch.zeros(2, 3, 64, dtype=F16).cuda()
    w, pos, f = torch.ones(64, dtype=F16).cuda(), torch.arange(2, dtype=torch.int32).cuda(), freqs(32).cuda()
    assert torch.equal(tk.kv_rotate(x, None, pos, f, q_norm=w)[0], x)
    assert torch.isnan(tk.kv_rotate(x, None, pos, f, q_norm=w, eps=0.0)[0]).all()


def test_keys_alone_and_one_norm(tk):
    x = torch.randn(9, 3, 64, generator=gen(6)).to(F16)
    w = norm_of("shared", 3, 64, F16, 7)
    pos, f = torch.arange(9), freqs(32)
    none, got = tk.kv_rotate(None, x.cuda(), pos.int().cuda(), f.cuda(), k_norm=w.cuda())
    assert none is None
    _rotate.close(got, *_rotate.rotate(x, pos.numpy(), f, w))
    # A norm for one of the two only.
    qo, ko = tk.kv_rotate(x.cuda(), x.cuda(), pos.int().cuda(), f.cuda(), q_norm=w.cuda())
    _rotate.close(qo, *_rotate.rotate(x, pos.numpy(), f, w))
    _rotate.close(ko, *_rotate.rotate(x, pos.numpy(), f))


@pytest.mark.parametrize("dim,pairs", [(128, 64), (72, 36)])
def test_in_place_on_a_fused_projection(tk, dim, pairs):
    full = torch.randn(33, 12, dim, generator=gen(8)).to(BF16)
    there = full.cuda()
    q, k, v = there.split([6, 3, 3], 1)
    got = tk.kv_rotate(q, k, torch.arange(33, dtype=torch.int32).cuda(), freqs(pairs).cuda(), q_out=q, k_out=k)
    assert got[0] is q and got[1] is k
    want, tol = _rotate.rotate(full[:, :9], np.arange(33), freqs(pairs))
    _rotate.close(there[:, :9], want, tol)
    assert torch.equal(there[:, 9:].cpu(), full[:, 9:])


def test_head_major_outputs_and_inputs(tk):
    x = torch.randn(4, 50, 64, generator=gen(9)).to(F16)  # [heads, tokens, dim]
    out = torch.full((7, 50, 64), 5.0, dtype=F16).cuda()
    tk.kv_rotate(x.cuda().transpose(0, 1), None, torch.arange(50, dtype=torch.int32).cuda(), freqs(32).cuda(),
                 q_out=out[2:6].transpose(0, 1))
    want, tol = _rotate.rotate(x.transpose(0, 1), np.arange(50), freqs(32))
    _rotate.close(out[2:6].transpose(0, 1), want, tol)
    assert (out[:2] == 5).all() and (out[6:] == 5).all()


def test_refusals(tk):
    x = torch.zeros(4, 6, 64, dtype=F16).cuda()
    pos, f = torch.zeros(4, dtype=torch.int32).cuda(), freqs(32).cuda()
    w = torch.ones(64, dtype=F16).cuda()
    with pytest.raises(TypeError):
        tk.kv_rotate(x.float(), None, pos, f)
    with pytest.raises(TypeError):
        tk.kv_rotate(x, x.to(BF16), pos, f)
    with pytest.raises(TypeError):
        tk.kv_rotate(x, None, pos.long(), f)
    with pytest.raises(TypeError):
        tk.kv_rotate(x, None, pos, f.double())
    with pytest.raises(TypeError):
        tk.kv_rotate(x, None, pos, f, q_norm=w.float())
    with pytest.raises(ValueError):
        tk.kv_rotate(None, None, pos, f)
    with pytest.raises(ValueError):
        tk.kv_rotate(x, None, pos[:3], f)
    with pytest.raises(ValueError):
        tk.kv_rotate(x, None, pos, freqs(33).cuda())
    with pytest.raises(ValueError):
        tk.kv_rotate(x, None, pos, f[:0])
    with pytest.raises(ValueError):
        tk.kv_rotate(x, None, pos, f, pairing="pairs")
    with pytest.raises(ValueError):
        tk.kv_rotate(x, None, pos, f, q_norm=torch.ones(5, 64, dtype=F16).cuda())
    with pytest.raises(ValueError):
        tk.kv_rotate(x, None, pos, f, k_norm=w)
    with pytest.raises(ValueError):
        tk.kv_rotate(x, None, pos, f, q_out=x[:3])
    with pytest.raises(ValueError):
        tk.kv_rotate(x, None, pos.cpu(), f)
    with pytest.raises(ValueError):
        tk.kv_rotate(x.transpose(1, 2), None, pos, f)
    for kw in (dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))):
        with pytest.raises(tk.TopKError):
            tk.kv_rotate(x, None, pos, f, q_norm=w, **kw)
    with pytest.raises(tk.TopKError):  # strides that are no multiple of 16 bytes
        tk.kv_rotate(torch.zeros(4, 6, 68, dtype=F16).cuda()[..., :64], None, pos, f)
    with pytest.raises(tk.TopKError):
        tk.kv_rotate(torch.zeros(4 * 6 * 64 + 4, dtype=F16).cuda()[4:].view(4, 6, 64), None, pos, f)
    with pytest.raises(tk.TopKError):  # an output over its input, shifted
        big = torch.zeros(5, 6, 64, dtype=F16).cuda()
        tk.kv_rotate(big[:4], None, pos, f, q_out=big[1:])
    with pytest.raises(tk.TopKError):  # over the other's
        out = torch.zeros(4, 8, 64, dtype=F16).cuda()
        tk.kv_rotate(x, x, pos, f, q_out=out[:, :6], k_out=out[:, 2:])
    with pytest.raises(tk.TopKError):  # over itself
        tk.kv_rotate(x, None, pos, f, q_out=torch.zeros(4, 1, 64, dtype=F16).cuda().expand(4, 6, 64))
    with pytest.raises(tk.TopKError):
        tk.kv_rotate(torch.zeros(4, 2, 264, dtype=F16).cuda(), None, pos, f)


def test_nothing_to_do(tk):
    q, k = tk.kv_rotate(torch.zeros(0, 4, 64, dtype=F16).cuda(), torch.zeros(0, 2, 64, dtype=F16).cuda(),
                        torch.zeros(0, dtype=torch.int32).cuda(), freqs(32).cuda())
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)


def test_gradients_are_refused_or_say_so(tk):
    x = torch.randn(2, 2, 64, device="cuda").to(F16).requires_grad_()
    pos, f = torch.zeros(2, dtype=torch.int32).cuda(), freqs(32).cuda()
    q, _ = tk.kv_rotate(x, None, pos, f)
    with pytest.raises(RuntimeError, match="not implemented"):
        q.float().sum().backward()
    with pytest.raises(RuntimeError, match="kv_rotate has no gradient"):
        tk.kv_rotate(x, None, pos, f, q_out=torch.empty_like(x))
    with torch.no_grad():
        tk.kv_rotate(x, None, pos, f, q_out=torch.empty_like(x))
    # What autograd saved of an output before the call is known to be stale.
    y = torch.randn(2, 2, 64, device="cuda").to(F16)
    z = (y.requires_grad_(False) * torch.ones(1, device="cuda", dtype=F16).requires_grad_()).sum()
    tk.kv_rotate(y, None, pos, f, q_out=y)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.backward()


def test_streams_and_graphs(tk):
    x = torch.randn(40, 8, 128, generator=gen(10)).to(BF16)
    pos = torch.arange(40)
    xd, posd, f = x.cuda(), pos.int().cuda(), freqs(64).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = tk.kv_rotate(xd, None, posd, f, stream=side)[0]
    torch.cuda.current_stream().wait_stream(side)
    _rotate.close(out, *_rotate.rotate(x, pos.numpy(), freqs(64)))
    out.record_stream(torch.cuda.current_stream())
    q_out = torch.empty_like(xd)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tk.kv_rotate(xd, None, posd, f, q_out=q_out)
    posd += 77
    q_out.zero_()
    graph.replay()
    _rotate.close(q_out, *_rotate.rotate(x, pos.numpy() + 77, freqs(64)))


# --- on the way to the pages


def check_append(tk, lens, new, heads, q_heads, dim, pairs, page, dtype, layout, pairing="halves", kind="shared",
                 ahead=0, positions=True, starts_past=0, sides=True, seed=20):
    """Appends new[b] tokens behind lens[b] held ones, and looks at every element of the pools, the side arrays and q_out."""
    cache = _kv.Cache(lens, heads, dim, page, dtype, layout, room=max(new), seed=seed)
    seqs, total = len(lens), sum(new) + starts_past
    qkv = torch.randn(total, q_heads + 2 * heads, dim, generator=gen(seed + 1)).to(dtype)
    q, k_new, v_new = qkv.split([q_heads, heads, heads], 1)
    qn, kn = norm_of(kind, q_heads, dim, dtype, 22) if q_heads else None, norm_of(kind, heads, dim, dtype, 23)
    starts = np.concatenate([[0], np.cumsum(new)])
    next_pos = torch.tensor([n + (ahead * (b + 1)) for b, n in enumerate(lens)], dtype=torch.int32)
    weight = torch.full((seqs, heads, cache.capacity), 3.0)
    pos = torch.full((seqs, heads, cache.capacity), -9, dtype=torch.int32)
    k, v, table, lens_d = cache.dev()
    w_d, p_d = weight.cuda(), pos.cuda()
    q_out = torch.full((total, q_heads, dim), 7.0, dtype=dtype).cuda() if q_heads else None
    there = qkv.cuda().split([q_heads, heads, heads], 1)
    f = freqs(pairs)
    got = tk.kv_append_rotated(k, v, table, lens_d, there[1], there[2], f.cuda(),
                               starts=None if all(n == 1 for n in new) and not starts_past else
                               torch.tensor(starts, dtype=torch.int32).cuda(),
                               weight=w_d if sides else None, pos=p_d if sides and positions else None,
                               next_pos=next_pos.cuda() if positions else None, k_norm=cuda(kn), pairing=pairing,
                               q=there[0] if q_heads else None, q_norm=cuda(qn), q_out=q_out)
    assert got is q_out
    at = np.concatenate([(next_pos[b].item() if positions else lens[b]) + np.arange(n) for b, n in enumerate(new)]
                        or [np.zeros(0)]).astype(np.int64)
    n_all = int(starts[-1])
    want_k, tol_k = _rotate.rotate(k_new[:n_all], at, f, kn, 1e-6, pairing)
    ek, ev = cache.k.clone(), cache.v.clone()
    kk, vv = k.cpu(), v.cpu()
    seen = torch.zeros(kk.shape[:2], dtype=torch.bool)
    for b in range(seqs):
        for i in range(new[b]):
            s = lens[b] + i
            p, o = cache.table[b, s // page].item(), s % page
            _rotate.close(kk[p, o], want_k[starts[b] + i], tol_k[starts[b] + i])
            assert torch.equal(vv[p, o], v_new[starts[b] + i])
            seen[p, o] = True
            if sides:
                weight[b, :, s] = 0
                if positions:
                    pos[b, :, s] = int(at[starts[b] + i])
    as_bits = lambda t: t.contiguous().view(torch.int16)
    assert torch.equal(as_bits(kk)[~seen], as_bits(ek)[~seen]) and torch.equal(as_bits(vv)[~seen], as_bits(ev)[~seen])
    assert torch.equal(w_d.cpu(), weight) and torch.equal(p_d.cpu(), pos)
    if q_heads:
        _rotate.close(q_out[:n_all], *_rotate.rotate(q[:n_all], at, f, qn, 1e-6, pairing))
        assert (q_out[n_all:] == 7).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("layout", ["head", "token"])
@pytest.mark.parametrize("lens,new", [([0], [1]), ([5, 0, 300], [1, 1, 1]), ([16, 15, 17, 1], [33, 0, 1, 16]),
                                      ([7, 9], [0, 0]), ([100], [700]), ([3] * 40, [2, 0, 5, 1] * 10)])
def test_append_lengths(tk, lens, new, layout, dtype):
    check_append(tk, lens, new, 2, 4, 64, 32, 16, dtype, layout, ahead=1000)


@pytest.mark.parametrize("pairing", ["halves", "neighbours"])
@pytest.mark.parametrize("kind", [None, "shared", "own"])
@pytest.mark.parametrize("dim,pairs,heads,q_heads", [(128, 64, 8, 32), (128, 16, 8, 0), (72, 36, 3, 3), (80, 10, 2, 6),
                                                     (8, 1, 1, 1), (256, 128, 5, 10), (96, 48, 4, 0), (40, 7, 1, 12)])
def test_append_dims(tk, dim, pairs, heads, q_heads, kind, pairing):
    check_append(tk, [9, 0, 40], [3, 20, 1], heads, q_heads, dim, pairs, 8, BF16, "token", pairing, kind, ahead=5)


@pytest.mark.parametrize("sides,positions", [(True, False), (False, True), (False, False)])
def test_append_without_side_arrays(tk, sides, positions):
    """Without next_pos a token's position is its slot; next_pos may come without pos."""
    check_append(tk, [9, 130], [3, 5], 2, 2, 64, 32, 16, F16, "head", sides=sides, positions=positions, ahead=100000)


def test_append_ignores_tokens_behind_the_last_sequence(tk):
    check_append(tk, [9, 3], [3, 0], 2, 2, 64, 32, 16, F16, "head", starts_past=6)


def test_append_drops_what_has_no_place(tk):
    """Beyond the capacity, or on a page that the table does not name: the query is turned all the same."""
    cache = _kv.Cache([30, 16], 1, 16, 16, F16, "token", seed=30)
    k, v, table, lens = cache.dev()
    table[1, 1] = -1
    before = k.clone(), v.clone()
    x = torch.randn(3, 8, 1, 16, generator=gen(31)).to(F16)
    q_out = torch.zeros(8, 1, 16, dtype=F16).cuda()
    tk.kv_append_rotated(k, v, table, lens, x[0].cuda(), x[1].cuda(), freqs(8).cuda(),
                         starts=torch.tensor([0, 5, 8], dtype=torch.int32).cuda(), q=x[2].cuda(), q_out=q_out)
    at = np.array([30, 31, 32, 33, 34, 16, 17, 18])
    _rotate.close(q_out, *_rotate.rotate(x[2], at, freqs(8)))
    p = cache.table[0, 1].item()
    want, tol = _rotate.rotate(x[0][:2], at[:2], freqs(8))
    _rotate.close(k[p, 14:16], want, tol)
    for new, old in zip((k, v), before):
        new[p, 14:16] = old[p, 14:16]
        assert torch.equal(new.view(torch.int16), old.view(torch.int16))


def test_append_matches_rotate_and_append(tk):
    """The same as kv_rotate and then kv_append, bit for bit."""
    lens, new = [40, 3, 0], [70, 1, 33]
    cache = _kv.Cache(lens, 4, 128, 16, BF16, "head", room=70, seed=32)
    k, v, table, lens_d = cache.dev()
    k2, v2 = k.clone(), v.clone()
    qkv = torch.randn(sum(new), 24, 128, generator=gen(33)).to(BF16).cuda()
    q, kn, vn = qkv.split([16, 4, 4], 1)
    starts = torch.tensor([0, 70, 71, 104], dtype=torch.int32).cuda()
    w = norm_of("shared", 4, 128, BF16, 34).cuda()
    f = freqs(64).cuda()
    q_out = tk.kv_append_rotated(k, v, table, lens_d, kn, vn, f, starts=starts, k_norm=w, q=q, q_norm=w)
    pos = torch.cat([torch.arange(a, a + n) for a, n in zip(lens, new)]).int().cuda()
    q2, kr = tk.kv_rotate(q, kn, pos, f, q_norm=w, k_norm=w)
    tk.kv_append(k2, v2, table, lens_d, kr, vn, starts=starts)
    assert torch.equal(q_out, q2)
    assert torch.equal(k.view(torch.int16), k2.view(torch.int16)) and torch.equal(v.view(torch.int16), v2.view(torch.int16))


def test_append_refusals(tk):
    cache = _kv.Cache([9, 3], 2, 64, 16, F16, "head", room=4, seed=35)
    k, v, table, lens = cache.dev()
    x = torch.zeros(2, 2, 64, dtype=F16).cuda()
    f = freqs(32).cuda()
    pos = torch.zeros(2, 2, cache.capacity, dtype=torch.int32).cuda()

    def call(**kw):
        a = dict(k_new=x, v_new=x, freq=f)
        a.update(kw)
        return tk.kv_append_rotated(k, v, table, lens, **a)

    for kw in (dict(pos=pos), dict(q_out=x), dict(q_norm=x[0, 0]), dict(k_new=torch.zeros(3, 2, 64, dtype=F16).cuda()),
               dict(k_new=x[:1], v_new=x[:1]), dict(pairing=3), dict(freq=freqs(33).cuda()), dict(q=x[:1])):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(tk.TopKError):  # q_out over k_new
        y = torch.zeros(2, 2, 64, dtype=F16).cuda()
        call(q=y, q_out=x)
    with pytest.raises(RuntimeError, match="no gradient"):
        call(q=x.clone().requires_grad_(), q_out=torch.empty_like(x))
    with pytest.warns(UserWarning, match="no gradient"):
        call(k_new=x.clone().requires_grad_())
    out = call(q=x.clone().requires_grad_())
    with pytest.raises(RuntimeError, match="not implemented"):
        out.float().sum().backward()


@pytest.mark.parametrize("tokens", [1, 2, 17])
@pytest.mark.parametrize("heads,parts", [(5, 3), (4, 4), (1, 3)])
def test_in_place_where_heads_lie_between_one_another(tk, tokens, heads, parts):
    """A projection that has each head's query, key and value side by side: q, k and v share every row of tokens, and no
    element."""
    full = torch.randn(tokens, heads, parts, 64, generator=gen(40)).to(F16)
    there = full.cuda()
    q, k, v = (there[:, :, i] for i in range(3))
    tk.kv_rotate(q, k, torch.arange(tokens, dtype=torch.int32).cuda(), freqs(32).cuda(), q_out=q, k_out=k)
    want, tol = _rotate.rotate(full[:, :, :2].reshape(tokens, -1, 64), np.arange(tokens), freqs(32))
    _rotate.close(there[:, :, :2].reshape(tokens, -1, 64), want, tol)
    assert torch.equal(there[:, :, 2:].cpu(), full[:, :, 2:])
    # On the way to the pages, the queries in place.
    cache = _kv.Cache([9], heads, 64, 16, F16, "head", room=tokens, seed=41)
    kp, vp, table, lens = cache.dev()
    there = full.cuda()
    q, k, v = (there[:, :, i] for i in range(3))
    tk.kv_append_rotated(kp, vp, table, lens, k, v, freqs(32).cuda(),
                         starts=torch.tensor([0, tokens], dtype=torch.int32).cuda(), q=q, q_out=q)
    at = 9 + np.arange(tokens)
    want, tol = _rotate.rotate(full[:, :, 0], at, freqs(32))
    _rotate.close(there[:, :, 0], want, tol)
    assert torch.equal(there[:, :, 1:].cpu(), full[:, :, 1:])
    want, tol = _rotate.rotate(full[:, :, 1], at, freqs(32))
    for i in range(tokens):
        p, o = cache.table[0, (9 + i) // 16].item(), (9 + i) % 16
        _rotate.close(kp[p, o], want[i], tol[i])
        assert torch.equal(vp[p, o].cpu(), full[i, :, 2])


def test_heads_that_meet_are_refused(tk):
    """Rows of heads in which two tensors do share elements."""
    full = torch.zeros(3, 4, 192 + 64, dtype=F16).cuda()
    pos, f = torch.zeros(3, dtype=torch.int32).cuda(), freqs(32).cuda()
    q = full[..., :64]
    for first in (8, 32, 56, 200, 248):  # a head on from there, in these rows or into the next ones
        k = full.view(-1)[first:].as_strided((3, 4, 64), (1024, 256, 1)) if first < 200 else \
            full.view(-1).as_strided((2, 4, 64), (1024, 256, 1), first)
        n = k.shape[0]
        with pytest.raises(tk.TopKError):
            tk.kv_rotate(q[:n], k, pos[:n], f, q_out=q[:n], k_out=k)
    with pytest.raises(tk.TopKError):  # one token
        tk.kv_rotate(q[:1], full[:1, :, 32:96], pos[:1], f, q_out=q[:1], k_out=full[:1, :, 32:96])


def test_outputs_that_are_no_tensors_are_refused(tk):
    """Before anything is asked of them, with gradients on and off."""
    x = torch.zeros(2, 2, 64, dtype=F16).cuda()
    pos, f = torch.zeros(2, dtype=torch.int32).cuda(), freqs(32).cuda()
    cache = _kv.Cache([9, 3], 2, 64, 16, F16, "head", room=4, seed=42)
    k, v, table, lens = cache.dev()
    for bad in (5, "q", [x], x.cpu().numpy(), object()):
        for mode in (torch.enable_grad(), torch.no_grad()):
            with mode:
                with pytest.raises(TypeError, match="q_out must be a torch.Tensor"):
                    tk.kv_rotate(x, None, pos, f, q_out=bad)
                with pytest.raises(TypeError, match="k_out must be a torch.Tensor"):
                    tk.kv_rotate(x, x, pos, f, k_out=bad)
                with pytest.raises(TypeError, match="q_out must be a torch.Tensor"):
                    tk.kv_append_rotated(k, v, table, lens, x, x, f, q=x, q_out=bad)
