"""sample_rows where one entry is sure and all others are equal, far below it:
every border is known in closed form, and each weight's error counts as often
as there are equal ones.  The token has to be the definition's wherever u is
not within 2^-36 of a border, as the header says (the forms here, in float64,
are right to some 2^-50)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def tk():
    import topk_selection_gb300

    yield topk_selection_gb300
    topk_selection_gb300.check_stream()


def check(tk, cols, value, dtype, top_p=1.0, rows=24, sure=5, seed=0):
    """Every second u is next to a border, the others are anywhere in the equal entries' share."""
    value = torch.tensor(value).to(dtype).double().item()
    w = np.exp(value)
    top_p = float(np.float32(top_p))
    # Kept: the sure entry, and so many of the equal ones.
    kept = cols - 1 if top_p >= 1 else int(np.ceil((top_p * (1 + (cols - 1) * w) - 1) / w))
    total = 1 + kept * w
    g = np.random.default_rng(seed)
    u = np.float32((1 + g.uniform(0, kept, rows) * w) / total)
    u[::2] = np.float32((1 + g.integers(1, kept, rows)[::2] * w) / total)
    u[::4] = np.nextafter(u[::4], np.float32(0))
    u = np.minimum(u, np.float32(1 - 2.0 ** -24))
    x = torch.full((rows, cols), value, dtype=dtype, device="cuda")
    x[:, sure] = 0
    token, logp = tk.sample_rows(x, torch.from_numpy(u).cuda(), top_p=top_p)
    at = (u.astype(np.float64) * total - 1) / w  # the equal entries that are passed, and a part of one
    near = np.abs(at - np.rint(at)) * w / total
    rank = np.floor(at).astype(np.int64)
    want = np.where(at < 0, sure, np.where(rank < sure, rank, rank + 1))
    got = token.cpu().numpy()
    wrong = (got != want) & (near > 2.0 ** -36)
    assert not wrong.any(), [(float(u[i]), int(got[i]), int(want[i]), float(np.log2(near[i]))) for i in np.flatnonzero(wrong)]
    lp = np.where(got == sure, 0.0, value) - np.log(total)
    assert np.abs(logp.cpu().numpy() - lp).max() <= 2.0 ** -18 + 2.0 ** -22 * np.abs(lp).max()


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("value", [-12.0, -13.9, -14.05, -14.5, -15.1, -16.7, -18.3, -21.0])
@pytest.mark.parametrize("cols", [20011, 131072, 262144])
def test_equal_entries_far_below_a_sure_one(tk, cols, value, dtype):
    check(tk, cols, value, dtype, seed=cols)


@pytest.mark.parametrize("value", [-14.5, -14.56, -14.75, -15.1, -20.8])
def test_as_many_as_there_can_be(tk, value):
    check(tk, 2 ** 21, value, F32, seed=1)
    check(tk, 2 ** 21, value, BF16, rows=12, seed=2)


@pytest.mark.parametrize("top_p", [0.999, 0.95])
@pytest.mark.parametrize("cols,value", [(262144, -11.3), (2 ** 21, -13.1), (2 ** 21, -15.1)])
def test_cut_by_top_p(tk, cols, value, top_p):
    check(tk, cols, value, F32, top_p=top_p, sure=cols // 2, seed=3)


def octaves_with_parts_of_a_unit(g, cols, last, past, low=None):
    """A row and a u.  The largest entry has 2^40.5 units of 2^-41 of its octave's weight 1; each of the octaves from 7 to
    `last` below it has nearly a unit more than a whole number of them; u times all is `past` units past the largest.
    low: the value of the other columns, not counted."""
    values = [np.float32(-0.4999 * np.log(2))]
    for o in range(7, min(last, 41) + 1):  # an entry each
        while True:
            x = np.float32((g.uniform(-0.45, 0.45) - o) * np.log(2))
            if 0.85 < np.exp(float(x)) * 2.0 ** 41 % 1 < 0.95:
                break
        values.append(x)
    for o in range(42, last + 1):  # so many that they are nearly a unit
        values += [np.float32(-o * np.log(2))] * int(0.97 * 2 ** (o - 41))
    w = np.exp(np.float64(values))
    u = np.float32(w[0] / w.sum() * (1 - 2.0 ** -12 * g.uniform(1, 2)))
    left = (w[0] + past * 2.0 ** -41) / float(u) - w.sum()  # three entries bring all to where u is
    for share in (0.9, 1 - 2.0 ** -18, 1.0):
        values.append(np.float32(np.log(left * share)))
        left -= np.exp(float(values[-1]))
    x = np.full(cols, -np.inf if low is None else low, dtype=np.float32)
    x[g.permutation(cols)[:len(values)]] = values
    w = np.sort(np.exp(np.float64(values)))[::-1]
    share = (float(u) * w.sum() - w[0]) / w.sum()
    assert 2.0 ** -36 < share < 2.0 ** -35
    return x, u, np.argsort(-x, kind="stable")[1]


def made(seed, rows, *args, **kw):
    g = np.random.default_rng(seed)
    return [np.stack(v) for v in zip(*(octaves_with_parts_of_a_unit(g, *args, **kw) for _ in range(rows)))]


def test_sums_over_the_octaves(tk):
    """What each octave has below a whole unit counts too: with 46 units less, u would still be in the largest entry's
    weight, by more than 2^-36 of all."""
    x, u, want = made(4, 64, 20000, 52, 32)
    token, _ = tk.sample_rows(torch.from_numpy(x).cuda(), torch.from_numpy(u).cuda())
    assert token.tolist() == want.tolist()


def test_sums_over_the_octaves_down_to_min_p(tk):
    """The same of what min_p keeps of a prefix that top_p cut: 2^20 entries of octave 40 are more than top_p leaves out."""
    x, u, want = made(5, 16, 2 ** 20, 38, 25, low=np.float32(-40 * np.log(2)))
    token, _ = tk.sample_rows(torch.from_numpy(x).cuda(), torch.from_numpy(u).cuda(), top_p=1 - 2.0 ** -22,
                              min_p=2.0 ** -38.5)  # 2^-39 of the largest: between the two
    assert token.tolist() == want.tolist()
