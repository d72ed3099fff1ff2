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


def fill(cache, b, slot, pool, head, value):
    """pool's vector of a slot that sequence b holds."""
    pool[cache.table[b, slot // cache.page], slot % cache.page, head] = value


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
