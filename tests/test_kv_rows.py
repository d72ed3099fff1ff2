"""Which side arrays the key-value cache operators take: their rows, each a
stretch of memory, are laid out in numpy and looked at for overlaps.  Refusals
come before any CUDA call, and what is accepted goes on to one, so this runs
without a GPU (the addresses are never used)."""
import ctypes
import random

import numpy as np
import pytest

from test_kv_abi import addr, attend, cache, rows, tk  # noqa: F401

INVALID = 1


def stretches(seqs, heads, seq, head, slots, first=0):
    return [(first + b * seq + h * head, first + b * seq + h * head + slots) for b in range(seqs) for h in range(heads)]


def overlap(a, b):
    return any(x0 < y1 and y0 < x1 for x0, x1 in a for y0, y1 in b)


def refused(tk, c, weight, weight_out):
    """Whether the call is refused for its arguments (a call that is not ends at the first look at an address)."""
    real = tk._KvRows
    got = attend(tk, c=c, weight=ctypes.byref(real(*weight)), weight_out=ctypes.byref(real(*weight_out)))
    return got == INVALID


@pytest.fixture(scope="module")
def no_gpu():
    import torch

    if torch.cuda.is_available():
        pytest.skip("on a machine with a GPU the made-up addresses are refused too")


def test_rows_inside_one_another(tk, no_gpu):  # noqa: F811
    """Of one array: sequence 0's second head where sequence 1's first one is, and the like."""
    c = dict(seqs=2, heads=2, table_width=5, table_stride=5)
    out = (addr(9), 160, 80, 80)
    assert refused(tk, cache(tk, **c), (addr(8), 80, 80, 80), out)
    assert refused(tk, cache(tk, **c), (addr(8), 120, 199, 80), out)  # 199 to 279 and 120 to 200
    assert not refused(tk, cache(tk, **c), (addr(8), 120, 200, 80), out)
    assert not refused(tk, cache(tk, **c), (addr(8), 80, 160, 80), out)
    assert not refused(tk, cache(tk, **c), (addr(8), 160, 80, 80), out)


def test_every_layout(tk, no_gpu):  # noqa: F811
    """Random strides and places of two arrays against a look at each pair of rows."""
    rng = random.Random(1)
    seen = np.zeros(2, int)
    for _ in range(4000):
        seqs, heads, slots = rng.choice([1, 2, 3, 5]), rng.choice([1, 2, 3, 4]), 80
        own = slots + rng.choice([0, 0, 7, 40])
        steps = [(own * heads, own), (own, own * seqs), (2 * own * heads, 2 * own), (rng.randrange(80, 700),
                                                                                     rng.randrange(80, 700))]
        seq, head = rng.choice(steps)
        many = slots + rng.choice([0, 0, 1, 30])
        apart = rng.choice([own, -own, 3 * own, rng.randrange(-3000, 3000), 10 ** 6, 0])
        a, b = stretches(seqs, heads, seq, head, slots), stretches(seqs, heads, seq, head, many, apart)
        itself = any(overlap(x[:i] + x[i + 1:], [x[i]]) for x in (a, b) for i in range(len(x)))
        want = itself or (apart != 0 and overlap(a, b))
        anywhere = 12345 * 80  # a dimension of one element has any stride
        put = (anywhere if seqs == 1 else seq, anywhere if heads == 1 else head)
        weight, weight_out = (addr(8), *put, slots), (addr(8) + 4 * apart, seq, head, many)
        got = refused(tk, cache(tk, seqs=seqs, heads=heads, k_stride=(8192, 64, 1024), v_stride=(8192, 64, 1024)),
                      weight, weight_out) if 4 % heads == 0 else None
        if got is not None:
            assert got == want, (seqs, heads, weight, weight_out)
            seen[int(want)] += 1
    assert seen.min() > 500
