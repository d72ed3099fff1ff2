"""Argument checks of topk_kv_rotate, topk_kv_append_rotated and
topk_sample_rows: made on the host before any CUDA call, so these run without a
GPU (the addresses are never used)."""
import ctypes

import pytest

from test_kv_abi import addr, cache, rows, tk  # noqa: F401

INVALID, UNSUPPORTED = 1, 2


class Rotation(ctypes.Structure):
    _fields_ = [("freq", ctypes.c_void_p), ("pairs", ctypes.c_int), ("pairing", ctypes.c_int), ("q_norm", ctypes.c_void_p),
                ("q_norm_stride", ctypes.c_int64), ("k_norm", ctypes.c_void_p), ("k_norm_stride", ctypes.c_int64),
                ("eps", ctypes.c_float)]


class Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride", ctypes.c_int64 * 2), ("heads", ctypes.c_int)]


class Sampling(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_float), ("temperatures", ctypes.c_void_p), ("top_k", ctypes.c_int),
                ("top_ks", ctypes.c_void_p), ("top_p", ctypes.c_float), ("top_ps", ctypes.c_void_p),
                ("min_p", ctypes.c_float), ("min_ps", ctypes.c_void_p)]


def rotation(**kw):
    r = Rotation(addr(20), 32, 0, addr(21), 0, addr(22), 64, 1e-6)
    for name, value in kw.items():
        setattr(r, name, value)
    return ctypes.byref(r)


def heads(i, token=512, head=64, n=4, first=0):
    return ctypes.byref(Heads(addr(i) + first, (ctypes.c_int64 * 2)(token, head), n))


def rotate(tk, dtype=1, tokens=8, dim=64, r=None, pos=addr(9), q="q", k="k", q_out="qo", k_out="ko"):  # noqa: F811
    pick = {"q": heads(5), "k": heads(6), "qo": heads(7), "ko": heads(8)}
    return tk._lib.topk_kv_rotate(dtype, tokens, dim, r or rotation(), pos, pick.get(q, q), pick.get(k, k),
                                  pick.get(q_out, q_out), pick.get(k_out, k_out), None)


def append(tk, c=None, r=None, tokens=2, starts=None, k="k", v="v", weight=None, pos=None, next_pos=None, q=None,  # noqa: F811
           q_out=None):
    pick = {"k": heads(5, 128, 64, 2), "v": heads(6, 128, 64, 2)}
    return tk._lib.topk_kv_append_rotated(c or cache(tk), r or rotation(), tokens, starts, pick.get(k, k), pick.get(v, v),
                                          weight, pos, next_pos, q, q_out, None)


def sample(tk, logits=addr(1), dtype=2, stride=1000, rows=4, cols=1000, s=None, u=addr(2), token=addr(3),  # noqa: F811
           logp=addr(4)):
    s = ctypes.byref(s or Sampling(1.0, None, 0, None, 1.0, None, 0.0, None))
    return tk._lib.topk_sample_rows(logits, dtype, stride, rows, cols, s, u, token, logp, None)


ROTATIONS = [dict(freq=None), dict(freq=addr(20) + 2), dict(pairs=0), dict(pairs=33), dict(pairing=2), dict(pairing=-1),
             dict(q_norm=addr(21) + 8), dict(k_norm=addr(22) + 2), dict(q_norm_stride=4), dict(k_norm_stride=-64),
             dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(k_norm_stride=2 ** 34)]


@pytest.mark.parametrize("kw", ROTATIONS, ids=str)
def test_rotations(tk, kw):  # noqa: F811
    assert rotate(tk, r=rotation(**kw)) == INVALID
    assert append(tk, r=rotation(**kw)) == INVALID


def test_rotate_refusals(tk):  # noqa: F811
    assert rotate(tk, dtype=2) == INVALID
    assert rotate(tk, tokens=-1) == INVALID
    assert rotate(tk, pos=None) == INVALID
    assert rotate(tk, pos=addr(9) + 2) == INVALID
    assert rotate(tk, q=None, k=None, q_out=None, k_out=None) == INVALID
    assert rotate(tk, q_out=None) == INVALID
    assert rotate(tk, k=None) == INVALID
    assert rotate(tk, dim=68) == UNSUPPORTED
    assert rotate(tk, dim=264) == UNSUPPORTED
    assert rotate(tk, q=heads(5, 512, 68)) == INVALID       # strides of 16 bytes
    assert rotate(tk, q=heads(5, 0)) == INVALID
    assert rotate(tk, q=heads(5, first=8)) == INVALID       # addresses too
    assert rotate(tk, q=heads(5, n=3)) == INVALID           # as many heads out as in
    assert rotate(tk, q=heads(5, 2 ** 34)) == UNSUPPORTED
    assert rotate(tk, tokens=2 ** 20, q=heads(5, 2 ** 33)) == INVALID
    assert rotate(tk, tokens=0) == 0


def test_rotate_overlaps(tk):  # noqa: F811
    assert rotate(tk, q_out=heads(7, 512, 32)) == INVALID            # heads over one another
    assert rotate(tk, q_out=heads(7, 128, 64)) == INVALID            # tokens over one another
    assert rotate(tk, q_out=heads(5, first=1024)) == INVALID         # a token behind its input
    assert rotate(tk, q_out=heads(5, first=128)) == INVALID          # a head behind it
    assert rotate(tk, k_out=heads(7)) == INVALID                     # both outputs in one place
    assert rotate(tk, k_out=heads(5)) == INVALID                     # over the other's input
    assert rotate(tk, q_out=heads(5, 512, 128)) == INVALID           # its own place with other strides


def test_append_refusals(tk):  # noqa: F811
    assert append(tk, c=cache(tk, dim=62)) == UNSUPPORTED
    assert append(tk, tokens=3) == INVALID
    assert append(tk, k=None) == INVALID
    assert append(tk, v=None) == INVALID
    assert append(tk, k=heads(5, 128, 64, 3)) == INVALID
    assert append(tk, pos=rows(tk, 8)) == INVALID                    # positions need next_pos
    assert append(tk, next_pos=addr(9) + 1) == INVALID
    assert append(tk, weight=rows(tk, 7, slots=79, head=79, seq=158)) == INVALID
    assert append(tk, q=heads(10)) == INVALID
    assert append(tk, q=heads(10), q_out=heads(10, n=2)) == INVALID
    assert append(tk, q=heads(10), q_out=heads(5)) == INVALID        # over k_new
    assert append(tk, q=heads(10), q_out=heads(6, 1024, 64, 4)) == INVALID
    assert append(tk, tokens=0, starts=addr(11)) == 0


def test_sample_refusals(tk):  # noqa: F811
    for kw in (dict(logits=None), dict(u=None), dict(token=None), dict(logp=None), dict(rows=0), dict(cols=0),
               dict(stride=999), dict(dtype=3), dict(dtype=-1), dict(logits=addr(1) + 2), dict(u=addr(2) + 1),
               dict(token=addr(3) + 2), dict(logp=addr(4) + 3)):
        assert sample(tk, **kw) == INVALID, kw
    nan = float("nan")
    for s in (Sampling(-1.0, None, 0, None, 1.0, None, 0.0, None), Sampling(nan, None, 0, None, 1.0, None, 0.0, None),
              Sampling(1.0, None, 0, None, nan, None, 0.0, None), Sampling(1.0, None, 0, None, 1.0, None, nan, None),
              Sampling(1.0, addr(5) + 2, 0, None, 1.0, None, 0.0, None),
              Sampling(1.0, None, 0, addr(5) + 1, 1.0, None, 0.0, None)):
        assert sample(tk, s=s) == INVALID
    assert sample(tk, cols=2 ** 21 + 1, stride=2 ** 22) == UNSUPPORTED
    assert sample(tk, stride=2 ** 39) == UNSUPPORTED


def test_python_checks_without_a_gpu(tk):  # noqa: F811
    import torch

    half = torch.zeros(2, 4, 64, dtype=torch.float16)
    pos, freq = torch.zeros(2, dtype=torch.int32), torch.zeros(32)
    with pytest.raises(ValueError, match="CUDA"):
        tk.kv_rotate(half, None, pos, freq)
    with pytest.raises(ValueError, match="absent"):
        tk.kv_rotate(None, None, pos, freq)
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        tk.kv_rotate(half.float(), None, pos, freq)
    with pytest.raises(ValueError, match="CUDA"):
        tk.sample_rows(torch.zeros(2, 8), torch.zeros(2))
    with pytest.raises(TypeError, match="logits must be"):
        tk.sample_rows(torch.zeros(2, 8, dtype=torch.float64), torch.zeros(2))
    with pytest.raises(TypeError, match="k_pages"):
        tk.kv_append_rotated(None, None, None, None, half, half, freq)
