"""Argument checks of the key-value cache operators: made on the host before
any CUDA call, so these run without a GPU (the addresses are never used)."""
import ctypes

import pytest
import torch

A = 0x10000000


@pytest.fixture(scope="module")
def tk():
    import __graft_entry__

    __graft_entry__._load_build_module().build()
    import topk_selection_gb300

    return topk_selection_gb300


def addr(i):
    return A + i * 0x10000000


def cache(tk, **kw):
    d = dict(k=addr(1), v=addr(2), dtype=1, pages=10, page_size=16, heads=2, dim=64, table=addr(3), table_stride=5,
             table_width=5, seqs=2, lens=addr(4), k_stride=(2048, 64, 1024), v_stride=(2048, 64, 1024))
    d.update(kw)
    c = tk._KvCache()
    for name, value in d.items():
        setattr(c, name, (ctypes.c_int64 * 3)(*value) if "k_stride" == name or "v_stride" == name else value)
    return ctypes.byref(c)


def rows(tk, i, slots=80, head=80, seq=160):
    return ctypes.byref(tk._KvRows(addr(i), seq, head, slots))


def strides(*s):
    return (ctypes.c_int64 * len(s))(*s)


def append(tk, c=None, k_new=addr(5), ks=(128, 64), v_new=addr(6), vs=(128, 64), tokens=2, starts=None, weight=None,
           pos=None, next_pos=None):
    return tk._lib.topk_kv_append(c or cache(tk), k_new, strides(*ks), v_new, strides(*vs), tokens, starts, weight,
                                  pos, next_pos, None)


def attend(tk, c=None, q=addr(5), qs=(256, 64), q_heads=4, scale=0.125, out=addr(6), lse=addr(7), weight=None,
           weight_out=None):
    return tk._lib.topk_kv_attend(c or cache(tk), q, strides(*qs), q_heads, scale, out, lse, weight, weight_out, None)


def evict(tk, c=None, weight="w", pos="p", next_pos=addr(9), budget=32, sink=1, recent=3, weight_out="o",
          pos_out="q", lens_out=addr(12)):
    pick = {"w": rows(tk, 7), "p": rows(tk, 8), "o": rows(tk, 10, 32, 32, 64), "q": rows(tk, 11, 32, 32, 64)}
    return tk._lib.topk_kv_evict(c or cache(tk), pick.get(weight, weight), pick.get(pos, pos), next_pos, budget, sink,
                                 recent, pick.get(weight_out, weight_out), pick.get(pos_out, pos_out), lens_out, None)


BAD_CACHES = [
    (dict(k=None), 1), (dict(v=None), 1), (dict(table=None), 1), (dict(lens=None), 1),
    (dict(dtype=2), 1), (dict(dtype=-1), 1), (dict(pages=0), 1), (dict(page_size=0), 1), (dict(heads=0), 1),
    (dict(dim=0), 1), (dict(table_width=0), 1), (dict(seqs=0), 1), (dict(table_stride=4), 1),
    (dict(k=addr(1) + 8), 1), (dict(v=addr(2) + 2), 1), (dict(table=addr(3) + 2), 1), (dict(lens=addr(4) + 1), 1),
    (dict(k_stride=(2048, 60, 1024)), 1), (dict(v_stride=(2048, 64, 0)), 1), (dict(k_stride=(-2048, 64, 1024)), 1),
    (dict(page_size=12), 2), (dict(page_size=65544), 2), (dict(dim=60), 2), (dict(dim=264), 2),
    (dict(table_width=1 << 26, table_stride=1 << 26), 2), (dict(seqs=65536), 2), (dict(heads=4097), 2),
]


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_cache_errors(tk, change, status):
    for call in (append, attend, evict):
        assert call(tk, cache(tk, **change)) == status


def test_append_errors(tk):
    assert append(tk, k_new=None) == 1
    assert append(tk, v_new=None) == 1
    assert append(tk, k_new=addr(5) + 8) == 1
    assert append(tk, ks=(128, 60)) == 1
    assert append(tk, vs=(0, 64)) == 1
    assert append(tk, tokens=-1) == 1
    assert append(tk, tokens=3) == 1                               # one token each, but there are two sequences
    assert append(tk, tokens=3, starts=addr(7) + 2) == 1
    assert append(tk, pos=rows(tk, 8)) == 1                        # positions without next_pos
    assert append(tk, next_pos=addr(9)) == 1
    assert append(tk, weight=rows(tk, 8, slots=79)) == 1           # fewer slots than the capacity
    assert append(tk, weight=rows(tk, 8, head=40)) == 1            # rows inside one another
    assert append(tk, pos=rows(tk, 8, seq=40), next_pos=addr(9)) == 1
    assert append(tk, tokens=0, starts=addr(7)) == 0               # nothing to do


def test_attend_errors(tk):
    assert attend(tk, q=None) == 1
    assert attend(tk, q=addr(5) + 4) == 1
    assert attend(tk, qs=(256, 63)) == 1
    assert attend(tk, q_heads=0) == 1
    assert attend(tk, q_heads=3) == 1
    assert attend(tk, scale=float("nan")) == 1
    assert attend(tk, scale=float("inf")) == 1
    assert attend(tk, out=None) == 1
    assert attend(tk, out=addr(6) + 8) == 1
    assert attend(tk, lse=addr(7) + 2) == 1
    assert attend(tk, weight=rows(tk, 8)) == 1                     # no place for the sums
    assert attend(tk, weight_out=rows(tk, 8)) == 1
    assert attend(tk, weight=rows(tk, 8), weight_out=rows(tk, 9, slots=79)) == 1
    near = ctypes.byref(tk._KvRows(addr(8) + 64, 160, 80, 80))
    assert attend(tk, weight=rows(tk, 8), weight_out=near) == 1    # overlapping, and not the same
    assert attend(tk, c=cache(tk, seqs=60000), q_heads=400) == 2
    assert attend(tk, c=cache(tk, seqs=1000, table_width=1 << 20, table_stride=1 << 20), q_heads=64) == 2  # tiles


def test_evict_errors(tk):
    for name in ("weight", "pos", "next_pos", "weight_out", "pos_out", "lens_out"):
        assert evict(tk, **{name: None}) == 1
    assert evict(tk, budget=0) == 1
    assert evict(tk, sink=-1) == 1
    assert evict(tk, recent=-1) == 1
    assert evict(tk, sink=16, recent=17) == 1                      # more protected than kept
    assert evict(tk, sink=2 ** 31 - 1, recent=2 ** 31 - 1) == 1
    assert evict(tk, next_pos=addr(9) + 1) == 1
    assert evict(tk, weight=rows(tk, 7, slots=79)) == 1
    assert evict(tk, budget=33) == 1                               # the outputs have room for 32
    assert evict(tk, weight_out=ctypes.byref(tk._KvRows(addr(7) + 64, 64, 32, 32))) == 1
    assert evict(tk, lens_out=addr(4) + 4) == 1


def test_binding_refusals(tk):
    half = torch.zeros(4, 16, 2, 64, dtype=torch.float16)
    table, lens = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        tk.kv_attend(half[:2], half.float(), half.float(), table, lens)
    with pytest.raises(ValueError):  # the pools are device memory
        tk.kv_attend(half[:2, 0], half, half, table, lens)
    with pytest.raises(ValueError):
        tk.kv_append(half, half, table, lens, half[:2, 0], half[:2, 0])
    with pytest.raises(ValueError):
        w = torch.zeros(2, 2, 32)
        tk.kv_evict(half, half, table, lens, w, w.int(), lens, 8)


def test_header_limit_matches_binding(tk):
    import os
    import re

    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "topk.h")).read()
    assert re.search(r"#define TOPK_KV_MAX_DIM\s+%d\b" % tk.KV_MAX_DIM, text)
