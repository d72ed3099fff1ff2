"""A decoder's attention over a bounded key-value cache.

Prompts go into a paged cache; every step appends one token per sequence,
attends to what the cache holds while adding up how much attention each slot
got, and whenever the sequences reach `--limit` slots keeps the `--budget`
most attended ones (and the first and newest tokens).  The queries, keys and
values are random: what a model would compute around these calls is left out.

    python examples/kv_decode.py --seqs 16 --prompt 3000 --steps 2000
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import topk_selection_gb300 as tk  # noqa: E402


class BoundedCache:
    """One layer's cache: pages for `limit` slots of every sequence, all allocated up front."""

    def __init__(self, seqs, heads, dim, limit, budget, sink, recent, page=16, dtype=torch.bfloat16):
        width = -(-limit // page)
        pool = torch.zeros(2, seqs * width, heads, page, dim, dtype=dtype, device="cuda")
        self.k, self.v = pool[0].transpose(1, 2), pool[1].transpose(1, 2)  # [pages, page, heads, dim]
        self.table = torch.arange(seqs * width, dtype=torch.int32, device="cuda").reshape(seqs, width)
        self.lens, self.seen = (torch.zeros(seqs, dtype=torch.int32, device="cuda") for _ in range(2))
        self.weight = torch.zeros(seqs, heads, width * page, device="cuda")
        self.pos = torch.zeros(seqs, heads, width * page, dtype=torch.int32, device="cuda")
        self.limit, self.budget, self.sink, self.recent = limit, budget, sink, recent
        self.held = 0  # the longest sequence's slots, known without asking the GPU

    def append(self, k, v, counts=None):
        """counts: tokens of each sequence, or None for one each."""
        add = torch.ones_like(self.lens) if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
        longest = 1 if counts is None else max(counts)
        if self.held + longest > self.limit:
            tk.kv_evict(self.k, self.v, self.table, self.lens, self.weight, self.pos, self.seen, self.budget,
                        sink=self.sink, recent=self.recent)
            self.held = min(self.held, self.budget)
        if self.held + longest > self.limit:
            raise ValueError("more new tokens than the cache has room for")
        starts = None
        if counts is not None:
            starts = torch.zeros(len(counts) + 1, dtype=torch.int32, device="cuda")
            starts[1:] = torch.cumsum(add, 0)
        tk.kv_append(self.k, self.v, self.table, self.lens, k, v, starts=starts, weight=self.weight, pos=self.pos,
                     next_pos=self.seen)
        self.lens += add
        self.seen += add
        self.held += longest

    def attend(self, q):
        return tk.kv_attend(q, self.k, self.v, self.table, self.lens, weight=self.weight)[0]


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("seqs", 16), ("q-heads", 32), ("heads", 8), ("dim", 128), ("prompt", 3000), ("steps", 2000),
                        ("limit", 4096), ("budget", 2048), ("sink", 4), ("recent", 256)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args(argv)
    torch.manual_seed(0)
    cache = BoundedCache(a.seqs, a.heads, a.dim, a.limit, a.budget, a.sink, a.recent)

    def rand(*shape):
        return torch.randn(*shape, device="cuda").to(torch.bfloat16)

    counts = [max(1, a.prompt - 17 * b) for b in range(a.seqs)]
    cache.append(rand(sum(counts), a.heads, a.dim), rand(sum(counts), a.heads, a.dim), counts)
    new = [rand(a.seqs, a.heads, a.dim) for _ in range(2)]
    q = 2 * rand(a.seqs, a.q_heads, a.dim)
    for _ in range(3):
        cache.append(*new)
        out = cache.attend(q)
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(a.steps):
        cache.append(*new)
        out = cache.attend(q)
    torch.cuda.synchronize()
    took = time.perf_counter() - start
    tk.check_stream()
    assert torch.isfinite(out).all()
    print(f"{a.steps} steps of {a.seqs} sequences: {took / a.steps * 1e6:.1f} us a step and layer, at most "
          f"{int(cache.lens.max())} of {int(cache.seen.max())} tokens held, "
          f"{a.seqs * a.steps / took:.0f} tokens/s and layer")


if __name__ == "__main__":
    main()
