"""A paged cache on the CPU and the key-value cache operators' definitions in
64 bits, for tests.  Nothing here is shared with the CUDA path."""
import numpy as np
import torch

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # half an ulp, relative, of a rounded output


class Cache:
    """Pools in which every slot that no sequence holds is NaN, and a table
    whose entries past a sequence's slots name no page."""

    def __init__(self, lens, heads, dim, page, dtype, layout="head", room=0, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.heads, self.dim, self.page, self.dtype = list(lens), heads, dim, page, dtype
        n = len(lens)
        width = max(1, max(-(-(x + room) // page) for x in lens))
        used = [-(-(x + room) // page) for x in lens]
        pages = sum(used) + 3
        order = torch.randperm(pages, generator=g).tolist()
        self.table = torch.full((n, width), 2 ** 30, dtype=torch.int32)
        for b in range(n):
            for i in range(used[b]):
                self.table[b, i] = order.pop()
        shape = (pages, heads, page, dim) if layout == "head" else (pages, page, heads, dim)
        self.k, self.v = (torch.full(shape, float("nan"), dtype=dtype) for _ in range(2))
        if layout == "head":
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        for b in range(n):
            for s0 in range(0, lens[b], page):
                c = min(page, lens[b] - s0)
                for p in (self.k, self.v):
                    p[self.table[b, s0 // page], :c] = torch.randn(c, heads, dim, generator=g).to(dtype)
        self.capacity = width * page
        self.device = device

    def rows(self, b, pool):
        """Sequence b's slots of a pool (its own k or v, or a copy), [slots, heads, dim]."""
        n = self.lens[b]
        return pool[self.table[b, :-(-n // self.page)].long()].reshape(-1, self.heads, self.dim)[:n]

    def dev(self):
        """(k, v, table, lens) on the device, with the pools' strides kept."""
        def put(t):
            if t.is_contiguous():
                return t.to(self.device)
            return t.transpose(1, 2).to(self.device).transpose(1, 2)
        return (put(self.k), put(self.v), self.table.to(self.device),
                torch.tensor(self.lens, dtype=torch.int32, device=self.device))


def attend(cache, q, scale, weight=None):
    """(out, lse, weight) of the definition in float64, with the bounds on
    each that float32 arithmetic of 16-bit inputs keeps.

    A score's float32 sum of dim products is within dim * 2^-24 of
    scale * sum |q_i k_i|, times 2 for the rounding of products, scale and
    exponent: d.  A share then has the relative error 2d + 2^-20 (its own and
    its sum's exponentials, at most 4 ulp each) + n * 2^-24 (the sum), and is
    carried into the product with the values to 2^-15, and with 2^-30 of the
    largest where it is smaller.  An output is rounded to its type once."""
    seqs, q_heads, dim = q.shape
    group = q_heads // cache.heads
    out = np.zeros((seqs, q_heads, dim))
    lse = np.full((seqs, q_heads), -np.inf)
    out_tol, lse_tol = np.zeros_like(out), np.zeros_like(lse)
    w_out = None if weight is None else weight.double().numpy().copy()
    w_tol = None if weight is None else np.zeros_like(w_out)
    for b in range(seqs):
        n = cache.lens[b]
        if n == 0:
            continue
        k, v = (cache.rows(b, p).double().numpy() for p in (cache.k, cache.v))
        for j in range(q_heads):
            h = j // group
            qq = q[b, j].double().numpy()
            with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
                s = scale * (k[:, h] @ qq)
                d = 2 * dim * 2.0 ** -24 * abs(scale) * (np.abs(k[:, h]) @ np.abs(qq)).max()
                if np.all(s == -np.inf):
                    continue
                top = s.max()
                e = np.exp(s - top)
                total = e.sum()
                p = e / total
                out[b, j] = p @ v[:, h]
                lse[b, j] = top + np.log(total)
                rel = 2 * d + 2.0 ** -20 + n * 2.0 ** -24
                out_tol[b, j] = UNIT[cache.dtype] * np.abs(out[b, j]) + 2.0 ** -25 + \
                    (rel + 2.0 ** -15 + n * 2.0 ** -30) * (p @ np.abs(v[:, h])) + \
                    n * 2.0 ** -30 * np.abs(v[:, h]).max(0)
                lse_tol[b, j] = rel + 2.0 ** -22 * abs(lse[b, j])
                if w_out is not None:
                    w_out[b, h, :n] += p
                    w_tol[b, h, :n] += p * rel + 2.0 ** -23 * np.abs(w_out[b, h, :n])
    return out, lse, w_out, out_tol, lse_tol, w_tol


def close(got, want, tol):
    """Equal where `want` is not finite, within tol elsewhere."""
    got = got.double().cpu().numpy()
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
    off = np.abs(got[fine] - want[fine]) - (tol[fine] if isinstance(tol, np.ndarray) else tol)
    assert off.size == 0 or off.max() <= 0, f"off by {off.max():.3g} more than the bound"


def evict_sources(weight, pos, n, next_pos, budget, sink, recent):
    """For each slot below min(n, budget), the slot whose token it holds
    afterwards: one row's definition, by a full sort."""
    if n <= budget:
        return np.arange(n)
    w = weight[:n].astype(np.float64)
    p = pos[:n].astype(np.int64)
    safe = (p < sink) | (p >= int(next_pos) - recent)
    nan = np.isnan(w)
    w = np.where(nan, 0.0, w)  # -0.0 sorts as 0.0: np.lexsort compares numbers
    key = np.where(nan, 1, 0)
    kept = np.lexsort((np.arange(n), -w, -key, ~safe))
    # protected slots are equal among each other
    guarded = np.flatnonzero(safe)
    others = kept[~safe[kept]]
    kept = np.concatenate([guarded, others])[:budget]
    source = np.arange(budget)
    holes = np.setdiff1d(source, kept)
    source[holes] = np.sort(kept[kept >= budget])
    return source
