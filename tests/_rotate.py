"""The norm and rotation of heads, and the sampling of rows, in 64 bits, for
tests.  Nothing here is shared with the CUDA path."""
import numpy as np
import torch

UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # half an ulp, relative, of a rounded output


def rotate(x, pos, freq, norm=None, eps=1e-6, pairing="halves"):
    """(result, bound) of [tokens, heads, dim] in float64.

    A norm's factor is off by the sum's dim * 2^-24 (halved by the root), its
    root's 2^-22 and three roundings; a cosine or sine by 2^-22 (2^-32 of a
    turn, 2^-28 of the series, roundings of its argument and terms); products
    and the sum by 2^-23.  The result is rounded to its type once."""
    y = x.double().cpu().numpy().copy()
    dim = y.shape[-1]
    rel = 2.0 ** -21
    if norm is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + np.float64(np.float32(eps))) * norm.double().cpu().numpy()
        rel += dim * 2.0 ** -25 + 2.0 ** -21
    f = freq.double().cpu().numpy()
    half = f.size
    angle = np.asarray(pos, dtype=np.longdouble)[:, None] * f.astype(np.longdouble)
    c, s = (fn(angle).astype(np.float64)[:, None, :] for fn in (np.cos, np.sin))
    at = (np.arange(half), np.arange(half) + half) if pairing == "halves" else (np.arange(half) * 2, np.arange(half) * 2 + 1)
    a, b = y[..., at[0]].copy(), y[..., at[1]].copy()
    tol = np.abs(y) * rel
    y[..., at[0]] = a * c - b * s
    y[..., at[1]] = b * c + a * s
    tol[..., at[0]] = tol[..., at[1]] = (np.abs(a) + np.abs(b)) * (rel + 2.0 ** -22)
    return y, tol + UNIT[x.dtype] * np.abs(y) + 2.0 ** -25


def close(got, want, tol):
    got = got.double().cpu().numpy()
    off = np.abs(got - want) - tol
    assert off.size == 0 or off.max() <= 0, f"off by {off.max():.3g} more than the bound"


def order(x):
    """Columns of a row in TopK order."""
    x = x.double().cpu().numpy()
    return np.lexsort((np.arange(x.size), -(x + 0.0)))


def sample(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logp, distance of u from the nearest border that decided) of one
    row: the definition by a full sort.  Parameters are float32 numbers."""
    x = x.double().cpu().numpy()
    u, temperature, top_p, min_p = (float(np.float32(v)) for v in (u, temperature, top_p, min_p))
    n = x.size
    best = np.lexsort((np.arange(n), -(x + 0.0)))
    x = x[best]
    if np.isnan(x).any() or np.isinf(x[0]) or np.isnan([u, temperature, top_p, min_p]).any() or temperature < 0:
        return -1, np.nan, 1.0
    if temperature == 0:
        return int(best[0]), 0.0, 1.0
    z = (x - x[0]) / min(max(temperature, 2.0 ** -60), 2.0 ** 60)
    w = np.exp(z)
    run = np.cumsum(w)
    near = 1.0
    keep = last = top_k if 0 < top_k < n else n
    if top_p < 1:
        t = top_p * run[last - 1]
        i = int(np.searchsorted(run[:last], t, "left"))
        # A border that u falls on exactly decides as well as any other.
        near = min(abs(run[i] - t) or 9.0, abs(run[i] - w[i] - t) or 9.0) / run[last - 1] if i else 1.0
        keep = min(keep, i + 1)
    if min_p > 0:
        keep = min(keep, max(1, int((z >= np.log(min(min_p, 1.0))).sum())))
    t = min(max(u, 0.0), 1 - 2.0 ** -24) * run[keep - 1]
    i = min(int(np.searchsorted(run[:keep], t, "right")), keep - 1)
    near = min(near, (abs(run[i] - t) or 9.0) / run[keep - 1], (abs(run[i] - w[i] - t) or 9.0) / run[keep - 1])
    return int(best[i]), z[i] - np.log(run[keep - 1]), near
