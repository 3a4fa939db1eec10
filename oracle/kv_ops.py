"""Float64 definitions of the full-attention operators of include/gdn_kv.h (numpy, one
request and head at a time).  Test infrastructure only; shares no code with the library.

Caches are given as values (float64 arrays of what the stored elements stand for, before
k_scale / v_scale), tables as integer arrays.
"""
from __future__ import annotations

import numpy as np

F8_MAX = 448.0


def e4m3_values() -> np.ndarray:
    """The 256 values of OCP e4m3 by their bits (0x7f and 0xff are NaN)."""
    b = np.arange(256)
    sign = np.where(b & 0x80, -1.0, 1.0)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[(b & 0x7f) == 0x7f] = np.nan
    return sign * v


def e4m3_round(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value, ties to the even mantissa, limited to +-448; NaN stays."""
    grid = e4m3_values()[:0x7f]  # non-negative and increasing; the index's parity is the mantissa's
    a = np.minimum(np.abs(np.asarray(x, np.float64)), F8_MAX)
    nan = np.isnan(a)
    a = np.where(nan, 0.0, a)
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    pick = np.where(dl < dh, lo, np.where(dl > dh, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.where(nan, np.nan, np.copysign(grid[pick], x))


def places(table, slot, page_size, pages, lo, hi):
    """(page, row, valid) of token places lo .. hi-1 of a slot."""
    i = np.arange(lo, hi)
    page = table[slot, i // page_size]
    return page, i % page_size, (page > 0) & (page < pages)


def attend(k, v, table, slot, begin, length, q, scale, k_scale=1.0, v_scale=1.0):
    """One request of one layer: k, v [pages, H, page_size, D], q [Hq, D].  Returns
    (out [Hq, D], lse [Hq], weights [H, length - begin], bound), where ``bound`` holds,
    per query head, sum p |v| [Hq, D] and the largest scale * sum |q k| [Hq]."""
    P, H, S, D = k.shape
    Hq = q.shape[0]
    G = Hq // H
    n = max(0, length - begin)
    out, lse = np.zeros((Hq, D)), np.full(Hq, -np.inf)
    weights, spread, size = np.zeros((H, n)), np.zeros((Hq, D)), np.zeros(Hq)
    if n == 0:
        return out, lse, weights, (spread, size)
    page, row, ok = places(table, slot, S, P, begin, length)
    page = np.where(ok, page, 0)
    for h in range(H):
        kk = np.where(ok[:, None], k[page, h, row], 0.0) * k_scale
        vv = np.where(ok[:, None], v[page, h, row], 0.0) * v_scale
        for j in range(h * G, (h + 1) * G):
            s = np.where(ok, scale * (kk @ q[j]), -np.inf)
            top = s.max()
            if top == -np.inf:
                continue
            p = np.exp(s - top)
            total = p.sum()
            p /= total
            out[j] = p @ vv
            lse[j] = top + np.log(total)
            weights[h] += p
            spread[j] = p @ np.abs(vv)
            size[j] = abs(scale) * (np.abs(kk) @ np.abs(q[j])).max()
    return out, lse, weights, (spread, size)


def plan(mass, pos, n, next_pos, budget, sink, recent):
    """Moves (list of (source, destination)) of one cache of n tokens; mass, pos [>= n]."""
    if n <= budget:
        return []

    def rank(i):
        if pos[i] < sink or pos[i] >= next_pos - recent:
            return -1, 0.0, i
        return 0, -(float(mass[i]) if mass[i] > 0 else 0.0), i

    order = sorted(range(n), key=rank)
    keep = set(order[:budget])
    freed = [i for i in range(budget) if i not in keep]
    moved = [i for i in range(budget, n) if i in keep]
    assert len(freed) == len(moved)
    return list(zip(moved, freed))


def rms(x, eps):
    return x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)


def block_norm(y, w_post=None, gate=None, act="none", scale=1.0, residual=None, w_pre=None, eps=1e-6,
               plus_one=False):
    """(out, residual_out) in float64; residual_out is None without a residual."""
    one = 1.0 if plus_one else 0.0
    u = np.asarray(y, np.float64)
    if w_post is not None:
        u = rms(u, eps) * (one + w_post)
    if gate is not None:
        z = np.asarray(gate, np.float64)
        with np.errstate(over="ignore"):
            sg = 1.0 / (1.0 + np.exp(-z))
        u = u * {"none": z, "silu": z * sg, "sigmoid": sg}[act]
    u = scale * u
    r = u if residual is None else residual + u
    return (rms(r, eps) * (one + w_pre) if w_pre is not None else r), (None if residual is None else r)
