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


def attend_chunk(k, v, table, slot, begin, length, q, scale, window=0, late=0, k_scale=1.0, v_scale=1.0):
    """A chunk of one request of one layer: the n queries q [n, Hq, D] stand at the last n of
    `length` places, each seeing the places up to its own, from `begin` on and, with a window, the
    last `window` of them.  Returns (out [n, Hq, D], lse [n, Hq], weights [H, length] of the last
    `late` queries, (sum p |v| [n, Hq, D], largest scale * sum |q k| [n, Hq]))."""
    P, H, S, D = k.shape
    n, Hq = q.shape[:2]
    G = Hq // H
    out, lse = np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf)
    weights, spread, size = np.zeros((H, length)), np.zeros((n, Hq, D)), np.zeros((n, Hq))
    page, row, ok = places(table, slot, S, P, 0, length)
    page = np.where(ok, page, 0)
    t = np.arange(length)
    at = np.arange(length - n, length)[:, None]
    seen = ok & (t <= at) & (t >= begin)
    if window:
        seen &= t > at - window
    any_seen = (seen.any(axis=0))[:, None]
    for h in range(H):
        kk = np.where(any_seen, k[page, h, row], 0.0) * k_scale
        vv = np.where(any_seen, v[page, h, row], 0.0) * v_scale
        for j in range(h * G, (h + 1) * G):
            s = np.where(seen, scale * (q[:, j] @ kk.T), -np.inf)
            top = s.max(axis=1)
            live = top > -np.inf
            p = np.exp(s - np.where(live, top, 0.0)[:, None])
            total = p.sum(axis=1)
            p /= np.where(live, total, 1.0)[:, None]
            out[:, j] = p @ vv
            lse[live, j] = top[live] + np.log(total[live])
            weights[h] += p[n - min(n, late):].sum(axis=0)
            spread[:, j] = p @ np.abs(vv)
            size[:, j] = np.where(seen, abs(scale) * (np.abs(q[:, j]) @ np.abs(kk).T), 0.0).max(axis=1)
    return out, lse, weights, (spread, size)


def turn(x, position, freqs, amplitude, adjacent):
    """Heads x [n, H, D] turned by position [n] (float64); the first 2 len(freqs) values of each."""
    rot = 2 * len(freqs)
    a = np.asarray(position, np.float64)[:, None, None] * np.asarray(freqs)
    c, s = amplitude * np.cos(a), amplitude * np.sin(a)
    y = np.array(x, np.float64)
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if adjacent else (slice(0, rot // 2), slice(rot // 2, rot))
    u, w = x[..., i], x[..., j]
    y[..., i], y[..., j] = u * c - w * s, w * c + u * s
    return y


def batch_map(table, slots, lens, new, pos, free, n_free, page_size, max_tokens):
    """kv_batch_map for lists; table (a copy is changed) and free as lists.  Returns a dict of the
    outputs and the error bits' names."""
    table = [list(r) for r in table]
    cap = len(table[0]) * page_size
    B = len(slots)
    out = dict(cu=[0], slot=[], len=[], pos=[], token_slot=[0] * max_tokens, token_index=[0] * max_tokens,
               token_pos=[0] * max_tokens, errors=set())
    if n_free != max(0, min(n_free, len(free))):
        out["errors"].add("lens")
    left = n_free = max(0, min(n_free, len(free)))
    total = lacked = 0
    for b in range(B):
        s, n, L, p = slots[b], new[b], lens[b], pos[b]
        first = total
        total += max(n, 0)
        live = 0 < s < len(table)
        if s >= len(table):
            out["errors"].add("slot")
        valid = live and n >= 0 and L >= 0 and L + n <= cap and total <= max_tokens and p + n < 2 ** 31
        served = valid
        if valid:
            need = -(-(L + n) // page_size) - -(-L // page_size)
            lacked += need
            served = need == 0 or lacked <= n_free
            if not served:
                out["errors"].add("pages")
        elif live:
            out["errors"].add("lens")
        if served:
            for e in range(-(-L // page_size), -(-(L + n) // page_size)):
                left -= 1
                table[s][e] = free[left]
            for i in range(n):
                out["token_slot"][first + i] = s
                out["token_index"][first + i] = L + i
                out["token_pos"][first + i] = p + i
        out["cu"].append(min(total, max_tokens))
        out["slot"].append(s if served else 0)
        out["len"].append(L + n if served else L)
        out["pos"].append(p + n if served else p)
    return dict(out, table=table, n_free=left)


def release(table, slots, lens, keep, free, n_free, page_size, pages):
    """kv_release for lists: (table, free, n_free, error names)."""
    table, free, errors = [list(r) for r in table], list(free), set()
    cap = len(table[0]) * page_size
    if n_free != max(0, min(n_free, len(free))):
        errors.add("lens")
    n_free = max(0, min(n_free, len(free)))
    for b, s in enumerate(slots):
        if s >= len(table):
            errors.add("slot")
        if not 0 < s < len(table):
            continue
        if lens[b] < 0 or lens[b] > cap or keep[b] < 0:
            errors.add("lens")
            continue
        for e in range(-(-keep[b] // page_size), -(-lens[b] // page_size)):
            if not 0 < table[s][e] < pages or n_free >= len(free):
                errors.add("page")
                continue
            free[n_free] = table[s][e]
            table[s][e] = 0
            n_free += 1
    return table, free, n_free, errors
