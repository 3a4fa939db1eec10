"""Inputs of the full-attention operators' tests, and their tolerances.

Caches are filled with NaN wherever no visible token lies (unused pages, the rest of a last
page, places before the first visible token), so a value read from there shows.
"""
from __future__ import annotations

from types import SimpleNamespace

import numpy as np
import torch

from oracle import kv_ops


def stored(x: torch.Tensor, f8: bool) -> torch.Tensor:
    return x.clamp(-448, 448).to(torch.float8_e4m3fn) if f8 else x.to(torch.bfloat16)


def make_cache(seed, lens, begins=None, kv_heads=2, dim=64, page=16, f8=False, layers=1, layer=0, extra_pages=3,
               slots=None, k_std=1.0, capacity=None):
    """A cache whose requests b = 0.. use slots[b] (default: a permutation of 1..B)."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    begins = begins or [0] * B
    slots = list(slots) if slots is not None else (torch.randperm(B, generator=g) + 1).tolist()
    n_slots = max([2] + [s + 1 for s in slots])
    max_pages = -(-max(max(lens + [1]), capacity or 0) // page)
    need = [-(-n // page) for n in lens]
    pages = 1 + sum(need) + extra_pages
    ids = (torch.randperm(pages - 1, generator=g) + 1).tolist()
    table = torch.zeros(n_slots, max_pages, dtype=torch.int32)
    shape = (layers, pages, kv_heads, page, dim)
    k = torch.full(shape, float("nan"))
    v = torch.full(shape, float("nan"))
    at = 0
    for b in range(B):
        if slots[b] <= 0 or slots[b] >= n_slots:
            continue
        mine = ids[at:at + need[b]]
        at += need[b]
        table[slots[b], :need[b]] = torch.tensor(mine, dtype=torch.int32)
        for i in range(begins[b], lens[b]):
            k[layer, mine[i // page], :, i % page] = k_std * torch.randn(kv_heads, dim, generator=g)
            v[layer, mine[i // page], :, i % page] = torch.randn(kv_heads, dim, generator=g) + 0.5
    k, v = stored(k, f8), stored(v, f8)
    cap = max_pages * page
    mass = torch.rand(layers, n_slots, kv_heads, cap, generator=g)
    pos = torch.arange(cap, dtype=torch.int32).expand(layers, n_slots, kv_heads, cap).contiguous()
    return SimpleNamespace(k=k, v=v, table=table, mass=mass, pos=pos, slots=slots, lens=lens, begins=begins,
                           kv_heads=kv_heads, dim=dim, page=page, f8=f8, layer=layer, cap=cap, n_slots=n_slots,
                           k_scale=0.5 if f8 else 1.0, v_scale=1.75 if f8 else 1.0, g=g)


def device_pool(c, mass=True, err=True):
    import gated_delta_rule_slot_amd as gdn

    e = torch.zeros(1, dtype=torch.int32, device="cuda") if err else None
    return gdn.kv_pool_create(c.k.cuda(), c.v.cuda(), c.table.cuda(), mass=c.mass.cuda() if mass else None,
                              pos=c.pos.cuda() if mass else None, err_word=e, k_scale=c.k_scale,
                              v_scale=c.v_scale)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def attend_all(c, q, scale):
    """oracle results of every request: (out, lse, [weights], spread, size)"""
    k, v = (t[c.layer].float().double().numpy() for t in (c.k, c.v))
    table = c.table.numpy()
    qd = q.float().double().numpy()
    B, Hq, D = qd.shape
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    spread, size, weights = np.zeros((B, Hq, D)), np.zeros((B, Hq)), []
    for b in range(B):
        live = 0 < c.slots[b] < c.n_slots
        o = kv_ops.attend(k, v, table, c.slots[b] if live else 0, c.begins[b], c.lens[b] if live else 0, qd[b],
                          scale, c.k_scale, c.v_scale)
        out[b], lse[b] = o[0], o[1]
        weights.append(o[2])
        spread[b], size[b] = o[3]
    return out, lse, weights, spread, size


def attn_slack(size, dim, n):
    """Relative error of a softmax weight, and of a sum of them, before the output's own
    rounding.

    A score is a sum of `dim` exact products of bf16 values accumulated in fp32: at most
    dim roundings (each up to one unit, 2^-23, as the matrix unit may truncate) of partial sums
    bounded by `size` = scale * sum |q k|; two more for the factor scale * log2(e) and the
    difference to the maximum, and the same again in the denominator: 2 (dim + 8) 2^-23 size.
    A weight is carried as two bf16 parts: 2^-8 of 2^-8, and 2^exp costs 2 units: 2^-15 in
    all.  Sums of n weights run over tiles of 32 (each one rounding), then over waves,
    lanes and splits: (n / 32 + 64) 2^-23."""
    return 2 * (dim + 8) * 2.0 ** -23 * size + 2.0 ** -15 + (n / 32 + 64) * 2.0 ** -23


def check_attention(c, q, scale, out, lse=None, mass=None, mass0=None):
    want, wlse, weights, spread, size = attend_all(c, q, scale)
    got = out.float().cpu().double().numpy()
    n = max(c.lens + [1])
    slack = attn_slack(size, c.dim, n)
    # bf16 rounds by at most 2^-8 of the value
    tol = 2.0 ** -8 * np.abs(want) + slack[..., None] * spread + 1e-38
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])
    if lse is not None:
        gl = lse.cpu().double().numpy()
        seen = np.isfinite(wlse)
        assert np.array_equal(np.isneginf(gl), ~seen)
        tl = slack[seen] + 2.0 ** -22 * (np.abs(wlse[seen]) + size[seen])
        assert (np.abs(gl[seen] - wlse[seen]) <= tl).all()
    if mass is not None:
        gm = mass.cpu().double().numpy()
        wm = mass0.double().numpy().copy()
        tm = np.zeros_like(wm)
        G = q.shape[1] // c.kv_heads
        for b, w in enumerate(weights):
            if w.shape[1] == 0 or not 0 < c.slots[b] < c.n_slots:
                continue
            at = (c.layer, c.slots[b], slice(None), slice(c.begins[b], c.lens[b]))
            wm[at] += w
            sl = slack[b].reshape(c.kv_heads, G).max(axis=1)[:, None]
            tm[at] = w * (sl + G * 2.0 ** -23) + 2.0 ** -24 * wm[at]  # the sum's own rounding
        assert (np.abs(gm - wm) <= tm).all(), np.abs(gm - wm).max()
