"""The measured cases of the prompt side of the full-attention layers: page tables and token
maps from request lengths, pages given back, rotary positions with the append to the paged
cache, and attention of chunks of new tokens over it.

With ``own`` false, ``run`` computes each operator from elementary torch operations;
with ``own`` true it calls the package.
"""
import math
import random

import torch

own = False

DEV = "cuda"
F8_MAX = 448.0


# ------------------------------------------------------------------- cases --
def _attn(name, batch, kv_heads, group, dim, page, new, cached, dtype, window=0, mass=0, begin=False, pad=0):
    return dict(name=name, op="attn", batch=batch, kv_heads=kv_heads, group=group, dim=dim, page=page,
                new_lo=new[0], new_hi=new[1], cached_lo=cached[0], cached_hi=cached[1], dtype=dtype,
                window=window, mass=mass, begin=begin, pad=pad)


def _rope(name, tokens, batch, q_heads, kv_heads, dim, rot, layout, scaling, page, dtype, far):
    return dict(name=name, op="rope", tokens=tokens, batch=batch, q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                rot=rot, layout=layout, scaling=scaling, page=page, dtype=dtype, far=far)


def _pages(name, op, batch, page, new, cached, pad=0, short=False):
    return dict(name=name, op=op, batch=batch, page=page, new_lo=new[0], new_hi=new[1], cached_lo=cached[0],
                cached_hi=cached[1], pad=pad, short=short)


def listed():
    return [
        # one 6144-token prompt, nothing cached
        _attn("attn_prompt", 1, 2, 8, 256, 64, (6144, 6144), (0, 0), "bf16"),
        # a server's mixed batch: prompts, their later chunks and single tokens over an 8-bit cache in 16-token pages
        _attn("attn_ragged_fp8", 24, 8, 4, 128, 16, (1, 1500), (0, 12000), "fp8", pad=2),
        # one chunk of a very long document
        _attn("attn_long_chunk", 1, 2, 8, 256, 64, (512, 512), (131072, 131072), "bf16"),
        # a few drafted tokens per request checked at once
        _attn("attn_drafts", 32, 2, 8, 256, 64, (1, 7), (500, 8192), "bf16"),
        # sliding-window layers, small heads, an odd number of query heads per key-value head
        _attn("attn_window", 8, 4, 3, 64, 128, (1111, 4099), (0, 0), "bf16", window=1024),
        # prompts that are cut right afterwards: the last 512 queries' weights are added up
        _attn("attn_prompt_mass", 2, 8, 4, 128, 32, (4099, 4099), (0, 0), "bf16", mass=512),
        # the new tokens of one decode step, a quarter of each head turned
        _rope("rope_step", 128, 128, 16, 2, 256, 64, "half", "plain", 64, "bf16", 131072),
        # a 6144-token chunk far into a long context, adjacent pairs, into an 8-bit cache
        _rope("rope_prompt_fp8", 6144, 1, 32, 8, 128, 128, "interleaved", "yarn", 64, "fp8", 1000000),
        # a decode step of a padded batch: now and then a request starts a page
        _pages("map_step", "map", 128, 64, (1, 1), (150, 4099), pad=3),
        # the prompts and chunks of one prefill step
        _pages("map_prompts", "map", 64, 16, (1, 1500), (0, 12000)),
        # after an eviction: each request gives back the page behind its budget
        _pages("release_step", "release", 32, 64, (64, 64), (1024, 1024)),
        # finished requests give back everything
        _pages("release_finished", "release", 64, 16, (150, 8192), (0, 0), pad=1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "rope", "map", "release"])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "fp8"])
    dim = rng.choice([64, 128, 256])
    if op == "attn":
        kv_heads = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
        batch = _log(rng, 1, 48)
        new = _log(rng, 1, 8192)
        cached = rng.choice([0, _log(rng, 1, 65536)])
        # 4 dim flops a pair of query head and place: at most 0.8 Tflop, and a cache of at most 2 GB
        while batch > 1 and (batch * new * (cached + new) * 4 * dim * kv_heads * group > 8e11
                             or batch * (cached + new) * kv_heads * dim > 1 << 29):
            batch //= 2
        while new * (cached + new) * 4 * dim * kv_heads * group > 8e11:
            new, cached = max(1, new // 2), cached // 2
        c = _attn("", batch, kv_heads, group, dim, page, (new // 5, new), (cached // 4, cached), dtype,
                  window=rng.choice([0, 0, _log(rng, 16, 4096)]), mass=rng.choice([0, 0, _log(rng, 1, 300)]),
                  begin=rng.random() < 0.2, pad=batch // 9)
    elif op == "rope":
        tokens = _log(rng, 1, 9000)
        kv_heads = rng.choice([1, 2, 4, 8])
        q_heads = kv_heads * rng.choice([1, 2, 3, 4])
        rot = rng.choice([r for r in (16, 32, 48, 64, 96, 128, 192, 256) if r <= dim])
        c = _rope("", tokens, rng.choice([1, min(tokens, 7), min(tokens, 64)]), q_heads, kv_heads, dim, rot,
                  rng.choice(["half", "interleaved"]), rng.choice(["plain", "linear", "ntk", "yarn", "bands"]),
                  page, dtype, _log(rng, 1, 1000000))
    elif op == "map":
        batch = _log(rng, 1, 300)
        new = _log(rng, 1, 60000 // batch)
        cached = rng.choice([0, _log(rng, 1, 12000)])
        c = _pages("", op, batch, page, (new // 4, new), (cached // 3, cached), batch // 9, rng.random() < 0.2)
    else:
        batch = _log(rng, 1, 128)
        new = _log(rng, 1, 500000 // batch)
        cached = rng.choice([0, _log(rng, 1, 4096)])
        c = _pages("", op, batch, page, (new // 4, new), (cached // 3, cached), batch // 9)
    del c["name"]
    return c


def _lengths(c):
    """(new, cached) tokens of each request: a matter of the case, so that its work is known."""
    r = random.Random(repr(sorted((k, v) for k, v in c.items() if k != "name")))
    new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["batch"])]
    cached = [r.randint(c["cached_lo"], c["cached_hi"]) for _ in range(c["batch"])]
    new[0], cached[-1] = c["new_hi"], c["cached_hi"]
    return new, cached


def _begins(c, new, cached):
    """First visible place: some requests see the last 4096 places before their new tokens."""
    return [max(0, m - 4096) if c["begin"] and b % 2 == 0 else 0 for b, m in enumerate(cached)]


# ------------------------------------------------------------------ inputs --
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, device=DEV, generator=g)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _stored(x, dtype):
    return x.to(torch.bfloat16) if dtype == "bf16" else x.clamp(-F8_MAX, F8_MAX).to(torch.float8_e4m3fn)


def _cache(g, slots, need, kv_heads, dim, page, dtype):
    """One layer's random cache; slot i + 1 has need[i] pages, scattered (page 0 is reserved)."""
    pages = 1 + sum(need)
    ids = (torch.randperm(pages - 1, device=DEV, generator=g) + 1).to(torch.int32)
    table = torch.zeros(slots, max(need), dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(need):
        table[i + 1, :n] = ids[at:at + n]
        at += n
    shape = (1, pages, kv_heads, page, dim)
    k, v = (_stored(_randn(g, *shape), dtype) for _ in range(2))
    one = dtype == "bf16"
    return dict(k=k, v=v, table=table, kscale=1.0 if one else 0.75, vscale=1.0 if one else 1.25)


def _handle(s):
    import gated_delta_rule_slot_amd as gdn

    return gdn.kv_pool_create(s["k"], s["v"], s["table"], mass=s.get("mass"), pos=s.get("pos"),
                              err_word=torch.zeros(1, dtype=torch.int32, device=DEV),
                              k_scale=s["kscale"], v_scale=s["vscale"])


def _prepare_attn(c, g):
    B, H, G, D, ps = c["batch"], c["kv_heads"], c["group"], c["dim"], c["page"]
    new, cached = _lengths(c)
    total = [n + m for n, m in zip(new, cached)]
    s = _cache(g, B + 1, [-(-n // ps) for n in total], H, D, ps, c["dtype"])
    s["new"], s["total"], s["begins"] = new, total, _begins(c, new, cached)
    slots = list(range(1, B + 1))
    if c["pad"]:  # a batch padded to its captured size
        slots[B - c["pad"]:] = [0] * c["pad"]
    s["slots_host"], s["slots"], s["len"] = slots, _i32(slots), _i32(total)
    s["cu"] = _i32([sum(new[:b]) for b in range(B + 1)])
    s["begin"] = _i32(s["begins"]) if c["begin"] else None
    T = sum(new)
    # queries whose scores spread the softmax over some tokens, as trained heads do
    s["q"] = (1.5 * _randn(g, T, H * G, D)).to(torch.bfloat16)
    s["scale"] = 1.0 / math.sqrt(D)
    s["cap"] = s["table"].shape[1] * ps
    s["mass"] = torch.rand(1, B + 1, H, s["cap"], device=DEV, generator=g) if c["mass"] else None
    if own:
        import gated_delta_rule_slot_amd as gdn

        s["pool"] = _handle(s)
        s["out"] = torch.empty(T, H * G, D, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(T, H * G, device=DEV)
        nbytes = gdn.attn_prefill_workspace_bytes(s["pool"], B, T, H * G, max(total), c["mass"])
        s["ws"] = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    return s


def _frequencies(c):
    """Angle per position of each pair (float64) and the factor of the turned values."""
    rot, base, factor, orig = c["rot"], 10000.0, 8.0, 8192.0
    i = torch.arange(rot // 2, dtype=torch.float64)
    kind = c["scaling"]
    if kind == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if kind == "linear":
        f = f / factor
    if kind == "yarn":
        at = [rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
        lo, hi = max(0.0, math.floor(at[0])), min(rot - 1.0, math.ceil(at[1]))
        ramp = torch.clamp((i - lo) / max(hi - lo, 1e-3), 0, 1)
        f = f / factor * ramp + f * (1 - ramp)
    if kind == "bands":
        turns = orig * f / (2 * math.pi)
        keep = torch.clamp((turns - 1.0) / (4.0 - 1.0), 0, 1)
        f = f / factor * (1 - keep) + f * keep
    return f, 0.1 * math.log(factor) + 1 if kind == "yarn" else 1.0


def _prepare_rope(c, g):
    T, B, H, D = c["tokens"], c["batch"], c["kv_heads"], c["dim"]
    per = -(-T // B)
    s = _cache(g, B + 1, [-(-(2 * per + 70) // c["page"])] * B, H, D, c["page"], c["dtype"])
    s["cap"] = s["table"].shape[1] * c["page"]
    i = torch.arange(T, device=DEV)
    s["slots"] = (i % B + 1).to(torch.int32)
    start = torch.randint(0, per + 60, (B,), device=DEV, generator=g)
    s["index"] = (start[i % B] + i // B).to(torch.int32)
    first = torch.randint(0, c["far"] + 1, (B,), device=DEV, generator=g)
    s["position"] = (first[i % B] + i // B).to(torch.int32)
    # queries, keys and values lie side by side in the projection's rows, as a fused product leaves them
    Hq = c["q_heads"]
    x = (2.0 * _randn(g, T, (Hq + 2 * H) * D)).to(torch.bfloat16)
    s["q"] = x[:, :Hq * D].view(T, Hq, D)
    s["kn"] = x[:, Hq * D:(Hq + H) * D].view(T, H, D)
    s["vn"] = x[:, (Hq + H) * D:].view(T, H, D)
    s["q_out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
    s["mass"] = torch.rand(1, B + 1, H, s["cap"], device=DEV, generator=g)
    s["pos"] = torch.zeros(1, B + 1, H, s["cap"], dtype=torch.int32, device=DEV)
    s["kdiv"], s["vdiv"] = (torch.tensor(s[n], device=DEV) for n in ("kscale", "vscale"))
    f, s["amp"] = _frequencies(c)
    if own:
        import gated_delta_rule_slot_amd as gdn

        s["pool"] = _handle(s)
        s["layout"] = gdn.ROPE_HALF if c["layout"] == "half" else gdn.ROPE_INTERLEAVED
        kind = {"plain": gdn.ROPE_PLAIN, "linear": gdn.ROPE_LINEAR, "ntk": gdn.ROPE_NTK, "yarn": gdn.ROPE_YARN,
                "bands": gdn.ROPE_BANDS}[c["scaling"]]
        f, s["amp"] = gdn.rope_frequencies(c["rot"], base=10000.0, scaling=kind, factor=8.0, original_len=8192.0,
                                           low=1.0, high=32.0 if c["scaling"] == "yarn" else 4.0)
    s["freqs"] = f.to(DEV)
    return s


def _prepare_pages(c, g):
    B, ps = c["batch"], c["page"]
    new, cached = _lengths(c)
    if c["op"] == "release":
        cached, new = [n + m for n, m in zip(new, cached)], cached  # (length, what is kept)
    need = [-(-n // ps) for n in cached]
    most = max(-(-(n + m) // ps) for n, m in zip(new, cached))
    extra = sum(-(-(n + m) // ps) for n, m in zip(new, cached)) - sum(need) if c["op"] == "map" else 40
    pages = 1 + sum(need) + extra + 100
    ids = (torch.randperm(pages - 1, device=DEV, generator=g) + 1).to(torch.int32)
    order = (torch.randperm(B, device=DEV, generator=g) + 1).tolist()
    table = torch.zeros(B + 1, max(1, most) + 2, dtype=torch.int32, device=DEV)
    at = 0
    for slot, n in zip(order, need):
        table[slot, :n] = ids[at:at + n]
        at += n
    if c["pad"]:
        order[B - c["pad"]:] = [0] * c["pad"]
    # the heads' sizes do not matter here: one head of one layer
    s = dict(k=torch.zeros(1, pages, 1, ps, 64, dtype=torch.bfloat16, device=DEV), kscale=1.0, vscale=1.0,
             table=table, table0=table.clone(), slots=_i32(order), len=_i32(cached), cap=table.shape[1] * ps)
    s["v"] = s["k"]
    free = torch.zeros(pages, dtype=torch.int32, device=DEV)
    free[:pages - 1 - at] = ids[at:]
    s["free"], s["n_free_out"] = free, _i32([0])
    have = pages - 1 - at
    if c["short"]:  # a list that runs out before the batch does
        have = extra // 2
    s["n_free"] = _i32([have])
    if c["op"] == "map":
        T = -(-(sum(new)) // 64) * 64  # a captured size: the rest is padding
        s["new"], s["tokens"] = _i32(new), max(64, T)
        s["next"] = s["len"] + torch.randint(0, 1000, (B,), device=DEV, generator=g, dtype=torch.int32)
        for n, size in (("cu", B + 1), ("slot_out", B), ("len_out", B), ("next_out", B)):
            s[n] = torch.zeros(size, dtype=torch.int32, device=DEV)
        for n in ("token_slot", "token_index", "token_pos"):
            s[n] = torch.zeros(s["tokens"], dtype=torch.int32, device=DEV)
    else:
        s["keep"] = _i32(new)
    if own:
        s["pool"] = _handle(s)
    return s


def prepare(case, seed):
    make = {"attn": _prepare_attn, "rope": _prepare_rope, "map": _prepare_pages, "release": _prepare_pages}
    s = make[case["op"]](case, _gen(seed))
    s["case"] = case
    return s


# ------------------------------------------------------------- plain forms --
def _rows(pool, ids, n):
    """[H, n, D] rows of the first n places of the pages ids, in 32 bits."""
    x = pool[0].view(torch.uint8 if pool.dtype == torch.float8_e4m3fn else torch.int16)[ids]
    P, H, S, D = x.shape
    return x.transpose(0, 1).reshape(H, P * S, D)[:, :n].contiguous().view(pool.dtype).float()


def _plain_attn(s):
    c = s["case"]
    B, H, G, D, ps = c["batch"], c["kv_heads"], c["group"], c["dim"], c["page"]
    T = sum(s["new"])
    out = torch.zeros(T, H * G, D, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, H * G), -math.inf, device=DEV)
    at = 0
    for b in range(B):
        n, L, slot = s["new"][b], s["total"][b], s["slots_host"][b]
        rows = slice(at, at + n)
        at += n
        if slot <= 0 or n == 0:
            continue
        ids = s["table"][slot, :-(-L // ps)].long()
        q = s["q"][rows].float().view(n, H, G, D).permute(1, 0, 2, 3).reshape(H, n * G, D)
        t = torch.arange(L, device=DEV)
        place = torch.arange(L - n, L, device=DEV)[:, None]
        seen = (t <= place) & (t >= s["begins"][b])
        if c["window"]:
            seen = seen & (t > place - c["window"])
        seen = seen[:, None, :].expand(n, G, L).reshape(n * G, L)
        k = _rows(s["k"], ids, L).transpose(1, 2).contiguous()
        v = _rows(s["v"], ids, L)
        x = torch.matmul(q, k).mul_(s["scale"] * s["kscale"])
        x.masked_fill_(~seen, -math.inf)
        m = x.amax(dim=-1, keepdim=True)
        m = torch.where(torch.isneginf(m), torch.zeros_like(m), m)
        p = x.sub_(m).exp_()
        l = p.sum(dim=-1, keepdim=True)
        p = p.mul_(torch.where(l > 0, 1.0 / l, torch.zeros_like(l)))
        o = torch.matmul(p, v) * s["vscale"]
        out[rows] = o.view(H, n, G, D).permute(1, 0, 2, 3).reshape(n, H * G, D).to(torch.bfloat16)
        lse[rows] = (m + torch.log(l)).view(H, n, G).permute(1, 0, 2).reshape(n, H * G)
        if c["mass"]:
            w = min(n, c["mass"])
            s["mass"][0, slot, :, :L] += p.view(H, n, G, L)[:, n - w:].sum(dim=(1, 2))
    r = {"out": out, "lse": lse}
    if c["mass"]:
        r["mass"] = s["mass"]
    return r


def _plain_turn(x, cos, sin, rot, layout):
    x = x.float()
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = x[..., :rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def _plain_rope(s):
    c = s["case"]
    # the angles of far positions need more than 32 bits
    angle = s["position"].double()[:, None, None] * s["freqs"]
    cos, sin = (torch.cos(angle) * s["amp"]).float(), (torch.sin(angle) * s["amp"]).float()
    q = _plain_turn(s["q"], cos, sin, c["rot"], c["layout"]).to(torch.bfloat16)
    k = _plain_turn(s["kn"], cos, sin, c["rot"], c["layout"])
    s["q_out"].copy_(q)
    slot, i = s["slots"].long(), s["index"].long()
    page, off = s["table"][slot, i // c["page"]].long(), i % c["page"]
    for pool, x, div in (("k", k, "kdiv"), ("v", s["vn"].float(), "vdiv")):
        if c["dtype"] == "fp8":
            s[pool][0].view(torch.uint8)[page, :, off] = _stored(x / s[div], "fp8").view(torch.uint8)
        else:
            s[pool][0][page, :, off] = x.to(torch.bfloat16)
    s["mass"][0][slot, :, i] = 0.0
    s["pos"][0][slot, :, i] = s["position"][:, None].expand(-1, c["kv_heads"])
    return {n: s[n] for n in ("q_out", "k", "v", "mass", "pos")}


def _before(x):
    return torch.cumsum(x, 0) - x


def _plain_map(s):
    c = s["case"]
    B, ps, T = c["batch"], c["page"], s["tokens"]
    slot, n, L, nf = s["slots"].long(), s["new"].long(), s["len"].long(), s["n_free"].long()
    end = torch.cumsum(n, 0)
    valid = (slot > 0) & (L + n <= s["cap"]) & (end <= T)
    have = (L + ps - 1) // ps
    need = torch.where(valid, (L + n + ps - 1) // ps - have, torch.zeros_like(n))
    rank = _before(need)
    served = valid & ((need == 0) | (rank + need <= nf))
    took = torch.where(served, need, torch.zeros_like(need))
    # pages: entry e of the flat list belongs to the request whose run holds it
    most = s["table"].shape[1]
    j = torch.arange(most, device=DEV)
    takes = j < took[:, None]
    row = torch.where(takes, slot[:, None], torch.zeros_like(slot)[:, None]).reshape(-1)
    col = torch.where(takes, have[:, None] + j, torch.zeros_like(j)).reshape(-1)
    src = torch.where(takes, nf - 1 - rank[:, None] - j, torch.zeros_like(j))
    page = torch.where(takes, s["free"][src.clamp(min=0)], torch.zeros_like(s["free"][:1])).reshape(-1)
    s["table"][row, col] = page  # what is not taken writes 0 to the reserved slot's first entry
    s["n_free_out"].copy_(nf - took.sum())
    add = torch.where(served, n, torch.zeros_like(n))
    s["cu"][1:] = end.clamp(max=T)
    s["slot_out"].copy_(torch.where(served, slot, torch.zeros_like(slot)))
    s["len_out"].copy_(L + add)
    s["next_out"].copy_(s["next"] + add)
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(end, t, right=True)
    live = b < B
    b = b.clamp(max=B - 1)
    live = live & served[b]
    i = t - (end - n)[b]
    zero = torch.zeros_like(t)
    s["token_slot"].copy_(torch.where(live, slot[b], zero))
    s["token_index"].copy_(torch.where(live, L[b] + i, zero))
    s["token_pos"].copy_(torch.where(live, s["next"].long()[b] + i, zero))
    return _map_outputs(s)


def _map_outputs(s):
    return {n: s[n] for n in ("table", "n_free_out", "cu", "slot_out", "len_out", "next_out", "token_slot",
                              "token_index", "token_pos")}


def _plain_release(s):
    ps = s["case"]["page"]
    slot = s["slots"].long()
    lo, hi = (s["keep"].long() + ps - 1) // ps, (s["len"].long() + ps - 1) // ps
    j = torch.arange(s["table"].shape[1], device=DEV)
    mine = (j >= lo[:, None]) & (j < hi[:, None]) & (slot > 0)[:, None]
    rows = s["table"][slot]
    at = torch.cumsum(mine.reshape(-1).long(), 0) - 1 + s["n_free"]
    # what is not given back goes to a place behind the list
    spare = s["free"].numel()
    list_ = torch.cat([s["free"], s["free"][:1]])
    list_[torch.where(mine.reshape(-1), at, torch.full_like(at, spare))] = rows.reshape(-1)
    s["free"].copy_(list_[:spare])
    s["n_free_out"].copy_(s["n_free"] + mine.sum())
    row = torch.where(mine, slot[:, None], torch.zeros_like(slot)[:, None])
    s["table"][row, torch.where(mine, j, torch.zeros_like(j))] = 0
    return {n: s[n] for n in ("table", "free", "n_free_out")}


# --------------------------------------------------------------------- run --
def _run_own(s):
    import gated_delta_rule_slot_amd as gdn

    c = s["case"]
    if c["op"] == "attn":
        gdn.attn_prefill_paged(s["pool"], 0, s["cu"], s["slots"], s["len"], s["q"], s["out"], max(s["total"]),
                               kv_begin=s["begin"], window=c["window"], scale=s["scale"], mass_tokens=c["mass"],
                               lse=s["lse"], workspace=s["ws"])
        r = {"out": s["out"], "lse": s["lse"]}
        if c["mass"]:
            r["mass"] = s["mass"]
        return r
    if c["op"] == "rope":
        gdn.rope_append(s["pool"], 0, s["slots"], s["index"], s["position"], s["q"], s["q_out"], s["kn"], s["vn"],
                        s["freqs"], layout=s["layout"], amplitude=s["amp"])
        return {n: s[n] for n in ("q_out", "k", "v", "mass", "pos")}
    if c["op"] == "map":
        gdn.kv_batch_map(s["pool"], s["slots"], s["len"], s["free"], s["n_free"], s["cu"], s["slot_out"],
                         s["len_out"], s["token_slot"], s["token_index"], new_len=s["new"], next_pos=s["next"],
                         next_pos_out=s["next_out"], token_pos=s["token_pos"], n_free_out=s["n_free_out"])
        return _map_outputs(s)
    gdn.kv_release(s["pool"], s["slots"], s["len"], s["free"], s["n_free"], keep=s["keep"],
                   n_free_out=s["n_free_out"])
    return {n: s[n] for n in ("table", "free", "n_free_out")}


def run(state):
    op = state["case"]["op"]
    if op == "release":  # a pass gives the entries away: they are put back for the next
        state["table"].copy_(state["table0"])
    if own:
        return _run_own(state)
    return {"attn": _plain_attn, "rope": _plain_rope, "map": _plain_map, "release": _plain_release}[op](state)


# -------------------------------------------------------------------- work --
def work(case):
    c = case
    size = 2 if c.get("dtype") == "bf16" else 1
    if c["op"] == "rope":
        row = c["tokens"] * c["dim"]
        turned = 6 * row // c["dim"] * c["rot"] * (c["q_heads"] + c["kv_heads"]) // 2
        return {"bytes": 4 * row * c["q_heads"] + 2 * row * c["kv_heads"] * (2 + size)
                + c["tokens"] * (12 + 8 * c["kv_heads"]), "flops": turned}
    new, cached = _lengths(c)
    if c["op"] == "map":
        ps = c["page"]
        pages = sum(-(-(n + m) // ps) - -(-m // ps) for n, m in zip(new, cached))
        return {"bytes": 12 * sum(new) + 36 * c["batch"] + 8 * pages, "flops": 0}
    if c["op"] == "release":
        ps = c["page"]
        pages = sum(-(-(n + m) // ps) - -(-m // ps) for n, m in zip(new, cached))
        return {"bytes": 12 * c["batch"] + 12 * pages, "flops": 0}
    pairs = rows = late = 0  # visible pairs, places seen by any query, pairs of the late queries
    for b, (n, m) in enumerate(list(zip(new, cached))[:c["batch"] - c["pad"]]):
        begin = _begins(c, new, cached)[b]
        first = max(begin, m - c["window"] + 1) if c["window"] else begin
        rows += n + m - first
        for i in range(n):
            got = m + i + 1 - max(begin, m + i + 1 - c["window"] if c["window"] else 0)
            pairs += got
            late += got if i >= n - c["mass"] else 0
    heads = c["kv_heads"] * c["group"]
    T = sum(new)
    moved = rows * c["kv_heads"] * (2 * c["dim"] * size + (8 if c["mass"] else 0)) + T * heads * (4 * c["dim"] + 4)
    return {"bytes": moved, "flops": heads * c["dim"] * (4 * pairs + 2 * late)}


# ------------------------------------------------------- 64-bit definitions --
def _exact_attn(c, s):
    B, H, G, D, ps = c["batch"], c["kv_heads"], c["group"], c["dim"], c["page"]
    T = sum(s["new"])
    out = torch.zeros(T, H * G, D, dtype=torch.float64, device=DEV)
    lse = torch.full((T, H * G), -math.inf, dtype=torch.float64, device=DEV)
    mass = s["mass"].double() if c["mass"] else None
    bits = torch.uint8 if c["dtype"] == "fp8" else torch.int16
    cu, slots, lens = s["cu"].tolist(), s["slots"].tolist(), s["len"].tolist()
    for b in range(B):
        r0, r1, L = cu[b], cu[b + 1], lens[b]
        n = r1 - r0
        if slots[b] <= 0:
            continue
        ids = s["table"][slots[b], :-(-L // ps)].long()
        for h in range(H):
            k, v = (s[x][0, :, h].view(bits)[ids].view(s[x].dtype).reshape(-1, D)[:L].double() for x in ("k", "v"))
            step = max(1, (1 << 28) // max(1, L * G))  # queries at a time
            for a in range(0, n, step):
                e = min(n, a + step)
                hidden = torch.ones(e - a, L, dtype=torch.bool, device=DEV).triu(L - n + a + 1)
                if c["window"]:
                    hidden |= torch.ones(e - a, L, dtype=torch.bool, device=DEV).tril(L - n + a - c["window"])
                hidden[:, :s["begins"][b]] = True
                q = s["q"][r0 + a:r0 + e, h * G:(h + 1) * G].double().reshape(-1, D)
                x = (q @ k.t()) * (s["scale"] * s["kscale"])
                x.view(e - a, G, L).masked_fill_(hidden[:, None, :], -math.inf)
                z = torch.logsumexp(x, dim=-1)
                w = torch.exp(x - torch.where(torch.isneginf(z), torch.zeros_like(z), z)[:, None])
                out[r0 + a:r0 + e, h * G:(h + 1) * G] = ((w @ v) * s["vscale"]).view(e - a, G, D)
                lse[r0 + a:r0 + e, h * G:(h + 1) * G] = z.view(e - a, G)
                if mass is not None and e > n - c["mass"]:
                    from_ = max(a, n - c["mass"]) - a
                    mass[0, slots[b], h, :L] += w.view(e - a, G, L)[from_:].sum(dim=(0, 1))
    r = {"out": out, "lse": lse}
    if mass is not None:
        r["mass"] = mass
    return r


def _exact_rope(c, s):
    r = {n: s[n].double() for n in ("k", "v", "mass")}
    rot = c["rot"]
    f, amp = _frequencies(c)
    a = s["position"].double()[:, None] * f.to(DEV)
    turn = torch.polar(torch.full_like(a, amp), a)[:, None]  # amp e^(i a)
    new = {}
    for n in ("q", "kn"):
        x = s[n].double().clone()
        if c["layout"] == "half":
            z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * turn
            x[..., :rot // 2], x[..., rot // 2:rot] = z.real, z.imag
        else:
            z = torch.view_as_complex(x[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * turn
            x[..., :rot] = torch.view_as_real(z).flatten(-2)
        new[n] = x
    new["vn"] = s["vn"].double()
    r["q_out"] = new["q"]
    slots, index = s["slots"].long(), s["index"].long()
    page, off = s["table"][slots, index // c["page"]].long(), index % c["page"]
    for h in range(c["kv_heads"]):
        for n, x, scale in (("k", "kn", "kscale"), ("v", "vn", "vscale")):
            y = new[x][:, h] / s[scale]
            r[n][0, page, h, off] = y.clamp(-F8_MAX, F8_MAX) if c["dtype"] == "fp8" else y
        r["mass"][0, slots, h, index] = 0
    r["pos"] = None
    return {n: r[n] for n in ("q_out", "k", "v", "mass", "pos")}


def exact(case, seed):
    if case["op"] in ("map", "release"):
        return None  # whole numbers only
    s = prepare(case, seed)
    return _exact_attn(case, s) if case["op"] == "attn" else _exact_rope(case, s)
