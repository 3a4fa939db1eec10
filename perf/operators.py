"""The measured cases of the full-attention operators: append to the paged key-value
cache, attention of one new token over it, eviction from it by accumulated attention
weight (the plan and the moves), and the norm / gate / residual step between blocks.

With ``own`` false, ``run`` computes each operator from elementary torch operations;
with ``own`` true it calls the package.
"""
import math

import torch

own = False

DEV = "cuda"
F8_MAX = 448.0


# ------------------------------------------------------------------- cases --
def _attn(name, batch, kv_heads, group, dim, page, lo, hi, dtype, mass, begin=False, pad=0):
    return dict(name=name, op="attn", batch=batch, kv_heads=kv_heads, group=group, dim=dim,
                page=page, lo=lo, hi=hi, dtype=dtype, mass=mass, begin=begin, pad=pad)


def _append(name, tokens, batch, kv_heads, dim, page, dtype):
    return dict(name=name, op="append", tokens=tokens, batch=batch, kv_heads=kv_heads, dim=dim,
                page=page, dtype=dtype)


def _evict(name, op, layers, batch, kv_heads, dim, page, n, budget, sink, recent, dtype):
    return dict(name=name, op=op, layers=layers, batch=batch, kv_heads=kv_heads, dim=dim,
                page=page, n=n, budget=budget, sink=sink, recent=recent, dtype=dtype)


def _norm(name, tokens, groups, dim, post, gate, residual, pre, wdtype):
    return dict(name=name, op="norm", tokens=tokens, groups=groups, dim=dim, post=post, gate=gate,
                residual=residual, pre=pre, wdtype=wdtype)


def listed():
    return [
        # one short chat request: what a single user waits for at each token
        _attn("attn_one_short", 1, 2, 8, 256, 64, 777, 777, "bf16", False),
        # a busy server: 128 requests of mixed lengths, weights accumulated for a later eviction
        _attn("attn_batch_ragged_mass", 128, 2, 8, 256, 64, 150, 4099, "bf16", True, pad=3),
        # few requests over very long documents
        _attn("attn_long", 4, 2, 8, 256, 64, 90001, 131072, "bf16", False),
        # 8-bit cache, 16-token pages, sliding-window starts
        _attn("attn_fp8_pages16", 64, 8, 4, 128, 16, 1000, 8192, "fp8", False, begin=True),
        # the new tokens of one decode step
        _append("append_step", 128, 128, 2, 256, 64, "bf16"),
        # the keys and values of one 6144-token prefill into an 8-bit cache
        _append("append_prefill_fp8", 6144, 1, 8, 128, 64, "fp8"),
        # a block of 64 new tokens over the budget, all 8 full layers of a batch at once
        _evict("evict_plan_block", "plan", 8, 32, 2, 256, 64, 1088, 1024, 4, 128, "bf16"),
        # a long prompt cut to a quarter
        _evict("evict_plan_long", "plan", 8, 2, 8, 128, 64, 32769, 8192, 4, 512, "bf16"),
        _evict("evict_apply_block", "apply", 8, 32, 2, 256, 64, 1088, 1024, 4, 128, "bf16"),
        _evict("evict_apply_long", "apply", 8, 2, 8, 128, 64, 32769, 8192, 4, 512, "fp8"),
        # after a block and before the next one, 128 tokens of one decode step
        _norm("norm_step", 128, 1, 2048, True, "sigmoid", "bf16", True, "bf16"),
        # the gated norm of the recurrence's heads, one 6144-token prefill
        _norm("norm_heads_prefill", 6144, 32, 128, True, "silu", "none", False, "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "append", "plan", "apply", "norm"])
    dim = rng.choice([64, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "fp8"])
    if op == "attn":
        batch = _log(rng, 1, 192)
        group = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
        most = min(131072, (1 << 28) // (batch * kv_heads * dim))
        hi = _log(rng, 24, max(25, most))
        c = _attn("", batch, kv_heads, group, dim, page, max(1, int(hi * rng.uniform(0.1, 1))), hi,
                  dtype, rng.random() < 0.4, rng.random() < 0.3, batch // 9)
    elif op == "append":
        tokens = _log(rng, 1, 9000)
        c = _append("", tokens, rng.choice([1, min(tokens, 7), min(tokens, 64)]), kv_heads, dim, page, dtype)
    elif op in ("plan", "apply"):
        budget = _log(rng, 100, 8192)
        n = budget + _log(rng, 1, 3 * budget)
        layers = rng.choice([1, 3, 8])
        batch = max(1, min(_log(rng, 1, 32), (1 << 22) // (n * layers * kv_heads)))
        recent = rng.choice([0, budget // 8, budget // 3])
        c = _evict("", op, layers, batch, kv_heads, dim, page, n, budget, rng.choice([0, 4]), recent, dtype)
    else:
        heads = rng.random() < 0.4
        groups = rng.choice([12, 16, 32]) if heads else 1
        d = rng.choice([64, 128, 256]) if heads else 8 * _log(rng, 32, 1024)
        tokens = _log(rng, 1, max(2, (1 << 24) // (groups * d)))
        residual = "none" if heads else rng.choice(["bf16", "f32"])
        c = _norm("", tokens, groups, d, heads or rng.random() < 0.6, rng.choice(["none", "silu", "sigmoid"]),
                  residual, residual != "none", rng.choice(["bf16", "f32"]))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs --
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, device=DEV, generator=g)


def _stored(x, dtype):
    return x.to(torch.bfloat16) if dtype == "bf16" else x.clamp(-F8_MAX, F8_MAX).to(torch.float8_e4m3fn)


def _pool(g, layers, slots, cap, used, kv_heads, dim, page, dtype):
    """Random pool with every slot's pages scattered over it (page 0 stays unused)."""
    max_pages = -(-cap // page)
    need = -(-used // page)
    pages = 1 + slots * need
    table = torch.zeros(slots, max_pages, dtype=torch.int32, device=DEV)
    table[:, :need] = (torch.randperm(pages - 1, device=DEV, generator=g) + 1).to(torch.int32).view(slots, need)
    shape = (layers, pages, kv_heads, page, dim)
    k, v = (_stored(_randn(g, *shape), dtype) for _ in range(2))
    mp = max_pages * page
    return dict(k=k, v=v, table=table, cap=mp, kscale=1.0 if dtype == "bf16" else 0.75,
                vscale=1.0 if dtype == "bf16" else 1.25)


def _handle(s):
    if not own:
        return None
    import gated_delta_rule_slot_amd as gdn

    return gdn.kv_pool_create(s["k"], s["v"], s["table"], mass=s.get("mass"), pos=s.get("pos"),
                              err_word=torch.zeros(1, dtype=torch.int32, device=DEV),
                              k_scale=s["kscale"], v_scale=s["vscale"])


def _prepare_attn(c, g):
    B, H, G, D = c["batch"], c["kv_heads"], c["group"], c["dim"]
    s = _pool(g, 1, B + 1, c["hi"], c["hi"], H, D, c["page"], c["dtype"])
    s["len"] = torch.randint(c["lo"], c["hi"] + 1, (B,), device=DEV, generator=g, dtype=torch.int32)
    s["len"][0] = c["hi"]
    slots = torch.randperm(B, device=DEV, generator=g) + 1
    if c["pad"]:  # a batch padded to its captured size
        slots[B - c["pad"]:] = 0
    s["slots"] = slots.to(torch.int32)
    s["begin"] = torch.clamp(s["len"] - 4096, min=0) if c["begin"] else None
    # queries whose scores spread the softmax over some tokens, as trained heads do
    s["q"] = (1.5 * _randn(g, B, H * G, D)).to(torch.bfloat16)
    s["scale"] = 1.0 / math.sqrt(D)
    s["mass"] = torch.rand(1, B + 1, H, s["cap"], device=DEV, generator=g) if c["mass"] else None
    if own:
        import gated_delta_rule_slot_amd as gdn

        s["pool"] = _handle(s)
        s["flags"] = gdn.ATTN_ACCUM_MASS if c["mass"] else 0
        s["out"] = torch.empty(B, H * G, D, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(B, H * G, device=DEV)
        nbytes = gdn.attn_workspace_bytes(s["pool"], B, H * G, c["hi"], s["flags"])
        s["ws"] = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    return s


def _prepare_append(c, g):
    T, B, H, D = c["tokens"], c["batch"], c["kv_heads"], c["dim"]
    per = -(-T // B)
    s = _pool(g, 1, B + 1, 2 * per + 70, 2 * per + 70, H, D, c["page"], c["dtype"])
    i = torch.arange(T, device=DEV)
    s["slots"] = (i % B + 1).to(torch.int32) if B > 1 else torch.ones(T, dtype=torch.int32, device=DEV)
    start = torch.randint(0, per + 60, (B,), device=DEV, generator=g)
    s["index"] = (start[i % B] + i // B).to(torch.int32)
    s["position"] = s["index"] + 1000
    # keys and values lie side by side in the projection's rows, as a fused product leaves them
    kv = (2.0 * _randn(g, T, 2 * H * D)).to(torch.bfloat16)
    s["kn"], s["vn"] = kv[:, :H * D].view(T, H, D), kv[:, H * D:].view(T, H, D)
    s["mass"] = torch.rand(1, B + 1, H, s["cap"], device=DEV, generator=g)
    s["pos"] = torch.zeros(1, B + 1, H, s["cap"], dtype=torch.int32, device=DEV)
    s["kdiv"], s["vdiv"] = (torch.tensor(s[n], device=DEV) for n in ("kscale", "vscale"))
    s["pool"] = _handle(s)
    return s


def _prepare_evict(c, g):
    L, B, H, n = c["layers"], c["batch"], c["kv_heads"], c["n"]
    used = n if c["op"] == "apply" else 1  # the plan reads no keys or values
    s = _pool(g, L, B + 1, n, used, H, c["dim"], c["page"], c["dtype"])
    s["len"] = torch.randint(max(1, n - n // 16), n + 1, (B,), device=DEV, generator=g, dtype=torch.int32)
    s["len"][0] = n
    s["slots"] = (torch.randperm(B, device=DEV, generator=g) + 1).to(torch.int32)
    # weights as a softmax spreads them: few large, many small, some never attended to
    w = torch.exp(3.0 * _randn(g, L, B + 1, H, s["cap"]) - 4.0)
    s["mass"] = torch.where(torch.rand(w.shape, device=DEV, generator=g) < 0.02, torch.zeros_like(w), w)
    # positions of a cache that was cut before: distinct, out of order in the first `budget` places
    gap = 3 * n
    order = torch.argsort(torch.rand(L, B + 1, H, c["budget"], device=DEV, generator=g), dim=-1)
    tail = torch.arange(c["budget"], s["cap"], device=DEV).expand(L, B + 1, H, -1)
    pos = torch.cat([order, tail], dim=-1)
    s["pos"] = torch.where(pos < 8, pos, pos + gap).to(torch.int32)
    s["next"] = s["len"] + gap
    s["most"] = min(c["budget"], n - c["budget"])
    s["n_moves"] = torch.zeros(L, B, H, dtype=torch.int32, device=DEV)
    s["moves"] = torch.full((L, B, H, s["most"], 2), -1, dtype=torch.int32, device=DEV)
    s["len_out"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    if c["op"] == "apply":
        r = _plain_plan(dict(s, case=c))
        s["n_moves"], s["moves"] = r["n_moves"], r["moves"]
    s["pool"] = _handle(s)
    return s


def _prepare_norm(c, g):
    T, N, D = c["tokens"], c["groups"], c["dim"]
    wt = torch.bfloat16 if c["wdtype"] == "bf16" else torch.float32
    s = dict(y=(0.3 * _randn(g, T, N, D)).to(torch.bfloat16), eps=1e-6)
    s["w_post"] = (1.0 + 0.2 * _randn(g, D)).to(wt) if c["post"] else None
    s["w_pre"] = (1.0 + 0.2 * _randn(g, D)).to(wt) if c["pre"] else None
    s["scale"] = 0.25 if c["residual"] != "none" else 1.0
    s["gate"] = s["residual"] = s["res_out"] = None
    if c["gate"] != "none":  # the gate is a slice of a wider projection
        s["gate"] = _randn(g, T, N * D + 64).to(torch.bfloat16)[:, 64:].view(T, N, D)
    if c["residual"] != "none":
        rt = torch.bfloat16 if c["residual"] == "bf16" else torch.float32
        s["residual"] = (2.0 * _randn(g, T, N, D)).to(rt)
        s["res_out"] = torch.empty_like(s["residual"])
    s["out"] = torch.empty(T, N, D, dtype=torch.bfloat16, device=DEV)
    if own:
        import gated_delta_rule_slot_amd as gdn

        s["act"] = {"none": gdn.ACT_NONE, "silu": gdn.ACT_SILU, "sigmoid": gdn.ACT_SIGMOID}[c["gate"]]
    return s


def prepare(case, seed):
    make = {"attn": _prepare_attn, "append": _prepare_append, "plan": _prepare_evict,
            "apply": _prepare_evict, "norm": _prepare_norm}[case["op"]]
    s = make(case, _gen(seed))
    s["case"] = case
    return s


# ------------------------------------------------------------- plain forms --
def _rows(pool, page, off):
    """[B, T, H, D] rows of one layer's [P, H, page, D] at (page, off) [B, T], in 32 bits."""
    if pool.dtype == torch.float8_e4m3fn:
        return pool.view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn).float()
    return pool[page, :, off].float()


def _plain_attn(s):
    c = s["case"]
    B, H, G, D, T = c["batch"], c["kv_heads"], c["group"], c["dim"], c["hi"]
    t = torch.arange(T, device=DEV)
    slot = s["slots"].long()
    page = s["table"][slot].long()[:, t // c["page"]]
    off = (t % c["page"]).expand(B, T)
    seen = (t < s["len"][:, None]) & (slot > 0)[:, None]
    if s["begin"] is not None:
        seen = seen & (t >= s["begin"][:, None])
    k = _rows(s["k"][0], page, off).permute(0, 2, 3, 1) * s["kscale"]
    q = s["q"].float().view(B, H, G, D)
    x = torch.matmul(q, k) * s["scale"]
    del k
    x = x.masked_fill(~seen[:, None, None, :], -math.inf)
    m = x.amax(dim=-1, keepdim=True)
    m = torch.where(torch.isneginf(m), torch.zeros_like(m), m)
    p = torch.exp(x - m)
    total = p.sum(dim=-1, keepdim=True)
    p = torch.where(total > 0, p / total, torch.zeros_like(p))
    v = _rows(s["v"][0], page, off).permute(0, 2, 1, 3) * s["vscale"]
    o = torch.matmul(p, v)
    r = {"out": o.view(B, H * G, D).to(torch.bfloat16), "lse": (m + torch.log(total)).view(B, H * G)}
    if c["mass"]:
        s["mass"][0].index_put_((slot[:, None, None], torch.arange(H, device=DEV)[:, None], t),
                                p.sum(dim=2), accumulate=True)
        r["mass"] = s["mass"]
    return r


def _plain_append(s):
    c = s["case"]
    slot, i = s["slots"].long(), s["index"].long()
    page, off = s["table"][slot, i // c["page"]].long(), i % c["page"]
    for pool, new, div in (("k", "kn", "kdiv"), ("v", "vn", "vdiv")):
        x = s[new]
        if c["dtype"] == "fp8":
            x = _stored(x.float() / s[div], "fp8")
            s[pool][0].view(torch.uint8)[page, :, off] = x.view(torch.uint8)
        else:
            s[pool][0][page, :, off] = x
    s["mass"][0][slot, :, i] = 0.0
    s["pos"][0][slot, :, i] = s["position"][:, None].expand(-1, c["kv_heads"])
    return {n: s[n] for n in ("k", "v", "mass", "pos")}


def _plain_plan(s):
    c = s["case"]
    n, budget, T, most = s["len"], c["budget"], c["n"], s["most"]
    slot = s["slots"].long()
    mass, pos = s["mass"][:, slot, :, :T], s["pos"][:, slot, :, :T]
    t = torch.arange(T, device=DEV)
    safe = (pos < c["sink"]) | (pos >= (s["next"] - c["recent"])[None, :, None, None])
    key = torch.where(mass > 0, mass, torch.zeros_like(mass)).view(torch.int32).long()
    key = torch.where(safe, torch.full_like(key, 0xFFFFFFFF), key)
    key = torch.where(t < n[None, :, None, None], key, torch.full_like(key, -1))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, t.expand_as(order).contiguous())
    over = (n > budget)[None, :, None, None]
    keep = rank < budget
    free = ~keep & (t < budget) & over
    move = keep & (t >= budget) & over
    count = move.sum(dim=-1)
    lists = []
    for flag in (move, free):
        at = torch.where(flag, flag.cumsum(-1) - 1, torch.full_like(rank, most)).clamp(max=most)
        got = torch.zeros(*flag.shape[:3], most + 1, dtype=torch.long, device=DEV)
        lists.append(got.scatter_(-1, at, t.expand_as(at).contiguous())[..., :most])
    moves = torch.stack(lists, dim=-1)
    moves = torch.where((t[:most] < count[..., None])[..., None], moves, torch.full_like(moves, -1))
    return {"n_moves": count.to(torch.int32), "moves": moves.to(torch.int32),
            "len_out": torch.clamp(n, max=budget)}


def _plain_apply(s):
    c = s["case"]
    L, B, H, most = c["layers"], c["batch"], c["kv_heads"], s["most"]
    used = torch.arange(most, device=DEV) < s["n_moves"][..., None]
    slot = s["slots"].long()[None, :, None, None]
    layer = torch.arange(L, device=DEV)[:, None, None, None]
    head = torch.arange(H, device=DEV)[None, None, :, None]
    at = []
    for j in range(2):
        # an unused entry copies the first row of the unused page 0 onto itself
        i = torch.where(used, s["moves"][..., j].long(), torch.zeros((), dtype=torch.long, device=DEV))
        page = torch.where(used, s["table"][slot, i // c["page"]].long(), torch.zeros_like(i))
        at.append((torch.where(used, slot, torch.zeros_like(slot)), i, page, i % c["page"]))
    (ss, si, sp, so), (ds, di, dp, do) = at
    for n in ("k", "v"):
        x = s[n].view(torch.uint8) if c["dtype"] == "fp8" else s[n]
        x[layer, dp, head, do] = x[layer, sp, head, so]
    for n in ("mass", "pos"):
        s[n][layer, ds, head, di] = s[n][layer, ss, head, si]
    return {n: s[n] for n in ("k", "v", "mass", "pos")}


def _rms(x, eps):
    return x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + eps)


def _plain_norm(s):
    c = s["case"]
    u = s["y"].float()
    if s["w_post"] is not None:
        u = _rms(u, s["eps"]) * s["w_post"].float()
    if s["gate"] is not None:
        z = s["gate"].float()
        e = 1.0 / (1.0 + torch.exp(-z))
        u = u * (z * e if c["gate"] == "silu" else e)
    u = u * s["scale"]
    r = {}
    if s["residual"] is not None:
        u = s["residual"].float() + u
        r["residual"] = u.to(s["residual"].dtype)
    if s["w_pre"] is not None:
        u = _rms(u, s["eps"]) * s["w_pre"].float()
    r["out"] = u.to(torch.bfloat16)
    return r


# --------------------------------------------------------------------- run --
def _run_own(s):
    import gated_delta_rule_slot_amd as gdn

    c = s["case"]
    if c["op"] == "attn":
        gdn.attn_decode_paged(s["pool"], 0, s["slots"], s["len"], s["q"], s["out"], c["hi"],
                              kv_begin=s["begin"], scale=s["scale"], flags=s["flags"], lse=s["lse"],
                              workspace=s["ws"])
        r = {"out": s["out"], "lse": s["lse"]}
        if c["mass"]:
            r["mass"] = s["mass"]
        return r
    if c["op"] == "append":
        gdn.kv_append(s["pool"], 0, s["slots"], s["index"], s["kn"], s["vn"], position=s["position"])
        return {n: s[n] for n in ("k", "v", "mass", "pos")}
    if c["op"] == "plan":
        gdn.kv_evict_plan(s["pool"], 0, c["layers"], s["slots"], s["len"], s["next"], c["n"],
                          c["budget"], c["sink"], c["recent"], s["n_moves"], s["moves"], s["len_out"])
        return {n: s[n] for n in ("n_moves", "moves", "len_out")}
    if c["op"] == "apply":
        gdn.kv_evict_apply(s["pool"], 0, c["layers"], s["slots"], s["n_moves"], s["moves"])
        return {n: s[n] for n in ("k", "v", "mass", "pos")}
    gdn.block_norm(s["y"], s["out"], w_post=s["w_post"], gate=s["gate"], act=s["act"],
                   scale=s["scale"], residual=s["residual"], residual_out=s["res_out"],
                   w_pre=s["w_pre"], eps=s["eps"])
    r = {"out": s["out"]}
    if s["residual"] is not None:
        r["residual"] = s["res_out"]
    return r


def run(state):
    if own:
        return _run_own(state)
    return {"attn": _plain_attn, "append": _plain_append, "plan": _plain_plan, "apply": _plain_apply,
            "norm": _plain_norm}[state["case"]["op"]](state)


# -------------------------------------------------------------------- work --
def work(case):
    c = case
    size = 2 if c.get("dtype") == "bf16" else 1
    if c["op"] == "attn":
        mean = (c["lo"] + c["hi"]) / 2  # lengths are uniform in [lo, hi], the first one is hi
        if c["begin"]:  # the last 4096 tokens are seen
            lens = range(c["lo"], c["hi"] + 1, max(1, (c["hi"] - c["lo"]) // 1000))
            mean = sum(min(n, 4096) for n in lens) / len(lens)
        tokens = mean * (c["batch"] - c["pad"])
        row = c["kv_heads"] * c["dim"]
        rows = c["batch"] * row * c["group"]
        return {"bytes": tokens * (2 * row * size + (8 * c["kv_heads"] if c["mass"] else 0)) + 4 * rows
                + 4 * rows / c["dim"], "flops": 4 * tokens * row * c["group"]}
    if c["op"] == "append":
        row = c["tokens"] * c["kv_heads"] * c["dim"]
        return {"bytes": 2 * row * (2 + size) + c["tokens"] * (12 + 8 * c["kv_heads"]), "flops": 2 * row}
    if c["op"] in ("plan", "apply"):
        units = c["layers"] * c["batch"] * c["kv_heads"]
        # the weights hold no order: the kept are spread evenly over what is neither recent nor first
        free = max(1, c["n"] - c["recent"] - c["sink"])
        tail = max(0, c["n"] - c["budget"] - c["recent"])
        kept = max(0, c["budget"] - c["recent"] - c["sink"])
        moves = min(c["recent"], c["n"] - c["budget"]) + tail * kept / free
        if c["op"] == "plan":
            return {"bytes": units * (8 * c["n"] + 8 * moves), "flops": 0}
        return {"bytes": units * moves * (4 * c["dim"] * size + 16 + 8), "flops": 0}
    elements = c["tokens"] * c["groups"] * c["dim"]
    res = {"none": 0, "bf16": 4, "f32": 8}[c["residual"]]
    return {"bytes": elements * (2 + 2 + res + (2 if c["gate"] != "none" else 0)), "flops": 10 * elements}


# ------------------------------------------------------- 64-bit definitions --
def _exact_attn(c, s):
    B, H, G, D, ps = c["batch"], c["kv_heads"], c["group"], c["dim"], c["page"]
    out = torch.zeros(B, H * G, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, H * G), -math.inf, dtype=torch.float64, device=DEV)
    mass = s["mass"].double() if c["mass"] else None
    slots, lens = s["slots"].tolist(), s["len"].tolist()
    begins = s["begin"].tolist() if s["begin"] is not None else [0] * B
    for b in range(B):
        lo, hi = begins[b], lens[b]
        if slots[b] <= 0 or lo >= hi:
            continue
        first = lo // ps
        ids = s["table"][slots[b], first:-(-hi // ps)].long()
        for h in range(H):
            k, v = (s[n][0, :, h].view(torch.uint8 if c["dtype"] == "fp8" else torch.int16)[ids]
                    .view(s[n].dtype).reshape(-1, D)[lo - first * ps:hi - first * ps].double()
                    for n in ("k", "v"))
            q = s["q"][b, h * G:(h + 1) * G].double()
            x = (k @ q.t()).t() * (s["kscale"] * s["scale"])
            p = torch.softmax(x, dim=-1)
            out[b, h * G:(h + 1) * G] = (p @ v) * s["vscale"]
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(x, dim=-1)
            if mass is not None:
                mass[0, slots[b], h, lo:hi] += p.sum(dim=0)
    r = {"out": out, "lse": lse}
    if mass is not None:
        r["mass"] = mass
    return r


def _exact_append(c, s):
    r = {n: s[n].double() for n in ("k", "v", "mass")}
    slots, index = s["slots"].long(), s["index"].long()
    page, off = s["table"][slots, index // c["page"]].long(), index % c["page"]
    for h in range(c["kv_heads"]):
        for n, new, scale in (("k", "kn", "kscale"), ("v", "vn", "vscale")):
            x = s[new][:, h].double() / s[scale]
            r[n][0, page, h, off] = x.clamp(-F8_MAX, F8_MAX) if c["dtype"] == "fp8" else x
        r["mass"][0, slots, h, index] = 0
    r["pos"] = None
    return r


def _exact_apply(c, s):
    r = {n: s[n].double() for n in ("k", "v", "mass")}
    slots, ps = s["slots"].tolist(), c["page"]
    counts = s["n_moves"].tolist()
    for la in range(c["layers"]):
        for b in range(c["batch"]):
            for h in range(c["kv_heads"]):
                mv = s["moves"][la, b, h, :counts[la][b][h]].long()
                src, dst = mv[:, 0], mv[:, 1]
                row = s["table"][slots[b]].long()
                for n in ("k", "v"):
                    r[n][la, row[dst // ps], h, dst % ps] = r[n][la, row[src // ps], h, src % ps]
                r["mass"][la, slots[b], h, dst] = r["mass"][la, slots[b], h, src]
    r["pos"] = None
    return r


def _exact_norm(c, s):
    x = s["y"].double()
    if c["post"]:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["dim"] + s["eps"]) * s["w_post"].double()
    if c["gate"] != "none":
        z = s["gate"].double()
        x = x * torch.sigmoid(z) * (z if c["gate"] == "silu" else 1.0)
    x = x * s["scale"]
    r = {}
    if c["residual"] != "none":
        x = x + s["residual"].double()
        r["residual"] = x
    if c["pre"]:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["dim"] + s["eps"]) * s["w_pre"].double()
    r["out"] = x
    return r


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers only
    s = prepare(case, seed)
    return {"attn": _exact_attn, "append": _exact_append, "apply": _exact_apply,
            "norm": _exact_norm}[case["op"]](case, s)
