"""GPU: the paged cache's append, attention and eviction against their float64 definitions
(oracle/kv_ops.py).  Tolerances: tests/kv_helpers.py."""
import numpy as np
import pytest
import torch

from oracle import kv_ops
from tests.kv_helpers import attend_all, check_attention, device_pool, i32, make_cache, stored

pytestmark = pytest.mark.gpu


def run_attention(c, group, seed=1, mass=False, lse=True, q_pad=0, scale=None, max_len=None, stream=None, pool=None,
                  q_std=1.0):
    import gated_delta_rule_slot_amd as gdn

    B, Hq = len(c.lens), c.kv_heads * group
    g = torch.Generator().manual_seed(seed)
    wide = (q_std * torch.randn(B, Hq * c.dim + q_pad, generator=g)).to(torch.bfloat16).cuda()
    q = wide[:, q_pad:].view(B, Hq, c.dim)
    pool = pool or device_pool(c)
    out = torch.full((B, Hq, c.dim), -7.0, dtype=torch.bfloat16, device="cuda")
    lv = torch.full((B, Hq), -7.0, device="cuda") if lse else None
    ml = max(c.lens) if max_len is None else max_len
    flags = gdn.ATTN_ACCUM_MASS if mass else 0
    n = gdn.attn_workspace_bytes(pool, B, Hq, ml, flags)
    ws = torch.full((n,), 0xff, dtype=torch.uint8, device="cuda") if n else None
    sc = c.dim ** -0.5 if scale is None else scale
    begin = i32(c.begins) if any(c.begins) else None
    gdn.attn_decode_paged(pool, c.layer, i32(c.slots), i32(c.lens), q, out, ml, kv_begin=begin, scale=sc,
                          flags=flags, lse=lv, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    return pool, q.cpu(), out, lv, sc


CASES = [
    # dim, kv_heads, group, page, fp8, lens, begins
    (64, 1, 1, 16, False, [1], None),
    (64, 2, 3, 1, False, [33, 64, 2], None),
    (128, 2, 4, 16, False, [0, 31, 32, 129], None),
    (128, 1, 16, 32, False, [500, 7], [0, 6]),
    (128, 3, 5, 8, False, [127, 128, 255], [100, 128, 33]),
    (256, 2, 8, 64, False, [300, 65, 1], None),
    (256, 1, 12, 128, False, [777], [31]),
    (64, 1, 17, 4, False, [90, 40], None),
    (128, 1, 40, 64, False, [140], None),
    (64, 1, 64, 2, False, [70], [3]),
    (64, 2, 2, 16, True, [100, 1, 45], None),
    (128, 2, 7, 32, True, [64, 333], [0, 300]),
    (256, 1, 16, 1024, True, [1100, 90], None),
    (256, 2, 1, 2, True, [61], [60]),
]


@pytest.mark.parametrize("mass", [False, True])
@pytest.mark.parametrize("dim,kv_heads,group,page,f8,lens,begins", CASES)
def test_attention_parity(dim, kv_heads, group, page, f8, lens, begins, mass):
    c = make_cache(dim + group + page, lens, begins, kv_heads, dim, page, f8)
    pool, q, out, lse, sc = run_attention(c, group, mass=mass, q_pad=8 * (group % 3))
    check_attention(c, q, sc, out, lse, pool.mass if mass else None, c.mass)
    if not mass:
        assert torch.equal(pool.mass.cpu(), c.mass)
    assert int(pool.err_word.item()) == 0


@pytest.mark.parametrize("f8,dim,group", [(False, 128, 8), (False, 256, 8), (True, 128, 4), (False, 64, 2)])
def test_attention_many_splits(f8, dim, group):
    """One request of thousands of tokens (many splits, several tiles a wave) beside short
    and empty ones, with a bound far above the lengths, and a second layer."""
    c = make_cache(5, [5003, 0, 70], [0, 0, 64], 1, dim, 64, f8, layers=2, layer=1, capacity=9000)
    pool, q, out, lse, sc = run_attention(c, group, mass=True, max_len=9000)
    check_attention(c, q, sc, out, lse, pool.mass, c.mass)
    # the same without weights, and with the closest bound: another number of splits
    _, q2, out2, lse2, _ = run_attention(c, group, mass=False, max_len=5003)
    check_attention(c, q2, sc, out2, lse2)


@pytest.mark.parametrize("seed", range(8))
def test_attention_random_cases(seed):
    r = np.random.default_rng(900 + seed)
    dim = int(r.choice([64, 128, 256]))
    kv_heads, group = int(r.integers(1, 4)), int(r.integers(1, 20))
    lens = [int(x) for x in r.integers(0, 700, size=r.integers(1, 6))]
    if max(lens) == 0:
        lens[0] = 1
    begins = [int(r.integers(0, n + 2)) if r.random() < 0.4 else 0 for n in lens]
    c = make_cache(seed, lens, begins, kv_heads, dim, int(2 ** r.integers(0, 9)), bool(r.random() < 0.5),
                   k_std=float(r.choice([0.1, 1.0, 3.0])))
    pool, q, out, lse, sc = run_attention(c, group, seed=seed, mass=True, q_pad=16)
    check_attention(c, q, sc, out, lse, pool.mass, c.mass)


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_attention_scales(scale):
    """A zero scale averages the values, a negative one turns the order, a large one picks
    nearly one token."""
    c = make_cache(11, [77, 200], None, 2, 128, 16)
    pool, q, out, lse, sc = run_attention(c, 4, mass=True, scale=scale)
    check_attention(c, q, sc, out, lse, pool.mass, c.mass)


def test_attention_infinite_scores():
    """A key of -inf scores leaves its token out; where all are -inf the row is empty; a
    +inf or NaN score makes that head's row NaN."""
    c = make_cache(3, [40, 40, 40], None, 1, 64, 8)
    c.mass.zero_()
    t = c.table[c.slots[0]]
    c.k[0, int(t[0]), 0, 3, 0] = float("inf")
    for i in range(40):
        c.k[0, int(c.table[c.slots[1]][i // 8]), 0, i % 8, 0] = float("inf")
    c.k[0, int(c.table[c.slots[2]][2]), 0, 1, 0] = float("inf")
    import gated_delta_rule_slot_amd as gdn

    pool = device_pool(c)
    g = torch.Generator().manual_seed(0)
    q = torch.randn(3, 2, 64, generator=g).to(torch.bfloat16)
    q[:, :, 0] = -1.0
    q[2, 0, 0], q[2, 1, 0] = 1.0, -1.0
    out = torch.empty(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(3, 2, device="cuda")
    ws = torch.empty(gdn.attn_workspace_bytes(pool, 3, 2, 40, 1), dtype=torch.uint8, device="cuda")
    gdn.attn_decode_paged(pool, 0, i32(c.slots), i32(c.lens), q.cuda(), out, 40, scale=0.125, flags=1, lse=lse,
                          workspace=ws)
    w = pool.mass.cpu()
    assert torch.isfinite(out[0].float()).all() and float(w[0, c.slots[0], 0, 3]) == 0.0
    assert abs(float(w[0, c.slots[0], 0, :40].sum()) - 2) < 1e-4
    assert not out[1].float().any() and torch.isneginf(lse[1]).all() and not w[0, c.slots[1]].any()
    assert torch.isnan(out[2, 0].float()).all() and torch.isnan(lse[2, 0])
    assert torch.isfinite(out[2, 1].float()).all() and torch.isfinite(lse[2, 1])


def test_attention_skips_and_flags():
    """Padding and bad slots, bad lengths and begins, bad pages."""
    import gated_delta_rule_slot_amd as gdn

    lens = [50, 60, 70, 80, 90, 100]
    c = make_cache(21, lens, None, 2, 128, 16, slots=[1, 0, 3, 2, 4, 5])
    c.table[5, 2] = 0             # places 32..47 of the last request
    c.table[5, 4] = c.k.shape[1]  # and 64..79
    pool = device_pool(c)
    slots = [1, 0, c.n_slots + 4, 2, -3, 5]
    B, Hq = 6, 8
    q = torch.randn(B, Hq, 128, generator=c.g).to(torch.bfloat16)

    def call(kv_len, begin, max_len):
        pool.err_word.zero_()
        pool.mass.copy_(c.mass)
        out = torch.full((B, Hq, 128), -7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((B, Hq), -7.0, device="cuda")
        ws = torch.empty(gdn.attn_workspace_bytes(pool, B, Hq, max_len, 1), dtype=torch.uint8, device="cuda")
        gdn.attn_decode_paged(pool, 0, i32(slots), i32(kv_len), q.cuda(), out, max_len, kv_begin=begin, scale=0.1,
                              flags=1, lse=lse, workspace=ws)
        return out, lse

    out, lse = call(lens, None, 112)
    c.slots = slots
    check_attention(c, q, 0.1, out, lse, pool.mass, c.mass)
    assert int(pool.err_word.item()) == gdn.ERRW_BAD_SLOT | gdn.ERRW_BAD_PAGE
    # too long, negative, negative begin: skipped like padding
    out, lse = call([50, 60, 70, -1, 90, 100], i32([-1, 0, 0, 0, 0, 0]), 99)
    assert not out.float().any() and torch.isneginf(lse).all() and torch.equal(pool.mass.cpu(), c.mass)
    assert int(pool.err_word.item()) & gdn.ERRW_BAD_SEQLENS


def test_attention_all_requests_empty():
    c = make_cache(2, [0, 0], None, 2, 64, 16)
    pool, q, out, lse, _ = run_attention(c, 2, mass=True)
    assert not out.float().any() and torch.isneginf(lse).all()
    assert torch.equal(pool.mass.cpu(), c.mass) and int(pool.err_word.item()) == 0


def test_attention_runs_are_bit_identical():
    c = make_cache(8, [3000, 40], None, 2, 128, 32)
    first = None
    for _ in range(3):
        pool, _, out, lse, _ = run_attention(c, 8, mass=True)
        now = (out.cpu(), lse.cpu(), pool.mass.cpu())
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))


def test_attention_without_err_word_and_lse():
    c = make_cache(4, [20], None, 1, 64, 16, slots=[1])
    c.table[1, 1] = -5
    pool = device_pool(c, mass=False, err=False)
    _, q, out, _, sc = run_attention(c, 1, lse=False, pool=pool)
    check_attention(c, q, sc, out)


@pytest.mark.parametrize("batch,mass", [(255, True), (257, False), (700, True)])
def test_attention_many_requests(batch, mass):
    """More requests than one step of the length scan takes, with empty and skipped ones
    between them."""
    r = np.random.default_rng(batch)
    lens = [int(x) for x in r.integers(0, 60, size=batch)]
    lens[batch // 2] = 900
    slots = [int(x) + 1 for x in r.permutation(batch)]
    for b in range(3, batch, 7):
        slots[b] = -(b % 2)
    c = make_cache(batch, lens, None, 1, 64, 16, slots=slots)
    pool, q, out, lse, sc = run_attention(c, 3, mass=mass)
    check_attention(c, q, sc, out, lse, pool.mass if mass else None, c.mass)
    assert int(pool.err_word.item()) == 0


def test_attention_largest_batch():
    """65535 requests of 64 heads (more joins than one grid dimension takes) over the same
    rows, against a float64 softmax on the device for some of them."""
    import gated_delta_rule_slot_amd as gdn

    B, Hq, D, n = 65535, 64, 64, 130
    g = torch.Generator(device="cuda").manual_seed(3)
    k = torch.randn(1, 20, 1, 16, D, device="cuda", generator=g).to(torch.bfloat16)
    v = torch.randn(1, 20, 1, 16, D, device="cuda", generator=g).to(torch.bfloat16)
    table = (torch.arange(9, device="cuda", dtype=torch.int32) + 2).expand(B + 1, 9).contiguous()
    pool = gdn.kv_pool_create(k, v, table)
    q = torch.randn(B, Hq, D, device="cuda", generator=g).to(torch.bfloat16)
    lens = (torch.arange(B, device="cuda", dtype=torch.int32) % (n + 1))
    out = torch.full((B, Hq, D), -7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(gdn.attn_workspace_bytes(pool, B, Hq, n), dtype=torch.uint8, device="cuda")
    gdn.attn_decode_paged(pool, 0, torch.arange(1, B + 1, dtype=torch.int32, device="cuda"), lens, q, out, n, scale=0.125,
                          workspace=ws)
    rows_k, rows_v = (t[0, 2:11, 0].reshape(-1, D).double() for t in (k, v))
    for b in list(range(0, 262)) + list(range(0, B, 997)) + list(range(B - 132, B)):
        m = int(lens[b])
        got = out[b].double()
        if m == 0:
            assert not got.any(), b
            continue
        p = torch.softmax(0.125 * q[b].double() @ rows_k[:m].t(), -1)
        want = p @ rows_v[:m]
        # 2^-8 for bf16; 2^-12 of sum p |v| covers kv_helpers.attn_slack for these sizes
        assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -12 * (p @ rows_v[:m].abs())).all(), b


@pytest.mark.parametrize("f8", [False, True])
def test_offsets_past_32_bits(f8):
    """Pages at the far end of a cache of more than 2^32 bytes, through append, attention
    and an eviction's moves."""
    import gated_delta_rule_slot_amd as gdn

    H, S, D = 2, 64, 256
    pages = 150000 if f8 else 70000   # 4.9 / 4.6 GB each for k and v; fp8 rows * D pass 2^32 too
    dt = torch.float8_e4m3fn if f8 else torch.bfloat16
    k = torch.empty(1, pages, H, S, D, dtype=dt, device="cuda")
    v = torch.empty(1, pages, H, S, D, dtype=dt, device="cuda")
    ids = [pages - 1, pages - 3]
    table = i32([[0, 0], ids])
    mass = torch.zeros(1, 2, H, 128, device="cuda")
    pos = torch.zeros(1, 2, H, 128, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pool = gdn.kv_pool_create(k, v, table, mass=mass, pos=pos, err_word=err)
    n = 100
    g = torch.Generator().manual_seed(6)
    kn, vn = (torch.randn(n, H, D, generator=g).to(torch.bfloat16) for _ in range(2))
    at = torch.arange(n, dtype=torch.int32).cuda()
    gdn.kv_append(pool, 0, torch.ones(n, dtype=torch.int32).cuda(), at, kn.cuda(), vn.cuda(), position=at)
    got = torch.cat([k[0, i].view(torch.uint8 if f8 else torch.int16) for i in ids], 1)[:, :n].cpu()
    want = (stored(kn.float(), f8)).transpose(0, 1).contiguous()
    assert torch.equal(got, want.view(torch.uint8 if f8 else torch.int16))
    q = torch.randn(1, 2 * H, D, generator=g).to(torch.bfloat16)
    out = torch.empty(1, 2 * H, D, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(gdn.attn_workspace_bytes(pool, 1, 2 * H, n), dtype=torch.uint8, device="cuda")
    gdn.attn_decode_paged(pool, 0, i32([1]), i32([n]), q.cuda(), out, n, scale=D ** -0.5, workspace=ws)
    c = make_cache(1, [n], None, H, D, S, f8, slots=[1])
    c.k_scale = c.v_scale = 1.0
    for i in range(n):
        c.k[0, c.table[1, i // S], :, i % S] = stored(kn[i].float(), f8)
        c.v[0, c.table[1, i // S], :, i % S] = stored(vn[i].float(), f8)
    check_attention(c, q, D ** -0.5, out)
    moves = i32([[[[[99, 0], [70, 5]]] * H]])
    gdn.kv_evict_apply(pool, 0, 1, i32([1]), i32([[[2] * H]]), moves)
    b = k.view(torch.uint8) if f8 else k.view(torch.int16)
    assert torch.equal(b[0, ids[0], :, 0], b[0, ids[1], :, 35]) and torch.equal(b[0, ids[0], :, 5], b[0, ids[1], :, 6])
    assert int(err.item()) == 0


# ------------------------------------------------------------------ append --
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("dim,kv_heads,page,n,pad", [(64, 1, 1, 1, 0), (128, 3, 16, 77, 8), (256, 2, 64, 300, 0)])
def test_append_matches_definition_and_touches_nothing_else(f8, dim, kv_heads, page, n, pad):
    import gated_delta_rule_slot_amd as gdn

    lens = [max(n, 5), 40, 33]
    c = make_cache(n, lens, None, kv_heads, dim, page, f8, layers=2)
    c.k_scale, c.v_scale = (0.37, 2.9) if f8 else (1.0, 1.0)
    pool = device_pool(c)
    g = torch.Generator().manual_seed(n)
    pick = torch.randperm(sum(lens), generator=g)[:n]
    where = [(c.slots[b], i) for b in range(3) for i in range(lens[b])]
    where = [where[j] for j in pick.tolist()]
    wide = 40.0 * torch.randn(n, 2 * kv_heads * dim + pad, generator=g)
    wide[torch.rand(wide.shape, generator=g) < 0.05] = 1e6
    wide[torch.rand(wide.shape, generator=g) < 0.02] = float("nan")
    wide[torch.rand(wide.shape, generator=g) < 0.1] *= 1e-4
    wide = wide.to(torch.bfloat16)
    kn = wide[:, :kv_heads * dim].view(n, kv_heads, dim)
    vn = wide[:, kv_heads * dim + pad:].view(n, kv_heads, dim)
    position = torch.randint(0, 1 << 30, (n,), generator=g, dtype=torch.int32)
    dev = wide.cuda()
    gdn.kv_append(pool, 1, i32([s for s, _ in where]), i32([i for _, i in where]),
                  dev[:, :kv_heads * dim].view(n, kv_heads, dim),
                  dev[:, kv_heads * dim + pad:].view(n, kv_heads, dim), position=position.cuda())
    raw = torch.uint8 if f8 else torch.int16
    for name, new, scale in (("k", kn, c.k_scale), ("v", vn, c.v_scale)):
        want = getattr(c, name).clone()
        for j, (s, i) in enumerate(where):
            x = new[j]
            if f8:
                x = (x.float().numpy() / np.float32(scale)).astype(np.float64)  # divided in fp32
                x = torch.from_numpy(kv_ops.e4m3_round(x)).float().to(torch.float8_e4m3fn)
            want[1, c.table[s, i // page], :, i % page] = x
        got = getattr(pool, name).cpu()
        nan = torch.isnan(want.float())
        assert torch.equal(torch.isnan(got.float()), nan)
        assert torch.equal(got.view(raw)[~nan], want.view(raw)[~nan])
    mass, pos = c.mass.clone(), c.pos.clone()
    for j, (s, i) in enumerate(where):
        mass[1, s, :, i], pos[1, s, :, i] = 0.0, position[j]
    assert torch.equal(pool.mass.cpu(), mass) and torch.equal(pool.pos.cpu(), pos)
    assert int(pool.err_word.item()) == 0


@pytest.mark.parametrize("k_scale,v_scale", [(1.0, 1.0 / 3), (0.0123, 7.77), (2.0 ** -9, 1.9999999), (1e-3, 448.0),
                                             (1e-30, 1e30), (1.17e-38, 3e38), (1e20, 2.0 ** -60)])
def test_append_divides_every_bf16_value_as_fp32_does(k_scale, v_scale):
    """All 65536 bf16 values by several scales, against numpy's fp32 division."""
    import gated_delta_rule_slot_amd as gdn

    bits = torch.arange(65536, dtype=torch.int32)
    x = (bits << 16).view(torch.float32).to(torch.bfloat16).view(512, 1, 128)
    pages, S = 33, 16
    k = torch.zeros(1, pages, 1, S, 128, dtype=torch.float8_e4m3fn, device="cuda")
    v = torch.zeros_like(k)
    table = torch.zeros(2, 32, dtype=torch.int32)
    table[1] = torch.arange(32) + 1
    pool = gdn.kv_pool_create(k, v, table.cuda(), k_scale=k_scale, v_scale=v_scale)
    at = torch.arange(512, dtype=torch.int32).cuda()
    gdn.kv_append(pool, 0, torch.ones(512, dtype=torch.int32).cuda(), at, x.cuda(), x.cuda())
    xf = x.float().numpy().reshape(-1)
    for t, s in ((k, k_scale), (v, v_scale)):
        with np.errstate(over="ignore", invalid="ignore"):
            want = kv_ops.e4m3_round((xf / np.float32(s)).astype(np.float64))
        got = t[0, 1:].float().cpu().double().numpy().reshape(-1)
        nan = np.isnan(want)
        assert np.array_equal(np.isnan(got), nan)
        assert np.array_equal(got[~nan], want[~nan])


def test_append_skips_and_flags():
    import gated_delta_rule_slot_amd as gdn

    c = make_cache(9, [40, 40], None, 2, 64, 16, slots=[1, 2])
    c.table[2, 1] = 0
    pool = device_pool(c)
    x = torch.ones(6, 2, 64, dtype=torch.bfloat16, device="cuda")
    p = torch.arange(6, dtype=torch.int32, device="cuda")
    for slots, index, bit in (([0, -1, 0, 0, 0, 0], [1] * 6, 0), ([c.n_slots] * 6, [1] * 6, gdn.ERRW_BAD_SLOT),
                              ([1] * 6, [-1, c.cap, 2 ** 31 - 1, -2 ** 31, -1, c.cap], gdn.ERRW_BAD_SEQLENS),
                              ([2] * 6, [16, 17, 20, 31, 30, 29], gdn.ERRW_BAD_PAGE)):
        pool.err_word.zero_()
        gdn.kv_append(pool, 0, i32(slots), i32(index), x, x, position=p)
        assert int(pool.err_word.item()) == bit
        assert torch.equal(pool.k.cpu().view(torch.int16), c.k.view(torch.int16))
        assert torch.equal(pool.mass.cpu(), c.mass) and torch.equal(pool.pos.cpu(), c.pos)
    gdn.kv_append(pool, 0, i32([]), i32([]), x[:0], x[:0], position=i32([]))


# ---------------------------------------------------------------- eviction --
def plan_case(seed, n_list, budget, sink, recent, kv_heads=2, layers=2, weights="exp", cap=None, dim=64, page=16):
    g = torch.Generator().manual_seed(seed)
    c = make_cache(seed, n_list, None, kv_heads, dim, page, layers=layers, capacity=cap)
    shape = c.mass.shape
    if weights == "exp":
        c.mass = torch.exp(3 * torch.randn(shape, generator=g))
    elif weights == "few":       # many ties
        c.mass = torch.randint(0, 3, shape, generator=g).float()
    elif weights == "same":
        c.mass = torch.full(shape, 0.25)
    elif weights == "close":     # neighbours in fp32
        c.mass = (torch.randint(0, 40, shape, generator=g) + 0x3f800000).to(torch.int32).view(torch.float32)
    elif weights == "odd":       # NaN, negative, infinite, subnormal, zeros of both signs
        c.mass = torch.exp(torch.randn(shape, generator=g))
        for k, x in enumerate((float("nan"), -3.0, float("inf"), 1e-42, 0.0, -0.0, 1e38)):
            c.mass[torch.rand(shape, generator=g) < 0.12] = x
    c.pos = torch.argsort(torch.rand(shape, generator=g), dim=-1).to(torch.int32)
    return c


def run_plan(c, budget, sink, recent, next_pos, lb=0, le=None, max_len=None, max_moves=None, kv_len=None, pool=None):
    import gated_delta_rule_slot_amd as gdn

    pool = pool or device_pool(c)
    le = c.mass.shape[0] if le is None else le
    B, H = len(c.lens), c.kv_heads
    ml = max(c.lens) if max_len is None else max_len
    M = max(0, min(budget, ml - budget)) if max_moves is None else max_moves
    nm = torch.full((le - lb, B, H), -9, dtype=torch.int32, device="cuda")
    mv = torch.full((le - lb, B, H, M, 2), -9, dtype=torch.int32, device="cuda")
    lo = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    gdn.kv_evict_plan(pool, lb, le, i32(c.slots), i32(c.lens if kv_len is None else kv_len), i32(next_pos), ml,
                      budget, sink, recent, nm, mv, lo)
    return pool, nm.cpu(), mv.cpu(), lo.cpu()


def check_plan(c, budget, sink, recent, next_pos, nm, mv, lo, lb=0):
    mass, pos = c.mass.numpy(), c.pos.numpy()
    for b, n in enumerate(c.lens):
        live = 0 < c.slots[b] < c.n_slots
        assert int(lo[b]) == (min(n, budget) if live else n)
        for la in range(nm.shape[0]):
            for h in range(c.kv_heads):
                want = kv_ops.plan(mass[la + lb, c.slots[b], h], pos[la + lb, c.slots[b], h], n, next_pos[b], budget,
                                   sink, recent) if live else []
                assert int(nm[la, b, h]) == len(want), (la, b, h)
                got = mv[la, b, h]
                assert [tuple(x) for x in got[:len(want)].tolist()] == want, (la, b, h)
                assert (got[len(want):] == -9).all()


@pytest.mark.parametrize("weights", ["exp", "few", "same", "close", "odd"])
@pytest.mark.parametrize("n_list,budget,sink,recent", [
    ([1, 2, 0], 1, 0, 0), ([100, 64, 65], 64, 4, 10), ([2048, 2047, 1025], 700, 0, 0), ([1500, 3], 1024, 1000, 24),
    ([5000, 4100], 4096, 4, 64), ([9000], 100, 0, 33), ([33000, 32769], 8192, 4, 500), ([40000], 39999, 0, 0)])
def test_plan_parity(weights, n_list, budget, sink, recent):
    small = max(n_list) < 3000
    c = plan_case(len(n_list) + budget, n_list, budget, sink, recent, kv_heads=2 if small else 1,
                  layers=2 if small else 1, weights=weights)
    nxt = [c.cap] * len(n_list)
    pool, nm, mv, lo = run_plan(c, budget, sink, recent, nxt)
    check_plan(c, budget, sink, recent, nxt, nm, mv, lo)
    assert int(pool.err_word.item()) == 0


@pytest.mark.parametrize("n", [1100, 2048, 4200, 38000])
@pytest.mark.parametrize("budget", [1, 63, 64, 65, 127, 128, 129, 191, 255, 256, 257, 320, 511, 512, 513, 1023, 1024,
                                    1025])
def test_plan_budgets_inside_a_step(n, budget):
    """The budget's place in a wave's rounds, with few and with many tokens kept past it."""
    c = plan_case(n + budget, [n, n - 37], budget, 0, 0, kv_heads=1, layers=1)
    c.mass[0, c.slots[1], :, budget - budget // 4:] += 1e4  # most of the kept lie past the budget
    nxt = [c.cap] * 2
    _, nm, mv, lo = run_plan(c, budget, 0, min(budget, 5), nxt)
    check_plan(c, budget, 0, min(budget, 5), nxt, nm, mv, lo)


@pytest.mark.parametrize("n", [700, 2048, 9000, 36864, 36865])
def test_plan_runs_of_equal_weights(n):
    """Runs of one weight, of zeros and of protected tokens beside spread ones, of lengths
    that begin and end anywhere in a wave's rounds; subnormal weights; two large ones."""
    g = torch.Generator().manual_seed(n)
    for kind in range(4):
        c = plan_case(n + kind, [n], n // 3, 4, n // 9, kv_heads=2, layers=1)
        m = c.mass[0, c.slots[0]]
        if kind == 0:
            at = 0
            while at < n:
                run = int(torch.randint(1, 700, (1,), generator=g))
                v = (0.25, 0.0, None, 3.0)[int(torch.randint(0, 4, (1,), generator=g))]
                if v is not None:
                    m[:, at:at + run] = v
                at += run
        elif kind == 1:
            m.copy_(torch.randint(0, 1 << 12, m.shape, generator=g).to(torch.int32).view(torch.float32))
        elif kind == 2:
            m.copy_(torch.where(torch.rand(m.shape, generator=g) < 0.5, 3.4e38, float("inf")))
        else:
            c.pos = torch.arange(c.cap).expand(c.pos.shape).contiguous().to(torch.int32)
            m.fill_(0.5)
        _, nm, mv, lo = run_plan(c, n // 3, 4, n // 9, [n])
        check_plan(c, n // 3, 4, n // 9, [n], nm, mv, lo)


def test_plan_protected_alone_fill_the_budget():
    """Positions that repeat, or a next position too low: more protected than the budget."""
    c = plan_case(7, [900, 300], 128, 4, 60)
    c.pos.fill_(2)
    _, nm, mv, lo = run_plan(c, 128, 4, 60, [900, 300])
    check_plan(c, 128, 4, 60, [900, 300], nm, mv, lo)
    c = plan_case(8, [900, 300], 128, 4, 60)
    nxt = [400, -(2 ** 31)]  # next - recent passes the 32-bit range
    _, nm, mv, lo = run_plan(c, 128, 4, 60, nxt)
    check_plan(c, 128, 4, 60, nxt, nm, mv, lo)


def test_plan_layers_skips_and_flags():
    import gated_delta_rule_slot_amd as gdn

    c = plan_case(31, [200, 210, 220, 230], 100, 2, 8, layers=3)
    nxt = [c.cap] * 4
    pool, nm, mv, lo = run_plan(c, 100, 2, 8, nxt, lb=1, le=3, max_len=232, max_moves=140)
    check_plan(c, 100, 2, 8, nxt, nm, mv, lo, lb=1)
    c.slots = [c.slots[0], 0, c.n_slots + 1, -4]
    pool, nm, mv, lo = run_plan(c, 100, 2, 8, nxt, pool=pool)
    check_plan(c, 100, 2, 8, nxt, nm, mv, lo)
    assert int(pool.err_word.item()) == gdn.ERRW_BAD_SLOT
    pool.err_word.zero_()
    c.slots = [1, 2, 3, 4]
    _, nm, mv, lo = run_plan(c, 100, 2, 8, nxt, pool=pool, max_len=230, kv_len=[231, -1, 101, 100], max_moves=130)
    assert int(pool.err_word.item()) == gdn.ERRW_BAD_SEQLENS
    assert lo.tolist() == [231, -1, 100, 100]
    assert not nm[:, :2].any() and not nm[:, 3].any() and (mv[:, :2] == -9).all()


@pytest.mark.parametrize("f8,dim,page,kv_heads", [(False, 64, 16, 2), (True, 64, 1, 1), (False, 256, 64, 1),
                                                  (True, 256, 8, 3), (False, 128, 32, 2)])
def test_apply_moves_rows_and_nothing_else(f8, dim, page, kv_heads):
    import gated_delta_rule_slot_amd as gdn

    c = make_cache(dim, [500, 120, 90], None, kv_heads, dim, page, f8, layers=3)
    pool = device_pool(c)
    budget = 100
    nxt = [c.cap] * 3
    c.pos = torch.argsort(torch.rand(c.mass.shape, generator=c.g), dim=-1).to(torch.int32)
    pool.pos.copy_(c.pos)
    _, nm, mv, _ = run_plan(c, budget, 4, 20, nxt, lb=1, le=3, pool=pool, max_moves=110)
    gdn.kv_evict_apply(pool, 1, 3, i32(c.slots), nm.cuda(), mv.cuda())
    raw = torch.uint8 if f8 else torch.int16
    k, v, mass, pos = (t.clone() for t in (c.k.view(raw), c.v.view(raw), c.mass, c.pos))
    moved = 0
    for la in range(2):
        for b in range(3):
            row = c.table[c.slots[b]]
            for h in range(kv_heads):
                for s, d in mv[la, b, h, :int(nm[la, b, h])].tolist():
                    for t in (k, v):
                        t[la + 1, row[d // page], h, d % page] = t[la + 1, row[s // page], h, s % page]
                    for t in (mass, pos):
                        t[la + 1, c.slots[b], h, d] = t[la + 1, c.slots[b], h, s]
                    moved += 1
    assert moved > 0
    assert torch.equal(pool.k.cpu().view(raw), k) and torch.equal(pool.v.cpu().view(raw), v)
    assert torch.equal(pool.mass.cpu(), mass) and torch.equal(pool.pos.cpu(), pos)
    assert int(pool.err_word.item()) == 0


def test_apply_skips_and_flags():
    import gated_delta_rule_slot_amd as gdn

    c = make_cache(17, [64, 64], None, 1, 64, 16, slots=[1, 2])
    c.table[2, 3] = 0
    pool = device_pool(c)

    def call(slots, counts, moves):
        pool.err_word.zero_()
        gdn.kv_evict_apply(pool, 0, 1, i32(slots), i32([[[n] for n in counts]]), i32([[[m] for m in moves]]))
        same = torch.equal(pool.k.cpu().view(torch.int16), c.k.view(torch.int16)) \
            and torch.equal(pool.mass.cpu(), c.mass)
        return int(pool.err_word.item()), same

    two = [[[40, 1], [41, 2]], [[40, 1], [41, 2]]]
    assert call([0, -1], [2, 2], two) == (0, True)
    assert call([1, 2], [0, 0], two) == (0, True)
    assert call([c.n_slots, 0], [2, 2], two) == (gdn.ERRW_BAD_SLOT, True)
    assert call([1, 2], [3, -1], two) == (gdn.ERRW_BAD_SEQLENS, True)
    bad = [[[c.cap, 1], [40, -1]], [[-1, 1], [40, c.cap]]]
    assert call([1, 2], [2, 2], bad) == (gdn.ERRW_BAD_SEQLENS, True)
    assert call([0, 2], [0, 2], [two[0], [[50, 1], [2, 48]]]) == (gdn.ERRW_BAD_PAGE, True)
    assert call([1, 0], [1, 0], two) == (0, False)  # a good one moves


def test_append_and_eviction_of_more_workgroups_than_one_grid_dimension_takes():
    import gated_delta_rule_slot_amd as gdn

    # 2^21 workgroups of 256 threads and some: 67.2 M tokens of one head of 64
    n, S = (1 << 26) + 100000, 1024
    pages = -(-n // S) + 1
    x = torch.empty(n, 1, 64, dtype=torch.bfloat16, device="cuda")
    x.view(torch.int32).view(n, 32)[:] = torch.arange(n, dtype=torch.int32, device="cuda")[:, None]
    k = torch.zeros(1, pages, 1, S, 64, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(2, pages)[:, 1:].contiguous()
    pool = gdn.kv_pool_create(k, v, table)
    at = torch.arange(n, dtype=torch.int32, device="cuda")
    gdn.kv_append(pool, 0, torch.ones(n, dtype=torch.int32, device="cuda"), at, x, x)
    for t in (k, v):
        assert torch.equal(t[0, 1:].view(-1, 64)[:n].view(torch.int32), x.view(n, 64).view(torch.int32))
        assert not t[0, 1:].view(-1, 64)[n:].any()
    del k, v, x, pool, at, table
    torch.cuda.empty_cache()

    # 2.1 M lists of one move each: 64 layers, 4100 requests, 8 heads, 17 tokens, budget 16
    L, B, H = 64, 4100, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.zeros(L, 2, H, 32, 64, dtype=torch.float8_e4m3fn, device="cuda")
    mass = torch.rand(L, B + 1, H, 32, device="cuda", generator=g) + 0.1
    pos = torch.arange(32, dtype=torch.int32, device="cuda").expand(L, B + 1, H, 32).contiguous()
    low = torch.randint(0, 16, (L, B, H, 1), device="cuda", generator=g)
    mass[:, 1:, :, :17].scatter_(3, low, 0.01)
    table = torch.ones(B + 1, 1, dtype=torch.int32, device="cuda")
    pool = gdn.kv_pool_create(k, torch.zeros_like(k), table, mass=mass, pos=pos)
    slots = torch.arange(1, B + 1, dtype=torch.int32, device="cuda")
    nm = torch.zeros(L, B, H, dtype=torch.int32, device="cuda")
    mv = torch.zeros(L, B, H, 1, 2, dtype=torch.int32, device="cuda")
    lo = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens = torch.full((B,), 17, dtype=torch.int32, device="cuda")
    gdn.kv_evict_plan(pool, 0, L, slots, lens, lens + 100, 17, 16, 0, 0, nm, mv, lo)
    assert (nm == 1).all() and (lo == 16).all() and (mv[..., 0] == 16).all() and torch.equal(mv[..., 1].long(), low)
    want = pos[:, 1:].clone().scatter_(3, low, 16)
    # (the rows are all in one page and all zero: mass and pos show what was moved)
    gdn.kv_evict_apply(pool, 0, L, slots, nm, mv)
    assert torch.equal(pos[:, 1:], want) and (mass[:, 1:, :, :17] > 0.05).all()


# ------------------------------------------------------- together, as used --
def hybrid_steps(c, pool, layer, steps, budget, group, seed, stream=None):
    """Decode `steps` tokens: append, attend with weights, evict to the budget.  Returns the
    outputs, and everything a host model of the same steps needs."""
    import gated_delta_rule_slot_amd as gdn

    B, H, D = len(c.lens), c.kv_heads, c.dim
    g = torch.Generator().manual_seed(seed)
    kn, vn = (torch.randn(steps, B, H, D, generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(steps, B, H * group, D, generator=g).to(torch.bfloat16)
    slots, length, nxt = i32(c.slots), i32(c.lens), i32(c.lens)
    ml = c.cap
    ws = torch.empty(gdn.attn_workspace_bytes(pool, B, H * group, ml, 1), dtype=torch.uint8, device="cuda")
    nm = torch.zeros(1, B, H, dtype=torch.int32, device="cuda")
    mv = torch.zeros(1, B, H, max(1, min(budget, ml - budget)), 2, dtype=torch.int32, device="cuda")
    len_out = torch.empty_like(length)
    outs = torch.empty(steps, B, H * group, D, dtype=torch.bfloat16, device="cuda")
    kd, vd, qd = kn.cuda(), vn.cuda(), q.cuda()
    for t in range(steps):
        gdn.kv_append(pool, layer, slots, length, kd[t], vd[t], position=nxt)
        length += 1
        nxt += 1
        gdn.attn_decode_paged(pool, layer, slots, length, qd[t], outs[t], ml, scale=D ** -0.5, flags=1, workspace=ws)
        gdn.kv_evict_plan(pool, layer, layer + 1, slots, length, nxt, ml, budget, 2, 8, nm, mv, len_out)
        gdn.kv_evict_apply(pool, layer, layer + 1, slots, nm, mv)
        length.copy_(len_out)
    return kn, vn, q, outs, length


def test_decode_with_eviction_follows_a_host_model():
    """Append, attend and evict as a budgeted decode does, against a host model that keeps
    each head's tokens as a set (no places, no moves)."""
    steps, budget, group, D, H = 24, 40, 4, 64, 2
    c = make_cache(41, [30, 39, 5], None, H, D, 16, capacity=64)
    for b in range(3):  # pages up to the capacity
        c.table[c.slots[b]] = torch.arange(4) + 1 + 4 * b
    c.k = torch.zeros(1, 13, H, 16, D, dtype=torch.bfloat16)
    c.v = torch.zeros_like(c.k)
    g = torch.Generator().manual_seed(12)
    sets = []
    c.mass.zero_()
    for b in range(3):
        rows = []
        for i in range(c.lens[b]):
            kk, vv = (torch.randn(H, D, generator=g).to(torch.bfloat16) for _ in range(2))
            page = c.table[c.slots[b], i // 16]
            c.k[0, page, :, i % 16], c.v[0, page, :, i % 16] = kk, vv
            rows.append((kk.double().numpy(), vv.double().numpy()))
        sets.append([{i: [r[0][h], r[1][h], 0.0] for i, r in enumerate(rows)} for h in range(H)])
    pool = device_pool(c)
    kn, vn, q, outs, length = hybrid_steps(c, pool, 0, steps, budget, group, 77)
    assert length.tolist() == [budget, budget, 5 + steps]
    got = outs.float().cpu().double().numpy()
    gap = 1.0
    for b in range(3):
        nxt = c.lens[b]
        for t in range(steps):
            for h in range(H):
                s = sets[b][h]
                s[nxt] = [kn[t, b, h].double().numpy(), vn[t, b, h].double().numpy(), 0.0]
                ids = sorted(s)
                kk, vv = (np.stack([s[i][j] for i in ids]) for j in range(2))
                for j in range(group):
                    x = kk @ q[t, b, h * group + j].double().numpy() * D ** -0.5
                    p = np.exp(x - x.max())
                    p /= p.sum()
                    o = p @ vv
                    # 2^-8 of the value for bf16, 2^-12 of sum p |v| for the weights (kv_helpers)
                    tol = 2.0 ** -8 * np.abs(o) + 2.0 ** -12 * (p @ np.abs(vv))
                    assert (np.abs(got[t, b, h * group + j] - o) <= tol).all(), (b, t, h, j)
                    for i, w in zip(ids, p):
                        s[i][2] += w
                if len(s) > budget:
                    free = [i for i in ids if not (i < 2 or i >= nxt + 1 - 8)]
                    free.sort(key=lambda i: s[i][2])
                    gap = min(gap, s[free[1]][2] - s[free[0]][2])
                    del s[free[0]]
            nxt += 1
    assert gap > 1e-5  # the two least weights were never near enough for fp32 to swap them
    pos, mass = pool.pos.cpu().numpy(), pool.mass.cpu().numpy()
    for b in range(3):
        for h in range(H):
            n = int(length[b])
            assert sorted(pos[0, c.slots[b], h, :n].tolist()) == sorted(sets[b][h])
            for i in range(n):
                assert abs(mass[0, c.slots[b], h, i] - sets[b][h][int(pos[0, c.slots[b], h, i])][2]) < 1e-4
    assert int(pool.err_word.item()) == 0


def test_decode_step_in_graphs_that_share_a_workspace():
    """Two graphs captured over one workspace, replayed in turn between eager work and with
    new device lengths, against the eager calls."""
    import gated_delta_rule_slot_amd as gdn

    c = make_cache(51, [300, 70, 200], None, 2, 128, 32, capacity=512)
    for b in range(3):
        c.table[c.slots[b]] = torch.arange(16) + 1 + 16 * b
    c.k = torch.randn(1, 49, 2, 32, 128, generator=c.g).to(torch.bfloat16)
    c.v = torch.randn(1, 49, 2, 32, 128, generator=c.g).to(torch.bfloat16)
    B, Hq, D, budget = 3, 8, 128, 128
    ref, pool = device_pool(c), device_pool(c)
    kn, vn = (torch.randn(B, 2, D, generator=c.g).to(torch.bfloat16).cuda() for _ in range(2))
    qs = [torch.randn(B, Hq, D, generator=c.g).to(torch.bfloat16).cuda() for _ in range(2)]
    slots = i32(c.slots)
    ws = torch.empty(gdn.attn_workspace_bytes(pool, B, Hq, 512, 1), dtype=torch.uint8, device="cuda")

    def bufs():
        return dict(length=i32([0, 0, 0]), nxt=i32([0, 0, 0]), out=torch.zeros(B, Hq, D, dtype=torch.bfloat16, device="cuda"),
                    lse=torch.zeros(B, Hq, device="cuda"), nm=torch.zeros(1, B, 2, dtype=torch.int32, device="cuda"),
                    mv=torch.zeros(1, B, 2, 128, 2, dtype=torch.int32, device="cuda"), lo=i32([0, 0, 0]))

    def step(p, s, q):
        gdn.kv_append(p, 0, slots, s["length"], kn, vn, position=s["nxt"])
        gdn.attn_decode_paged(p, 0, slots, s["length"], q, s["out"], 512, scale=0.09, flags=1, lse=s["lse"], workspace=ws)
        gdn.kv_evict_plan(p, 0, 1, slots, s["length"], s["nxt"], 512, budget, 2, 16, s["nm"], s["mv"], s["lo"])
        gdn.kv_evict_apply(p, 0, 1, slots, s["nm"], s["mv"])

    sets = [bufs(), bufs()]
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s, q in zip(sets, qs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(pool, s, q)
        graphs.append(graph)
    torch.cuda.synchronize()
    for name in ("k", "v", "mass", "pos"):
        getattr(pool, name).copy_(getattr(ref, name))
    want = bufs()
    for turn in range(6):
        s, q = sets[turn % 2], qs[turn % 2]
        lens = [300 + turn, 70 * turn % 129, 200 - turn]
        for d in (s, want):
            d["length"].copy_(i32(lens))
            d["nxt"].copy_(i32([1000 + turn] * 3))
        graphs[turn % 2].replay()
        torch.cuda.synchronize()
        got = {n: s[n].clone() for n in ("out", "lse", "nm", "lo")}
        step(ref, want, q)
        torch.cuda.synchronize()
        for n in got:
            assert torch.equal(got[n], want[n]), (turn, n)
        for n in ("k", "v", "mass", "pos"):
            a, b = (getattr(p, n).view(torch.int16) if n in "kv" else getattr(p, n) for p in (pool, ref))
            assert torch.equal(a, b), (turn, n)
    assert int(pool.err_word.item()) == 0


def test_calls_on_other_streams():
    """Two streams with a workspace each, at once, give what one stream gives."""
    import gated_delta_rule_slot_amd as gdn

    c = make_cache(61, [2000, 900], None, 2, 128, 16)
    pool = device_pool(c, mass=False)
    q = [torch.randn(2, 8, 128, generator=c.g).to(torch.bfloat16).cuda() for _ in range(2)]
    ws = [torch.empty(gdn.attn_workspace_bytes(pool, 2, 8, 2000), dtype=torch.uint8, device="cuda") for _ in range(2)]
    out = [torch.zeros(2, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    slots, lens = i32(c.slots), i32(c.lens)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            gdn.attn_decode_paged(pool, 0, slots, lens, q[i], out[i], 2000, scale=0.1, workspace=ws[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        check_attention(c, q[i].cpu(), 0.1, out[i])


def test_attention_output_between_wide_q_rows():
    """out in the gap that q's rows leave in one buffer is apart from q."""
    import gated_delta_rule_slot_amd as gdn

    c = make_cache(77, [40, 129, 3], None, 2, 64, 16, False)
    B, Hq = 3, 6
    n = B * Hq * c.dim
    g = torch.Generator().manual_seed(78)
    buf = torch.randn(B, Hq * c.dim + n, generator=g).to(torch.bfloat16).cuda()
    q = buf[:, :Hq * c.dim].view(B, Hq, c.dim)
    keep = q.cpu()
    out = buf[1, Hq * c.dim:].view(B, Hq, c.dim)
    pool = device_pool(c)
    need = gdn.attn_workspace_bytes(pool, B, Hq, 129)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    gdn.attn_decode_paged(pool, c.layer, i32(c.slots), i32(c.lens), q, out, 129, scale=0.125, workspace=ws)
    check_attention(c, keep, 0.125, out)
    assert torch.equal(q.cpu(), keep)


@pytest.mark.parametrize("dim,kv_heads,group,page,lens,begins", [
    (64, 1, 2, 16, [1, 40, 131], None), (128, 2, 4, 4, [300, 77], [0, 5]), (256, 1, 8, 64, [700, 2], None),
    (128, 1, 17, 32, [513], [100]), (256, 2, 1, 8, [33, 260], None), (64, 1, 8, 64, [5003], None)])
def test_attention_infinite_values(dim, kv_heads, group, page, lens, begins):
    """An infinite value makes its column infinite whatever its weight's bits are, one of each
    sign or a NaN makes it NaN, and every other column, lse and the weights stay as they are."""
    c = make_cache(dim + lens[0], lens, begins, kv_heads, dim, page, layers=1)
    for b, n in enumerate(lens):
        lo = c.begins[b]
        for d in range(dim // 2):  # column d: one token's value, another token in each column
            i = lo + (d * 7) % (n - lo)
            c.v[0, c.table[c.slots[b], i // page], :, i % page, d] = float("-inf") if d % 3 == 0 else float("inf")
        i, j = lo + (n - lo) // 2, n - 1
        c.v[0, c.table[c.slots[b], i // page], :, i % page, dim - 1] = float("inf")
        c.v[0, c.table[c.slots[b], j // page], :, j % page, dim - 1] = float("-inf" if i != j else "nan")
        c.v[0, c.table[c.slots[b], i // page], :, i % page, dim - 2] = float("nan")
    pool, q, out, lse, sc = run_attention(c, group, mass=True)
    with np.errstate(invalid="ignore"):
        want, _, _, _, _ = attend_all(c, q, sc)
    odd = ~np.isfinite(want)
    assert odd[:, :, :dim // 2].all() and odd[:, :, dim - 2:].all() and not odd[:, :, dim // 2:dim - 2].any()
    got = out.float().cpu().double().numpy()
    assert np.array_equal(got[odd], want[odd], equal_nan=True)
    out[torch.from_numpy(odd).cuda()] = 0.0
    c.v[..., :dim // 2] = 0.0  # the other columns against the definition without these
    c.v[..., dim - 2:] = 0.0
    check_attention(c, q, sc, out, lse, pool.mass, c.mass)


def test_attention_arrays_side_by_side():
    """Inputs, outputs, weights and workspace back to back in one buffer are apart."""
    import gated_delta_rule_slot_amd as gdn

    c = make_cache(91, [40, 129, 300], None, 2, 64, 16)
    B, Hq, D = 3, 4, 64
    q = torch.randn(B, Hq, D, generator=c.g).to(torch.bfloat16)
    probe = device_pool(c)
    n = gdn.attn_workspace_bytes(probe, B, Hq, 300, 1)
    ints = c.table.numel() + 3 * B
    sizes = [q.numel() * 2, q.numel() * 2, n, c.mass.numel() * 4, B * Hq * 4, 4, ints * 4]
    buf = torch.zeros(256 + sum(sizes), dtype=torch.uint8, device="cuda")
    at = (-buf.data_ptr()) % 256  # the workspace lies after q and out: 3 * 4 * 64 * 2 * 2 bytes, 12 * 256
    parts = []
    for size in sizes:
        parts.append(buf[at:at + size])
        at += size
    qd, out = (t.view(torch.bfloat16).view(B, Hq, D) for t in parts[:2])
    ws, mass = parts[2], parts[3].view(torch.float32).view(c.mass.shape)
    lse, err, word = parts[4].view(torch.float32).view(B, Hq), parts[5].view(torch.int32), parts[6].view(torch.int32)
    table, slots, lens, begin = word[:c.table.numel()].view(c.table.shape), *word[c.table.numel():].split(B)
    qd.copy_(q), mass.copy_(c.mass), table.copy_(c.table), slots.copy_(i32(c.slots)), lens.copy_(i32(c.lens))
    pool = gdn.kv_pool_create(c.k.cuda(), c.v.cuda(), table, mass=mass, err_word=err)
    gdn.attn_decode_paged(pool, 0, slots, lens, qd, out, 300, kv_begin=begin, scale=0.125, flags=1, lse=lse, workspace=ws)
    check_attention(c, q, 0.125, out, lse, mass, c.mass)
    assert torch.equal(qd.cpu(), q) and lens.tolist() == c.lens and int(err.item()) == 0


@pytest.mark.parametrize("slots,counts,bit", [([0, -1], [7, -3], 0), ([9, 1], [0, 0], "ERRW_BAD_SLOT"),
                                              ([0, 9], [-1, 7], "ERRW_BAD_SLOT"), ([1, 0], [7, 0], "ERRW_BAD_SEQLENS")])
def test_apply_looks_at_the_slot_before_the_count(slots, counts, bit):
    """A padded request is skipped whatever its count holds, and a slot that is none is told
    with any count, as in the plan."""
    import gated_delta_rule_slot_amd as gdn

    c = make_cache(18, [64, 64], None, 1, 64, 16, slots=[1, 2])
    pool = device_pool(c)
    moves = torch.full((1, 2, 1, 2, 2), 3, dtype=torch.int32, device="cuda")
    gdn.kv_evict_apply(pool, 0, 1, i32(slots), i32([[[n] for n in counts]]), moves)
    assert int(pool.err_word.item()) == (getattr(gdn, bit) if bit else 0)
    assert torch.equal(pool.k.cpu().view(torch.int16), c.k.view(torch.int16)) and torch.equal(pool.mass.cpu(), c.mass)


@pytest.mark.parametrize("f8,dim,page,batch,max_len,workers", [
    (True, 64, 64, 16, 4096, 512), (True, 64, 64, 15, 4096, 256), (True, 128, 16, 32, 8192, 512),
    (True, 128, 16, 31, 8000, 256), (False, 64, 8, 16, 4096, 512), (True, 128, 64, 32, 8192, 256)])
def test_attention_with_one_and_two_workgroups_per_compute_unit(f8, dim, page, batch, max_len, workers):
    """Both sides of the rule for the number of workgroups: by the bytes of a row and of a
    head's run in a page, and by the blocks of 128 tokens that the bound allows."""
    import gated_delta_rule_slot_amd as gdn

    r = np.random.default_rng(dim + page + batch)
    lens = [int(x) for x in r.integers(0, 300, size=batch)]
    lens[0], lens[-1] = 1500, 1
    c = make_cache(batch, lens, None, 4, dim, page, f8, capacity=max_len)
    pool, q, out, lse, sc = run_attention(c, 2, mass=True, max_len=max_len)
    check_attention(c, q, sc, out, lse, pool.mass, c.mass)
    # the workspace's parts: units, O and (m, l) of 2 x 16 heads a workgroup
    units, parts = batch * 4 * 8, workers * 2 * 16
    pad = lambda n: -(-n // 256) * 256  # noqa: E731
    assert gdn.attn_workspace_bytes(pool, batch, 8, max_len) == pad(units) + pad(parts * dim * 4) + pad(parts * 8)


def test_attention_begin_counts_places_also_after_an_eviction():
    """kv_begin is a place: after a cut, the tokens in the places from it on are seen, whatever
    their positions, and the whole cache without it."""
    import gated_delta_rule_slot_amd as gdn

    c = make_cache(88, [200], None, 1, 64, 16, slots=[1])
    pool = device_pool(c)
    c.pos = torch.arange(c.cap, dtype=torch.int32).expand(c.mass.shape).contiguous()
    _, nm, mv, lo = run_plan(c, 100, 4, 50, [200], pool=pool)
    gdn.kv_evict_apply(pool, 0, 1, i32([1]), nm.cuda(), mv.cuda())
    assert int(nm.sum()) >= 50 and (pool.pos[0, 1, 0, :60].cpu() >= 150).any()  # recent ones in early places
    c.k, c.v, c.mass = pool.k.cpu(), pool.v.cpu(), pool.mass.cpu()
    c.lens = lo.tolist()
    for begin in (0, 60):
        c.begins = [begin]
        _, q, out, lse, sc = run_attention(c, 4, pool=pool)
        check_attention(c, q, sc, out, lse)


@pytest.mark.parametrize("dim,page,lens", [(64, 16, [1, 40, 128]), (128, 64, [3000, 5]), (256, 4, [700])])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_attention_of_nothing_seen_is_zero_whatever_the_values(dim, page, lens, value):
    """Every score -inf: out = 0 and lse = -inf also where the values are NaN or infinite."""
    c = make_cache(dim, lens, None, 2, dim, page)
    c.k[...] = 0.0
    c.k[..., 0] = float("-inf")
    c.v[...] = value
    import gated_delta_rule_slot_amd as gdn

    pool = device_pool(c)
    B, Hq = len(lens), 6
    q = torch.zeros(B, Hq, dim, dtype=torch.bfloat16)
    q[..., 0] = 1.0
    for flags in (0, 1):
        out = torch.full((B, Hq, dim), -7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((B, Hq), -7.0, device="cuda")
        ws = torch.empty(gdn.attn_workspace_bytes(pool, B, Hq, max(lens), flags), dtype=torch.uint8, device="cuda")
        gdn.attn_decode_paged(pool, 0, i32(c.slots), i32(lens), q.cuda(), out, max(lens), scale=0.125, flags=flags,
                              lse=lse, workspace=ws)
        assert not out.float().any() and torch.isneginf(lse).all()
        assert torch.equal(pool.mass.cpu(), c.mass)


def test_forms_of_much_shared_memory_in_a_graph():
    """Attention of head dim 256 (78 KB a workgroup) and a plan of 36864 tokens (156 KB)
    captured together, replayed with new lengths and weights between eager work."""
    import gated_delta_rule_slot_amd as gdn

    n, budget = 36864, 30000
    g = torch.Generator(device="cuda").manual_seed(5)
    k, v = (torch.randn(1, n // 128 + 1, 1, 128, 256, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    table = torch.zeros(2, n // 128, dtype=torch.int32, device="cuda")
    table[1] = torch.randperm(n // 128, device="cuda", generator=g) + 1
    mass = torch.rand(1, 2, 1, n, device="cuda", generator=g)
    pos = torch.arange(n, dtype=torch.int32, device="cuda").expand(1, 2, 1, n).contiguous()
    pool = gdn.kv_pool_create(k, v, table, mass=mass, pos=pos)
    q = torch.randn(1, 8, 256, device="cuda", generator=g).to(torch.bfloat16)
    slots, lens, nxt = i32([1]), i32([n]), i32([n])
    ws = torch.empty(gdn.attn_workspace_bytes(pool, 1, 8, n, 1), dtype=torch.uint8, device="cuda")
    out = torch.zeros(1, 8, 256, dtype=torch.bfloat16, device="cuda")
    nm, mv = (torch.zeros(1, 1, 1, *x, dtype=torch.int32, device="cuda") for x in ((), (budget, 2)))
    lo = torch.zeros_like(lens)

    def step():
        gdn.attn_decode_paged(pool, 0, slots, lens, q, out, n, scale=0.0625, flags=1, workspace=ws)
        gdn.kv_evict_plan(pool, 0, 1, slots, lens, nxt, n, budget, 4, 64, nm, mv, lo)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for turn in range(4):
        lens.fill_(n - 1001 * turn)
        mass.copy_(torch.rand(mass.shape, device="cuda", generator=g))
        m0 = mass.clone()
        step()
        want = out.clone(), nm.clone(), mv.clone()
        m1 = mass.clone()
        mass.copy_(m0)
        for t in (out, nm, lo):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(nm, want[1]) and torch.equal(mass, m1), turn
        assert torch.equal(mv, want[2]) and int(nm) > 0 and int(lo) == min(int(lens), budget)
