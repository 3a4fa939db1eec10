"""GPU: page tables and token maps, release of pages, rotary positions with the append, and
attention of chunks of new tokens, against their definitions (oracle/kv_ops.py)."""
import numpy as np
import pytest
import torch

from oracle import kv_ops
from tests.kv_helpers import attn_slack, device_pool, i32, make_cache, stored

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ attention --
def chunk_call(c, new, group, window=0, late=0, q_pad=0, scale=None, max_len=None, extra=0, lse=True, pool=None, q=None,
               q_std=1.0, seed=1, stream=None):
    """One call over cache c, whose last new[b] places are the new tokens'; `extra` rows behind the
    last request.  Returns (pool, q, out, lse, scale)."""
    import gated_delta_rule_slot_amd as gdn

    B, Hq, T = len(c.lens), c.kv_heads * group, sum(new) + extra
    g = torch.Generator().manual_seed(seed)
    if q is None:
        wide = (q_std * torch.randn(T, Hq * c.dim + q_pad, generator=g)).to(torch.bfloat16).cuda()
        q = wide[:, q_pad:].view(T, Hq, c.dim)
    pool = pool or device_pool(c)
    out = torch.full((T, Hq, c.dim), -7.0, dtype=torch.bfloat16, device="cuda")
    lv = torch.full((T, Hq), -7.0, device="cuda") if lse else None
    ml = max(c.lens) if max_len is None else max_len
    n = gdn.attn_prefill_workspace_bytes(pool, B, T, Hq, ml, late)
    ws = torch.full((n,), 0xff, dtype=torch.uint8, device="cuda") if n else None
    sc = c.dim ** -0.5 if scale is None else scale
    begin = i32(c.begins) if any(c.begins) else None
    cu = i32([sum(new[:b]) for b in range(B + 1)])
    gdn.attn_prefill_paged(pool, c.layer, cu, i32(c.slots), i32(c.lens), q, out, ml, kv_begin=begin, window=window,
                           scale=sc, mass_tokens=late, lse=lv, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    return pool, q.cpu(), out, lv, sc


def check_chunk(c, new, q, scale, out, lse, window=0, late=0, mass=None, errors=None):
    k, v = (t[c.layer].float().double().numpy() for t in (c.k, c.v))
    table = c.table.numpy()
    got, qd = out.float().cpu().double().numpy(), q.float().double().numpy()
    at = 0
    wm = c.mass.double().numpy().copy()
    tm = np.zeros_like(wm)
    for b, n in enumerate(new):
        rows = slice(at, at + n)
        at += n
        live = 0 < c.slots[b] < c.n_slots
        if not live or n == 0:
            assert not got[rows].any()
            if lse is not None:
                assert torch.isneginf(lse[rows]).all()
            continue
        L = c.lens[b]
        want, wl, w, (spread, size) = kv_ops.attend_chunk(k, v, table, c.slots[b], c.begins[b], L, qd[rows], scale,
                                                          window, late, c.k_scale, c.v_scale)
        slack = attn_slack(size, c.dim, 2 * L)  # (sums run over steps of 16 places)
        # the output's rounding, and the weights' before the product with the values: half a bf16
        # step each, 2^-8
        tol = 2.0 ** -8 * np.abs(want) + (slack[..., None] + 2.0 ** -8) * (1 + 2.0 ** -8) * spread + 1e-38
        bad = ~(np.abs(got[rows] - want) <= tol)
        assert not bad.any(), (b, np.argwhere(bad)[:4], got[rows][bad][:4], want[bad][:4])
        seen = np.isfinite(wl)
        tl = slack + 2.0 ** -22 * (np.abs(np.where(seen, wl, 0)) + size)
        if lse is not None:
            gl = lse[rows].cpu().double().numpy()
            assert np.array_equal(np.isneginf(gl), ~seen)
            assert (np.abs(gl[seen] - wl[seen]) <= tl[seen]).all()
        if late:
            # a weight is exp(s - lse): the score's error and the lse's
            m = min(n, late)
            sl = (slack + tl)[n - m:].max()
            idx = (c.layer, c.slots[b], slice(None), slice(0, L))
            wm[idx] += w
            tm[idx] = w * (sl + (m * q.shape[1] / c.kv_heads / 32 + 64) * 2.0 ** -23) + 2.0 ** -24 * wm[idx]
    assert (got[at:] == -7.0).all()
    if lse is not None:
        assert (lse[at:] == -7.0).all()
    if mass is not None:
        gm = mass.cpu().double().numpy()
        assert (np.abs(gm - wm) <= tm).all(), np.abs(gm - wm).max()


CASES = [
    # dim, kv_heads, group, page, fp8, new, cached, begins, window
    (64, 1, 1, 16, False, [1], [0], None, 0),
    (64, 2, 3, 1, False, [33, 64, 2], [0, 5, 0], None, 0),
    (128, 2, 4, 16, False, [0, 31, 32, 129], [4, 0, 1, 70], None, 0),
    (128, 1, 16, 32, False, [50, 7], [0, 300], [0, 6], 0),
    (128, 3, 5, 8, False, [127, 12, 25], [0, 128, 255], [100, 128, 33], 0),
    (256, 2, 8, 64, False, [300, 65, 1], [0, 0, 77], None, 0),
    (256, 1, 12, 128, False, [77], [700], [31], 0),
    (64, 1, 17, 4, False, [90, 40], [3, 0], None, 24),
    (128, 1, 40, 64, False, [14], [140], None, 0),
    (64, 1, 64, 2, False, [7], [70], [3], 9),
    (64, 2, 2, 16, True, [100, 1, 45], [0, 200, 64], None, 0),
    (128, 2, 7, 32, True, [64, 33], [0, 300], [0, 300], 0),
    (256, 1, 16, 1024, True, [110, 9], [1000, 0], None, 100),
    (256, 2, 1, 2, True, [61], [0], [60], 0),
    (256, 1, 4, 16, False, [130], [200], None, 1),
    (128, 1, 1, 64, False, [257], [64], None, 65),
]


@pytest.mark.parametrize("late", [0, 20])
@pytest.mark.parametrize("dim,kv_heads,group,page,f8,new,cached,begins,window", CASES)
def test_chunk_parity(dim, kv_heads, group, page, f8, new, cached, begins, window, late):
    lens = [n + m for n, m in zip(new, cached)]
    c = make_cache(dim + group + page, lens, begins, kv_heads, dim, page, f8)
    pool, q, out, lse, sc = chunk_call(c, new, group, window, late, q_pad=8 * (group % 3), extra=group % 2)
    check_chunk(c, new, q, sc, out, lse, window, late, pool.mass)
    assert int(pool.err_word.item()) == 0


@pytest.mark.parametrize("f8,dim,group,window", [(False, 128, 8, 0), (False, 256, 8, 0), (True, 128, 4, 0),
                                                 (False, 64, 2, 1500), (True, 256, 3, 0)])
def test_chunk_divided_places(f8, dim, group, window):
    """A few tokens over thousands of places (divided and joined) beside short and empty
    requests, with bounds above the lengths, in a second layer."""
    new, cached = [5, 0, 7, 1], [5003, 40, 64, 2999]
    c = make_cache(5, [n + m for n, m in zip(new, cached)], [0, 0, 64, 17], 1, dim, 64, f8, layers=2, layer=1,
                   capacity=9000)
    for max_len in (9000, 5008):
        pool, q, out, lse, sc = chunk_call(c, new, group, window, 3, max_len=max_len)
        check_chunk(c, new, q, sc, out, lse, window, 3, pool.mass)


@pytest.mark.parametrize("seed", range(8))
def test_chunk_random_cases(seed):
    r = np.random.default_rng(300 + seed)
    dim = int(r.choice([64, 128, 256]))
    kv_heads, group = int(r.integers(1, 4)), int(r.integers(1, 20))
    B = int(r.integers(1, 6))
    new = [int(x) for x in r.integers(0, 120, size=B)]
    new[0] += 1
    cached = [int(x) for x in r.integers(0, 500, size=B)]
    lens = [max(1, n + m) for n, m in zip(new, cached)]
    begins = [int(r.integers(0, n + 2)) if r.random() < 0.4 else 0 for n in lens]
    window, late = int(r.choice([0, 0, 1, 50, 200])), int(r.choice([0, 1, 33, 1000]))
    c = make_cache(seed, lens, begins, kv_heads, dim, int(2 ** r.integers(0, 9)), bool(r.random() < 0.5),
                   k_std=float(r.choice([0.1, 1.0, 3.0])))
    pool, q, out, lse, sc = chunk_call(c, new, group, window, late, q_pad=16, seed=seed)
    check_chunk(c, new, q, sc, out, lse, window, late, pool.mass)
    assert int(pool.err_word.item()) == 0


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_chunk_scales(scale):
    """A zero scale averages the values, a negative one turns the order, a large one picks nearly
    one place (and makes the running maximum jump)."""
    c = make_cache(11, [77, 200], None, 2, 128, 16)
    pool, q, out, lse, sc = chunk_call(c, [40, 70], 4, late=11, scale=scale)
    check_chunk(c, [40, 70], q, sc, out, lse, 0, 11, pool.mass)


def test_chunk_of_single_tokens_is_the_decode():
    """One token per request: the one-token attention's results within both tolerances."""
    import gated_delta_rule_slot_amd as gdn

    c = make_cache(4, [200, 1, 0, 333], None, 2, 128, 16)
    c.lens[2] = 1
    pool, q, out, lse, sc = chunk_call(c, [1] * 4, 4)
    want, wl = torch.empty_like(out), torch.empty_like(lse)
    ws = torch.empty(gdn.attn_workspace_bytes(pool, 4, 8, 333), dtype=torch.uint8, device="cuda")
    gdn.attn_decode_paged(pool, 0, i32(c.slots), i32(c.lens), q.cuda(), want, 333, scale=sc, lse=wl, workspace=ws)
    ok = torch.tensor([0, 1, 3], device="cuda")  # the third's only place has no page
    assert (lse[ok] - wl[ok]).abs().max() < 1e-4
    assert (out[ok].float() - want[ok].float()).abs().max() < 3 * 2.0 ** -8 * 4


def nan_free(c):
    """The cache with zeros for the NaN of its unused rows."""
    c.k, c.v = torch.nan_to_num(c.k.float()).to(c.k.dtype), torch.nan_to_num(c.v.float()).to(c.v.dtype)
    return c


@pytest.mark.parametrize("dim,group,window", [(64, 1, 0), (128, 4, 0), (256, 8, 0), (128, 4, 30), (256, 3, 7)])
def test_chunk_later_tokens_that_are_not_finite(dim, group, window):
    """Tokens of the chunk with NaN and infinite values and keys: tokens before them (and, with a
    window, far behind them) are as if they were not there."""
    n, L = 100, 150
    c = make_cache(dim + group, [L], None, 1, dim, 16)
    t = c.table[c.slots[0]]

    def row(x, i):
        return x[0, int(t[i // 16]), 0, i % 16]

    row(c.v, 90)[3] = float("nan")
    row(c.v, 97)[:] = float("inf")
    row(c.v, 110)[5] = float("-inf")
    row(c.k, 120)[:] = float("nan")
    pool, q, out, lse, sc = chunk_call(c, [n], group, window)
    got = out.float().cpu()
    clean = make_cache(dim + group, [L], None, 1, dim, 16)
    pool2, _, out2, lse2, _ = chunk_call(clean, [n], group, window, q=q.cuda())
    place = torch.arange(L - n, L)
    free = torch.ones(n, dtype=torch.bool)
    for bad in (90, 97, 110, 120):
        free &= (place < bad) | ((place >= bad + window) if window else torch.zeros(n, dtype=torch.bool))
    assert free.any()
    # both are within half a step and the weights' rounding of the same value: the walks differ
    tol = 4 * 2.0 ** -8 * (out2.float().cpu().abs() + 4)
    assert ((got - out2.float().cpu()).abs() <= tol)[free].all()
    assert torch.isfinite(got[free]).all() and torch.isfinite(lse.cpu()[free]).all()
    only_inf = (place >= 97) & (place < 110) & ((place < 97 + window) if window else True)
    cols = [d for d in range(dim) if d != 3]
    assert torch.isinf(got[only_inf][:, :, cols]).all()
    saw_nan = (place >= 90) & ((place < 90 + window) if window else True)
    assert torch.isnan(got[saw_nan][:, :, 3]).all()
    saw_key = (place >= 120) & ((place < 120 + window) if window else True)
    assert torch.isnan(got[saw_key]).all() and torch.isnan(lse.cpu()[saw_key]).all()


@pytest.mark.parametrize("dim,group,f8", [(64, 3, True), (128, 4, False), (256, 8, True), (256, 2, False)])
def test_chunk_values_that_are_not_finite_in_divided_places(dim, group, f8):
    """The same where the places are divided and joined, and in an e4m3 cache (which has NaN only)."""
    n, L = 20, 3000
    c = make_cache(dim + group, [L], None, 1, dim, 16, f8)
    t = c.table[c.slots[0]]
    bad = [(L - 7, 3)] if f8 else [(L - 7, 3), (L - 12, 9), (1000, 40)]
    for i, (place, column) in enumerate(bad):
        c.v[0, int(t[place // 16]), 0, place % 16, column] = float("nan") if i == 0 else float("inf")
    pool, q, out, lse, sc = chunk_call(c, [n], group, late=n)
    clean = make_cache(dim + group, [L], None, 1, dim, 16, f8)
    _, _, want, wl, _ = chunk_call(clean, [n], group, q=q.cuda())
    got, want = out.float().cpu(), want.float().cpu()
    assert torch.equal(lse, wl) and torch.isfinite(pool.mass).all()
    place = torch.arange(L - n, L)
    hit = torch.zeros(n, dim, dtype=torch.bool)
    for i, (at, column) in enumerate(bad):
        sees = place >= at
        hit[sees, column] = True
        v = got[sees][:, :, column]
        assert (torch.isnan(v) if i == 0 else torch.isposinf(v)).all()
    free = ~hit[:, None, :].expand_as(got)
    assert ((got - want).abs() <= 4 * 2.0 ** -8 * (want.abs() + 4))[free].all()


@pytest.mark.parametrize("rise", [0.1, 1.0, -1.0])
@pytest.mark.parametrize("dim,kv_heads,group,f8", [(64, 1, 3, False), (64, 32, 2, False), (128, 2, 2, False),
                                                   (256, 1, 4, False), (64, 1, 2, True), (128, 1, 8, True),
                                                   (256, 1, 1, True)])
def test_chunk_scores_that_rise_with_the_place(dim, kv_heads, group, f8, rise):
    """Every block of places has much larger scores than those before (or, falling, smaller ones), so that
    the reference of the exponent has to follow, for some rows of a wave and not for others."""
    new, L, rest = ([200, 70, 2], 333, 12288) if kv_heads > 2 else ([150, 40], 333, 0)  # (tiles of 256 rows)
    lens = [L] + [77] * (len(new) - 1)
    c = make_cache(dim, lens, None, kv_heads, dim, 16, f8)
    g = torch.Generator().manual_seed(dim + group)
    T = sum(new) + rest
    for b, n in enumerate(lens):
        at = torch.arange(n)
        page = c.table[c.slots[b]][at // 16].long()
        ramp = (at * rise).view(n, 1, 1) / dim
        k = ramp + 0.3 * torch.randn(n, kv_heads, dim, generator=g)
        c.k[0].view(torch.uint8 if f8 else torch.int16)[page, :, at % 16] = \
            stored(k, f8).view(torch.uint8 if f8 else torch.int16)
    # rows of one sign rise where those of the other fall
    sign = torch.where(torch.rand(T, kv_heads * group, 1, generator=g) < 0.7, 1.0, -1.0)
    q = (sign + 0.3 * torch.randn(T, kv_heads * group, dim, generator=g)).to(torch.bfloat16).cuda()
    pool, q, out, lse, sc = chunk_call(c, new, group, late=7, q=q, scale=1.0, extra=rest)
    check_chunk(c, new, q, sc, out, lse, 0, 7, pool.mass)


@pytest.mark.parametrize("f8,page,window,late", [(False, 16, 0, 70), (True, 32, 0, 5), (False, 4, 90, 0),
                                                 (True, 2, 90, 400), (False, 64, 1, 3)])
def test_chunk_tiles_of_twice_the_rows(f8, page, window, late):
    """A call of so many rows of heads of 64 that a tile has 256 of them (most behind the last request):
    requests of one to a few hundred tokens, tiles and waves filled in part, values that are not finite in one."""
    H, G, B, late_place, rest = 32, 2, 6, 45, 12000
    r = np.random.default_rng(page)
    new, cached = [300, 87, 0, 129, 5, 1], [20, 0, 9, 70, 31, 200]
    lens = [max(1, n + m) for n, m in zip(new, cached)]
    begins = [int(r.integers(0, n)) if i % 5 == 3 else 0 for i, n in enumerate(lens)]
    c = make_cache(page, lens, begins, H, 64, page, f8)
    pool, q, clean, lse, sc = chunk_call(c, new, G, window, late, extra=rest)
    check_chunk(c, new, q, sc, clean, lse, window, late, pool.mass)
    at = lens[0] - late_place
    c.v[0, int(c.table[c.slots[0], at // page]), 7, at % page, 11] = float("nan") if f8 else float("inf")
    pool, _, out, lse2, _ = chunk_call(c, new, G, window, late, q=q.cuda(), extra=rest)
    assert torch.equal(lse, lse2) and torch.isfinite(pool.mass).all()
    first = 300 - late_place
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[first:min(300, first + window) if window else 300, 7 * G:8 * G, 11] = True
    assert (torch.isnan(out[hit]) if f8 else torch.isposinf(out[hit])).all()
    x, y = out[~hit].float(), clean[~hit].float()
    assert ((x - y).abs() <= 4 * 2.0 ** -8 * (y.abs() + 4)).all()
    assert int(pool.err_word.item()) == 0


@pytest.mark.parametrize("batch,dim,group", [(65, 64, 1), (300, 128, 3), (5000, 64, 2)])
def test_chunk_many_requests(batch, dim, group):
    """More requests than a wave has lanes, and than two steps of its search reach, some of them
    empty or padding, lengths of a few."""
    r = np.random.default_rng(batch)
    new = [int(x) for x in r.integers(0, 4, size=batch)]
    lens = [max(1, n + int(x)) for n, x in zip(new, r.integers(0, 6, size=batch))]
    slots = [int(x) + 1 for x in r.permutation(batch)]
    for b in range(0, batch, 11):
        slots[b] = 0
    c = make_cache(batch, lens, None, 1, dim, 4, slots=slots)
    pool, q, out, lse, sc = chunk_call(c, new, group, late=2, extra=3)
    check_chunk(c, new, q, sc, out, lse, 0, 2, pool.mass)
    assert int(pool.err_word.item()) == 0


def test_chunk_more_tiles_than_one_dimension_of_a_grid():
    """A prompt of 70000 tokens and 64 query heads in a narrow window (35000 tiles): rows from all over
    it against the definition."""
    import gated_delta_rule_slot_amd as gdn

    n, page, window = 70000, 64, 40
    g = torch.Generator(device="cuda").manual_seed(5)
    pages = -(-n // page) + 1
    k, v = (torch.randn(1, pages, 1, page, 64, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    table = torch.zeros(2, pages - 1, dtype=torch.int32)
    table[1] = torch.randperm(pages - 1, generator=torch.Generator().manual_seed(1)).to(torch.int32) + 1
    pool = gdn.kv_pool_create(k, v, table.cuda(), err_word=i32([0]))
    q = torch.randn(n, 64, 64, device="cuda", generator=g).to(torch.bfloat16)
    out = torch.full_like(q, -7.0)
    ws = torch.empty(gdn.attn_prefill_workspace_bytes(pool, 1, n, 64, n), dtype=torch.uint8, device="cuda")
    gdn.attn_prefill_paged(pool, 0, i32([0, n]), i32([1]), i32([n]), q, out, n, window=window, scale=0.125, workspace=ws)
    assert int(pool.err_word.item()) == 0
    kh, vh = (t[0].float().cpu().double().numpy() for t in (k, v))
    for i in (0, 1, 39, 40, 1999, 4463, 4464, 35000, 65535, 65536, n - 1):
        want, _, _, (spread, size) = kv_ops.attend(kh, vh, table.numpy(), 1, max(0, i - window + 1), i + 1,
                                                   q[i].float().cpu().double().numpy(), 0.125)
        slack = attn_slack(size, 64, 2 * window)
        tol = 2.0 ** -8 * np.abs(want) + (slack[:, None] + 2.0 ** -8) * (1 + 2.0 ** -8) * spread
        assert (np.abs(out[i].float().cpu().double().numpy() - want) <= tol).all(), i


def test_chunk_begins_past_every_place():
    """A first visible place at the end of the int32 range: rows that see nothing, no weights."""
    c = make_cache(2, [300, 40], None, 2, 64, 16)
    begins, c.begins = c.begins, [2 ** 31 - 1, 41]
    pool, q, out, lse, sc = chunk_call(c, [200, 40], 2, late=200)
    assert not out.float().any() and torch.isneginf(lse).all() and torch.equal(pool.mass.cpu(), c.mass)
    assert int(pool.err_word.item()) == 0
    pool, q, out, lse, sc = chunk_call(c, [200, 40], 2, window=2 ** 31 - 1, late=2 ** 31 - 1)
    assert not out.float().any() and torch.equal(pool.mass.cpu(), c.mass)
    c.begins = begins
    pool, q, out, lse, sc = chunk_call(c, [200, 40], 2, window=2 ** 31 - 1, late=2 ** 31 - 1)
    check_chunk(c, [200, 40], q, sc, out, lse, 0, 200, pool.mass)


def test_chunk_scores_that_are_not_finite():
    """-inf scores leave a place out, rows of nothing else are empty, +inf makes a row NaN."""
    c = nan_free(make_cache(3, [40, 40, 40], None, 1, 64, 8))
    t = c.table[c.slots[0]]
    c.k[0, int(t[0]), 0, 3, 0] = float("inf")
    for i in range(40):
        c.k[0, int(c.table[c.slots[1]][i // 8]), 0, i % 8, 0] = float("inf")
    c.k[0, int(c.table[c.slots[2]][2]), 0, 1, 0] = float("inf")
    c.mass.zero_()
    g = torch.Generator().manual_seed(0)
    q = torch.randn(30, 2, 64, generator=g).to(torch.bfloat16)
    q[:, :, 0] = -1.0
    q[20:, 0, 0] = 1.0
    pool, _, out, lse, _ = chunk_call(c, [10, 10, 10], 2, late=10, q=q.cuda(), scale=0.125)
    w = pool.mass.cpu()
    assert torch.isfinite(out[:10].float()).all() and float(w[0, c.slots[0], 0, 3]) == 0.0
    assert abs(float(w[0, c.slots[0], 0, :40].sum()) - 20) < 1e-3
    assert not out[10:20].float().any() and torch.isneginf(lse[10:20]).all() and not w[0, c.slots[1]].any()
    assert torch.isnan(out[20:, 0].float()).all() and torch.isnan(lse[20:, 0]).all()
    assert torch.isfinite(out[20:, 1].float()).all() and torch.isfinite(lse[20:, 1]).all()


@pytest.mark.parametrize("late", [0, 8])
def test_chunk_skips_and_flags(late):
    """Padding and bad slots, bad lengths and begins, ranges outside the rows, bad pages."""
    import gated_delta_rule_slot_amd as gdn

    lens = [50, 60, 70, 80, 90, 100, 40]
    new = [10, 11, 12, 13, 14, 15, 16]
    c = make_cache(21, lens, None, 2, 128, 16, slots=[1, 0, 3, 2, 4, 5, 6])
    base = c.table.clone()

    def run(**kw):
        c2 = make_cache(21, lens, None, 2, 128, 16, slots=[1, 0, 3, 2, 4, 5, 6])
        for n, x in kw.items():
            getattr(c2, n)[x[0]] = x[1]
        pool, q, out, lse, sc = chunk_call(c2, new, 4, late=late, max_len=100)
        return c2, pool, q, out, lse, sc, int(pool.err_word.item())

    c2, pool, q, out, lse, sc, e = run()
    check_chunk(c2, new, q, sc, out, lse, 0, late, pool.mass)
    assert e == 0
    for change, bit in ((dict(slots=(2, 7)), gdn.ERRW_BAD_SLOT), (dict(lens=(2, 11)), gdn.ERRW_BAD_SEQLENS),
                        (dict(lens=(2, 101)), gdn.ERRW_BAD_SEQLENS), (dict(lens=(2, -1)), gdn.ERRW_BAD_SEQLENS),
                        (dict(begins=(2, -1)), gdn.ERRW_BAD_SEQLENS)):
        c2, pool, q, out, lse, sc, e = run(**change)
        assert e == bit, change
        at = sum(new[:2])
        assert not out[at:at + 12].float().any() and torch.isneginf(lse[at:at + 12]).all()
        c2.slots[2], c2.lens[2], c2.begins[2] = 0, 70, 0
        check_chunk(c2, new, q, sc, out, lse, 0, late, pool.mass)
    # pages 2 and 4 of the sixth are none: their places are not there
    c2 = make_cache(21, lens, None, 2, 128, 16, slots=[1, 0, 3, 2, 4, 5, 6])
    c2.table[5, 2], c2.table[5, 4] = 0, c2.k.shape[1]
    pool, q, out, lse, sc = chunk_call(c2, new, 4, late=late)
    check_chunk(c2, new, q, sc, out, lse, 0, late, pool.mass)
    assert int(pool.err_word.item()) == gdn.ERRW_BAD_PAGE
    assert torch.equal(base[:5], c2.table[:5])
    # a range past the rows: that request's are left, the others' are there
    pool = device_pool(c)
    cu = i32([0, 10, 21, 33, 46, 60, 75, 92])
    T = 91
    q = torch.randn(T, 8, 128, generator=c.g).to(torch.bfloat16).cuda()
    out = torch.full((T, 8, 128), -7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(gdn.attn_prefill_workspace_bytes(pool, 7, T, 8, 100), dtype=torch.uint8, device="cuda")
    gdn.attn_prefill_paged(pool, 0, cu, i32(c.slots), i32(c.lens), q, out, 100, scale=0.1, workspace=ws)
    assert int(pool.err_word.item()) == gdn.ERRW_BAD_SEQLENS
    assert (out[75:] == -7.0).all() and torch.isfinite(out[:75].float()).all() and (out[:75] != -7.0).any(dim=-1).all()


def test_chunk_offsets_past_32_bits():
    """Pages beyond 4 GiB of a layer, and a second layer beyond 8."""
    import gated_delta_rule_slot_amd as gdn

    pages, H, page, D = 20000, 4, 128, 256
    k = torch.empty(2, pages, H, page, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    table = torch.zeros(2, 4, dtype=torch.int32)
    ids = [pages - 1, 17, pages - 2, 19000]
    table[1] = torch.tensor(ids)
    g = torch.Generator().manual_seed(0)
    kk, vv = (torch.randn(4, H, page, D, generator=g).to(torch.bfloat16) for _ in range(2))
    for layer in (0, 1):
        k[layer, torch.tensor(ids)] = kk.cuda()
        v[layer, torch.tensor(ids)] = vv.cuda()
    small = make_cache(1, [500], None, H, D, page)
    small.k[0, 1:5], small.v[0, 1:5] = kk, vv
    small.table[small.slots[0], :4] = torch.tensor([1, 2, 3, 4], dtype=torch.int32)
    _, q, want, wl, sc = chunk_call(small, [70], 2)
    pool = gdn.kv_pool_create(k, v, table.cuda())
    for layer in (0, 1):
        out = torch.empty_like(want)
        ws = torch.empty(gdn.attn_prefill_workspace_bytes(pool, 1, 70, 8, 500), dtype=torch.uint8, device="cuda")
        gdn.attn_prefill_paged(pool, layer, i32([0, 70]), i32([1]), i32([500]), q.cuda(), out, 500, scale=sc,
                               workspace=ws)
        assert torch.equal(out, want)
    del k, v, pool


def test_chunk_in_graphs_that_share_a_workspace():
    """Two captured calls over one workspace, replayed in turn with lengths that change, on a
    stream of their own, against eager calls."""
    import gated_delta_rule_slot_amd as gdn

    c = make_cache(8, [700, 300], None, 2, 128, 16, capacity=4000)
    nan_free(c)
    pool = device_pool(c)
    g = torch.Generator().manual_seed(3)
    q = torch.randn(60, 8, 128, generator=g).to(torch.bfloat16).cuda()
    lens, slots = i32([700, 300]), i32(c.slots)
    cus = [i32([0, 40, 60]), i32([0, 3, 50])]
    outs = [torch.zeros(60, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ws = torch.empty(gdn.attn_prefill_workspace_bytes(pool, 2, 60, 8, 4000), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0

    def call(i, out):
        gdn.attn_prefill_paged(pool, 0, cus[i], slots, lens, q, out, 4000, scale=0.1, workspace=ws)

    side = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(side):
        for i in range(2):
            call(i, outs[i])
        side.synchronize()
        for i in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                call(i, outs[i])
            graphs.append(graph)
    torch.cuda.synchronize()
    for step in range(4):
        lens.copy_(i32([700 - 90 * step, 300 - 60 * step]))
        for i in (0, 1):
            outs[i].zero_()
            graphs[i].replay()
            torch.cuda.synchronize()
            want = torch.zeros_like(outs[i])
            call(i, want)
            assert torch.equal(outs[i], want), (step, i)


# ----------------------------------------------------------------------- rope --
def rope_case(seed, n, q_heads, kv_heads, dim, page, f8, far=5000):
    g = torch.Generator().manual_seed(seed)
    c = make_cache(seed, [n + 20, 33], None, kv_heads, dim, page, f8, layers=2, layer=1, slots=[2, 1], capacity=n + 40)
    place = torch.randperm(n + 20, generator=g)[:n]
    slot = torch.full((n,), 2, dtype=torch.int32)
    if n > 3:
        slot[1], place[1] = 1, 7
    pos = torch.randint(0, far + 1, (n,), generator=g)
    x = (2 * torch.randn(n, (q_heads + 2 * kv_heads) * dim + 24, generator=g)).to(torch.bfloat16)
    return c, slot, place.to(torch.int32), pos.to(torch.int32), x


def split_rows(x, q_heads, kv_heads, dim):
    n, a, b = x.shape[0], q_heads * dim, (q_heads + kv_heads) * dim
    return (x[:, 8:8 + a].view(n, q_heads, dim), x[:, 8 + a:8 + b].view(n, kv_heads, dim),
            x[:, 8 + b:8 + b + kv_heads * dim].view(n, kv_heads, dim))


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("n,q_heads,kv_heads,dim,rot,page,f8,far", [
    (1, 1, 1, 64, 64, 16, False, 5000), (5, 3, 1, 64, 16, 1, True, 100), (33, 16, 2, 256, 64, 64, False, 131072),
    (70, 8, 8, 128, 128, 32, True, 10 ** 6), (200, 5, 5, 128, 48, 128, False, 2 ** 31 - 1),
    (7, 0, 3, 256, 256, 4, False, 12), (64, 12, 4, 256, 240, 16, True, 70000), (1030, 4, 1, 128, 96, 16, False, 9000),
])
def test_rope_append_parity(n, q_heads, kv_heads, dim, rot, page, f8, far, adjacent):
    import gated_delta_rule_slot_amd as gdn

    c, slot, place, pos, x = rope_case(n + dim, n, q_heads, kv_heads, dim, page, f8, far)
    pool = device_pool(c)
    amp = 1.25
    freqs, _ = gdn.rope_frequencies(rot, base=10000.0)
    xd = x.cuda()
    q, k, v = split_rows(xd, q_heads, kv_heads, dim)
    q_out = torch.full((n, q_heads, dim), -7.0, dtype=torch.bfloat16, device="cuda") if q_heads else None
    kb, vb = pool.k.clone(), pool.v.clone()
    gdn.rope_append(pool, 1, slot.cuda(), place.cuda(), pos.cuda(), q if q_heads else None, q_out, k, v, freqs.cuda(),
                    layout=gdn.ROPE_INTERLEAVED if adjacent else gdn.ROPE_HALF, amplitude=amp)
    torch.cuda.synchronize()
    assert torch.equal(xd.cpu(), x) and int(pool.err_word.item()) == 0
    qh, kh, vh = (t.float().double().numpy() for t in split_rows(x, q_heads, kv_heads, dim))
    # the angle is off by 2^-24 of a turn in fp32 and the sines by 4 units: 2^-21; products and the
    # sum add 3 units of the pair's size; then one rounding
    slack = 2.0 ** -20

    def check(got, want, size, step, least):
        tol = step * np.abs(want) + slack * size + least
        assert (np.abs(got - want) <= tol).all(), np.abs(got - want).max()

    if q_heads:
        want = kv_ops.turn(qh, pos.numpy(), freqs.numpy(), amp, adjacent)
        check(q_out.float().cpu().double().numpy(), want, 1.25 * 2 * np.abs(qh).max(), 2.0 ** -8, 1e-38)
    wk = kv_ops.turn(kh, pos.numpy(), freqs.numpy(), amp, adjacent) / c.k_scale
    p = c.table[slot.long(), place.long() // page].long()
    r = place.long() % page
    gk, gv = (t[1].float().cpu()[p, :, r].double().numpy() for t in (pool.k, pool.v))
    if f8:
        wk = np.clip(wk, -448, 448)
        check(gk, wk, 2.5 * np.abs(kh).max() / c.k_scale, 2.0 ** -4, 2.0 ** -10)
        want = kv_ops.e4m3_round((vh.astype(np.float32) / np.float32(c.v_scale)).astype(np.float64))
        assert np.array_equal(gv, want)
    else:
        check(gk, wk, 2.5 * np.abs(kh).max(), 2.0 ** -8, 1e-38)
        assert np.array_equal(gv, vh)
    # nothing else has changed
    kb[1].view(torch.uint8 if f8 else torch.int16)[p, :, r] = pool.k[1].view(torch.uint8 if f8 else torch.int16)[p, :, r]
    vb[1].view(torch.uint8 if f8 else torch.int16)[p, :, r] = pool.v[1].view(torch.uint8 if f8 else torch.int16)[p, :, r]
    bits = torch.uint8 if f8 else torch.int16
    assert torch.equal(kb.view(bits), pool.k.view(bits)) and torch.equal(vb.view(bits), pool.v.view(bits))
    mass, ps = c.mass.clone(), c.pos.clone()
    mass[1, slot.long(), :, place.long()] = 0
    ps[1, slot.long(), :, place.long()] = pos[:, None].expand(-1, kv_heads)
    assert torch.equal(pool.mass.cpu(), mass) and torch.equal(pool.pos.cpu(), ps)


def test_rope_in_place_negative_and_skipped():
    """Queries turned in place inside the projection's rows; negative positions; tokens that are
    skipped, or stored nowhere."""
    import gated_delta_rule_slot_amd as gdn

    c, slot, place, pos, x = rope_case(9, 12, 4, 2, 128, 16, False)
    pos = pos - 3000
    slot[3], slot[4], place[5] = 0, c.n_slots, c.cap
    c.table[2, int(place[6]) // 16] = 0
    bad_page = [i for i in range(12) if slot[i] == 2 and i not in (5,) and place[i] // 16 == place[6] // 16]
    pool = device_pool(c)
    freqs, amp = gdn.rope_frequencies(64, scaling=gdn.ROPE_YARN, factor=4.0, original_len=2048)
    xd = x.cuda()
    q, k, v = split_rows(xd, 4, 2, 128)
    before = pool.k.clone()
    gdn.rope_append(pool, 1, slot.cuda(), place.cuda(), pos.cuda(), q, q, k, v, freqs.cuda(), amplitude=amp)
    torch.cuda.synchronize()
    assert int(pool.err_word.item()) == gdn.ERRW_BAD_SLOT | gdn.ERRW_BAD_SEQLENS | gdn.ERRW_BAD_PAGE
    qh = split_rows(x, 4, 2, 128)[0].float().double().numpy()
    want = kv_ops.turn(qh, pos.numpy(), freqs.numpy(), amp, False)
    got = split_rows(xd.cpu(), 4, 2, 128)[0].float().double().numpy()
    on = [i for i in range(12) if i not in (3, 4)]
    assert (np.abs(got - want)[on] <= 2.0 ** -8 * np.abs(want)[on] + 2.0 ** -20 * 4 * np.abs(qh).max()).all()
    assert np.array_equal(got[3:5], qh[3:5])
    rest = x.clone()
    rest[:, 8:8 + 512] = xd.cpu()[:, 8:8 + 512]
    assert torch.equal(rest, xd.cpu())
    kept = torch.ones(12, dtype=torch.bool)
    kept[[3, 4, 5] + bad_page] = False
    same = pool.k[1].view(torch.int16) == before[1].view(torch.int16)
    changed = (~same).any(dim=-1)[:, 0].sum().item()
    assert changed == int(kept.sum())


def test_rope_offsets_past_32_bits():
    """Tokens whose rows lie past 4 GiB of the projection's buffer and of the layer."""
    import gated_delta_rule_slot_amd as gdn

    pages, D = 70000, 256
    k = torch.empty(1, pages, 2, 64, D, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(2, 2, dtype=torch.int32)
    table[1] = torch.tensor([3, pages - 1])
    pool = gdn.kv_pool_create(k, torch.empty_like(k), table.cuda())
    rows = 3
    wide = torch.empty(rows, (1 << 31) // 2 + 64, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(1)
    x = torch.randn(rows, 6 * D, generator=g).to(torch.bfloat16)
    wide[:, :6 * D] = x.cuda()
    freqs = gdn.rope_frequencies(64)[0].cuda()
    q, kn, vn = wide[:, :2 * D].view(rows, 2, D), wide[:, 2 * D:4 * D].view(rows, 2, D), wide[:, 4 * D:6 * D].view(rows, 2, D)
    args = (i32([1, 1, 1]), i32([5, 70, 127]), i32([9, 8, 7]))
    gdn.rope_append(pool, 0, *args, q, q, kn, vn, freqs)
    small = x.cuda()
    sq, sk, sv = (small[:, i * 2 * D:(i + 1) * 2 * D].view(rows, 2, D) for i in range(3))
    other = gdn.kv_pool_create(torch.zeros(1, 4, 2, 64, D, dtype=torch.bfloat16, device="cuda"),
                               torch.zeros(1, 4, 2, 64, D, dtype=torch.bfloat16, device="cuda"),
                               i32([[0, 0], [1, 2]]))
    out = torch.empty(rows, 2, D, dtype=torch.bfloat16, device="cuda")
    gdn.rope_append(other, 0, *args, sq, out, sk, sv, freqs)
    assert torch.equal(q, out)
    for i, (p, r) in enumerate(((3, 5), (pages - 1, 6), (pages - 1, 63))):
        assert torch.equal(pool.k[0, p, :, r], other.k[0, 1 if i == 0 else 2, :, r])
        assert torch.equal(pool.v[0, p, :, r], vn[i])
    del k, wide, pool


# ------------------------------------------------------------------ page tables --
def map_pool(slots, max_pages, page, pages, seed=0, lens=None, order=None):
    """A pool (one head) whose slots order[b] hold lens[b] places; the rest of the pages are free."""
    import gated_delta_rule_slot_amd as gdn

    g = torch.Generator().manual_seed(seed)
    ids = (torch.randperm(pages - 1, generator=g) + 1).tolist()
    table = torch.zeros(slots, max_pages, dtype=torch.int32)
    for s, n in zip(order or [], lens or []):
        for e in range(-(-n // page)):
            table[s, e] = ids.pop()
    k = torch.zeros(1, pages, 1, page, 64, dtype=torch.bfloat16, device="cuda")
    pool = gdn.kv_pool_create(k, k, table.cuda(), err_word=i32([0]))
    return pool, table, ids


def run_map(pool, table, free, n_free, slots, lens, new, pos, max_tokens, in_place=False, no_pos=False):
    import gated_delta_rule_slot_amd as gdn

    B = len(slots)
    want = kv_ops.batch_map(table.tolist(), slots, lens, new if new is not None else [1] * B,
                            pos if pos is not None else lens, free, n_free, pool.page_size, max_tokens)
    o = {n: torch.full((m,), -7, dtype=torch.int32, device="cuda")
         for n, m in (("cu", B + 1), ("slot", B), ("len", B), ("pos", B), ("token_slot", max_tokens),
                      ("token_index", max_tokens), ("token_pos", max_tokens), ("n_free", 1))}
    ld, pd, nf = i32(lens), i32(pos) if pos is not None else None, i32([n_free])
    if in_place:
        o["len"], o["pos"], o["n_free"] = ld, pd, nf
    pool.page_table.copy_(table)
    pool.err_word.zero_()
    fr = i32(free)
    gdn.kv_batch_map(pool, i32(slots), ld, fr, nf, o["cu"], o["slot"], o["len"], o["token_slot"], o["token_index"],
                     new_len=i32(new) if new is not None else None, next_pos=pd,
                     next_pos_out=o["pos"] if pd is not None else None, token_pos=None if no_pos else o["token_pos"],
                     n_free_out=o["n_free"])
    torch.cuda.synchronize()
    for n in ("cu", "slot", "len", "token_slot", "token_index"):
        assert o[n].tolist() == want[n], n
    if pd is not None:
        assert o["pos"].tolist() == want["pos"]
    if not no_pos:
        assert o["token_pos"].tolist() == want["token_pos"]
    assert pool.page_table.tolist() == want["table"] and o["n_free"].tolist() == [want["n_free"]]
    assert fr.tolist() == free
    bits = sum({"slot": gdn.ERRW_BAD_SLOT, "lens": gdn.ERRW_BAD_SEQLENS, "pages": gdn.ERRW_NO_PAGES}[e]
               for e in want["errors"])
    assert int(pool.err_word.item()) == bits
    return o, want


@pytest.mark.parametrize("B,page,lo,hi,cached,extra", [
    (1, 16, 1, 1, 0, 0), (1, 64, 700, 700, 63, 3), (5, 1, 0, 9, 20, 0), (7, 16, 0, 40, 33, 64),
    (128, 64, 1, 1, 300, 5), (300, 8, 0, 5, 30, 1), (257, 32, 0, 70, 100, 9), (40, 16, 200, 900, 500, 2),
    (700, 128, 0, 40, 10, 70), (3, 1024, 5000, 9000, 100, 1),
])
def test_batch_map(B, page, lo, hi, cached, extra):
    r = np.random.default_rng(B + page)
    new = [int(x) for x in r.integers(lo, hi + 1, size=B)]
    lens = [int(x) for x in r.integers(0, cached + 1, size=B)]
    pos = [int(x) for x in r.integers(0, 10 ** 6, size=B)]
    order = [int(x) + 1 for x in r.permutation(B)]
    most = -(-(max(n + m for n, m in zip(new, lens))) // page) + 1
    pages = 2 + sum(-(-(n + m) // page) for n, m in zip(new, lens)) + 7
    pool, table, free = map_pool(B + 1, most, page, pages, B, lens, order)
    for b in range(0, B, 9):
        if B > 9:
            order[b] = -(b % 2)
    T = sum(new) + extra
    run_map(pool, table, free, len(free), order, lens, new, pos, T)
    run_map(pool, table, free, len(free), order, lens, new, pos, T, in_place=True)
    run_map(pool, table, free, len(free), order, lens, new, None, T, no_pos=True)
    # a list that runs out on the way, an empty one
    run_map(pool, table, free, len(free) // 3, order, lens, new, pos, T)
    run_map(pool, table, free, 0, order, lens, new, pos, T)
    if lo == hi == 1:
        run_map(pool, table, free, len(free), order, lens, None, pos, T)


def test_batch_map_refusals_on_the_device():
    """Bad slots and lengths, positions past 31 bits, tokens past the arrays, counts outside the list."""
    B = 40
    lens, new, pos = [10] * B, [7] * B, [5] * B
    order = list(range(1, B + 1))
    pool, table, free = map_pool(B + 1, 4, 16, 400, 1, lens, order)
    n = len(free)
    for change in (dict(order=(3, B + 1)), dict(order=(3, 2 ** 31 - 1)), dict(order=(3, -5)), dict(lens=(4, -1)),
                   dict(lens=(4, 58)), dict(lens=(4, 2 ** 31 - 1)), dict(new=(9, -3)), dict(new=(9, 2 ** 31 - 1)),
                   dict(new=(9, 55)), dict(pos=(6, 2 ** 31 - 7)), dict(pos=(6, 2 ** 31 - 8))):
        a = dict(order=list(order), lens=list(lens), new=list(new), pos=list(pos))
        for name, (i, x) in change.items():
            a[name][i] = x
        for T in (7 * B + 3, 7 * 20 + 3, 0 if "new" in change else 7):
            run_map(pool, table, free, n, a["order"], a["lens"], a["new"], a["pos"], T)
    run_map(pool, table, free, -3, order, lens, new, pos, 7 * B)
    run_map(pool, table, free, n + 5, order, lens, new, pos, 7 * B)
    # more requests than one workgroup takes at a time, the sum passing the arrays early on
    B = 600
    pool, table, free = map_pool(B + 1, 4, 16, 4000, 1, [10] * B, list(range(1, B + 1)))
    new = [7] * B
    new[100] = 2 ** 31 - 1
    new[590] = 0
    run_map(pool, table, free, len(free), list(range(1, B + 1)), [10] * B, new, [0] * B, 7 * B)


def run_release(pool, table, free, n_free, slots, lens, keep, in_place=False):
    import gated_delta_rule_slot_amd as gdn

    wt, wf, wn, errors = kv_ops.release(table.tolist(), slots, lens, keep if keep is not None else [0] * len(slots),
                                        free, n_free, pool.page_size, pool.pages)
    pool.page_table.copy_(table)
    pool.err_word.zero_()
    fr, nf = i32(free), i32([n_free])
    out = nf if in_place else i32([-7])
    gdn.kv_release(pool, i32(slots), i32(lens), fr, nf, keep=i32(keep) if keep is not None else None, n_free_out=out)
    torch.cuda.synchronize()
    assert pool.page_table.tolist() == wt and fr.tolist() == wf and out.tolist() == [wn]
    bits = sum({"slot": gdn.ERRW_BAD_SLOT, "lens": gdn.ERRW_BAD_SEQLENS, "page": gdn.ERRW_BAD_PAGE}[e] for e in errors)
    assert int(pool.err_word.item()) == bits


@pytest.mark.parametrize("B,page,hi", [(1, 16, 0), (1, 16, 5000), (9, 1, 70), (64, 16, 3000), (33, 64, 64),
                                       (1100, 32, 90), (3, 1024, 9000), (1100, 16, 200),
                                       (2, 1, 3000)])
def test_release(B, page, hi):
    r = np.random.default_rng(B + page)
    lens = [int(x) for x in r.integers(0, hi + 1, size=B)]
    keep = [int(x) for x in r.integers(0, hi + 2, size=B)]
    order = [int(x) + 1 for x in r.permutation(B)]
    need = sum(-(-n // page) for n in lens)
    pool, table, ids = map_pool(B + 1, -(-hi // page) + 2, page, need + 40, B, lens, order)
    for b in range(0, B, 9):
        if B > 9:
            order[b] = 0
    free = ids[:20] + [0] * (need + 19)
    run_release(pool, table, free, 20, order, lens, keep)
    run_release(pool, table, free, 20, order, lens, None, in_place=True)
    run_release(pool, table, free[:20 + need // 2], 20, order, lens, None)  # a list with too little room
    run_release(pool, table, free, -4, order, lens, keep)
    run_release(pool, table, free[:20], 33, order, lens, keep)
    if B > 9:
        bad = table.clone()
        bad[order[1], 0], bad[order[2], 0] = 0, need + 40
        lens[3], lens[4], keep[5], order[6] = -1, 2 ** 31 - 1, -1, B + 1
        run_release(pool, bad, free, 20, order, lens, keep)


def test_maps_in_a_graph_count_on():
    """A captured decode step's map that updates lengths, positions and the list in place: every
    replay goes on where the last ended, as the host's model does."""
    import gated_delta_rule_slot_amd as gdn

    B, page = 6, 4
    lens, pos, order = [0, 3, 4, 7, 8, 1], [9, 8, 7, 6, 5, 4], [2, 1, 4, 3, 0, 6]
    pool, table, free = map_pool(8, 12, page, 60, 2, [n if s else 0 for n, s in zip(lens, order)], order)
    sl, ln, ps, fr, nf = i32(order), i32(lens), i32(pos), i32(free), i32([len(free)])
    cu, so, ts, ti, tp = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (B + 1, B, 8, 8, 8))

    def step():
        gdn.kv_batch_map(pool, sl, ln, fr, nf, cu, so, ln, ts, ti, next_pos=ps, next_pos_out=ps, token_pos=tp)

    step()  # (loads the code)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    pool.page_table.copy_(table)
    ln.copy_(i32(lens)), ps.copy_(i32(pos)), nf.fill_(len(free))
    t, n = table.tolist(), len(free)
    for _ in range(5):
        graph.replay()
        torch.cuda.synchronize()
        w = kv_ops.batch_map(t, order, lens, [1] * B, pos, free, n, page, 8)
        t, n, lens, pos = w["table"], w["n_free"], w["len"], w["pos"]
        assert pool.page_table.tolist() == t and nf.tolist() == [n] and ln.tolist() == lens and ps.tolist() == pos
        assert ts.tolist() == w["token_slot"] and ti.tolist() == w["token_index"] and tp.tolist() == w["token_pos"]


# ---------------------------------------------------------------------- together --
class Steps:
    """A layer's decode steps with buffers of their own, all of it on the device: lengths, positions
    and the free list go on from step to step.  With 600 pages a request the attention divides its places."""

    def __init__(self, page=4, B=5, H=2, G=3, dim=64, most=60):
        import gated_delta_rule_slot_amd as gdn

        self.gdn, self.cap, self.scale = gdn, most * page, dim ** -0.5
        g = torch.Generator().manual_seed(7)
        pages = 1 + B * most // 2
        k = torch.full((1, pages, H, page, dim), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.pool = gdn.kv_pool_create(k, k.clone(), torch.zeros(B + 1, most, dtype=torch.int32, device="cuda"),
                                       err_word=i32([0]))
        self.free, self.n_free = i32(list(range(pages - 1, 0, -1))), i32([pages - 1])
        self.slots, self.lens, self.nxt = i32([3, 1, 5, 2, 4]), i32([0] * B), i32([0, 9, 100, 7, 1])
        self.new = i32([1, 2, 0, 3, 1])
        T = 9
        self.x = torch.randn(T, (H * G + 2 * H) * dim, generator=g).to(torch.bfloat16).cuda()
        self.q, self.k, self.v = (t.view(T, -1, dim) for t in self.x.split([H * G * dim, H * dim, H * dim], dim=1))
        self.cu, self.so = i32([0] * (B + 1)), i32([0] * B)
        self.ts, self.ti, self.tp = (i32([0] * T) for _ in range(3))
        self.qr, self.out = (torch.zeros(T, H * G, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        f, self.amp = gdn.rope_frequencies(32)
        self.freqs = f.cuda()
        n = gdn.attn_prefill_workspace_bytes(self.pool, B, T, H * G, self.cap)
        self.ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def step(self, stream=None):
        self.gdn.kv_batch_map(self.pool, self.slots, self.lens, self.free, self.n_free, self.cu, self.so, self.lens,
                              self.ts, self.ti, new_len=self.new, next_pos=self.nxt, next_pos_out=self.nxt,
                              token_pos=self.tp, stream=stream)
        self.gdn.rope_append(self.pool, 0, self.ts, self.ti, self.tp, self.q, self.qr, self.k, self.v, self.freqs,
                             amplitude=self.amp, stream=stream)
        self.gdn.attn_prefill_paged(self.pool, 0, self.cu, self.so, self.lens, self.qr, self.out, self.cap,
                                    scale=self.scale, workspace=self.ws, stream=stream)

    def release(self, stream=None):
        self.gdn.kv_release(self.pool, self.slots, self.lens, self.free, self.n_free, stream=stream)

    def state(self):
        torch.cuda.synchronize()
        return [t.clone() for t in (self.lens, self.nxt, self.n_free, self.free, self.pool.page_table, self.ts, self.ti,
                                    self.tp, self.cu, self.so, self.qr, self.out, self.pool.err_word)]


def same(a, b):
    for i, (x, y) in enumerate(zip(a, b)):
        assert torch.equal(x, y), i


@pytest.mark.parametrize("most", [60, 600])
def test_whole_steps_replayed(most):
    """Steps of map, append and attention, captured once, replayed with eager work between: every
    replay's state and outputs are those of eager steps on another pool."""
    a, b = Steps(most=most), Steps(most=most)
    assert (a.ws.numel() > 0) == (most == 600)
    graph = torch.cuda.CUDAGraph()
    start = [t.clone() for t in (a.lens, a.nxt, a.n_free, a.pool.page_table)]
    a.step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        a.step()
    for t, s in zip((a.lens, a.nxt, a.n_free, a.pool.page_table), start):
        t.copy_(s)
    for _ in range(12):
        x = torch.randn_like(a.x)
        a.x.copy_(x), b.x.copy_(x)
        graph.replay()
        b.step()
        same(a.state(), b.state())
    assert a.out.float().abs().sum() > 0 and a.lens.tolist() == [12, 24, 0, 36, 12]
    a.release(), b.release()
    same(a.state(), b.state())
    assert not a.pool.page_table.any()


@pytest.mark.parametrize("most", [60, 600])
def test_steps_on_streams_at_once(most):
    """Two pools' steps on streams of their own, neither the current one, running at the same time."""
    want = Steps(most=most)
    for _ in range(10):
        want.step()
    want.release()
    got, streams = [Steps(most=most), Steps(most=most)], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, st in zip(got, streams):
            s.step(stream=st)
    for s, st in zip(got, streams):
        s.release(stream=st)
    for s in got:
        same(s.state(), want.state())


@pytest.mark.parametrize("f8,dim,rot,adjacent", [(False, 128, 128, False), (True, 64, 32, True), (False, 256, 64, False)])
def test_prompts_then_decode_follow_a_host_model(f8, dim, rot, adjacent):
    """Prompts in chunks, then decode steps, eviction and the release of pages, all tables made on
    the device, against a host model that keeps every request's keys and values as plain lists."""
    import gated_delta_rule_slot_amd as gdn

    H, G, page, B, budget = 2, 3, 16, 3, 60
    slots, pages, most = [2, 3, 1], 40, 12
    g = torch.Generator().manual_seed(dim)
    dt = torch.float8_e4m3fn if f8 else torch.bfloat16
    ks, vs = (0.5, 0.75) if f8 else (1.0, 1.0)
    k = torch.full((1, pages, H, page, dim), float("nan")).to(dt).cuda()
    mass = torch.zeros(1, 4, H, most * page, device="cuda")
    pool = gdn.kv_pool_create(k, k.clone(), torch.zeros(4, most, dtype=torch.int32, device="cuda"), mass=mass,
                              pos=torch.zeros(1, 4, H, most * page, dtype=torch.int32, device="cuda"),
                              err_word=i32([0]), k_scale=ks, v_scale=vs)
    freqs, amp = gdn.rope_frequencies(rot, scaling=gdn.ROPE_LINEAR, factor=2.0)
    free, n_free = i32(list(range(pages - 1, 0, -1)) + [0]), i32([pages - 1])
    lens, nxt, sl = i32([0] * B), i32([0] * B), i32(slots)
    model = [[] for _ in range(B)]  # per request: (key [H, D], value [H, D], position)
    host = dict(len=[0] * B, pos=[0] * B)
    sc = dim ** -0.5
    layout = gdn.ROPE_INTERLEAVED if adjacent else gdn.ROPE_HALF
    for step, new in enumerate([[40, 17, 1], [30, 60, 33], [1, 1, 1], [1, 1, 1], [5, 0, 2]]):
        T = sum(new) + 4
        x = torch.randn(T, (H * G + 2 * H) * dim, generator=g).to(torch.bfloat16)
        q, kn, vn = (t.view(T, -1, dim) for t in x.cuda().split([H * G * dim, H * dim, H * dim], dim=1))
        cu, so = i32([0] * (B + 1)), i32([0] * B)
        ts, ti, tp = (i32([0] * T) for _ in range(3))
        gdn.kv_batch_map(pool, sl, lens, free, n_free, cu, so, lens, ts, ti, new_len=i32(new), next_pos=nxt,
                         next_pos_out=nxt, token_pos=tp)
        qr = torch.empty(T, H * G, dim, dtype=torch.bfloat16, device="cuda")
        gdn.rope_append(pool, 0, ts, ti, tp, q, qr, kn, vn, freqs.cuda(), layout=layout, amplitude=amp)
        out = torch.empty(T, H * G, dim, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(T, H * G, device="cuda")
        cap = most * page
        ws = torch.empty(gdn.attn_prefill_workspace_bytes(pool, B, T, H * G, cap, T), dtype=torch.uint8, device="cuda")
        gdn.attn_prefill_paged(pool, 0, cu, so, lens, qr, out, cap, scale=sc, mass_tokens=T, lse=lse, workspace=ws)
        torch.cuda.synchronize()
        assert int(pool.err_word.item()) == 0
        # the model: rotation in fp64 of the same inputs, rounded to what the cache holds
        xq, xk, xv = (t.float().double().numpy().reshape(T, -1, dim)
                      for t in x.split([H * G * dim, H * dim, H * dim], dim=1))
        at = 0
        for b in range(B):
            n = new[b]
            p = np.arange(host["pos"][b], host["pos"][b] + n)
            kk = stored(torch.tensor(kv_ops.turn(xk[at:at + n], p, freqs.numpy(), amp, adjacent) / ks).float(), f8)
            vv = stored(torch.tensor(xv[at:at + n] / vs).float(), f8)
            for i in range(n):
                model[b].append((kk[i].double().numpy() * ks, vv[i].double().numpy() * vs, int(p[i])))
            old = len(model[b]) - n
            qd = kv_ops.turn(xq[at:at + n], p, freqs.numpy(), amp, adjacent)
            for i in range(n):
                for j in range(H * G):
                    h = j // G
                    K = np.stack([m[0][h] for m in model[b][:old + i + 1]])
                    V = np.stack([m[1][h] for m in model[b][:old + i + 1]])
                    s = sc * (K @ qd[i, j])
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    # a key may round the other way where fp32 and fp64 fall on either side of a
                    # border: one step of the stored type for each, beside the bf16 roundings
                    step_ = 2.0 ** -3 if f8 else 2.0 ** -7
                    err = sc * step_ * (np.abs(K) @ np.abs(qd[i, j])).max() * 0.25 + 2.0 ** -6
                    tol = 2.0 ** -7 * np.abs(w @ V) + 2 * err * (w @ np.abs(V)) + 1e-6
                    assert (np.abs(out[at + i, j].float().cpu().double().numpy() - w @ V) <= tol).all(), (step, b, i, j)
            at += n
            host["len"][b] += n
            host["pos"][b] += n
        assert lens.tolist() == host["len"] and nxt.tolist() == host["pos"]
        if max(host["len"]) > budget:  # cut, and give the pages behind the budget back
            used = [-(-n // page) for n in host["len"]]
            nm = torch.zeros(1, B, H, dtype=torch.int32, device="cuda")
            mv = torch.zeros(1, B, H, budget, 2, dtype=torch.int32, device="cuda")
            cut = i32([0] * B)
            gdn.kv_evict_plan(pool, 0, 1, sl, lens, nxt, 2 * budget, budget, 2, 20, nm, mv, cut)
            gdn.kv_evict_apply(pool, 0, 1, sl, nm, mv)
            before = int(n_free.item())
            gdn.kv_release(pool, sl, lens, free, n_free, keep=cut)
            lens.copy_(cut)
            torch.cuda.synchronize()
            host["len"] = cut.tolist()
            freed = sum(u - -(-n // page) for u, n in zip(used, host["len"]))
            assert int(n_free.item()) == before + freed and freed > 0
            t = pool.page_table.cpu()
            in_use = [int(t[s, e]) for s, n in zip(slots, host["len"]) for e in range(-(-n // page))]
            assert sorted(in_use + free[:int(n_free.item())].tolist()) == list(range(1, pages))
            # every head's kept set, by position, is what remains of the model
            pos = pool.pos.cpu()
            for b in range(B):
                kept = [set(pos[0, slots[b], h, :host["len"][b]].tolist()) for h in range(H)]
                assert all(len(s) == host["len"][b] for s in kept)
                model[b] = [(np.stack([m[0][h] if m[2] in kept[h] else np.full(dim, np.nan) for h in range(H)]),
                             np.stack([m[1][h] if m[2] in kept[h] else np.full(dim, np.nan) for h in range(H)]), m[2])
                            for m in model[b]]
            break
    # after the cut the kept keys attend the same: a decode step by both attentions
    x = torch.randn(B, H * G, dim, generator=g).to(torch.bfloat16).cuda()
    o1, o2 = torch.empty_like(x), torch.empty_like(x)
    ws = torch.empty(gdn.attn_workspace_bytes(pool, B, H * G, most * page), dtype=torch.uint8, device="cuda")
    gdn.attn_decode_paged(pool, 0, sl, lens, x, o1, most * page, scale=sc, workspace=ws)
    ws = torch.empty(gdn.attn_prefill_workspace_bytes(pool, B, B, H * G, most * page), dtype=torch.uint8, device="cuda")
    gdn.attn_prefill_paged(pool, 0, i32([0, 1, 2, 3]), sl, lens, x, o2, most * page, scale=sc, workspace=ws)
    xd = x.float().cpu().double().numpy()
    for b in range(B):
        for j in range(H * G):
            rows = [m for m in model[b] if not np.isnan(m[0][j // G]).any()]
            K, V = np.stack([m[0][j // G] for m in rows]), np.stack([m[1][j // G] for m in rows])
            s = sc * (K @ xd[b, j])
            w = np.exp(s - s.max())
            w /= w.sum()
            tol = 2.0 ** -7 * np.abs(w @ V) + (2.0 ** -2 if f8 else 2.0 ** -5) * (w @ np.abs(V)) + 1e-6
            for o in (o1, o2):
                assert (np.abs(o[b, j].float().cpu().double().numpy() - w @ V) <= tol).all()
