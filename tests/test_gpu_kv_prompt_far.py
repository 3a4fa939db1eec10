"""GPU: attention of chunks with scores of any size: keys and queries are small whole numbers, so
that a score is exact in fp32 and, times a large scale, only the largest ones have a weight."""
import numpy as np
import pytest
import torch

from tests.kv_helpers import i32, make_cache, stored
from tests.test_gpu_kv_prompt import check_chunk, chunk_call

pytestmark = pytest.mark.gpu


def whole_numbers(seed, lens, kv_heads, dim, page, f8, group, tokens, begins=None, capacity=None):
    c = make_cache(seed, lens, begins, kv_heads, dim, page, f8, capacity=capacity)
    k = torch.randint(-2, 3, c.k.shape, generator=c.g).float()
    c.k = stored(torch.where(torch.isnan(c.k.float()), c.k.float(), k), f8)
    q = torch.randint(-2, 3, (tokens, kv_heads * group, dim), generator=c.g).to(torch.bfloat16)
    return c, q


def check_sharp(c, new, q, scale, out, lse, window=0, late=0, mass=None, mass0=None):
    """out is the mean of the values at the largest scores, lse that score and the logarithm of their
    number, a weight 1 / number."""
    f32scale = float(np.float32(scale))
    k, v = (t[c.layer].float().double().numpy() for t in (c.k, c.v))
    got, gl = out.float().cpu().double().numpy(), lse.cpu().double().numpy()
    qd, G = q.float().double().numpy(), q.shape[1] // c.kv_heads
    wm = (c.mass if mass0 is None else mass0).double().numpy().copy()
    added = np.zeros_like(wm)
    at = 0
    for b, n in enumerate(new):
        L, t = c.lens[b], c.table[c.slots[b]].numpy()
        i = np.arange(L)
        K, V = (x[t[i // c.page], :, i % c.page] for x in (k, v))  # [L, H, D]
        for r in range(n):
            place = L - n + r
            lo = max(c.begins[b], place - window + 1 if window else 0)
            for j in range(q.shape[1]):
                s = K[lo:place + 1, j // G] @ qd[at + r, j]
                s = s if f32scale >= 0 else -s
                top = s == s.max()
                vv = c.v_scale * V[lo:place + 1, j // G][top]
                want, spread = vv.mean(axis=0), np.abs(vv).mean(axis=0)
                # the weights are all the same: their rounding to bf16, the sums' roundings, the output's
                tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + (L / 32 + 64) * 2.0 ** -23) * (1 + 2.0 ** -8) * spread
                assert (np.abs(got[at + r, j] - want) <= tol).all(), (b, r, j, got[at + r, j][:4], want[:4])
                wl = s.max() * abs(f32scale) * c.k_scale + np.log(top.sum())
                # fp32: scale * k_scale * log2(e), its product with the score, the logarithm's sum, ln 2
                assert abs(gl[at + r, j] - wl) <= 2.0 ** -21 * abs(wl) + 2.0 ** -20, (b, r, j, gl[at + r, j], wl)
                if n - r <= late:
                    added[c.layer, c.slots[b], j // G, lo:place + 1] += top / top.sum()
        at += n
    if mass is not None:
        # 2^x, 1 / l and the product: a few units each; sums of up to late * G weights
        tol = added * (16 + late * G) * 2.0 ** -23 + 2.0 ** -23 * (wm + added)
        err = np.abs(mass.cpu().double().numpy() - wm - added)
        assert (err <= tol).all(), err.max()


SCALES = [1e3, 1e6, 1e9, 1e12, -1e30]
LATE = [0, 20]  # queries whose weights are added to mass


@pytest.mark.parametrize("late", LATE)
@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("dim,group,f8,window", [(64, 3, False, 0), (64, 2, True, 60), (128, 4, False, 70),
                                                 (128, 1, True, 0), (256, 8, False, 0), (256, 2, True, 33)])
def test_far_scores(dim, group, f8, window, scale, late):
    new, lens = [70, 9, 1], [200, 150, 70]
    c, q = whole_numbers(dim, lens, 2, dim, 16, f8, group, 80)
    pool, _, out, lse, sc = chunk_call(c, new, group, window, late, q=q.cuda(), scale=scale)
    check_sharp(c, new, q, scale, out, lse, window, late, pool.mass)
    assert int(pool.err_word.item()) == 0


@pytest.mark.parametrize("late", LATE)
@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("dim,f8", [(64, False), (128, True), (256, False), (256, True)])
def test_far_scores_divided(dim, f8, scale, late):
    new, lens = [2, 3], [3000, 4100]
    c, q = whole_numbers(dim, lens, 1, dim, 64, f8, 2, 5, [0, 17], 9000)
    pool, _, out, lse, sc = chunk_call(c, new, 2, 0, late, q=q.cuda(), scale=scale, max_len=9000)
    check_sharp(c, new, q, scale, out, lse, 0, late, pool.mass)


@pytest.mark.parametrize("late", LATE)
@pytest.mark.parametrize("scale", [1e6, -1e9])
@pytest.mark.parametrize("f8", [False, True])
def test_far_scores_in_tiles_of_twice_the_rows(f8, scale, late):
    new, rest = [130, 1], 12288
    c, q = whole_numbers(3, [200, 33], 32, 64, 16, f8, 2, 131 + rest)
    pool, _, out, lse, sc = chunk_call(c, new, 2, 0, late, q=q.cuda(), scale=scale, extra=rest)
    check_sharp(c, new, q, scale, out, lse, 0, late, pool.mass)


@pytest.mark.parametrize("late", LATE)
@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("dim,group,f8", [(64, 3, False), (128, 4, True), (256, 8, False)])
def test_far_scores_of_single_tokens_are_the_decodes(dim, group, f8, scale, late):
    import gated_delta_rule_slot_amd as gdn
    from tests.kv_helpers import device_pool

    lens = [333, 1, 64, 900]
    c, q = whole_numbers(dim, lens, 2, dim, 16, f8, group, 4)
    pool, _, out, lse, sc = chunk_call(c, [1] * 4, group, 0, late, q=q.cuda(), scale=scale)
    check_sharp(c, [1] * 4, q, scale, out, lse, 0, late, pool.mass)
    other = device_pool(c)
    one, ol = torch.empty_like(out), torch.empty_like(lse)
    flags = gdn.ATTN_ACCUM_MASS if late else 0
    n = gdn.attn_workspace_bytes(other, 4, 2 * group, 900, flags)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    gdn.attn_decode_paged(other, 0, i32(c.slots), i32(lens), q.cuda(), one, 900, scale=scale, lse=ol, workspace=ws,
                          flags=flags)
    check_sharp(c, [1] * 4, q, scale, one, ol, 0, late, other.mass)


@pytest.mark.parametrize("far", [2e3, 1e5, 1e7, 1e10])
@pytest.mark.parametrize("dim,f8", [(64, False), (128, False), (256, True)])
def test_far_and_near_rows_of_a_wave(dim, f8, far):
    """Every third row's scores are `far` times the others': the others are as they are alone."""
    new, lens = [60, 9], [200, 120]
    c, q = whole_numbers(dim + 1, lens, 1, dim, 16, f8, 4, 69)
    grow = torch.ones(69, 4, 1)
    grow.view(-1)[::3] = float(2 ** int(np.log2(far)))
    q = torch.where(grow > 1, q, 0.1 * torch.randn(q.shape, generator=c.g))
    big, small = (q * grow).to(torch.bfloat16), (q * (grow == 1)).to(torch.bfloat16)
    pool, _, out, lse, sc = chunk_call(c, new, 4, q=big.cuda(), scale=1.0)
    near = (grow == 1).expand(69, 4, 1)[..., 0]
    _, _, alone, al, _ = chunk_call(c, new, 4, q=small.cuda(), scale=1.0)
    check_chunk(c, new, small, sc, alone, al)
    # both within the weights' and the output's rounding of the same value
    v = stored(torch.nan_to_num(c.v.float()), False).abs().max().float() * c.v_scale
    assert ((out - alone).float().abs().cpu()[near] <= 4 * 2.0 ** -8 * v).all()
    assert ((lse - al).abs().cpu()[near] <= 2.0 ** -18 * (1 + al.abs().cpu()[near])).all()
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    # a far row's scores differ by `far` or not at all
    at = 0
    for b, n in enumerate(new):
        rows = [(r, j) for r in range(n) for j in range(4) if not near[at + r, j]]
        t = c.table[c.slots[b]].numpy()
        i = np.arange(lens[b])
        K, V = (x[0].float().double().numpy()[t[i // 16], 0, i % 16] for x in (c.k, c.v))
        for r, j in rows:
            place = lens[b] - n + r
            s = K[:place + 1] @ big[at + r, j].float().double().numpy()
            top = s == s.max()
            vv = c.v_scale * V[:place + 1][top]
            want, spread = vv.mean(axis=0), np.abs(vv).mean(axis=0)
            tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -16) * (1 + 2.0 ** -8) * spread
            assert (np.abs(out[at + r, j].float().cpu().double().numpy() - want) <= tol).all(), (b, r, j)
        at += n


@pytest.mark.parametrize("scale", [0.3, 1e4, 1e8, 3e20])
def test_far_scores_of_ordinary_heads(scale):
    """Scores of any fraction: finite results, the logarithm of their sum within its roundings, and
    weights that sum to one for every row."""
    for dim, f8 in ((64, False), (128, True), (256, False), (256, True)):
        c = make_cache(dim, [300, 90], None, 2, dim, 16, f8)
        c.mass.zero_()
        pool, q, out, lse, sc = chunk_call(c, [100, 3], 3, late=9, scale=float(np.float32(scale)))
        check_chunk(c, [100, 3], q, sc, out, lse)
        assert torch.isfinite(out.float()).all()
        total = pool.mass.sum(dim=-1).cpu()[0]
        for b, rows in ((0, 9), (1, 3)):
            assert ((total[c.slots[b]] - 3 * rows).abs() <= 3 * rows * 2.0 ** -12).all(), (dim, total[c.slots[b]])
