"""GPU: attention of chunks over values at the ends of their range, joined from many pieces, and of
requests without new tokens."""
import pytest
import torch

from tests.kv_helpers import make_cache, stored
from tests.test_gpu_kv_prompt import check_chunk, chunk_call

pytestmark = pytest.mark.gpu


def set_rows(x, c, b, at, rows):
    """rows [n, H, D] at the places `at` of request b."""
    page = c.table[c.slots[b]][at // c.page].long()
    bits = torch.uint8 if c.f8 else torch.int16
    x[0].view(bits)[page, :, at % c.page] = stored(rows, c.f8).view(bits)


@pytest.mark.parametrize("max_len", [None, 9000])
@pytest.mark.parametrize("dim,n,new", [(64, 950, 3), (128, 700, 30), (256, 470, 5)])
def test_sums_of_the_largest_values(dim, n, new, max_len):
    """Visible places times the largest value just below the end of fp32, and scores that rise by
    almost as much as the exponent's reference may stay behind: the mean is finite, and there."""
    c = make_cache(dim, [n], None, 1, dim, 16, capacity=max_len)
    block = 32 if dim == 256 else 64
    at = torch.arange(n)
    k = torch.zeros(n, 1, dim)
    # a lane has half of a block's places: 16 e^2.75 or 32 e^2 are just below 256
    k[:, 0, 0] = torch.where(at % (5 * block) < block, 0.0, 2.75 if dim == 256 else 2.0)
    v = torch.full((n, 1, dim), 3.3e38 / n)
    v[:, 0, 1::2] *= -1
    v[:, 0, 2] = torch.randn(n, generator=c.g)
    set_rows(c.k, c, 0, at, k)
    set_rows(c.v, c, 0, at, v)
    q = torch.zeros(new, 2, dim, dtype=torch.bfloat16)
    q[:, :, 0] = 1.0
    pool, _, out, lse, sc = chunk_call(c, [new], 2, late=2, q=q.cuda(), scale=1.0, max_len=max_len)
    assert torch.isfinite(out.float()).all()
    check_chunk(c, [new], q, sc, out, lse, 0, 2, pool.mass)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("n", [900, 5000, 27000])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("first", [True, False])
def test_values_that_are_not_finite_and_have_no_weight(dim, n, first, value):
    """A value that is not finite and whose weight is below 2^-100 of the largest makes its column so too or is
    as if it were not there; never NaN from an infinite one.  Divided or not, and whichever piece comes first."""
    new = 3
    c, clean = (make_cache(dim, [n], None, 1, dim, 64) for _ in range(2))
    at = torch.arange(n)
    low = at < n // 2 if first else (at >= n // 2) & (at < n - new)
    k = torch.zeros(n, 1, dim)
    k[:, 0, 0] = torch.where(low, -200.0, 0.0)
    for x in (c, clean):
        set_rows(x.k, x, 0, at, k)
    bad = at[low][17:18]
    set_rows(c.v, c, 0, bad, torch.full((1, 1, dim), value))
    q = torch.randn(new, 2, dim, generator=c.g).to(torch.bfloat16)
    q[:, :, 0] = 1.0
    pool, _, out, lse, sc = chunk_call(c, [new], 2, late=2, q=q.cuda(), scale=1.0)
    _, _, want, wl, _ = chunk_call(clean, [new], 2, q=q.cuda(), scale=1.0)
    check_chunk(clean, [new], q, sc, want, wl)
    assert torch.equal(lse, wl) and torch.isfinite(pool.mass).all()
    o, w = out.float(), want.float()
    shown = torch.isnan(o) if value != value else o == value
    assert (shown | ((o - w).abs() <= 4 * 2.0 ** -8 * (w.abs() + 4))).all()


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("dim,new,group", [(64, 1, 1), (64, 4, 2), (128, 2, 3), (256, 3, 1)])
def test_join_of_hundreds_of_pieces(dim, new, group, f8):
    """One request over so many places that the pieces of a tile take several rounds of a wave's lanes:
    maxima that rise over the pieces, that fall, and first pieces that see nothing."""
    import gated_delta_rule_slot_amd as gdn

    n = 27000
    for kind in ("rises", "falls", "late"):
        c = make_cache(dim, [n], None, 1, dim, 64, f8)
        at = torch.arange(n)
        ramp = 12.0 * at / n if kind == "rises" else 12.0 * (1 - at / n)
        if kind != "late":
            k = 0.3 * torch.randn(n, 1, dim, generator=c.g)
            k[:, 0, 0] = ramp
            set_rows(c.k, c, 0, at, k)
        else:
            c.table[c.slots[0], :21000 // 64] = 0
        q = torch.randn(new, group, dim, generator=c.g).to(torch.bfloat16)
        q[:, :, 0] = 2.0
        pool, _, out, lse, sc = chunk_call(c, [new], group, late=2, q=q.cuda(), scale=0.8 if kind != "late" else 0.1)
        assert gdn.attn_prefill_workspace_bytes(pool, 1, new, group, n) >= 65 * new * group * (dim + 2) * 4
        check_chunk(c, [new], q, sc, out, lse, 0, 2, pool.mass)
        assert int(pool.err_word.item()) == (gdn.ERRW_BAD_PAGE if kind == "late" else 0)


@pytest.mark.parametrize("where", [0, 2, 4])
def test_requests_without_new_tokens_are_checked_too(where):
    """Bad slots, lengths and begins of a request that has no rows set their bit; the others' rows are there."""
    import gated_delta_rule_slot_amd as gdn

    new = [9, 20, 30, 5, 6]
    new[where] = 0
    lens, slots = [50, 60, 70, 80, 90], [1, 4, 3, 2, 5]
    for change, bit in ((dict(), 0), (dict(slots=0), 0), (dict(slots=-3), 0), (dict(slots=6), gdn.ERRW_BAD_SLOT),
                        (dict(lens=-1), gdn.ERRW_BAD_SEQLENS), (dict(lens=97), gdn.ERRW_BAD_SEQLENS),
                        (dict(begins=-1), gdn.ERRW_BAD_SEQLENS), (dict(lens=0), 0),
                        (dict(slots=0, lens=-1), 0)):
        c = make_cache(3, lens, None, 2, 128, 16, slots=slots, capacity=96)
        for name, x in change.items():
            getattr(c, name)[where] = x
        pool, q, out, lse, sc = chunk_call(c, new, 4, late=3, max_len=96)
        assert int(pool.err_word.item()) == bit, change
        c.slots[where] = 0
        check_chunk(c, new, q, sc, out, lse, 0, 3, pool.mass)


def test_attention_leaves_the_table_and_the_cache_alone():
    """Bad pages, slots and lengths among the requests: table, keys and values as they were."""
    c = make_cache(21, [50, 60, 70, 80], None, 2, 128, 16, slots=[1, 0, 3, 2])
    c.table[3, 2], c.table[2, 1] = 0, c.k.shape[1]
    c.lens[0] = 200
    table = c.table.clone()
    pool, q, out, lse, sc = chunk_call(c, [10, 11, 12, 13], 4, late=5, max_len=80)
    assert torch.equal(pool.page_table.cpu(), table) and int(pool.err_word.item()) != 0
    assert torch.equal(pool.k.cpu().view(torch.int16), c.k.view(torch.int16))
    assert torch.equal(pool.v.cpu().view(torch.int16), c.v.view(torch.int16))
