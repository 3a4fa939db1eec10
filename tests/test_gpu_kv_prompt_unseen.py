"""GPU: attention of chunks over page tables whose entries before the first visible place are no
pages (a sliding window that gave its front pages back, a cache cut at its front)."""
import pytest
import torch

from tests.kv_helpers import make_cache
from tests.test_gpu_kv_prompt import check_chunk, chunk_call

pytestmark = pytest.mark.gpu


def without_front(c, new, window):
    """The cache's table with entries that are no pages wherever a page lies wholly before the first
    place that a request's new tokens see; how many."""
    dropped = 0
    for b, n in enumerate(new):
        L = c.lens[b]
        first = max(c.begins[b], L - n - window + 1 if window else 0)
        for e in range(min(first // c.page, c.table.shape[1])):
            c.table[c.slots[b], e] = (0, c.k.shape[1], -1, 2 ** 31 - 1)[e % 4]
            dropped += 1
    return dropped


def both_tables(seed, new, cached, begins, kv_heads, dim, page, f8, group, window, late, max_len=None):
    lens = [n + m for n, m in zip(new, cached)]
    full, cut = (make_cache(seed, lens, begins, kv_heads, dim, page, f8, capacity=max_len) for _ in range(2))
    assert without_front(cut, new, window) > 0
    pool, q, want, wl, sc = chunk_call(full, new, group, window, late, max_len=max_len)
    assert int(pool.err_word.item()) == 0
    cut_pool, _, out, lse, _ = chunk_call(cut, new, group, window, late, max_len=max_len, q=q.cuda())
    assert int(cut_pool.err_word.item()) == 0
    assert torch.equal(out, want) and torch.equal(lse, wl) and torch.equal(cut_pool.mass, pool.mass)
    assert torch.equal(cut_pool.page_table.cpu(), cut.table)
    check_chunk(cut, new, q, sc, out, lse, window, late, cut_pool.mass)


@pytest.mark.parametrize("by_window", [False, True])
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("page", [1, 4, 16, 64])
@pytest.mark.parametrize("dim,group", [(64, 3), (128, 4), (256, 16)])
def test_pages_before_the_first_visible_place(dim, group, page, f8, by_window):
    begins, window = ([0, 0, 0], 50) if by_window else ([117, 76, 230], 0)
    both_tables(page + dim, [40, 7, 1], [200, 133, 240], begins, 2, dim, page, f8, group, window, 5)


@pytest.mark.parametrize("by_window", [False, True])
@pytest.mark.parametrize("dim,page,f8", [(64, 4, True), (128, 16, False), (256, 1, False), (256, 16, True)])
def test_pages_before_the_first_visible_place_divided(dim, page, f8, by_window):
    """The same where the places are divided over workgroups."""
    begins, window = ([0, 0], 2777) if by_window else ([1001, 47], 0)
    both_tables(page, [3, 1], [5000, 2990], begins, 1, dim, page, f8, 2, window, 2, max_len=9000)


@pytest.mark.parametrize("page", [1, 16])
def test_tables_of_requests_that_see_nothing(page):
    """No place is visible to any new token, or to the first tiles' (16 query heads: 8 tokens a tile):
    entries that are no pages are not looked at."""
    c = make_cache(page, [40, 60], [41, 48], 1, 128, page)
    c.table[c.slots[0]] = 0
    c.table[c.slots[1], :48 // page] = 0
    pool, q, out, lse, sc = chunk_call(c, [40, 60], 16, late=9)
    assert int(pool.err_word.item()) == 0
    assert not out[:88].float().any() and torch.isneginf(lse[:88]).all()
    check_chunk(c, [40, 60], q, sc, out, lse, 0, 9, pool.mass)


@pytest.mark.parametrize("page", [4, 16])
def test_the_first_visible_place_in_no_page(page):
    """The page of the first visible place itself is looked at: the bit is set, the place left out."""
    import gated_delta_rule_slot_amd as gdn

    c = make_cache(page, [150], [70], 1, 128, page)
    c.table[c.slots[0], :70 // page + 1] = 0
    pool, q, out, lse, sc = chunk_call(c, [20], 4, late=3)
    assert int(pool.err_word.item()) == gdn.ERRW_BAD_PAGE
    check_chunk(c, [20], q, sc, out, lse, 0, 3, pool.mass)
