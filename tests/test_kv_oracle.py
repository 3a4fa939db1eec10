"""Pins of the float64 definitions of the full-attention operators against things other
than themselves (CPU)."""
import numpy as np
import pytest
import torch

from oracle import kv_ops


def test_e4m3_values_and_rounding_match_torch():
    bits = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    want = bits.view(torch.float8_e4m3fn).float().double().numpy()
    got = kv_ops.e4m3_values()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])
    grid = got[:0x7f]
    mid = (grid[1:] + grid[:-1]) / 2  # every tie, and its two neighbours in fp32
    x = np.concatenate([grid, mid, np.nextafter(mid.astype(np.float32), np.float32(1e9)).astype(np.float64),
                        np.nextafter(mid.astype(np.float32), np.float32(0)).astype(np.float64),
                        np.random.default_rng(1).normal(0, 60, 4000).astype(np.float32), [447.9, 500.0, 1e30]])
    x = np.concatenate([x, -x])
    want = torch.from_numpy(x).float().clamp(-448, 448).to(torch.float8_e4m3fn).float().double().numpy()
    assert np.array_equal(kv_ops.e4m3_round(x), want)
    assert np.isnan(kv_ops.e4m3_round(np.array([np.nan]))).all()


@pytest.mark.parametrize("begin,length", [(0, 1), (0, 37), (5, 37), (36, 37), (9, 9), (12, 9)])
def test_attend_matches_torch_softmax_over_gathered_rows(begin, length):
    g = torch.Generator().manual_seed(3)
    P, H, S, D, G = 9, 2, 8, 16, 3
    k, v = (torch.randn(P, H, S, D, generator=g, dtype=torch.float64) for _ in range(2))
    table = torch.zeros(3, 6, dtype=torch.int64)
    table[2, :5] = torch.tensor([4, 1, 8, 3, 6])
    q = torch.randn(H * G, D, generator=g, dtype=torch.float64)
    out, lse, w, _ = kv_ops.attend(k.numpy(), v.numpy(), table.numpy(), 2, begin, length, q.numpy(), 0.25)
    if begin >= length:
        assert not out.any() and np.isneginf(lse).all() and w.shape == (H, 0)
        return
    rows_k = torch.stack([k[table[2, i // S], :, i % S] for i in range(begin, length)], 1)
    rows_v = torch.stack([v[table[2, i // S], :, i % S] for i in range(begin, length)], 1)
    s = 0.25 * torch.einsum("hgd,htd->hgt", q.view(H, G, D), rows_k)
    p = torch.softmax(s, -1)
    assert np.allclose(out, torch.einsum("hgt,htd->hgd", p, rows_v).reshape(H * G, D).numpy(), atol=1e-13)
    assert np.allclose(lse, torch.logsumexp(s, -1).reshape(-1).numpy(), atol=1e-13)
    assert np.allclose(w, p.sum(1).numpy(), atol=1e-13)


def test_attend_skips_bad_pages():
    g = np.random.default_rng(0)
    k, v = g.normal(size=(2, 4, 1, 4, 8))
    q = g.normal(size=(2, 8))
    table = np.array([[0, 0, 0], [2, 9, 3]])
    out, lse, w, _ = kv_ops.attend(k, v, table, 1, 0, 12, q, 1.0)
    good = np.array([[0, 0], [2, 3]])
    o2, l2, w2, _ = kv_ops.attend(k, v, good, 1, 0, 8, q, 1.0)
    assert np.allclose(out, o2) and np.allclose(lse, l2)
    assert not w[0, 4:8].any() and np.allclose(np.delete(w, range(4, 8), 1), w2)
    none, lse, _, _ = kv_ops.attend(k, v, np.array([[0], [0]]), 1, 0, 3, q, 1.0)
    assert not none.any() and np.isneginf(lse).all()


def test_plan_worked_by_hand():
    # 7 tokens, budget 4; sink position 0 (at index 5), the newest position 11 (at index 1)
    mass = np.array([0.5, 0.0, 0.9, 0.5, np.nan, 0.1, 0.5])
    pos = np.array([3, 11, 5, 6, 7, 0, 9])
    # protected: indices 5 and 1; then 2 (0.9), then 0 (0.5, the lowest of three equal)
    assert kv_ops.plan(mass, pos, 7, 12, 4, 1, 1) == [(5, 3)]
    assert kv_ops.plan(mass, pos, 4, 12, 4, 1, 1) == []
    # nothing protected: 2, 0, 3, 6 stay
    assert kv_ops.plan(mass, pos, 7, 100, 4, 0, 0) == [(6, 1)]
    # more protected than the budget: the lowest indices
    assert kv_ops.plan(mass, pos, 7, 12, 2, 100, 0) == []


def test_block_norm_worked_by_hand():
    y = np.array([[3.0, 4.0]])
    w = np.array([2.0, 1.0])
    out, r = kv_ops.block_norm(y, w_post=w, eps=0.5)  # mean square 12.5, + 0.5 = 13
    assert r is None and np.allclose(out, [[6 / 13 ** 0.5, 4 / 13 ** 0.5]])
    out, r = kv_ops.block_norm(y, gate=np.array([[0.0, 0.0]]), act="sigmoid", scale=2.0,
                               residual=np.array([[1.0, -4.0]]))
    assert np.allclose(r, [[4.0, 0.0]]) and np.allclose(out, r)
    out, r = kv_ops.block_norm(y, residual=np.array([[0.0, -4.0]]), w_pre=np.zeros(2), eps=1e-12, plus_one=True)
    assert np.allclose(r, [[3.0, 0.0]]) and np.allclose(out, [[2 ** 0.5, 0.0]])
    out, _ = kv_ops.block_norm(y, gate=np.array([[1.0, -800.0]]), act="silu")
    assert np.allclose(out, [[3 / (1 + np.exp(-1.0)), 0.0]])
