"""GPU: whole steps (page tables, rotary append, attention) that go on after an eviction and after a
release, on pages that were given back, against a host model of every request."""
import numpy as np
import pytest
import torch

from oracle import kv_ops
from tests.kv_helpers import i32, stored
from tests.test_gpu_kv_prompt import Steps, same

pytestmark = pytest.mark.gpu


class Server:
    """A layer's requests in slots, and per request and key-value head the keys, values and positions
    that its cache should hold, in any order."""

    def __init__(self, f8, dim, rot, adjacent, slots=(2, 3, 1), H=2, G=3, page=16, pages=40, most=12):
        import gated_delta_rule_slot_amd as gdn

        self.gdn, self.f8, self.dim, self.adjacent = gdn, f8, dim, adjacent
        self.H, self.G, self.page, self.pages, self.cap = H, G, page, pages, most * page
        self.slots, self.B = list(slots), len(slots)
        self.g = torch.Generator().manual_seed(dim + page)
        self.ks, self.vs = (0.5, 0.75) if f8 else (1.0, 1.0)
        dt = torch.float8_e4m3fn if f8 else torch.bfloat16
        k = torch.full((1, pages, H, page, dim), float("nan")).to(dt).cuda()
        n = max(slots) + 1
        self.pool = gdn.kv_pool_create(
            k, k.clone(), torch.zeros(n, most, dtype=torch.int32, device="cuda"),
            mass=torch.zeros(1, n, H, self.cap, device="cuda"),
            pos=torch.zeros(1, n, H, self.cap, dtype=torch.int32, device="cuda"), err_word=i32([0]),
            k_scale=self.ks, v_scale=self.vs)
        self.freqs, self.amp = gdn.rope_frequencies(rot, scaling=gdn.ROPE_LINEAR, factor=2.0)
        self.free, self.n_free = i32(list(range(pages - 1, 0, -1)) + [0]), i32([pages - 1])
        self.lens, self.nxt, self.sl = i32([0] * self.B), i32([0] * self.B), i32(self.slots)
        self.model = [[[] for _ in range(H)] for _ in range(self.B)]
        self.at, self.length = [0] * self.B, [0] * self.B

    def mapped(self):
        t = self.pool.page_table.cpu()
        return [{int(p) for p in t[s, :-(-n // self.page)]} for s, n in zip(self.slots, self.length)]

    def check_pages(self):
        """Every page is in one request's row or in the list."""
        used = [p for s in self.mapped() for p in s]
        listed = self.free[:int(self.n_free.item())].tolist()
        assert sorted(used + listed) == list(range(1, self.pages))

    def step(self, new, name):
        gdn, H, G, dim, B = self.gdn, self.H, self.G, self.dim, self.B
        T, sc = sum(new) + 4, dim ** -0.5
        x = torch.randn(T, (H * G + 2 * H) * dim, generator=self.g).to(torch.bfloat16)
        widths = [H * G * dim, H * dim, H * dim]
        q, kn, vn = (t.view(T, -1, dim) for t in x.cuda().split(widths, dim=1))
        cu, so = i32([0] * (B + 1)), i32([0] * B)
        ts, ti, tp = (i32([0] * T) for _ in range(3))
        gdn.kv_batch_map(self.pool, self.sl, self.lens, self.free, self.n_free, cu, so, self.lens, ts, ti,
                         new_len=i32(new), next_pos=self.nxt, next_pos_out=self.nxt, token_pos=tp)
        qr, out = (torch.full((T, H * G, dim), -7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        gdn.rope_append(self.pool, 0, ts, ti, tp, q, qr, kn, vn, self.freqs.cuda(), amplitude=self.amp,
                        layout=gdn.ROPE_INTERLEAVED if self.adjacent else gdn.ROPE_HALF)
        lse = torch.empty(T, H * G, device="cuda")
        n = gdn.attn_prefill_workspace_bytes(self.pool, B, T, H * G, self.cap, T)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        gdn.attn_prefill_paged(self.pool, 0, cu, so, self.lens, qr, out, self.cap, scale=sc, mass_tokens=T, lse=lse,
                               workspace=ws)
        torch.cuda.synchronize()
        assert int(self.pool.err_word.item()) == 0, name
        xq, xk, xv = (t.float().double().numpy().reshape(T, -1, dim) for t in x.split(widths, dim=1))
        got, at = out.float().cpu().double().numpy(), 0
        for b, n in enumerate(new):
            p = np.arange(self.at[b], self.at[b] + n)
            rows = slice(at, at + n)
            kk = stored(torch.tensor(kv_ops.turn(xk[rows], p, self.freqs.numpy(), self.amp, self.adjacent) / self.ks)
                        .float(), self.f8).double().numpy() * self.ks
            vv = stored(torch.tensor(xv[rows] / self.vs).float(), self.f8).double().numpy() * self.vs
            qd = kv_ops.turn(xq[rows], p, self.freqs.numpy(), self.amp, self.adjacent)
            for i in range(n):
                for h in range(H):
                    self.model[b][h].append((kk[i, h], vv[i, h], int(p[i])))
                    K, V = (np.stack([m[e] for m in self.model[b][h]]) for e in (0, 1))
                    for j in range(h * G, (h + 1) * G):
                        s = sc * (K @ qd[i, j])
                        w = np.exp(s - s.max())
                        w /= w.sum()
                        # a key may round the other way where fp32 and fp64 fall on either side of a border: one
                        # step of the stored type for each, beside the bf16 roundings
                        step = 2.0 ** -3 if self.f8 else 2.0 ** -7
                        err = sc * step * (np.abs(K) @ np.abs(qd[i, j])).max() * 0.25 + 2.0 ** -6
                        tol = 2.0 ** -7 * np.abs(w @ V) + 2 * err * (w @ np.abs(V)) + 1e-6
                        assert (np.abs(got[at + i, j] - w @ V) <= tol).all(), (name, b, i, j)
            at += n
            self.at[b] += n
            self.length[b] += n
        assert self.lens.tolist() == self.length and self.nxt.tolist() == self.at
        assert (got[at:] == -7.0).all()
        self.check_pages()

    def cut(self, budget):
        """Evict down to the budget, and give the pages behind it back; these."""
        gdn, B, H = self.gdn, self.B, self.H
        nm = torch.zeros(1, B, H, dtype=torch.int32, device="cuda")
        mv = torch.zeros(1, B, H, budget, 2, dtype=torch.int32, device="cuda")
        kept = i32([0] * B)
        gdn.kv_evict_plan(self.pool, 0, 1, self.sl, self.lens, self.nxt, 2 * budget, budget, 2, 20, nm, mv, kept)
        gdn.kv_evict_apply(self.pool, 0, 1, self.sl, nm, mv)
        return self.give_back(kept)

    def give_back(self, keep):
        before = int(self.n_free.item())
        self.gdn.kv_release(self.pool, self.sl, self.lens, self.free, self.n_free, keep=keep)
        self.lens.copy_(keep)
        self.length = keep.tolist()
        given = set(self.free[before:int(self.n_free.item())].tolist())
        pos = self.pool.pos.cpu()
        for b, s in enumerate(self.slots):
            for h in range(self.H):
                kept = set(pos[0, s, h, :self.length[b]].tolist())
                assert len(kept) == self.length[b]
                self.model[b][h] = [m for m in self.model[b][h] if m[2] in kept]
                assert len(self.model[b][h]) == self.length[b]
        self.check_pages()
        return given


@pytest.mark.parametrize("f8,dim,rot,adjacent", [(False, 128, 128, False), (True, 64, 32, True),
                                                 (False, 256, 64, False)])
def test_steps_after_a_cut_and_after_a_release(f8, dim, rot, adjacent):
    s = Server(f8, dim, rot, adjacent)
    s.step([40, 17, 1], "prompts")
    s.step([30, 60, 33], "chunks")
    given = s.cut(60)
    assert s.length == [60, 60, 34] and s.at == [70, 77, 34] and given
    # decode steps and a chunk behind the kept tokens, at positions past their places
    s.step([1, 1, 1], "after the cut")
    s.step([1, 0, 2], "a request that waits")
    before = s.mapped()
    s.step([25, 0, 30], "chunks after the cut")
    taken = set().union(*s.mapped()) - set().union(*before)
    assert taken & given  # pages that were given back hold new tokens
    # again, and the first request ends: its slot begins anew on its own and others' pages
    given = s.cut(50)
    assert s.length == [50, 50, 50] and given
    s.step([1, 7, 0], "after the second cut")
    ends = s.give_back(i32([0, s.length[1], s.length[2]]))
    assert len(ends) == 4
    s.nxt[0] = 0
    s.at[0] = 0
    s.step([70, 1, 1], "a new request in the slot")
    assert s.mapped()[0] & ends
    s.step([1, 33, 1], "and on")
    s.give_back(i32([0, 0, 0]))
    assert int(s.n_free.item()) == s.pages - 1 and not s.pool.page_table[1:].any()


@pytest.mark.parametrize("most", [60, 600])
def test_steps_replayed_after_a_release(most):
    """A captured step goes on after everything was given back, on the pages in the order in which they came back."""
    a, b = Steps(most=most), Steps(most=most)
    start = [t.clone() for t in (a.lens, a.nxt, a.n_free, a.pool.page_table)]
    graph = torch.cuda.CUDAGraph()
    a.step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        a.step()
    for t, s in zip((a.lens, a.nxt, a.n_free, a.pool.page_table), start):
        t.copy_(s)
    for turn in range(3):
        table, before = b.pool.page_table.tolist(), b.free[:int(b.n_free.item())].tolist()
        taken = set()
        for _ in range(7):
            x = torch.randn_like(a.x)
            a.x.copy_(x), b.x.copy_(x)
            graph.replay()
            b.step()
            same(a.state(), b.state())
            taken |= {p for row in b.pool.page_table.tolist() for p in row if p}
        assert not any(any(r) for r in table) and taken == set(before[len(before) - len(taken):])
        assert a.out.float().abs().sum() > 0 and torch.isfinite(a.out.float()).all()
        for s in (a, b):
            s.release()
            s.lens.zero_()
        same(a.state(), b.state())
        assert int(a.n_free.item()) == len(before) and not a.pool.page_table.any()
        assert sorted(a.free.tolist()) == sorted(before)
