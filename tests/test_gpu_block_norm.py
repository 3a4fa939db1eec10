"""GPU: block_norm against its float64 definition (oracle/kv_ops.py)."""
import numpy as np
import pytest
import torch

from oracle import kv_ops

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def case(seed, tokens, groups, dim, post, gate, res, pre, wt="bf16", plus_one=False, scale=1.0, eps=1e-6, y_pad=0,
         g_pad=0, y_std=1.0):
    g = torch.Generator().manual_seed(seed)
    w = lambda: ((0.0 if plus_one else 1.0) + 0.3 * torch.randn(dim, generator=g)).to(DT[wt])  # noqa: E731
    y = (y_std * torch.randn(tokens, groups * dim + y_pad, generator=g)).to(torch.bfloat16)
    z = (2.0 * torch.randn(tokens, groups * dim + g_pad, generator=g)).to(torch.bfloat16)
    return dict(y=y, y_pad=y_pad, z=z if gate else None, g_pad=g_pad, act=gate, w_post=w() if post else None,
                w_pre=w() if pre else None, scale=scale, eps=eps, plus_one=plus_one,
                res=(3 * torch.randn(tokens, groups, dim, generator=g)).to(DT[res]) if res else None,
                shape=(tokens, groups, dim))


def run(c, in_place=False, stream=None):
    import gated_delta_rule_slot_amd as gdn

    T, G, D = c["shape"]
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    y = dev(c["y"])[:, c["y_pad"]:].view(T, G, D)
    z = dev(c["z"])[:, c["g_pad"]:].view(T, G, D) if c["z"] is not None else None
    res = dev(c["res"])
    out = y if in_place and not c["y_pad"] else torch.full((T, G, D), -7.0, dtype=torch.bfloat16, device="cuda")
    ro = None if res is None else res if in_place else torch.full_like(res, -7.0)
    act = {None: gdn.ACT_NONE, "none": gdn.ACT_NONE, "silu": gdn.ACT_SILU, "sigmoid": gdn.ACT_SIGMOID}[c["act"]]
    gdn.block_norm(y, out, w_post=dev(c["w_post"]), gate=z, act=act, scale=c["scale"], residual=res, residual_out=ro,
                   w_pre=dev(c["w_pre"]), eps=c["eps"], flags=gdn.NORM_PLUS_ONE if c["plus_one"] else 0, stream=stream)
    return out, ro


def check(c, out, ro):
    f = lambda t: None if t is None else t.float().double().numpy()  # noqa: E731
    T, G, D = c["shape"]
    y = f(c["y"])[:, c["y_pad"]:].reshape(T, G, D)
    z = f(c["z"])[:, c["g_pad"]:].reshape(T, G, D) if c["z"] is not None else None
    one = 1.0 if c["plus_one"] else 0.0
    want, wr = kv_ops.block_norm(y, f(c["w_post"]), z, c["act"], c["scale"], f(c["res"]), f(c["w_pre"]), c["eps"],
                                 c["plus_one"])
    u, _ = kv_ops.block_norm(y, f(c["w_post"]), z, c["act"], c["scale"], None, None, c["eps"], c["plus_one"])
    # u is a product of up to five factors, each within a few units of 2^-24 (the root's
    # argument is a sum of dim squares taken over 8 values a thread and a tree: under 30
    # roundings, halved by the root; exp within 2^-21 for |z| < 16): 2^-18 of it in all.  In r
    # the parts may cancel, so its error goes by |residual| + |u|; the second norm adds 2^-18
    # again.  Then each output is rounded once.
    part = np.abs(u) + (np.abs(f(c["res"])) if c["res"] is not None else 0.0)
    err = 2.0 ** -18 * part
    if c["w_pre"] is not None:
        r = u if wr is None else wr
        inv = 1.0 / np.sqrt((r * r).mean(-1, keepdims=True) + c["eps"])
        # an error e of each r moves the root mean square by at most its own root mean square
        rel = np.sqrt((err * err).mean(-1, keepdims=True)) * inv + 2.0 ** -18
        tol = np.abs(inv * (one + f(c["w_pre"]))) * err + np.abs(want) * rel
    else:
        tol = err
    got = out.float().cpu().double().numpy()
    assert (np.abs(got - want) <= tol + 2.0 ** -8 * np.abs(want) + 1e-38).all(), np.abs(got - want).max()
    if wr is not None:
        gr = ro.float().cpu().double().numpy()
        half = 2.0 ** -8 if ro.dtype == torch.bfloat16 else 2.0 ** -24
        assert (np.abs(gr - wr) <= err + half * np.abs(wr)).all(), np.abs(gr - wr).max()


FORMS = [  # post, gate, residual, pre
    (True, "silu", None, False), (True, "sigmoid", "bf16", True), (False, None, "f32", True),
    (True, None, "bf16", False), (False, "none", None, False), (False, "silu", "bf16", True), (True, None, None, True),
]


@pytest.mark.parametrize("post,gate,res,pre", FORMS)
@pytest.mark.parametrize("tokens,groups,dim", [(1, 1, 8), (3, 5, 64), (7, 3, 128), (5, 2, 136), (9, 1, 264), (4, 1, 512),
                                               (3, 1, 520), (2, 1, 2048), (3, 1, 2056), (2, 1, 5120), (2, 1, 8200),
                                               (1, 1, 16392), (1, 1, 32768)])
def test_block_norm_parity(tokens, groups, dim, post, gate, res, pre):
    for wt, plus in (("bf16", False), ("f32", True)):
        c = case(dim + tokens, tokens, groups, dim, post, gate, res, pre, wt, plus, scale=0.37, y_pad=8, g_pad=24)
        check(c, *run(c))


def test_block_norm_many_rows_and_in_place():
    """The recurrence's heads (odd row counts), and residual_out = residual, out = y."""
    c = case(3, 131, 32, 128, True, "silu", None, False, "f32")
    check(c, *run(c))
    c = case(4, 129, 1, 2048, True, "sigmoid", "bf16", True, scale=0.25)
    check(c, *run(c, in_place=True))
    c = case(5, 33, 3, 72, True, None, "f32", True)
    check(c, *run(c, in_place=True))


def test_block_norm_streamed():
    """Tensors past the size from which they are not kept in the caches."""
    c = case(11, 3101, 1, 4096, True, "silu", "f32", True, scale=0.5, g_pad=8)
    check(c, *run(c))
    c = case(12, 12001, 8, 136, True, "sigmoid", "bf16", False, "f32")
    check(c, *run(c, in_place=True))


def test_block_norm_of_more_rows_than_one_grid_dimension_takes():
    """2.1 M rows of a workgroup each, bit for bit what smaller calls give."""
    import gated_delta_rule_slot_amd as gdn

    T, D = (1 << 21) + 3, 520
    y = torch.randn(T, 1, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)).to(torch.bfloat16)
    w = torch.rand(D, device="cuda")
    out = torch.full_like(y, -7.0)
    gdn.block_norm(y, out, w_post=w)
    part = torch.empty(4096, 1, D, dtype=torch.bfloat16, device="cuda")
    for t in (0, 1 << 20, T - 4096):
        gdn.block_norm(y[t:t + 4096], part, w_post=w)
        assert torch.equal(out[t:t + 4096], part), t
    assert not (out == -7.0).all(dim=-1).any()


@pytest.mark.parametrize("std,eps", [(1e-18, 1e-6), (1e-3, 1e-5), (1e15, 1e-6), (0.0, 1e-6)])
def test_block_norm_small_large_and_zero_rows(std, eps):
    """Rows whose squares leave bf16's comfortable range, and rows of zeros."""
    c = case(6, 5, 2, 256, True, "sigmoid", None, False, eps=eps, y_std=std)
    check(c, *run(c))
    c = case(7, 5, 1, 1024, False, None, "f32", True, eps=eps, y_std=std)
    check(c, *run(c))


def test_block_norm_gates_at_the_ends():
    c = case(8, 4, 1, 64, False, "silu", None, False)
    c["z"][:, ::4], c["z"][:, 1::4], c["z"][:, 2::4] = -200.0, 200.0, 0.0
    check(c, *run(c))


def test_block_norm_rows_do_not_touch_their_neighbours():
    """A NaN row stays alone, and nothing behind the last row is written."""
    import gated_delta_rule_slot_amd as gdn

    for dim in (64, 136, 2056):
        y = torch.randn(6, 1, dim, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
        y[2] = float("nan")
        store = torch.full((8, 1, dim), -7.0, dtype=torch.bfloat16, device="cuda")
        w = torch.ones(dim, device="cuda")
        gdn.block_norm(y, store[:6], w_post=w)
        got = store.float().cpu()
        assert torch.isnan(got[2]).all() and torch.isfinite(got[[0, 1, 3, 4, 5]]).all() and (got[6:] == -7).all()


def test_block_norm_in_a_graph():
    c = case(9, 40, 1, 2048, True, "silu", "f32", True)
    import gated_delta_rule_slot_amd as gdn

    y, z = c["y"].cuda().view(40, 1, 2048), c["z"].cuda().view(40, 1, 2048)
    res, wp, wq = c["res"].cuda(), c["w_post"].cuda(), c["w_pre"].cuda()
    out, ro = torch.empty_like(y), torch.empty_like(res)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.block_norm(y, out, w_post=wp, gate=z, act=gdn.ACT_SILU, residual=res, residual_out=ro, w_pre=wq)
    for turn in range(4):
        y.mul_(-1.5)
        graph.replay()
        a, b = out.clone(), ro.clone()
        gdn.block_norm(y, out, w_post=wp, gate=z, act=gdn.ACT_SILU, residual=res, residual_out=ro, w_pre=wq)
        assert torch.equal(a, out) and torch.equal(b, ro), turn


def test_output_norm_of_the_recurrence():
    """A decode step of the recurrence, then its gated output norm, as a linear layer uses
    them: the norm's input is the step's own output."""
    import gated_delta_rule_slot_amd as gdn
    import workloads as wl

    H, D, B = 4, 64, 3
    g = wl.generator(5)
    ssm, conv = wl.warm_pool(g, 1, 5, H, D, D, False)
    pool = gdn.state_pool_create(ssm.cuda(), conv.cuda())
    x = wl.projected_inputs(g, B, H, D, D, wl.ALPHA_PER_HEAD)
    o = torch.empty(B, H, D, dtype=torch.bfloat16, device="cuda")
    gdn.gdn_decode_step(pool, 0, torch.tensor([1, 2, 3], dtype=torch.int32).cuda(), x["x"].cuda(),
                        wl.conv_weights(g, 3 * H * D).cuda(), x["alpha"].cuda(), wl.ALPHA_PER_HEAD, x["beta"].cuda(), o)
    c = case(10, B, H, D, True, "silu", None, False)
    c["y"] = o.cpu().view(B, H * D)
    check(c, *run(c))


def test_block_norm_output_between_wide_rows():
    """out in the gap that y's rows leave in one buffer is apart from y, and equals the
    result of memory of its own; one that reaches into the next row is refused."""
    import gated_delta_rule_slot_amd as gdn

    T, G, D = 3, 2, 64
    n = T * G * D
    g = torch.Generator().manual_seed(31)
    buf = torch.randn(T, G * D + n + 8, generator=g).to(torch.bfloat16).cuda()
    y = buf[:, :G * D].view(T, G, D)
    w = torch.rand(D, generator=g).cuda()
    keep, own = buf.clone(), torch.empty(T, G, D, dtype=torch.bfloat16, device="cuda")
    gdn.block_norm(y, own, w_pre=w)
    gap = buf[1, G * D:G * D + n]
    gdn.block_norm(y, gap.view(T, G, D), w_pre=w)
    assert torch.equal(gap.view(T, G, D), own)
    keep[1, G * D:G * D + n] = own.flatten()
    assert torch.equal(buf, keep)
    with pytest.raises(Exception, match="out overlaps y"):
        gdn.block_norm(y, buf.flatten()[G * D + 16:G * D + 16 + n].view(T, G, D), w_pre=w)
    assert torch.equal(buf, keep)
