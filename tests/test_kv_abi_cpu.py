"""Host-side checks of include/gdn_kv.h that need no GPU: sizes, and every refusal before a
launch (pointers are made-up numbers that nothing reads)."""
import ctypes as ct

import pytest
import torch

import gated_delta_rule_slot_amd as gdn
from gated_delta_rule_slot_amd import _binding as B
from gated_delta_rule_slot_amd import _kv as K

P = 0x100000  # a 256-byte aligned made-up address


def desc(**kw):
    d = dict(layers=2, pages=9, kv_heads=2, page_size=16, head_dim=64, slots=4, max_pages=5,
             kv_dtype=B.GDN_BF16, k_scale=1.0, v_scale=1.0, k_base=P, v_base=P, page_table=P, mass=P, pos=P,
             err_word=None)
    d.update(kw)
    return K.KvDesc(*[d[f] for f, _ in K.KvDesc._fields_])


def make(**kw):
    h = ct.c_void_p()
    return B._lib.kv_pool_create(ct.byref(desc(**kw)), ct.byref(h)), h


@pytest.fixture
def pool():
    st, h = make()
    assert st == 0, B.last_error()
    yield h
    B._lib.kv_pool_destroy(h)


def test_sizes():
    assert gdn.kv_pool_bytes(2, 9, 2, 16, 64, 4, 5, B.GDN_BF16) == (2 * 9 * 2 * 16 * 64 * 2, 2 * 4 * 2 * 80)
    assert gdn.kv_pool_bytes(2, 9, 2, 16, 64, 4, 5, gdn.GDN_F8_E4M3)[0] == 2 * 9 * 2 * 16 * 64
    # past 32 bits
    assert gdn.kv_pool_bytes(8, 100000, 8, 64, 256, 4, 5, B.GDN_BF16)[0] == 8 * 100000 * 8 * 64 * 256 * 2


@pytest.mark.parametrize("kw,status", [
    (dict(), 0), (dict(kv_dtype=gdn.GDN_F8_E4M3, k_scale=0.5, v_scale=3.0), 0), (dict(mass=None, pos=None), 0),
    (dict(page_size=1), 0), (dict(page_size=1024), 0),
    (dict(layers=0), -1), (dict(kv_heads=0), -1), (dict(max_pages=0), -1), (dict(pages=1), -1),
    (dict(slots=1), -1), (dict(kv_dtype=B.GDN_F32), -1), (dict(kv_dtype=7), -1),
    (dict(head_dim=32), -3), (dict(head_dim=96), -3), (dict(page_size=24), -3), (dict(page_size=2048), -3),
    (dict(page_size=0), -3), (dict(max_pages=1 << 26), -3), (dict(pages=1 << 26), -3),
    (dict(pages=1 << 30, kv_heads=4), -3), (dict(kv_heads=70000), -3),
    (dict(k_base=None), -1), (dict(v_base=None), -1), (dict(page_table=None), -1),
    (dict(k_base=P + 8), -3), (dict(page_table=P + 2), -1), (dict(mass=P + 1), -1), (dict(err_word=P + 2), -1),
    (dict(k_scale=2.0), -1), (dict(kv_dtype=2, k_scale=0.0), -1), (dict(kv_dtype=2, v_scale=-1.0), -1),
    (dict(kv_dtype=2, v_scale=float("inf")), -1), (dict(kv_dtype=2, k_scale=float("nan")), -1),
])
def test_pool_create_validation(kw, status):
    st, h = make(**kw)
    assert st == status, B.last_error()
    if st == 0:
        B._lib.kv_pool_destroy(h)
    else:
        assert B.last_error()


APPEND = dict(layer=0, n=3, slot_ids=P, index=P, position=P, k=P, ks=128, v=P, vs=128, stream=None)
ATTN = dict(layer=0, batch=2, q_heads=4, max_len=80, slot_table=P, kv_len=P, kv_begin=None, q=P, qs=256,
            scale=1.0, flags=0, out=P, lse=None, ws=P, ws_bytes=1 << 30, stream=None)
PLAN = dict(lb=0, le=2, batch=2, max_len=80, slot_table=P, kv_len=P, next_pos=P, budget=32, sink=2, recent=8,
            max_moves=32, n_moves=P, moves=P, out=P + 4096, stream=None)
APPLY = dict(lb=0, le=2, batch=2, max_moves=32, slot_table=P, n_moves=P, moves=P, stream=None)
NORM = dict(tokens=4, groups=2, dim=64, y=P, ys=128, w_post=P, gate=P, gs=128, act=1, scale=1.0, res=P, res_out=P,
            rt=B.GDN_BF16, w_pre=P, wt=B.GDN_F32, eps=1e-6, flags=0, out=P, stream=None)


@pytest.mark.parametrize("fn,base,kw,status", [
    ("kv_append", APPEND, dict(layer=2), -2), ("kv_append", APPEND, dict(layer=-1), -2),
    ("kv_append", APPEND, dict(layer=2 ** 31 - 1), -2),
    ("kv_append", APPEND, dict(n=-1), -2), ("kv_append", APPEND, dict(n=0, k=None), 0),
    ("kv_append", APPEND, dict(slot_ids=None), -1), ("kv_append", APPEND, dict(index=None), -1),
    ("kv_append", APPEND, dict(position=None), -1), ("kv_append", APPEND, dict(v=None), -1),
    ("kv_append", APPEND, dict(ks=120), -1), ("kv_append", APPEND, dict(vs=132), -3),
    ("kv_append", APPEND, dict(k=P + 8), -3),
    ("attn_decode_paged", ATTN, dict(layer=2), -2), ("attn_decode_paged", ATTN, dict(batch=-1), -2),
    ("attn_decode_paged", ATTN, dict(batch=65536), -2), ("attn_decode_paged", ATTN, dict(batch=0, q=None), 0),
    ("attn_decode_paged", ATTN, dict(q_heads=3), -1), ("attn_decode_paged", ATTN, dict(q_heads=0), -1),
    ("attn_decode_paged", ATTN, dict(q_heads=130, qs=1 << 14), -3),
    ("attn_decode_paged", ATTN, dict(max_len=81), -2), ("attn_decode_paged", ATTN, dict(max_len=-1), -2),
    ("attn_decode_paged", ATTN, dict(flags=2), -1), ("attn_decode_paged", ATTN, dict(scale=float("nan")), -1),
    ("attn_decode_paged", ATTN, dict(scale=float("-inf")), -1), ("attn_decode_paged", ATTN, dict(scale=-2e30), -1),
    ("attn_decode_paged", ATTN, dict(slot_table=None), -1), ("attn_decode_paged", ATTN, dict(kv_len=None), -1),
    ("attn_decode_paged", ATTN, dict(q=None), -1), ("attn_decode_paged", ATTN, dict(out=None), -1),
    ("attn_decode_paged", ATTN, dict(qs=248), -1), ("attn_decode_paged", ATTN, dict(qs=260), -3),
    ("attn_decode_paged", ATTN, dict(q=P + 2), -3), ("attn_decode_paged", ATTN, dict(out=P + 8), -3),
    ("attn_decode_paged", ATTN, dict(flags=1, ws=None), -1),
    ("attn_decode_paged", ATTN, dict(flags=1, ws_bytes=64), -1),
    ("attn_decode_paged", ATTN, dict(flags=1, ws=P + 128), -3),
    ("kv_evict_plan", PLAN, dict(le=3), -2), ("kv_evict_plan", PLAN, dict(lb=1, le=0), -2),
    ("kv_evict_plan", PLAN, dict(lb=1, le=1, moves=None), 0), ("kv_evict_plan", PLAN, dict(batch=0), 0),
    ("kv_evict_plan", PLAN, dict(max_len=81), -2), ("kv_evict_plan", PLAN, dict(budget=0), -1),
    ("kv_evict_plan", PLAN, dict(sink=25), -1), ("kv_evict_plan", PLAN, dict(sink=-1), -1),
    ("kv_evict_plan", PLAN, dict(recent=-1), -1), ("kv_evict_plan", PLAN, dict(recent=2 ** 31 - 1), -1),
    ("kv_evict_plan", PLAN, dict(max_moves=31), -1), ("kv_evict_plan", PLAN, dict(moves=None), -1),
    ("kv_evict_plan", PLAN, dict(next_pos=None), -1), ("kv_evict_plan", PLAN, dict(n_moves=None), -1),
    ("kv_evict_plan", PLAN, dict(out=None), -1), ("kv_evict_plan", PLAN, dict(out=P + 4), -1),
    ("kv_evict_apply", APPLY, dict(le=3), -2), ("kv_evict_apply", APPLY, dict(max_moves=-1), -2),
    ("kv_evict_apply", APPLY, dict(max_moves=81), -2), ("kv_evict_apply", APPLY, dict(max_moves=0, moves=None), 0),
    ("kv_evict_apply", APPLY, dict(moves=None), -1), ("kv_evict_apply", APPLY, dict(slot_table=None), -1),
])
def test_calls_refuse_before_launch(pool, fn, base, kw, status):
    a = dict(base, **kw)
    assert getattr(B._lib, fn)(pool, *a.values()) == status, B.last_error()
    assert bool(B.last_error()) == (status != 0)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=0, y=None), 0), (dict(tokens=-1), -2), (dict(tokens=1 << 31), -2), (dict(groups=0), -1),
    (dict(dim=0), -1), (dict(dim=60), -3), (dict(dim=32776, ys=1 << 20, gs=1 << 20), -3), (dict(act=3), -1),
    (dict(gate=None), -1), (dict(rt=gdn.GDN_F8_E4M3), -1), (dict(wt=5), -1), (dict(flags=2), -1),
    (dict(eps=0.0), -1), (dict(eps=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(res=None), -1),
    (dict(res_out=None), -1), (dict(y=None), -1), (dict(out=None), -1), (dict(ys=120), -1), (dict(gs=120), -1),
    (dict(ys=132), -3), (dict(gs=140), -3), (dict(y=P + 8), -3), (dict(w_post=P + 4), -3), (dict(w_pre=P + 2), -3),
    (dict(res=P + 8), -3), (dict(res_out=P + 8), -3), (dict(out=P + 8), -3), (dict(gate=P + 8), -3),
])
def test_block_norm_refuses_before_launch(kw, status):
    assert B._lib.block_norm(*dict(NORM, **kw).values()) == status, B.last_error()


Q, F = 4 * 128 * 2, 4 * 128 * 4  # bytes of NORM's rows in bf16 and fp32
APART = dict(y=P, w_post=P + 0x10000, gate=P + 0x20000, res=P + 0x30000, res_out=P + 0x30000, w_pre=P + 0x40000,
             out=P + 0x50000)


@pytest.mark.parametrize("kw,what", [
    (dict(out=P, ys=136), "out overlaps y"), (dict(out=P + 16), "out overlaps y"),
    (dict(out=P - 16), "out overlaps y"), (dict(out=P + Q - 16), "out overlaps y"),
    (dict(out=P - Q + 16), "out overlaps y"), (dict(tokens=1, out=P + 240), "out overlaps y"),
    (dict(out=P + 1792, ys=1024, tokens=2), "out overlaps y"),
    (dict(out=P, res=None, res_out=None, y=P + 16), "out overlaps y"),
    (dict(out=APART["gate"]), "out overlaps gate"), (dict(out=APART["res"]), "out overlaps gate"),
    (dict(out=APART["res"], res=P + 0x60000), "out overlaps gate"),
    (dict(out=APART["res"] + F - 16, rt=B.GDN_F32), "out overlaps gate"),
    (dict(out=APART["w_post"] + 240), "out overlaps gate"), (dict(out=APART["w_pre"]), "out overlaps gate"),
    (dict(res_out=P), "residual_out overlaps"), (dict(res_out=APART["gate"]), "residual_out overlaps"),
    (dict(res_out=APART["res"] + 16), "residual_out overlaps"),
    (dict(res_out=APART["res"] + F - 16, rt=B.GDN_F32), "residual_out overlaps"),
    (dict(res_out=APART["w_pre"] - 16), "residual_out overlaps"),
])
def test_block_norm_refuses_overlaps(kw, what):
    a = {**NORM, **APART, **kw}
    assert B._lib.block_norm(*a.values()) == -1
    assert B.last_error().startswith(what)


@pytest.mark.parametrize("off,qs", [(0, 256), (16, 256), (1024 - 16, 256), (-1024 + 16, 256), (1024 - 16, 512),
                                    (512, 512), (0, 512)])
def test_attention_refuses_out_over_q(pool, off, qs):
    a = dict(ATTN, q=P, qs=qs, out=P + off, ws=P + 0x100000)
    assert B._lib.attn_decode_paged(pool, *a.values()) == -1
    assert "out overlaps q" in B.last_error()


def test_apply_refuses_lists_past_any_grid():
    st, h = make(layers=1 << 14, pages=2, kv_heads=2, max_pages=1 << 25, page_size=16)
    assert st == 0, B.last_error()
    try:
        a = dict(APPLY, le=1 << 14, batch=1 << 10, max_moves=1 << 20)
        assert B._lib.kv_evict_apply(h, *a.values()) == -2 and "2^40" in B.last_error()
    finally:
        B._lib.kv_pool_destroy(h)


def test_null_pool_and_missing_mass():
    st, h = make(mass=None, pos=None)
    assert st == 0
    try:
        for fn, base in (("kv_append", APPEND), ("attn_decode_paged", ATTN), ("kv_evict_plan", PLAN),
                         ("kv_evict_apply", APPLY)):
            assert getattr(B._lib, fn)(None, *base.values()) == -1
        assert B._lib.kv_evict_plan(h, *PLAN.values()) == -1 and "mass" in B.last_error()
        assert B._lib.attn_decode_paged(h, *dict(ATTN, flags=1).values()) == -1
        n = ct.c_size_t()
        assert B._lib.attn_workspace_bytes(h, 2, 4, 80, 1, ct.byref(n)) == -1
        assert B._lib.attn_workspace_bytes(h, 2, 4, 80, 0, None) == -1
    finally:
        B._lib.kv_pool_destroy(h)
    B._lib.kv_pool_destroy(None)


def test_workspace_grows_with_the_weights(pool):
    n, m = ct.c_size_t(), ct.c_size_t()
    assert B._lib.attn_workspace_bytes(pool, 2, 4, 80, 0, ct.byref(n)) == 0
    assert B._lib.attn_workspace_bytes(pool, 2, 4, 80, 1, ct.byref(m)) == 0
    assert m.value >= n.value + 2 * 4 * 80 * 4
    assert B._lib.attn_workspace_bytes(pool, 0, 4, 0, 1, ct.byref(n)) == 0


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    k = torch.zeros(1, 3, 1, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        gdn.kv_pool_create(k, k, torch.zeros(2, 2, dtype=torch.int32))  # not on the GPU
    with pytest.raises(ValueError):
        gdn.kv_pool_create(k, k[:, :2], torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(TypeError):
        gdn.kv_pool_create(k.float(), k.float(), torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        gdn.block_norm(torch.zeros(2, 64), None)
    with pytest.raises(ValueError):
        gdn.block_norm(torch.zeros(2, 1, 64, dtype=torch.bfloat16), None)


# every array of an attention call at a place of its own: (address, bytes)
AT = {n: P + 0x200000 * (i + 1) for i, n in enumerate(
    ("q", "slot_table", "kv_len", "kv_begin", "page_table", "mass", "err_word", "out", "lse", "ws"))}


def attention_at(**kw):
    """The call over a pool with every array apart but for `kw`."""
    at = {**AT, **kw}
    st, h = make(page_table=at["page_table"], mass=at["mass"], err_word=at["err_word"])
    assert st == 0, B.last_error()
    n = ct.c_size_t()
    assert B._lib.attn_workspace_bytes(h, 2, 4, 80, 1, ct.byref(n)) == 0
    a = dict(ATTN, flags=1, ws_bytes=n.value, layer=1,
             **{k: at[k] for k in ("q", "slot_table", "kv_len", "kv_begin", "out", "lse", "ws")})
    try:
        return B._lib.attn_decode_paged(h, *a.values()), n.value
    finally:
        B._lib.kv_pool_destroy(h)


# bytes of each: q and out 2 x 4 x 64 bf16, page_table 4 x 5, a layer's mass (of two) 4 x 2 x 80
SIZE = dict(q=1024, slot_table=8, kv_len=8, kv_begin=8, page_table=80, mass=2560, err_word=4, out=1024, lse=32)


@pytest.mark.parametrize("written,name", [("out", "out"), ("lse", "lse"), ("ws", "workspace"), ("mass", "mass"),
                                          ("err_word", "err_word")])
@pytest.mark.parametrize("read", ["q", "slot_table", "kv_len", "kv_begin", "page_table"])
def test_attention_refuses_outputs_over_inputs(written, name, read):
    """The read array's first and last 4 bytes (or its first 16 or 256, by the alignment)
    inside the written one, and the written one's inside it."""
    ws = attention_at(lse=AT["slot_table"])[1]
    size = dict(SIZE, ws=ws)
    base = AT[written] + (2560 if written == "mass" else 0)  # layer 1 is called
    offs = [0, size[written] - 4] if read not in ("q",) else [0, (size[written] - 1) // 16 * 16]
    for off in offs:
        if base + off != AT[read]:
            assert attention_at(**{read: base + off})[0] == -1, off
            assert B.last_error() == f"{name} overlaps {read}", off


@pytest.mark.parametrize("a,b,text", [("lse", "out", "lse overlaps out"), ("ws", "out", "workspace overlaps out"),
                                      ("ws", "lse", "workspace overlaps lse"), ("mass", "out", "mass overlaps out"),
                                      ("mass", "ws", "mass overlaps workspace"),
                                      ("err_word", "lse", "err_word overlaps lse")])
def test_attention_refuses_outputs_over_each_other(a, b, text):
    at = AT[b] - (2560 if a == "mass" else 0)
    assert attention_at(**{a: at})[0] == -1 and B.last_error() == text


PLAN_AT = {n: P + 0x200000 * (i + 1) for i, n in enumerate(
    ("slot_table", "kv_len", "next_pos", "mass", "pos", "err_word", "n_moves", "moves", "out"))}
# bytes: 2 layers x 2 requests x 2 heads, 32 moves; mass and pos of two layers, 4 slots x 2 heads x 80
PLAN_SIZE = dict(slot_table=8, kv_len=8, next_pos=8, mass=5120, pos=5120, err_word=4, n_moves=32, moves=2048, out=8)


def plan_at(**kw):
    at = {**PLAN_AT, **kw}
    st, h = make(mass=at["mass"], pos=at["pos"], err_word=at["err_word"], layers=3)
    assert st == 0, B.last_error()
    a = dict(PLAN, lb=1, le=3, **{k: at[k] for k in ("slot_table", "kv_len", "next_pos", "n_moves", "moves", "out")})
    try:
        return B._lib.kv_evict_plan(h, *a.values())
    finally:
        B._lib.kv_pool_destroy(h)


@pytest.mark.parametrize("written,name", [("out", "kv_len_out"), ("n_moves", "n_moves"), ("moves", "moves"),
                                          ("err_word", "err_word")])
@pytest.mark.parametrize("read", ["slot_table", "kv_len", "next_pos", "mass", "pos"])
def test_plan_refuses_outputs_over_inputs(written, name, read):
    base = 2560 if read in ("mass", "pos") else 0  # the second layer of three is the first one called
    for off in (0, PLAN_SIZE[written] - 4, 4 - PLAN_SIZE[read]):
        at = PLAN_AT[written] + off - base
        assert plan_at(**{read: at}) == -1, off
        assert B.last_error() == f"{name} overlaps {read}", off


@pytest.mark.parametrize("a,b", [("n_moves", "out"), ("moves", "out"), ("moves", "n_moves"), ("err_word", "moves")])
def test_plan_refuses_outputs_over_each_other(a, b):
    assert plan_at(**{a: PLAN_AT[b] + PLAN_SIZE[b] - 4}) == -1
    assert B.last_error() == f"{a} overlaps {b}".replace("out", "kv_len_out")


def test_plan_refuses_lists_past_any_memory(pool):
    assert B._lib.kv_evict_plan(pool, *dict(PLAN, max_moves=1 << 30, batch=1 << 15).values()) == -2
    assert "2^40" in B.last_error()


@pytest.mark.parametrize("fn,base,names", [
    ("kv_append", APPEND, ["slot_ids", "index", "position"]),
    ("attn_decode_paged", {**ATTN, "out": P + 0x10000, "ws": P + 0x20000, "kv_begin": P, "lse": P + 0x30000},
     ["slot_table", "kv_len", "kv_begin", "lse"]),
    ("kv_evict_plan", PLAN, ["slot_table", "kv_len", "next_pos", "n_moves", "moves", "out"]),
    ("kv_evict_apply", APPLY, ["slot_table", "n_moves", "moves"])])
def test_word_arrays_off_their_alignment_are_refused(pool, fn, base, names):
    for name in names:
        for off in (1, 2, 3):
            assert getattr(B._lib, fn)(pool, *dict(base, **{name: base[name] + 0x100000 + off}).values()) == -1
            assert "4-byte aligned" in B.last_error(), name


BIG = 2 ** 31 - 1


@pytest.mark.parametrize("kw,status", [
    (dict(layers=BIG, slots=BIG, kv_heads=32, pages=1 << 20, page_size=32, max_pages=1 << 24, head_dim=256), -3),
    # k of 2^63 bytes, and a layer less; mass of 2^61 entries, and a slot less
    (dict(layers=1 << 24, pages=1 << 20, kv_heads=8, page_size=128, max_pages=1, head_dim=256), -3),
    (dict(layers=(1 << 24) - 1, pages=1 << 20, kv_heads=8, page_size=128, max_pages=1, head_dim=256), 0),
    (dict(layers=1 << 10, slots=1 << 19, kv_heads=8, page_size=128, max_pages=1 << 22), -3),
    (dict(layers=1 << 10, slots=(1 << 19) - 1, kv_heads=8, page_size=128, max_pages=1 << 22), 0),
])
def test_sizes_past_63_bits_are_refused(kw, status):
    d, n, m = desc(**kw), ct.c_size_t(), ct.c_size_t()
    assert B._lib.kv_pool_bytes(ct.byref(d), ct.byref(n), ct.byref(m)) == status
    if status == 0:
        rows = d.layers * d.pages * d.kv_heads * d.page_size
        assert n.value == rows * d.head_dim * 2 and m.value == d.layers * d.slots * d.kv_heads * d.max_pages * d.page_size
    st, h = make(**kw)
    assert st == status
    B._lib.kv_pool_destroy(h)


def test_binding_loads_without_torch_private_names(monkeypatch):
    """A torch build without the private device and stream calls (a CPU build) still loads
    the package, and the public calls stand in for them."""
    import importlib.util
    from types import SimpleNamespace

    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    spec = importlib.util.spec_from_file_location("gated_delta_rule_slot_amd._kv_again", K.__file__)
    again = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(again)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index: SimpleNamespace(cuda_stream=40 + index))
    assert again._on_stream(None, 3) == 43
    assert again._current_device is torch.cuda.current_device
