"""Host-side checks, without a GPU, of the prompt side of include/gdn_kv.h: sizes, frequencies, and
every refusal before a launch (pointers are made-up numbers that nothing reads)."""
import ctypes as ct
import math

import numpy as np
import pytest
import torch

import gated_delta_rule_slot_amd as gdn
from gated_delta_rule_slot_amd import _binding as B
from gated_delta_rule_slot_amd import _kv as K
from oracle import kv_ops
from tests.test_kv_abi_cpu import P, make

STEP = 0x200000


@pytest.fixture(autouse=True)
def own_descriptors():
    """The binding's own descriptor types, also after a test that has loaded the binding a second
    time (which leaves its types on the library's calls)."""
    for fn, t in (("kv_pool_bytes", K.KvDesc), ("kv_pool_create", K.KvDesc), ("rope_frequencies", K.RopeDesc)):
        f = getattr(B._lib, fn)
        f.argtypes = [ct.POINTER(t), *f.argtypes[1:]]


@pytest.fixture
def pool(own_descriptors):
    st, h = make()
    assert st == 0, B.last_error()
    yield h
    B._lib.kv_pool_destroy(h)


def apart(names):
    return {n: P + STEP * (i + 1) for i, n in enumerate(names)}


MAP_AT = apart(["slot_table", "kv_len", "new_len", "next_pos", "free_pages", "n_free", "n_free_out", "cu", "slot_out",
                "len_out", "pos_out", "token_slot", "token_index", "token_pos"])
MAP = dict(batch=3, max_tokens=40, slot_table=0, kv_len=0, new_len=0, next_pos=0, free_capacity=9, free_pages=0,
           n_free=0, n_free_out=0, cu=0, slot_out=0, len_out=0, pos_out=0, token_slot=0, token_index=0, token_pos=0,
           stream=None)
MAP.update(MAP_AT)
REL_AT = apart(["slot_table", "kv_len", "keep", "free_pages", "n_free", "n_free_out"])
REL = dict(batch=3, slot_table=REL_AT["slot_table"], kv_len=REL_AT["kv_len"], keep=REL_AT["keep"], free_capacity=9,
           free_pages=REL_AT["free_pages"], n_free=REL_AT["n_free"], n_free_out=REL_AT["n_free_out"], stream=None)
ROPE_AT = apart(["slot_ids", "index", "position", "q", "q_out", "k", "v", "freqs"])
ROPE = dict(layer=0, n=3, slot_ids=ROPE_AT["slot_ids"], index=ROPE_AT["index"], position=ROPE_AT["position"],
            q_heads=4, q=ROPE_AT["q"], qs=256, q_out=ROPE_AT["q_out"], qos=256, k=ROPE_AT["k"], ks=128,
            v=ROPE_AT["v"], vs=128, rot=64, layout=0, freqs=ROPE_AT["freqs"], amplitude=1.0, stream=None)
CHUNK_AT = apart(["cu", "slot_table", "kv_len", "kv_begin", "q", "out", "lse", "ws"])
CHUNK = dict(layer=0, batch=2, tokens=6, q_heads=4, max_len=80, cu=CHUNK_AT["cu"], slot_table=CHUNK_AT["slot_table"],
             kv_len=CHUNK_AT["kv_len"], kv_begin=CHUNK_AT["kv_begin"], q=CHUNK_AT["q"], qs=256, scale=1.0, window=0,
             mass=0, out=CHUNK_AT["out"], lse=CHUNK_AT["lse"], ws=CHUNK_AT["ws"], ws_bytes=1 << 30, stream=None)
CALLS = {"kv_batch_map": MAP, "kv_release": REL, "rope_append": ROPE, "attn_prefill_paged": CHUNK}


def call(pool, fn, **kw):
    return getattr(B._lib, fn)(pool, *dict(CALLS[fn], **kw).values())


REFUSED = [
    ("kv_batch_map", dict(batch=-1), -2), ("kv_batch_map", dict(batch=65536), -2),
    ("kv_batch_map", dict(max_tokens=-1), -2), ("kv_batch_map", dict(max_tokens=(1 << 26) - 1), -2),
    ("kv_batch_map", dict(free_capacity=-1), -2), ("kv_batch_map", dict(pos_out=MAP["pos_out"], next_pos=None), -1),
    ("kv_release", dict(batch=-1), -2), ("kv_release", dict(free_capacity=-1), -2),
    ("rope_append", dict(layer=2), -2), ("rope_append", dict(layer=-1), -2), ("rope_append", dict(layer=2 ** 31 - 1), -2),
    ("rope_append", dict(n=-1), -2), ("rope_append", dict(n=0, k=None), 0), ("rope_append", dict(q_heads=-1), -2),
    ("rope_append", dict(q_heads=65536), -2), ("rope_append", dict(rot=0), -3), ("rope_append", dict(rot=8), -3),
    ("rope_append", dict(rot=24), -3), ("rope_append", dict(rot=80), -3), ("rope_append", dict(rot=-16), -3),
    ("rope_append", dict(layout=2), -1), ("rope_append", dict(layout=-1), -1),
    ("rope_append", dict(amplitude=float("nan")), -1), ("rope_append", dict(amplitude=float("inf")), -1),
    ("rope_append", dict(ks=120), -1), ("rope_append", dict(vs=64), -1), ("rope_append", dict(qs=248), -1),
    ("rope_append", dict(qos=128), -1), ("rope_append", dict(ks=132), -3), ("rope_append", dict(qs=260), -3),
    ("rope_append", dict(qos=260), -3), ("rope_append", dict(k=ROPE["k"] + 8), -3),
    ("rope_append", dict(v=ROPE["v"] + 2), -3), ("rope_append", dict(q=ROPE["q"] + 8), -3),
    ("rope_append", dict(q_out=ROPE["q_out"] + 4), -3), ("rope_append", dict(freqs=ROPE["freqs"] + 4), -1),
    ("attn_prefill_paged", dict(layer=2), -2), ("attn_prefill_paged", dict(layer=-1), -2),
    ("attn_prefill_paged", dict(batch=-1), -2), ("attn_prefill_paged", dict(batch=65536), -2),
    ("attn_prefill_paged", dict(batch=0, q=None), 0), ("attn_prefill_paged", dict(tokens=0, q=None), 0),
    ("attn_prefill_paged", dict(tokens=-1), -2), ("attn_prefill_paged", dict(tokens=2 ** 31 - 1), -2),
    ("attn_prefill_paged", dict(q_heads=3), -1), ("attn_prefill_paged", dict(q_heads=0), -1),
    ("attn_prefill_paged", dict(q_heads=130, qs=1 << 14), -3), ("attn_prefill_paged", dict(max_len=81), -2),
    ("attn_prefill_paged", dict(max_len=-1), -2), ("attn_prefill_paged", dict(window=-1), -2),
    ("attn_prefill_paged", dict(mass=-1), -2), ("attn_prefill_paged", dict(scale=float("nan")), -1),
    ("attn_prefill_paged", dict(scale=float("inf")), -1), ("attn_prefill_paged", dict(scale=-2e30), -1),
    ("attn_prefill_paged", dict(qs=248), -1), ("attn_prefill_paged", dict(qs=260), -3),
    ("attn_prefill_paged", dict(q=CHUNK["q"] + 8), -3), ("attn_prefill_paged", dict(out=CHUNK["out"] + 8), -3),
    ("attn_prefill_paged", dict(mass=4, ws=None), -1), ("attn_prefill_paged", dict(mass=4, ws_bytes=64), -1),
    ("attn_prefill_paged", dict(mass=4, ws=CHUNK["ws"] + 128), -3),
]


@pytest.mark.parametrize("fn,kw,status", REFUSED)
def test_calls_refuse_before_launch(pool, fn, kw, status):
    assert call(pool, fn, **kw) == status, B.last_error()
    assert bool(B.last_error()) == (status != 0)


REQUIRED = [("kv_batch_map", n) for n in ("slot_table", "kv_len", "free_pages", "n_free", "n_free_out", "cu", "slot_out",
                                          "len_out", "token_slot", "token_index")]
REQUIRED += [("kv_release", n) for n in ("slot_table", "kv_len", "free_pages", "n_free", "n_free_out")]
REQUIRED += [("rope_append", n) for n in ("slot_ids", "index", "position", "q", "q_out", "k", "v", "freqs")]
REQUIRED += [("attn_prefill_paged", n) for n in ("cu", "slot_table", "kv_len", "q", "out")]


@pytest.mark.parametrize("fn,name", REQUIRED)
def test_required_pointers(pool, fn, name):
    assert call(pool, fn, **{name: None}) == -1 and "NULL" in B.last_error()


WORDS = [("kv_batch_map", n) for n in MAP_AT] + [("kv_release", n) for n in REL_AT]
WORDS += [("rope_append", n) for n in ("slot_ids", "index", "position")]
WORDS += [("attn_prefill_paged", n) for n in ("cu", "slot_table", "kv_len", "kv_begin", "lse")]


@pytest.mark.parametrize("fn,name", WORDS)
def test_word_arrays_off_their_alignment_are_refused(pool, fn, name):
    for off in (1, 2, 3):
        assert call(pool, fn, **{name: CALLS[fn][name] + off}) == -1 and "4-byte aligned" in B.last_error()


MAP_BYTES = dict(slot_table=12, kv_len=12, new_len=12, next_pos=12, free_pages=36, n_free=4, n_free_out=4, cu=16,
                 slot_out=12, len_out=12, pos_out=12, token_slot=160, token_index=160, token_pos=160)
MAP_NAMES = dict(cu="cu_seqlens", len_out="kv_len_out", pos_out="next_pos_out")
MAP_OUT = ["cu", "slot_out", "len_out", "pos_out", "n_free_out", "token_slot", "token_index", "token_pos"]


@pytest.mark.parametrize("written", MAP_OUT)
@pytest.mark.parametrize("other", [n for n in MAP_AT])
def test_map_refuses_overlaps(pool, written, other):
    """The other array's first word on the written one's last, and its last on the first; the same
    place too, but for the pairs that may be one array."""
    if written == other:
        return
    offs = [MAP_BYTES[written] - 4, 4 - MAP_BYTES[other]]
    pair = {written, other} in ({"len_out", "kv_len"}, {"pos_out", "next_pos"}, {"n_free_out", "n_free"})
    for off in offs + ([] if pair else [0]):
        if pair and off == 0:
            continue
        assert call(pool, "kv_batch_map", **{other: MAP_AT[written] + off}) == -1, off
        a, b = (MAP_NAMES.get(n, n) for n in (written, other))
        assert B.last_error() in (f"{a} overlaps {b}", f"{b} overlaps {a}")


@pytest.mark.parametrize("written", MAP_OUT + ["page_table"])
@pytest.mark.parametrize("other", ["page_table", "err_word"])
def test_map_refuses_overlaps_with_the_pool(written, other):
    if written == other:
        return
    at = dict(page_table=P, err_word=P + 0x100000)
    where = MAP_AT.get(written, at.get(written)) + (MAP_BYTES.get(written, 80) - 4)
    st, h = make(**dict(at, **{other: where}))
    assert st == 0
    try:
        assert call(h, "kv_batch_map") == -1 and "overlaps" in B.last_error()
    finally:
        B._lib.kv_pool_destroy(h)


@pytest.mark.parametrize("written,size", [("free_pages", 36), ("n_free_out", 4)])
@pytest.mark.parametrize("other,bytes_", [("slot_table", 12), ("kv_len", 12), ("keep", 12), ("n_free", 4),
                                          ("free_pages", 36), ("n_free_out", 4)])
def test_release_refuses_overlaps(pool, written, size, other, bytes_):
    if written == other:
        return
    for off in (size - 4, 4 - bytes_):
        if {written, other} == {"n_free", "n_free_out"}:
            continue
        assert call(pool, "kv_release", **{other: REL_AT[written] + off}) == -1
        assert "overlaps" in B.last_error()


@pytest.mark.parametrize("kw", [
    dict(q_out=ROPE["q"] + 16), dict(q_out=ROPE["q"] - 512 + 16), dict(q_out=ROPE["q"], qos=264),
    dict(q_out=ROPE["k"]), dict(q_out=ROPE["k"] + 2 * 128 * 2 + 240), dict(q_out=ROPE["v"]),
    dict(q_out=ROPE["v"] - 3 * 512 + 16), dict(q_out=ROPE["slot_ids"]), dict(q_out=ROPE["index"]),
    dict(q_out=ROPE["position"]), dict(q_out=ROPE["freqs"]), dict(q_out=ROPE["freqs"] + 240),
    # the projection's rows [q | k | v], turned in place: k one vector too early
    dict(q=P, q_out=P, qs=512, qos=512, k=P + 512 - 16, ks=512, v=P + 768, vs=512),
    dict(q=P, q_out=P, qs=512, qos=512, k=P + 512, ks=512, v=P + 768 + 16, vs=512),
    # keys or values in the place of the queries that are turned
    dict(q_out=ROPE["q"], k=ROPE["q"]), dict(q_out=ROPE["q"], k=ROPE["q"], ks=256),
    dict(q_out=ROPE["q"], v=ROPE["q"], vs=256),
    # other strides within the same range
    dict(q=P, q_out=P, qs=512, qos=512, k=P + 512, ks=256, v=P + 768, vs=512),
])
def test_rope_refuses_overlaps(pool, kw):
    assert call(pool, "rope_append", **kw) == -1, B.last_error()
    assert B.last_error().startswith("q_out overlaps")


CHUNK_BYTES = dict(q=6 * 512, cu=12, slot_table=8, kv_len=8, kv_begin=8, page_table=80, mass=2560, err_word=4,
                   out=6 * 512, lse=96)


def chunk_at(mass_tokens=3, **kw):
    at = dict(CHUNK_AT, page_table=P + 0x2000000, mass=P + 0x2100000, err_word=P + 0x2200000)
    at.update(kw)
    st, h = make(page_table=at["page_table"], mass=at["mass"], err_word=at["err_word"])
    assert st == 0, B.last_error()
    n = ct.c_size_t()
    assert B._lib.attn_prefill_workspace_bytes(h, 2, 6, 4, 80, mass_tokens, ct.byref(n)) == 0
    a = dict(CHUNK, mass=mass_tokens, layer=1, ws_bytes=n.value, **{k: at[k] for k in CHUNK_AT})
    try:
        return B._lib.attn_prefill_paged(h, *a.values()), n.value, at
    finally:
        B._lib.kv_pool_destroy(h)


@pytest.mark.parametrize("written,name", [("out", "out"), ("lse", "lse"), ("ws", "workspace"), ("mass", "mass"),
                                          ("err_word", "err_word")])
@pytest.mark.parametrize("read", ["q", "cu", "slot_table", "kv_len", "kv_begin", "page_table", "out", "lse"])
def test_chunk_refuses_overlaps(written, name, read):
    if read == written or (written, read) == ("out", "lse"):
        return
    _, ws, at = chunk_at(lse=CHUNK_AT["slot_table"])
    at["lse"] = CHUNK_AT["lse"]
    size = dict(CHUNK_BYTES, ws=ws)
    base = at[written] + (2560 if written == "mass" else 0)  # layer 1 is called
    offs = [0, size[written] - 4] if read not in ("q", "out") else [0, (size[written] - 1) // 16 * 16]
    for off in offs:
        assert chunk_at(**{read: base + off})[0] == -1, off
        assert B.last_error() == f"{name} overlaps {dict(cu='cu_seqlens').get(read, read)}", off


def test_workspace_sizes(pool):
    n = ct.c_size_t()

    def size(batch, tokens, heads, max_len, mass):
        assert B._lib.attn_prefill_workspace_bytes(pool, batch, tokens, heads, max_len, mass, ct.byref(n)) == 0
        return n.value

    assert size(0, 0, 4, 80, 0) == 0 and size(2, 6, 4, 80, 0) == 0
    assert size(2, 6, 4, 80, 1) >= 6 * 4 * 4
    assert B._lib.attn_prefill_workspace_bytes(pool, 2, 6, 4, 80, 0, None) == -1
    st, h = make(max_pages=1 << 13, mass=None, pos=None)
    assert st == 0
    try:
        assert B._lib.attn_prefill_workspace_bytes(h, 1, 1, 4, 1 << 17, 0, ct.byref(n)) == 0 and n.value > 0
        assert B._lib.attn_prefill_workspace_bytes(h, 1, 1, 4, 1 << 17, 1, ct.byref(n)) == -1  # no mass
    finally:
        B._lib.kv_pool_destroy(h)


def test_null_pool():
    for fn in CALLS:
        assert call(None, fn) == -1


# ------------------------------------------------------------------- frequencies --
@pytest.mark.parametrize("rot", [2, 16, 48, 64, 128, 256])
def test_frequencies(rot):
    i = np.arange(rot // 2)
    theta = 10000.0 ** (-2 * i / rot)
    f, a = gdn.rope_frequencies(rot)
    assert f.dtype == torch.float64 and a == 1.0
    np.testing.assert_allclose(f.numpy(), theta, rtol=1e-15)
    f, a = gdn.rope_frequencies(rot, scaling=gdn.ROPE_LINEAR, factor=4.0)
    np.testing.assert_allclose(f.numpy(), theta / 4, rtol=1e-15)
    if rot > 2:
        f, a = gdn.rope_frequencies(rot, scaling=gdn.ROPE_NTK, factor=4.0)
        # the slowest pair is slowed by the factor, the fastest not at all
        np.testing.assert_allclose(f.numpy()[-1], theta[-1] / 4, rtol=1e-13)
        assert f[0] == 1.0 and a == 1.0
    f, a = gdn.rope_frequencies(rot, scaling=gdn.ROPE_BANDS, factor=8.0, original_len=8192, low=1.0, high=4.0)
    turns = 8192 * theta / (2 * math.pi)
    keep = np.clip((turns - 1) / 3, 0, 1)
    np.testing.assert_allclose(f.numpy(), theta * (keep + (1 - keep) / 8), rtol=1e-14)
    assert a == 1.0
    f, a = gdn.rope_frequencies(rot, scaling=gdn.ROPE_YARN, factor=8.0, original_len=8192)
    r = f.numpy() / theta
    np.testing.assert_allclose(r[turns > 40], 1.0, rtol=1e-14)
    if rot >= 64:
        np.testing.assert_allclose(r[turns < 0.5], 1 / 8, rtol=1e-14)
    assert (np.diff(r) <= 1e-15).all() and abs(a - (0.1 * math.log(8.0) + 1)) < 1e-7
    for kind in (gdn.ROPE_LINEAR, gdn.ROPE_YARN):  # factor 1 changes nothing
        f, a = gdn.rope_frequencies(rot, scaling=kind, factor=1.0, original_len=4096)
        np.testing.assert_allclose(f.numpy(), theta, rtol=1e-15)
        assert a == 1.0


@pytest.mark.parametrize("kw,status", [
    (dict(rot_dim=0), -3), (dict(rot_dim=3), -3), (dict(rot_dim=258), -3), (dict(rot_dim=-2), -3),
    (dict(rot_dim=2, scaling=2), -3), (dict(scaling=5), -1), (dict(scaling=-1), -1), (dict(base=1.0), -1),
    (dict(base=float("inf")), -1), (dict(base=float("nan")), -1), (dict(scaling=1, factor=0.5), -1),
    (dict(scaling=1, factor=float("inf")), -1), (dict(scaling=3, factor=2.0, original_len=0.0), -1),
    (dict(scaling=4, factor=2.0, original_len=100.0, low=4.0, high=4.0), -1),
    (dict(scaling=4, factor=2.0, original_len=100.0, low=0.0), -1),
    (dict(scaling=3, factor=2.0, original_len=float("nan")), -1),
    (dict(scaling=3, factor=2.0, original_len=100.0, high=float("inf")), -1),
])
def test_frequencies_refuse(kw, status):
    with pytest.raises(gdn.GdnError) as e:
        gdn.rope_frequencies(**dict(dict(rot_dim=64), **kw))
    assert e.value.status == status
    assert B._lib.rope_frequencies(None, None, None) == -1


# -------------------------------------------------------------------- definitions --
def test_chunk_definition_against_torch():
    """attend_chunk on scattered pages against a masked softmax over gathered rows, and row by row
    against the one-token definition."""
    r = np.random.default_rng(0)
    H, G, D, page, n, L, begin, window = 2, 3, 8, 4, 5, 19, 2, 9
    k, v = r.standard_normal((2, 9, H, page, D))
    table = np.zeros((2, 6), np.int64)
    table[1, :5] = [7, 3, 8, 1, 5]
    q = r.standard_normal((n, H * G, D))
    out, lse, w, (spread, size) = kv_ops.attend_chunk(k, v, table, 1, begin, L, q, 0.4, window, 2, 1.5, 0.5)
    K, V = (x[table[1, :5]].transpose(1, 0, 2, 3).reshape(H, 20, D)[:, :L] for x in (k, v))
    for i in range(n):
        t = L - n + i
        for j in range(H * G):
            seen = slice(max(begin, t - window + 1), t + 1)
            s = torch.tensor(0.4 * 1.5 * (K[j // G, seen] @ q[i, j]))
            p = torch.softmax(s, 0).numpy()
            np.testing.assert_allclose(out[i, j], 0.5 * (p @ V[j // G, seen]), rtol=1e-12)
            np.testing.assert_allclose(lse[i, j], torch.logsumexp(s, 0).item(), rtol=1e-12)
        one = kv_ops.attend(k, v, table, 1, max(begin, t - window + 1), t + 1, q[i], 0.4, 1.5, 0.5)
        np.testing.assert_allclose(out[i], one[0], rtol=1e-12)
        np.testing.assert_allclose(spread[i], one[3][0], rtol=1e-12)
        np.testing.assert_allclose(size[i], one[3][1], rtol=1e-12)
    assert abs(w.sum() - 2 * H * G) < 1e-12 and not w[:, :max(begin, L - 2 - window + 1)].any()


def test_turn_definition():
    """A turn keeps lengths, turns by sums, and is a complex product; the rest of a head stays."""
    r = np.random.default_rng(1)
    x, f = r.standard_normal((4, 2, 10)), np.array([1.0, 0.1, 0.01])
    pos = np.array([0, 3, -7, 100])
    for adjacent in (False, True):
        y = kv_ops.turn(x, pos, f, 2.0, adjacent)
        i, j = ((slice(0, 6, 2), slice(1, 6, 2)) if adjacent else (slice(0, 3), slice(3, 6)))
        z = 2.0 * (x[..., i] + 1j * x[..., j]) * np.exp(1j * pos[:, None, None] * f)
        np.testing.assert_allclose(y[..., i] + 1j * y[..., j], z, rtol=1e-12)
        assert np.array_equal(y[..., 6:], x[..., 6:])
        twice = kv_ops.turn(kv_ops.turn(x, pos, f, 1.0, adjacent), -pos, f, 1.0, adjacent)
        np.testing.assert_allclose(twice, x, rtol=1e-12)


def test_map_and_release_definitions():
    """By hand: pages of 4, three requests, one refused; released again the list is whole."""
    table = [[0] * 4 for _ in range(4)]
    table[2][0] = 9
    o = kv_ops.batch_map(table, [2, 1, 3], [3, 0, 0], [2, 4, 8], [13, 0, 0], [5, 6, 7], 3, 4, 16)
    assert o["table"] == [[0] * 4, [6, 0, 0, 0], [9, 7, 0, 0], [0] * 4] and o["n_free"] == 1
    assert o["cu"] == [0, 2, 6, 14] and o["slot"] == [2, 1, 0] and o["len"] == [5, 4, 0] and o["pos"] == [15, 4, 0]
    assert o["token_slot"] == [2, 2, 1, 1, 1, 1] + [0] * 10 and o["token_index"][:6] == [3, 4, 0, 1, 2, 3]
    assert o["token_pos"][:6] == [13, 14, 0, 1, 2, 3] and o["errors"] == {"pages"}
    t, free, n, e = kv_ops.release(o["table"], [1, 2], [4, 5], [0, 3], [5, 0, 0, 0], 1, 4, 10)
    assert free == [5, 6, 7, 0] and n == 3 and not e and t[2][:2] == [9, 0] and t[1][0] == 0


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(AttributeError):
        gdn.kv_batch_map(None, x, x, x, x, x, x, x, x, x)
    assert K.RopeDesc._fields_[0][0] == "rot_dim"
