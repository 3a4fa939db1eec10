"""ctypes binding of include/gdn_kv.h: the paged key-value cache, its page tables, its attention
and its eviction, rotary positions, and the norm between blocks.  Argument marshalling only, as in _binding.py:
each function carries the C entry point's name and every step runs in the library's
kernels.  All tensors of a call live on the current HIP device.
"""
from __future__ import annotations

import ctypes as ct

import torch

from ._binding import GDN_BF16, GDN_F32, _check, _f32, _i32, _i64, _lib, _sz, _u32, _vp

# the current device and stream as plain numbers (torch.cuda's objects cost more than the
# launch of a small kernel); a torch build that lacks these takes the public way
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda index: torch.cuda.current_stream(index).cuda_stream)

GDN_F8_E4M3 = 2
ERRW_BAD_PAGE = 16
ATTN_ACCUM_MASS = 1
ACT_NONE, ACT_SILU, ACT_SIGMOID = 0, 1, 2
NORM_PLUS_ONE = 1
ERRW_NO_PAGES = 32
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_PLAIN, ROPE_LINEAR, ROPE_NTK, ROPE_YARN, ROPE_BANDS = 0, 1, 2, 3, 4


class KvDesc(ct.Structure):
    _fields_ = [
        ("layers", ct.c_int32), ("pages", ct.c_int32), ("kv_heads", ct.c_int32),
        ("page_size", ct.c_int32), ("head_dim", ct.c_int32), ("slots", ct.c_int32),
        ("max_pages", ct.c_int32), ("kv_dtype", ct.c_int32), ("k_scale", ct.c_float),
        ("v_scale", ct.c_float), ("k_base", ct.c_void_p), ("v_base", ct.c_void_p),
        ("page_table", ct.c_void_p), ("mass", ct.c_void_p), ("pos", ct.c_void_p),
        ("err_word", ct.c_void_p),
    ]


class RopeDesc(ct.Structure):
    _fields_ = [("rot_dim", ct.c_int32), ("scaling", ct.c_int32), ("base", ct.c_double), ("factor", ct.c_double),
                ("original_len", ct.c_double), ("low", ct.c_double), ("high", ct.c_double)]


_lib.kv_pool_bytes.argtypes = [ct.POINTER(KvDesc), ct.POINTER(_sz), ct.POINTER(_sz)]
_lib.kv_pool_create.argtypes = [ct.POINTER(KvDesc), ct.POINTER(_vp)]
_lib.kv_pool_destroy.argtypes = [_vp]
_lib.kv_pool_destroy.restype = None
_lib.kv_append.argtypes = [_vp, _i32, _i32, _vp, _vp, _vp, _vp, _i64, _vp, _i64, _vp]
_lib.attn_workspace_bytes.argtypes = [_vp, _i32, _i32, _i32, _u32, ct.POINTER(_sz)]
_lib.attn_decode_paged.argtypes = [_vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _i64, _f32, _u32,
                                   _vp, _vp, _vp, _sz, _vp]
_lib.kv_evict_plan.argtypes = [_vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp,
                               _vp, _vp, _vp]
_lib.kv_evict_apply.argtypes = [_vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp]
_lib.block_norm.argtypes = [_i64, _i32, _i32, _vp, _i64, _vp, _vp, _i64, _i32, _f32, _vp, _vp, _i32, _vp,
                            _i32, _f32, _u32, _vp, _vp]
_lib.kv_batch_map.argtypes = [_vp, _i32, _i32, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                              _vp, _vp, _vp]
_lib.kv_release.argtypes = [_vp, _i32, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp]
_lib.rope_frequencies.argtypes = [ct.POINTER(RopeDesc), ct.POINTER(ct.c_double), ct.POINTER(_f32)]
_lib.rope_append.argtypes = [_vp, _i32, _i32, _vp, _vp, _vp, _i32, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i32,
                             _i32, _vp, _f32, _vp]
_lib.attn_prefill_workspace_bytes.argtypes = [_vp, _i32, _i32, _i32, _i32, _i32, ct.POINTER(_sz)]
_lib.attn_prefill_paged.argtypes = [_vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _i64, _f32, _i32,
                                    _i32, _vp, _vp, _vp, _sz, _vp]
for _f in ("kv_pool_bytes", "kv_pool_create", "kv_append", "attn_workspace_bytes", "attn_decode_paged",
           "kv_evict_plan", "kv_evict_apply", "block_norm", "kv_batch_map", "kv_release", "rope_frequencies",
           "rope_append", "attn_prefill_workspace_bytes", "attn_prefill_paged"):
    getattr(_lib, _f).restype = ct.c_int


def _on(index) -> int:
    """The device that a call runs on, by number; every tensor of the call has to be there."""
    if index < 0:
        raise ValueError("tensor must be on the GPU")
    if index != _current_device():
        raise ValueError(f"tensors are on cuda:{index}, the current device is cuda:{_current_device()}")
    return index


def _on_stream(stream, index) -> int:
    if stream is None:
        return _current_raw_stream(index)
    if stream.device_index != index:
        raise ValueError(f"stream of cuda:{stream.device_index}, tensors on cuda:{index}")
    return stream.cuda_stream


def _arg(t, dtype, numel, name, index):
    """Pointer of a contiguous tensor of at least numel elements (None stays None)."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name}: on {t.device}, expected cuda:{index}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name}: needs at least {numel} elements, has {t.numel()}")
    return t.data_ptr()


def _rows(t, n, heads, dim, name, index):
    """(pointer, stride) of bf16 [n, heads, dim] whose rows [heads, dim] are contiguous
    at any distance."""
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name}: expected {torch.bfloat16}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name}: on {t.device}, expected cuda:{index}")
    if t.shape != (n, heads, dim):
        raise ValueError(f"{name}: expected {(n, heads, dim)}, got {tuple(t.shape)}")
    s0, s1, s2 = t.stride()
    if (dim > 1 and s2 != 1) or (heads > 1 and s1 != dim):
        raise ValueError(f"{name}: [heads, dim] must be contiguous within a row")
    return t.data_ptr(), s0 if n > 1 else heads * dim


def kv_pool_bytes(layers, pages, kv_heads, page_size, head_dim, slots, max_pages, kv_dtype):
    """(bytes of k and of v, elements of mass and of pos)."""
    d = KvDesc(layers, pages, kv_heads, page_size, head_dim, slots, max_pages, kv_dtype, 1.0, 1.0)
    b, e = _sz(), _sz()
    _check(_lib.kv_pool_bytes(ct.byref(d), ct.byref(b), ct.byref(e)))
    return b.value, e.value


class KvPool:
    """Handle over caller-owned cache tensors (see kv_pool_create)."""

    def __init__(self, handle, k, v, page_table, mass, pos, err_word):
        self.handle = handle
        self.k, self.v, self.page_table = k, v, page_table
        self.mass, self.pos, self.err_word = mass, pos, err_word
        self.layers, self.pages, self.kv_heads, self.page_size, self.head_dim = k.shape
        self.slots, self.max_pages = page_table.shape
        self.device = k.get_device()

    @property
    def capacity(self):
        return self.max_pages * self.page_size

    def destroy(self):
        if self.handle:
            _lib.kv_pool_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def kv_pool_create(k, v, page_table, mass=None, pos=None, err_word=None, k_scale=1.0, v_scale=1.0):
    """Wrap ``k``, ``v`` [layers, pages, kv_heads, page_size, head_dim] (bfloat16 or
    float8_e4m3fn), ``page_table`` int32 [slots, max_pages] and, optionally, ``mass``
    fp32 and ``pos`` int32 [layers, slots, kv_heads, max_pages * page_size]."""
    if k.dim() != 5 or k.shape != v.shape or k.dtype != v.dtype:
        raise ValueError("k and v must be [layers, pages, kv_heads, page_size, head_dim] of one type")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [slots, max_pages]")
    if k.dtype == torch.bfloat16:
        dt = GDN_BF16
    elif k.dtype == torch.float8_e4m3fn:
        dt = GDN_F8_E4M3
    else:
        raise TypeError("k and v must be bfloat16 or float8_e4m3fn")
    L, P, H, S, D = k.shape
    N, M = page_table.shape
    dev = _on(k.get_device())
    for t, name in ((mass, "mass"), (pos, "pos")):
        if t is not None and tuple(t.shape) != (L, N, H, M * S):
            raise ValueError(f"{name} must be [layers, slots, kv_heads, max_pages * page_size]")
    d = KvDesc(L, P, H, S, D, N, M, dt, float(k_scale), float(v_scale),
               _arg(k, k.dtype, 0, "k", dev), _arg(v, k.dtype, 0, "v", dev),
               _arg(page_table, torch.int32, 0, "page_table", dev),
               _arg(mass, torch.float32, 0, "mass", dev), _arg(pos, torch.int32, 0, "pos", dev),
               _arg(err_word, torch.int32, 1, "err_word", dev))
    h = _vp()
    _check(_lib.kv_pool_create(ct.byref(d), ct.byref(h)))
    return KvPool(h, k, v, page_table, mass, pos, err_word)


def kv_append(pool: KvPool, layer, slot_ids, index, k, v, position=None, stream=None):
    """Store ``k``, ``v`` bf16 [n, kv_heads, head_dim] (rows at any stride) at places
    ``index`` int32 [n] of slots ``slot_ids`` int32 [n]; ``position`` int32 [n]."""
    dev = _on(pool.device)
    n = slot_ids.numel()
    kp, ks = _rows(k, n, pool.kv_heads, pool.head_dim, "k", dev)
    vp, vs = _rows(v, n, pool.kv_heads, pool.head_dim, "v", dev)
    _check(_lib.kv_append(
        pool.handle, layer, n, _arg(slot_ids, torch.int32, n, "slot_ids", dev),
        _arg(index, torch.int32, n, "index", dev), _arg(position, torch.int32, n, "position", dev),
        kp, ks, vp, vs, _on_stream(stream, dev)))


def attn_workspace_bytes(pool: KvPool, batch, q_heads, max_len, flags=0) -> int:
    n = _sz()
    _check(_lib.attn_workspace_bytes(pool.handle, batch, q_heads, max_len, flags, ct.byref(n)))
    return n.value


def attn_decode_paged(pool: KvPool, layer, slot_table, kv_len, q, out, max_len, kv_begin=None, scale=1.0,
                      flags=0, lse=None, workspace=None, stream=None):
    """``q`` bf16 [batch, q_heads, head_dim] (rows at any stride), ``out`` the same,
    contiguous; ``slot_table``, ``kv_len``, ``kv_begin`` int32 [batch] (the first visible
    place: not for slots that kv_evict_apply has cut); ``lse`` fp32 [batch, q_heads];
    ``workspace`` uint8 (attn_workspace_bytes)."""
    dev = _on(pool.device)
    B = slot_table.numel()
    if q.dim() != 3:
        raise ValueError("q must be [batch, q_heads, head_dim]")
    H = q.shape[1]
    qp, qs = _rows(q, B, H, pool.head_dim, "q", dev)
    _check(_lib.attn_decode_paged(
        pool.handle, layer, B, H, max_len, _arg(slot_table, torch.int32, B, "slot_table", dev),
        _arg(kv_len, torch.int32, B, "kv_len", dev), _arg(kv_begin, torch.int32, B, "kv_begin", dev),
        qp, qs, scale, flags, _arg(out, torch.bfloat16, B * H * pool.head_dim, "out", dev),
        _arg(lse, torch.float32, B * H, "lse", dev), _arg(workspace, torch.uint8, 0, "workspace", dev),
        workspace.numel() if workspace is not None else 0, _on_stream(stream, dev)))


def _moves(pool, layers, batch, moves):
    if moves.dim() != 5 or tuple(moves.shape[:3]) != (layers, batch, pool.kv_heads) or moves.shape[4] != 2:
        raise ValueError("moves must be [layers, batch, kv_heads, max_moves, 2]")
    return moves.shape[3]


def kv_evict_plan(pool: KvPool, layer_begin, layer_end, slot_table, kv_len, next_pos, max_len, budget, sink,
                  recent, n_moves, moves, kv_len_out, stream=None):
    """Plan the eviction of layers [layer_begin, layer_end) to ``budget`` tokens:
    ``n_moves`` int32 [layers, batch, kv_heads], ``moves`` int32 [layers, batch, kv_heads,
    max_moves, 2] (source, destination), ``kv_len_out`` int32 [batch]."""
    dev = _on(pool.device)
    B, L = slot_table.numel(), layer_end - layer_begin
    M = _moves(pool, L, B, moves)
    _check(_lib.kv_evict_plan(
        pool.handle, layer_begin, layer_end, B, max_len, _arg(slot_table, torch.int32, B, "slot_table", dev),
        _arg(kv_len, torch.int32, B, "kv_len", dev), _arg(next_pos, torch.int32, B, "next_pos", dev), budget,
        sink, recent, M, _arg(n_moves, torch.int32, L * B * pool.kv_heads, "n_moves", dev),
        _arg(moves, torch.int32, 0, "moves", dev), _arg(kv_len_out, torch.int32, B, "kv_len_out", dev),
        _on_stream(stream, dev)))


def kv_evict_apply(pool: KvPool, layer_begin, layer_end, slot_table, n_moves, moves, stream=None):
    """Carry out the moves of kv_evict_plan in the cache, its mass and its positions."""
    dev = _on(pool.device)
    B, L = slot_table.numel(), layer_end - layer_begin
    M = _moves(pool, L, B, moves)
    _check(_lib.kv_evict_apply(
        pool.handle, layer_begin, layer_end, B, M, _arg(slot_table, torch.int32, B, "slot_table", dev),
        _arg(n_moves, torch.int32, L * B * pool.kv_heads, "n_moves", dev),
        _arg(moves, torch.int32, 0, "moves", dev), _on_stream(stream, dev)))


def kv_batch_map(pool: KvPool, slot_table, kv_len, free_pages, n_free, cu_seqlens, slot_out, kv_len_out,
                 token_slot, token_index, new_len=None, next_pos=None, next_pos_out=None, token_pos=None,
                 n_free_out=None, stream=None):
    """Pages, ``cu_seqlens`` int32 [batch + 1] and token maps ``token_slot``, ``token_index``, ``token_pos``
    int32 [max_tokens] of a step that gives request b ``new_len[b]`` tokens (default 1) behind its
    ``kv_len[b]``; ``slot_out``, ``kv_len_out`` (may be ``kv_len``), ``next_pos_out`` (may be ``next_pos``)
    int32 [batch].  Pages come from ``free_pages[:n_free]``; ``n_free_out`` defaults to ``n_free``."""
    dev = _on(pool.device)
    B, T = slot_table.numel(), token_slot.numel()
    n_free_out = n_free if n_free_out is None else n_free_out
    i32 = torch.int32
    _check(_lib.kv_batch_map(
        pool.handle, B, T, _arg(slot_table, i32, B, "slot_table", dev), _arg(kv_len, i32, B, "kv_len", dev),
        _arg(new_len, i32, B, "new_len", dev), _arg(next_pos, i32, B, "next_pos", dev), free_pages.numel(),
        _arg(free_pages, i32, 0, "free_pages", dev), _arg(n_free, i32, 1, "n_free", dev),
        _arg(n_free_out, i32, 1, "n_free_out", dev), _arg(cu_seqlens, i32, B + 1, "cu_seqlens", dev),
        _arg(slot_out, i32, B, "slot_out", dev), _arg(kv_len_out, i32, B, "kv_len_out", dev),
        _arg(next_pos_out, i32, B, "next_pos_out", dev), _arg(token_slot, i32, T, "token_slot", dev),
        _arg(token_index, i32, T, "token_index", dev), _arg(token_pos, i32, T, "token_pos", dev),
        _on_stream(stream, dev)))


def kv_release(pool: KvPool, slot_table, kv_len, free_pages, n_free, keep=None, n_free_out=None, stream=None):
    """Give the pages of the places from ``keep[b]`` (default 0) to ``kv_len[b]`` back to
    ``free_pages``; ``n_free_out`` defaults to ``n_free``."""
    dev = _on(pool.device)
    B, i32 = slot_table.numel(), torch.int32
    n_free_out = n_free if n_free_out is None else n_free_out
    _check(_lib.kv_release(
        pool.handle, B, _arg(slot_table, i32, B, "slot_table", dev), _arg(kv_len, i32, B, "kv_len", dev),
        _arg(keep, i32, B, "keep", dev), free_pages.numel(), _arg(free_pages, i32, 0, "free_pages", dev),
        _arg(n_free, i32, 1, "n_free", dev), _arg(n_free_out, i32, 1, "n_free_out", dev), _on_stream(stream, dev)))


def rope_frequencies(rot_dim, base=10000.0, scaling=ROPE_PLAIN, factor=1.0, original_len=0.0, low=1.0, high=32.0):
    """(float64 [rot_dim / 2] on the CPU: angle per position of each pair, amplitude)."""
    d = RopeDesc(rot_dim, scaling, base, factor, original_len, low, high)
    f = (ct.c_double * max(1, rot_dim // 2))()
    a = _f32()
    _check(_lib.rope_frequencies(ct.byref(d), f, ct.byref(a)))
    return torch.tensor(list(f), dtype=torch.float64), a.value


def rope_append(pool: KvPool, layer, slot_ids, index, position, q, q_out, k, v, freqs, layout=ROPE_HALF,
                amplitude=1.0, stream=None):
    """Turn ``q`` bf16 [n, q_heads, head_dim] into ``q_out`` (may be ``q``; both may be None) and ``k``
    bf16 [n, kv_heads, head_dim] by ``position`` int32 [n], and store ``k`` and ``v`` at places ``index``
    of slots ``slot_ids``; rows at any stride.  ``freqs`` float64 [rot_dim / 2] on the device."""
    dev = _on(pool.device)
    n = slot_ids.numel()
    kp, ks = _rows(k, n, pool.kv_heads, pool.head_dim, "k", dev)
    vp, vs = _rows(v, n, pool.kv_heads, pool.head_dim, "v", dev)
    H, qp, qs, op, os_ = 0, None, 0, None, 0
    if q is not None:
        if q.dim() != 3 or q_out is None:
            raise ValueError("q must be [n, q_heads, head_dim], and q_out be given with it")
        H = q.shape[1]
        qp, qs = _rows(q, n, H, pool.head_dim, "q", dev)
        op, os_ = _rows(q_out, n, H, pool.head_dim, "q_out", dev)
    _check(_lib.rope_append(
        pool.handle, layer, n, _arg(slot_ids, torch.int32, n, "slot_ids", dev),
        _arg(index, torch.int32, n, "index", dev), _arg(position, torch.int32, n, "position", dev), H, qp, qs, op,
        os_, kp, ks, vp, vs, 2 * freqs.numel(), layout, _arg(freqs, torch.float64, 0, "freqs", dev), amplitude,
        _on_stream(stream, dev)))


def attn_prefill_workspace_bytes(pool: KvPool, batch, tokens, q_heads, max_len, mass_tokens=0) -> int:
    n = _sz()
    _check(_lib.attn_prefill_workspace_bytes(pool.handle, batch, tokens, q_heads, max_len, mass_tokens,
                                             ct.byref(n)))
    return n.value


def attn_prefill_paged(pool: KvPool, layer, cu_seqlens, slot_table, kv_len, q, out, max_len, kv_begin=None,
                       window=0, scale=1.0, mass_tokens=0, lse=None, workspace=None, stream=None):
    """``q`` bf16 [tokens, q_heads, head_dim] (rows at any stride), ``out`` the same, contiguous;
    ``cu_seqlens`` int32 [batch + 1]; ``slot_table``, ``kv_len`` (with the new tokens), ``kv_begin`` int32
    [batch]; ``lse`` fp32 [tokens, q_heads]; ``workspace`` uint8 (attn_prefill_workspace_bytes)."""
    dev = _on(pool.device)
    B = slot_table.numel()
    if q.dim() != 3:
        raise ValueError("q must be [tokens, q_heads, head_dim]")
    T, H = q.shape[:2]
    qp, qs = _rows(q, T, H, pool.head_dim, "q", dev)
    _check(_lib.attn_prefill_paged(
        pool.handle, layer, B, T, H, max_len, _arg(cu_seqlens, torch.int32, B + 1, "cu_seqlens", dev),
        _arg(slot_table, torch.int32, B, "slot_table", dev), _arg(kv_len, torch.int32, B, "kv_len", dev),
        _arg(kv_begin, torch.int32, B, "kv_begin", dev), qp, qs, scale, window, mass_tokens,
        _arg(out, torch.bfloat16, T * H * pool.head_dim, "out", dev), _arg(lse, torch.float32, T * H, "lse", dev),
        _arg(workspace, torch.uint8, 0, "workspace", dev), workspace.numel() if workspace is not None else 0,
        _on_stream(stream, dev)))


def block_norm(y, out, w_post=None, gate=None, act=ACT_NONE, scale=1.0, residual=None, residual_out=None,
               w_pre=None, eps=1e-6, flags=0, stream=None):
    """``y``, ``gate`` bf16 [tokens, groups, dim] (a token's groups adjacent, tokens at any
    stride); ``residual``, ``residual_out`` bf16 or fp32, ``out`` bf16, all contiguous
    [tokens, groups, dim]; ``w_post``, ``w_pre`` bf16 or fp32 [dim]."""
    if y.dim() != 3:
        raise ValueError("y must be [tokens, groups, dim]")
    dev = _on(y.get_device())
    T, G, D = y.shape
    yp, ys = _rows(y, T, G, D, "y", dev)
    gp, gs = _rows(gate, T, G, D, "gate", dev) if gate is not None else (None, 0)
    n = T * G * D
    w = w_post if w_post is not None else w_pre
    wt = torch.bfloat16 if w is None else w.dtype
    rt = torch.bfloat16 if residual is None else residual.dtype
    if wt not in (torch.bfloat16, torch.float32) or rt not in (torch.bfloat16, torch.float32):
        raise TypeError("weights and residual must be bfloat16 or float32")
    _check(_lib.block_norm(
        T, G, D, yp, ys, _arg(w_post, wt, D, "w_post", dev), gp, gs, act, scale,
        _arg(residual, rt, n, "residual", dev), _arg(residual_out, rt, n, "residual_out", dev),
        GDN_F32 if rt == torch.float32 else GDN_BF16, _arg(w_pre, wt, D, "w_pre", dev),
        GDN_F32 if wt == torch.float32 else GDN_BF16, eps, flags,
        _arg(out, torch.bfloat16, n, "out", dev), _on_stream(stream, dev)))
