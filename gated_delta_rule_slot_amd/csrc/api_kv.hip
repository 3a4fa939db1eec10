// api_kv.hip -- the C ABI declared in include/gdn_kv.h: host-side validation and
// dispatch.  No device memory is allocated here; every buffer belongs to the caller.
#include <math.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <new>

#include "api.hpp"
#include "kv.hpp"

namespace {

using gdn::aligned;
using gdn::launched;
using gdn::ok;

// int32 and fp32 arrays (the kernels read some of them by scalar loads)
gdn_status check_words(std::initializer_list<const void *> arrays) {
  for (const void *p : arrays)
    if (!aligned(p, 4)) return fail(GDN_ERR_ARG, "int32 and fp32 arrays must be 4-byte aligned");
  return GDN_OK;
}

// Memory of n >= 1 rows of `row` bytes, one every `stride` (>= row) bytes
struct Rows {
  const void *base;
  int64_t n, row, stride;
};

// whether a row of `a` shares a byte with [p, p + bytes)
bool overlap(const Rows &a, const void *p, int64_t bytes) {
  if (!a.base || !p) return false;
  const __int128 base = reinterpret_cast<uintptr_t>(a.base), lo = reinterpret_cast<uintptr_t>(p);
  const __int128 last = base + __int128(a.n - 1) * a.stride;  // the last row's first byte
  if (last + a.row <= lo || lo + bytes <= base) return false;  // (mostly so, and no division)
  if (a.n == 1) return true;
  const __int128 before = lo - base - a.row;  // the first row that ends behind lo
  const __int128 i = before < 0 ? 0 : before / a.stride + 1;
  return i < a.n && base + i * a.stride < lo + bytes;
}

// An array of a call, for the message
struct Array {
  const char *name;
  Rows rows;
};
Array flat(const char *name, const void *p, int64_t bytes) { return {name, {bytes ? p : nullptr, 1, bytes, bytes}}; }

// Workgroups run in any order, so nothing that one writes may be read or written elsewhere:
// `out` (each flat) has to lie apart from `in` and from each other.
gdn_status check_apart(std::initializer_list<Array> out, std::initializer_list<Array> in) {
  for (const Array *w = out.begin(); w != out.end(); ++w) {
    for (const Array &r : in)
      if (overlap(r.rows, w->rows.base, w->rows.row)) return fail(GDN_ERR_ARG, "%s overlaps %s", w->name, r.name);
    for (const Array *x = out.begin(); x != w; ++x)
      if (overlap(x->rows, w->rows.base, w->rows.row)) return fail(GDN_ERR_ARG, "%s overlaps %s", w->name, x->name);
  }
  return GDN_OK;
}

// Two groups of rows, of which one is written: rows of one buffer at the same stride may lie
// between each other, others have to lie apart altogether.
bool rows_meet(const Rows &a, const Rows &b) {
  if (!a.base || !b.base) return false;
  const __int128 x = reinterpret_cast<uintptr_t>(a.base), y = reinterpret_cast<uintptr_t>(b.base);
  if (x + __int128(a.n - 1) * a.stride + a.row <= y || y + __int128(b.n - 1) * b.stride + b.row <= x) return false;
  if (a.stride != b.stride) return true;
  const int64_t d = int64_t(((y - x) % a.stride + a.stride) % a.stride);
  return d < a.row || a.stride - d < b.row;
}

gdn_status check_shape(const gdn_kv_desc *d) {
  if (!d) return fail(GDN_ERR_ARG, "descriptor is NULL");
  if (d->layers <= 0 || d->kv_heads <= 0 || d->max_pages <= 0)
    return fail(GDN_ERR_ARG, "need layers, kv_heads and max_pages >= 1");
  if (d->pages < 2 || d->slots < 2)
    return fail(GDN_ERR_ARG, "need pages >= 2 and slots >= 2 (page 0 and slot 0 are reserved)");
  if (d->kv_dtype != GDN_BF16 && d->kv_dtype != GDN_F8_E4M3)
    return fail(GDN_ERR_ARG, "kv_dtype must be GDN_BF16 or GDN_F8_E4M3");
  if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256)
    return fail(GDN_ERR_UNSUPPORTED, "head dim %d not in {64, 128, 256}", d->head_dim);
  if (d->page_size < 1 || d->page_size > 1024 || (d->page_size & (d->page_size - 1)))
    return fail(GDN_ERR_UNSUPPORTED, "page_size %d is not a power of two in [1, 1024]", d->page_size);
  if (int64_t(d->max_pages) * d->page_size >= (int64_t(1) << 30))
    return fail(GDN_ERR_UNSUPPORTED, "max_pages * page_size must be below 2^30");
  if (d->kv_heads > 65535 ||
      int64_t(d->pages) * d->page_size >= (int64_t(1) << 31) / d->kv_heads)
    return fail(GDN_ERR_UNSUPPORTED, "pages * kv_heads * page_size must be below 2^31");
  // (the products of all sizes pass 64 bits; offsets into the arrays are counted in them)
  const __int128 rows = __int128(d->layers) * d->pages * d->kv_heads * d->page_size;
  const __int128 entries = __int128(d->layers) * d->slots * d->kv_heads * d->max_pages * d->page_size;
  if (rows * d->head_dim * (d->kv_dtype == GDN_BF16 ? 2 : 1) > INT64_MAX || entries * 4 > INT64_MAX)
    return fail(GDN_ERR_UNSUPPORTED, "k, v, mass and pos must each be below 2^63 bytes");
  return GDN_OK;
}

gdn_status check_call(gdn_kv_pool_t p, int layer_begin, int layer_end, int batch) {
  if (!p) return fail(GDN_ERR_ARG, "pool handle is NULL");
  if (layer_begin < 0 || layer_end > p->d.layers || layer_begin > layer_end)
    return fail(GDN_ERR_RANGE, "layers [%d, %d) outside [0, %d)", layer_begin, layer_end, p->d.layers);
  if (batch < 0 || batch > 65535) return fail(GDN_ERR_RANGE, "batch %d outside [0, 65535]", batch);
  // (layer, request, head) is counted in 31 bits
  if (int64_t(layer_end - layer_begin) * batch * p->d.kv_heads >= (int64_t(1) << 31))
    return fail(GDN_ERR_RANGE, "layers * batch * kv_heads must be below 2^31");
  return GDN_OK;
}

gdn_status check_max_len(gdn_kv_pool_t p, int max_len) {
  if (max_len < 0 || max_len > p->capacity)
    return fail(GDN_ERR_RANGE, "max_len %d outside [0, %d]", max_len, p->capacity);
  return GDN_OK;
}

gdn_status check_heads(gdn_kv_pool_t p, int q_heads) {
  if (q_heads <= 0 || q_heads % p->d.kv_heads)
    return fail(GDN_ERR_ARG, "q_heads %d is not a positive multiple of kv_heads %d", q_heads,
                p->d.kv_heads);
  if (q_heads / p->d.kv_heads > 64)
    return fail(GDN_ERR_UNSUPPORTED, "more than 64 query heads per key-value head");
  return GDN_OK;
}

gdn_status check_attn(gdn_kv_pool_t p, int batch, int q_heads, int max_len, uint32_t flags) {
  gdn_status s = check_call(p, 0, 1, batch);
  if (s != GDN_OK) return s;
  if ((s = check_max_len(p, max_len)) != GDN_OK) return s;
  if ((s = check_heads(p, q_heads)) != GDN_OK) return s;
  if (flags & ~uint32_t(GDN_F_ACCUM_MASS)) return fail(GDN_ERR_ARG, "unknown flag bits 0x%x", flags);
  if ((flags & GDN_F_ACCUM_MASS) && !p->d.mass)
    return fail(GDN_ERR_ARG, "GDN_F_ACCUM_MASS needs a pool with mass");
  if (!gdn::attn_fits(p, batch, q_heads, max_len))
    return fail(GDN_ERR_RANGE, "batch * kv_heads * max_len too large (2^31 blocks of 128 tokens)");
  return GDN_OK;
}

}  // namespace

GDN_API gdn_status kv_pool_bytes(const gdn_kv_desc *d, size_t *kv_bytes, size_t *mass_elements) {
  gdn_status s = check_shape(d);
  if (s != GDN_OK) return s;
  if (kv_bytes)
    *kv_bytes = size_t(d->layers) * d->pages * d->kv_heads * d->page_size * d->head_dim *
                (d->kv_dtype == GDN_BF16 ? 2 : 1);
  if (mass_elements)
    *mass_elements = size_t(d->layers) * d->slots * d->kv_heads * d->max_pages * d->page_size;
  return ok();
}

GDN_API gdn_status kv_pool_create(const gdn_kv_desc *d, gdn_kv_pool_t *out) {
  if (!out) return fail(GDN_ERR_ARG, "out is NULL");
  *out = nullptr;
  gdn_status s = check_shape(d);
  if (s != GDN_OK) return s;
  if (!d->k_base || !d->v_base || !d->page_table)
    return fail(GDN_ERR_ARG, "k_base, v_base or page_table is NULL");
  if (!aligned(d->k_base, 16) || !aligned(d->v_base, 16))
    return fail(GDN_ERR_UNSUPPORTED, "pool base pointers must be 16-byte aligned");
  if ((s = check_words({d->page_table, d->mass, d->pos, d->err_word})) != GDN_OK) return s;
  if (!(d->k_scale > 0) || !(d->v_scale > 0) || !isfinite(d->k_scale) || !isfinite(d->v_scale))
    return fail(GDN_ERR_ARG, "k_scale and v_scale must be finite and positive");
  if (d->kv_dtype == GDN_BF16 && (d->k_scale != 1.f || d->v_scale != 1.f))
    return fail(GDN_ERR_ARG, "k_scale and v_scale must be 1 for a GDN_BF16 pool");
  gdn_kv_pool *p = new (std::nothrow) gdn_kv_pool;
  if (!p) return fail(GDN_ERR_ARG, "out of host memory");
  p->d = *d;
  p->capacity = d->max_pages * d->page_size;
  p->page_shift = __builtin_ctz(unsigned(d->page_size));
  p->layer_rows = int64_t(d->pages) * d->kv_heads * d->page_size;
  p->row_bytes = d->head_dim * (d->kv_dtype == GDN_BF16 ? 2 : 1);
  *out = p;
  return ok();
}

GDN_API void kv_pool_destroy(gdn_kv_pool_t pool) { delete pool; }

GDN_API gdn_status kv_append(gdn_kv_pool_t pool, int32_t layer, int32_t n, const int32_t *slot_ids,
                             const int32_t *index, const int32_t *position, const uint16_t *k,
                             int64_t k_stride, const uint16_t *v, int64_t v_stride, void *stream) {
  gdn_status s = check_call(pool, layer, layer < INT32_MAX ? layer + 1 : layer, 0);
  if (s != GDN_OK) return s;
  if (n < 0) return fail(GDN_ERR_RANGE, "n < 0");
  if (n == 0) return ok();
  if (!slot_ids || !index || !k || !v) return fail(GDN_ERR_ARG, "a required pointer is NULL");
  if ((s = check_words({slot_ids, index, position})) != GDN_OK) return s;
  if (pool->d.pos && !position) return fail(GDN_ERR_ARG, "the pool has pos: position is required");
  const int64_t row = int64_t(pool->d.kv_heads) * pool->d.head_dim;
  if (k_stride < row || v_stride < row)
    return fail(GDN_ERR_ARG, "k_stride or v_stride below kv_heads * head_dim");
  if (k_stride % 8 || v_stride % 8 || !aligned(k, 16) || !aligned(v, 16))
    return fail(GDN_ERR_UNSUPPORTED, "k and v rows must be 16-byte aligned");
  // one thread per 8 values of a row
  if (int64_t(n) * (row / 8) >= (int64_t(1) << 38))
    return fail(GDN_ERR_RANGE, "n * kv_heads * head_dim too large");
  gdn::AppendArgs a{n, slot_ids, index, position, k, v, k_stride, v_stride};
  return launched(gdn::launch_kv_append(pool, layer, a, static_cast<hipStream_t>(stream)),
                  "kv_append launch");
}

GDN_API gdn_status attn_workspace_bytes(gdn_kv_pool_t pool, int32_t batch, int32_t q_heads,
                                        int32_t max_len, uint32_t flags, size_t *bytes) {
  if (!bytes) return fail(GDN_ERR_ARG, "bytes is NULL");
  gdn_status s = check_attn(pool, batch, q_heads, max_len, flags);
  if (s != GDN_OK) return s;
  *bytes = gdn::attn_workspace(pool, batch, q_heads, max_len, flags);
  return ok();
}

GDN_API gdn_status attn_decode_paged(gdn_kv_pool_t pool, int32_t layer, int32_t batch,
                                     int32_t q_heads, int32_t max_len, const int32_t *slot_table,
                                     const int32_t *kv_len, const int32_t *kv_begin,
                                     const uint16_t *q, int64_t q_stride, float scale,
                                     uint32_t flags, uint16_t *out, float *lse, void *workspace,
                                     size_t workspace_bytes, void *stream) {
  gdn_status s = check_attn(pool, batch, q_heads, max_len, flags);
  if (s != GDN_OK) return s;
  if (layer < 0 || layer >= pool->d.layers)
    return fail(GDN_ERR_RANGE, "layer %d outside [0, %d)", layer, pool->d.layers);
  if (!(fabsf(scale) * pool->d.k_scale <= 1e30f))
    return fail(GDN_ERR_ARG, "scale * k_scale must be a number of at most 1e30");
  if (batch == 0) return ok();
  if (!slot_table || !kv_len || !q || !out) return fail(GDN_ERR_ARG, "a required pointer is NULL");
  if ((s = check_words({slot_table, kv_len, kv_begin, lse})) != GDN_OK) return s;
  if (q_stride < int64_t(q_heads) * pool->d.head_dim)
    return fail(GDN_ERR_ARG, "q_stride below q_heads * head_dim");
  if (q_stride % 8 || !aligned(q, 16) || !aligned(out, 16))
    return fail(GDN_ERR_UNSUPPORTED, "q rows and out must be 16-byte aligned");
  const size_t need = gdn::attn_workspace(pool, batch, q_heads, max_len, flags);
  if (need && (!workspace || workspace_bytes < need))
    return fail(GDN_ERR_ARG, "workspace of %zu bytes is below the needed %zu", workspace_bytes, need);
  if (need && !aligned(workspace, 256))
    return fail(GDN_ERR_UNSUPPORTED, "workspace must be 256-byte aligned");
  const int64_t row = int64_t(q_heads) * pool->d.head_dim * 2;
  const gdn::KvGeom g = gdn::kv_geom(pool, layer);
  const int64_t mass_bytes = flags & GDN_F_ACCUM_MASS ? int64_t(g.slots) * g.kv_heads * g.capacity * 4 : 0;
  s = check_apart({flat("out", out, batch * row), flat("lse", lse, int64_t(batch) * q_heads * 4),
                   flat("workspace", workspace, int64_t(need)), flat("mass", g.mass, mass_bytes),
                   flat("err_word", g.err, 4)},
                  {{"q", {q, batch, row, q_stride * 2}}, flat("slot_table", slot_table, batch * 4),
                   flat("kv_len", kv_len, batch * 4), flat("kv_begin", kv_begin, batch * 4),
                   flat("page_table", g.page_table, int64_t(g.slots) * g.max_pages * 4)});
  if (s != GDN_OK) return s;
  gdn::AttnArgs a{batch, q_heads, max_len, slot_table, kv_len, kv_begin, q,
                  q_stride, scale, flags, out, lse, workspace};
  return launched(gdn::launch_attn_decode(pool, layer, a, static_cast<hipStream_t>(stream)),
                  "attn_decode_paged launch");
}

GDN_API gdn_status kv_evict_plan(gdn_kv_pool_t pool, int32_t layer_begin, int32_t layer_end,
                                 int32_t batch, int32_t max_len, const int32_t *slot_table,
                                 const int32_t *kv_len, const int32_t *next_pos, int32_t budget,
                                 int32_t sink, int32_t recent, int32_t max_moves,
                                 int32_t *n_moves, int32_t *moves, int32_t *kv_len_out,
                                 void *stream) {
  gdn_status s = check_call(pool, layer_begin, layer_end, batch);
  if (s != GDN_OK) return s;
  if ((s = check_max_len(pool, max_len)) != GDN_OK) return s;
  if (!pool->d.mass || !pool->d.pos)
    return fail(GDN_ERR_ARG, "an eviction plan needs a pool with mass and pos");
  if (budget < 1 || sink < 0 || recent < 0 || int64_t(sink) + recent > budget)
    return fail(GDN_ERR_ARG, "need budget >= 1, sink, recent >= 0 and sink + recent <= budget");
  const int most = std::max(0, std::min(budget, max_len - budget));
  if (max_moves < most)
    return fail(GDN_ERR_ARG, "max_moves %d below min(budget, max_len - budget) = %d", max_moves, most);
  const int64_t lists = int64_t(layer_end - layer_begin) * batch * pool->d.kv_heads;
  if (lists * max_moves >= int64_t(1) << 40)
    return fail(GDN_ERR_RANGE, "layers * batch * kv_heads * max_moves must be below 2^40");
  if (batch == 0 || layer_begin == layer_end) return ok();
  if (!slot_table || !kv_len || !next_pos || !n_moves || !kv_len_out || (!moves && most > 0))
    return fail(GDN_ERR_ARG, "a required pointer is NULL");
  if ((s = check_words({slot_table, kv_len, next_pos, n_moves, moves, kv_len_out})) != GDN_OK) return s;
  const gdn::KvGeom g = gdn::kv_geom(pool, layer_begin);
  const int64_t mass_bytes = (layer_end - layer_begin) * (int64_t(g.slots) * g.kv_heads * g.capacity * 4);
  s = check_apart({flat("kv_len_out", kv_len_out, batch * 4), flat("n_moves", n_moves, lists * 4),
                   flat("moves", moves, lists * max_moves * 8), flat("err_word", g.err, 4)},
                  {flat("slot_table", slot_table, batch * 4), flat("kv_len", kv_len, batch * 4),
                   flat("next_pos", next_pos, batch * 4), flat("mass", g.mass, mass_bytes),
                   flat("pos", g.pos, mass_bytes)});
  if (s != GDN_OK) return s;
  gdn::EvictArgs a{layer_end - layer_begin, batch, max_len, budget, sink, recent, max_moves,
                   slot_table, kv_len, next_pos, n_moves, moves, kv_len_out};
  return launched(gdn::launch_kv_evict_plan(pool, layer_begin, a, static_cast<hipStream_t>(stream)),
                  "kv_evict_plan launch");
}

GDN_API gdn_status kv_evict_apply(gdn_kv_pool_t pool, int32_t layer_begin, int32_t layer_end,
                                  int32_t batch, int32_t max_moves, const int32_t *slot_table,
                                  const int32_t *n_moves, const int32_t *moves, void *stream) {
  gdn_status s = check_call(pool, layer_begin, layer_end, batch);
  if (s != GDN_OK) return s;
  if (max_moves < 0 || max_moves > pool->capacity)
    return fail(GDN_ERR_RANGE, "max_moves %d outside [0, %d]", max_moves, pool->capacity);
  if (int64_t(layer_end - layer_begin) * batch * pool->d.kv_heads * max_moves >= int64_t(1) << 40)
    return fail(GDN_ERR_RANGE, "layers * batch * kv_heads * max_moves must be below 2^40");
  if (batch == 0 || layer_begin == layer_end || max_moves == 0) return ok();
  if (!slot_table || !n_moves || !moves) return fail(GDN_ERR_ARG, "a required pointer is NULL");
  if ((s = check_words({slot_table, n_moves, moves})) != GDN_OK) return s;
  gdn::EvictArgs a{};
  a.layers = layer_end - layer_begin;
  a.batch = batch;
  a.max_moves = max_moves;
  a.slot_table = slot_table;
  a.n_moves = const_cast<int32_t *>(n_moves);
  a.moves = const_cast<int32_t *>(moves);
  return launched(gdn::launch_kv_evict_apply(pool, layer_begin, a, static_cast<hipStream_t>(stream)),
                  "kv_evict_apply launch");
}

GDN_API gdn_status kv_batch_map(gdn_kv_pool_t pool, int32_t batch, int32_t max_tokens,
                                const int32_t *slot_table, const int32_t *kv_len, const int32_t *new_len,
                                const int32_t *next_pos, int32_t free_capacity,
                                const int32_t *free_pages, const int32_t *n_free, int32_t *n_free_out,
                                int32_t *cu_seqlens, int32_t *slot_out, int32_t *kv_len_out,
                                int32_t *next_pos_out, int32_t *token_slot, int32_t *token_index,
                                int32_t *token_pos, void *stream) {
  gdn_status s = check_call(pool, 0, 1, batch);
  if (s != GDN_OK) return s;
  if (max_tokens < 0 || max_tokens > (1 << 26) - 2)
    return fail(GDN_ERR_RANGE, "max_tokens %d outside [0, 2^26 - 2]", max_tokens);
  if (free_capacity < 0) return fail(GDN_ERR_RANGE, "free_capacity < 0");
  if (!n_free || !n_free_out || !cu_seqlens || (!free_pages && free_capacity > 0))
    return fail(GDN_ERR_ARG, "a required pointer is NULL");
  if (batch > 0 && (!slot_table || !kv_len || !slot_out || !kv_len_out))
    return fail(GDN_ERR_ARG, "a required pointer is NULL");
  if (max_tokens > 0 && (!token_slot || !token_index)) return fail(GDN_ERR_ARG, "a required pointer is NULL");
  if (next_pos_out && !next_pos) return fail(GDN_ERR_ARG, "next_pos_out without next_pos");
  if ((s = check_words({slot_table, kv_len, new_len, next_pos, free_pages, n_free, n_free_out, cu_seqlens,
                        slot_out, kv_len_out, next_pos_out, token_slot, token_index, token_pos})) != GDN_OK)
    return s;
  const int64_t row = int64_t(batch) * 4, tok = int64_t(max_tokens) * 4;
  int32_t *const table = const_cast<int32_t *>(pool->d.page_table);
  // (an array that is updated in place is named as an output only)
  s = check_apart({flat("cu_seqlens", cu_seqlens, row + 4), flat("slot_out", slot_out, row),
                   flat("kv_len_out", kv_len_out, row), flat("next_pos_out", next_pos_out, row),
                   flat("n_free_out", n_free_out, 4), flat("token_slot", token_slot, tok),
                   flat("token_index", token_index, tok), flat("token_pos", token_pos, tok),
                   flat("page_table", table, int64_t(pool->d.slots) * pool->d.max_pages * 4),
                   flat("err_word", pool->d.err_word, 4)},
                  {flat("slot_table", slot_table, row),
                   flat("kv_len", kv_len == kv_len_out ? nullptr : kv_len, row),
                   flat("new_len", new_len, row),
                   flat("next_pos", next_pos == next_pos_out ? nullptr : next_pos, row),
                   flat("free_pages", free_pages, int64_t(free_capacity) * 4),
                   flat("n_free", n_free == n_free_out ? nullptr : n_free, 4)});
  if (s != GDN_OK) return s;
  gdn::MapArgs a{batch, max_tokens, free_capacity, slot_table, kv_len, new_len, next_pos, free_pages, n_free,
                 table, n_free_out, cu_seqlens, slot_out, kv_len_out, next_pos_out, token_slot, token_index,
                 token_pos};
  return launched(gdn::launch_kv_batch_map(pool, a, static_cast<hipStream_t>(stream)), "kv_batch_map launch");
}

GDN_API gdn_status kv_release(gdn_kv_pool_t pool, int32_t batch, const int32_t *slot_table,
                              const int32_t *kv_len, const int32_t *keep, int32_t free_capacity,
                              int32_t *free_pages, const int32_t *n_free, int32_t *n_free_out,
                              void *stream) {
  gdn_status s = check_call(pool, 0, 1, batch);
  if (s != GDN_OK) return s;
  if (free_capacity < 0) return fail(GDN_ERR_RANGE, "free_capacity < 0");
  if (!n_free || !n_free_out || (!free_pages && free_capacity > 0) || (batch > 0 && (!slot_table || !kv_len)))
    return fail(GDN_ERR_ARG, "a required pointer is NULL");
  if ((s = check_words({slot_table, kv_len, keep, free_pages, n_free, n_free_out})) != GDN_OK) return s;
  const int64_t row = int64_t(batch) * 4;
  int32_t *const table = const_cast<int32_t *>(pool->d.page_table);
  s = check_apart({flat("free_pages", free_pages, int64_t(free_capacity) * 4), flat("n_free_out", n_free_out, 4),
                   flat("page_table", table, int64_t(pool->d.slots) * pool->d.max_pages * 4),
                   flat("err_word", pool->d.err_word, 4)},
                  {flat("slot_table", slot_table, row), flat("kv_len", kv_len, row), flat("keep", keep, row),
                   flat("n_free", n_free == n_free_out ? nullptr : n_free, 4)});
  if (s != GDN_OK) return s;
  gdn::ReleaseArgs a{batch, free_capacity, slot_table, kv_len, keep, n_free, table, free_pages, n_free_out};
  return launched(gdn::launch_kv_release(pool, a, static_cast<hipStream_t>(stream)), "kv_release launch");
}

GDN_API gdn_status rope_frequencies(const gdn_rope_desc *d, double *freqs, float *amplitude) {
  if (!d || !freqs) return fail(GDN_ERR_ARG, "desc or freqs is NULL");
  if (d->rot_dim < 2 || d->rot_dim > 256 || d->rot_dim % 2)
    return fail(GDN_ERR_UNSUPPORTED, "rot_dim %d is not even and in [2, 256]", d->rot_dim);
  if (d->scaling < GDN_ROPE_PLAIN || d->scaling > GDN_ROPE_BANDS)
    return fail(GDN_ERR_ARG, "scaling %d unknown", d->scaling);
  if (d->scaling == GDN_ROPE_NTK && d->rot_dim < 4)
    return fail(GDN_ERR_UNSUPPORTED, "GDN_ROPE_NTK needs rot_dim >= 4");
  if (!(d->base > 1) || !std::isfinite(d->base)) return fail(GDN_ERR_ARG, "base must be finite and above 1");
  if (d->scaling != GDN_ROPE_PLAIN && (!(d->factor >= 1) || !std::isfinite(d->factor)))
    return fail(GDN_ERR_ARG, "factor must be finite and at least 1");
  const bool ramp = d->scaling == GDN_ROPE_YARN || d->scaling == GDN_ROPE_BANDS;
  if (ramp && (!(d->original_len > 0) || !(d->low > 0) || !(d->high > d->low) || !std::isfinite(d->original_len) ||
               !std::isfinite(d->high)))
    return fail(GDN_ERR_ARG, "need original_len > 0 and high > low > 0, all finite");
  const int rot = d->rot_dim;
  const double turn = 6.283185307179586476925, f = d->factor;
  const double base = d->scaling == GDN_ROPE_NTK ? d->base * std::pow(f, rot / (rot - 2.0)) : d->base;
  // the index at which a pair turns `times` over original_len
  auto index_of = [&](double times) {
    return rot * std::log(d->original_len / (times * turn)) / (2 * std::log(d->base));
  };
  double lo = 0, hi = 0;
  if (d->scaling == GDN_ROPE_YARN) {
    lo = std::max(0.0, std::floor(index_of(d->high)));
    hi = std::min(rot - 1.0, std::ceil(index_of(d->low)));
  }
  for (int i = 0; i < rot / 2; ++i) {
    const double theta = std::pow(base, -2.0 * i / rot);
    double slow = 0;  // how much of the angle is divided by the factor
    if (d->scaling == GDN_ROPE_LINEAR) slow = 1;
    if (d->scaling == GDN_ROPE_YARN) slow = (i - lo) / std::max(hi - lo, 1e-3);
    if (d->scaling == GDN_ROPE_BANDS) slow = 1 - (d->original_len * theta / turn - d->low) / (d->high - d->low);
    slow = std::min(1.0, std::max(0.0, slow));
    freqs[i] = slow == 0 ? theta : theta / f * slow + theta * (1 - slow);
  }
  if (amplitude) *amplitude = d->scaling == GDN_ROPE_YARN ? float(0.1 * std::log(f) + 1.0) : 1.f;
  return ok();
}

GDN_API gdn_status rope_append(gdn_kv_pool_t pool, int32_t layer, int32_t n, const int32_t *slot_ids,
                               const int32_t *index, const int32_t *position, int32_t q_heads,
                               const uint16_t *q, int64_t q_stride, uint16_t *q_out, int64_t q_out_stride,
                               const uint16_t *k, int64_t k_stride, const uint16_t *v, int64_t v_stride,
                               int32_t rot_dim, int32_t layout, const double *freqs, float amplitude,
                               void *stream) {
  gdn_status s = check_call(pool, layer, layer < INT32_MAX ? layer + 1 : layer, 0);
  if (s != GDN_OK) return s;
  if (n < 0) return fail(GDN_ERR_RANGE, "n < 0");
  if (q_heads < 0 || q_heads > 65535) return fail(GDN_ERR_RANGE, "q_heads %d outside [0, 65535]", q_heads);
  if (rot_dim < 16 || rot_dim > pool->d.head_dim || rot_dim % 16)
    return fail(GDN_ERR_UNSUPPORTED, "rot_dim %d is not a multiple of 16 in [16, head_dim]", rot_dim);
  if (layout != GDN_ROPE_HALF && layout != GDN_ROPE_INTERLEAVED) return fail(GDN_ERR_ARG, "layout %d unknown", layout);
  if (!std::isfinite(amplitude)) return fail(GDN_ERR_ARG, "amplitude must be finite");
  if (n == 0) return ok();
  if (!slot_ids || !index || !position || !k || !v || !freqs || (q_heads > 0 && (!q || !q_out)))
    return fail(GDN_ERR_ARG, "a required pointer is NULL");
  if ((s = check_words({slot_ids, index, position})) != GDN_OK) return s;
  if (!aligned(freqs, 8)) return fail(GDN_ERR_ARG, "freqs must be 8-byte aligned");
  const int64_t row = int64_t(pool->d.kv_heads) * pool->d.head_dim, qrow = int64_t(q_heads) * pool->d.head_dim;
  if (k_stride < row || v_stride < row || (q_heads > 0 && (q_stride < qrow || q_out_stride < qrow)))
    return fail(GDN_ERR_ARG, "a stride is below the values of a token");
  if (k_stride % 8 || v_stride % 8 || !aligned(k, 16) || !aligned(v, 16) ||
      (q_heads > 0 && (q_stride % 8 || q_out_stride % 8 || !aligned(q, 16) || !aligned(q_out, 16))))
    return fail(GDN_ERR_UNSUPPORTED, "rows of q, q_out, k and v must be 16-byte aligned");
  if (q_heads > 0) {
    const Rows to{q_out, n, qrow * 2, q_out_stride * 2};
    struct {
      const char *name;
      Rows rows;
    } in[] = {{"q", {q, n, qrow * 2, q_stride * 2}}, {"k", {k, n, row * 2, k_stride * 2}},
              {"v", {v, n, row * 2, v_stride * 2}}, {"slot_ids", {slot_ids, 1, n * int64_t(4), n * int64_t(4)}},
              {"index", {index, 1, n * int64_t(4), n * int64_t(4)}},
              {"position", {position, 1, n * int64_t(4), n * int64_t(4)}}, {"freqs", {freqs, 1, rot_dim * 4, rot_dim * 4}},
              {"err_word", {pool->d.err_word, 1, 4, 4}}};
    for (const auto &x : in) {
      if (&x == in && q_out == q && q_out_stride == q_stride) continue;  // in place
      const bool meet = x.rows.n == 1 && x.rows.row == x.rows.stride ? overlap(to, x.rows.base, x.rows.row)
                                                                     : rows_meet(to, x.rows);
      if (meet) return fail(GDN_ERR_ARG, "q_out overlaps %s", x.name);
    }
  }
  gdn::RopeArgs a{n, q_heads, slot_ids, index, position, q, q_stride, q_out, q_out_stride, k, v, k_stride, v_stride,
                  rot_dim, layout, freqs, amplitude};
  return launched(gdn::launch_rope_append(pool, layer, a, static_cast<hipStream_t>(stream)), "rope_append launch");
}

namespace {
gdn_status check_chunk(gdn_kv_pool_t p, int batch, int tokens, int q_heads, int max_len, int mass_tokens) {
  gdn_status s = check_call(p, 0, 1, batch);
  if (s != GDN_OK) return s;
  if ((s = check_max_len(p, max_len)) != GDN_OK) return s;
  if ((s = check_heads(p, q_heads)) != GDN_OK) return s;
  if (tokens < 0 || mass_tokens < 0) return fail(GDN_ERR_RANGE, "tokens or mass_tokens < 0");
  if (mass_tokens > 0 && !p->d.mass) return fail(GDN_ERR_ARG, "mass_tokens needs a pool with mass");
  if (!gdn::chunk_fits(p, batch, tokens, q_heads, max_len))
    return fail(GDN_ERR_RANGE, "tokens * q_heads or batch * kv_heads * max_len too large");
  return GDN_OK;
}
}  // namespace

GDN_API gdn_status attn_prefill_workspace_bytes(gdn_kv_pool_t pool, int32_t batch, int32_t tokens,
                                                int32_t q_heads, int32_t max_len, int32_t mass_tokens,
                                                size_t *bytes) {
  if (!bytes) return fail(GDN_ERR_ARG, "bytes is NULL");
  gdn_status s = check_chunk(pool, batch, tokens, q_heads, max_len, mass_tokens);
  if (s != GDN_OK) return s;
  *bytes = gdn::chunk_workspace(pool, batch, tokens, q_heads, max_len, mass_tokens);
  return ok();
}

GDN_API gdn_status attn_prefill_paged(gdn_kv_pool_t pool, int32_t layer, int32_t batch, int32_t tokens,
                                      int32_t q_heads, int32_t max_len, const int32_t *cu_seqlens,
                                      const int32_t *slot_table, const int32_t *kv_len,
                                      const int32_t *kv_begin, const uint16_t *q, int64_t q_stride,
                                      float scale, int32_t window, int32_t mass_tokens, uint16_t *out,
                                      float *lse, void *workspace, size_t workspace_bytes, void *stream) {
  gdn_status s = check_chunk(pool, batch, tokens, q_heads, max_len, mass_tokens);
  if (s != GDN_OK) return s;
  if (layer < 0 || layer >= pool->d.layers)
    return fail(GDN_ERR_RANGE, "layer %d outside [0, %d)", layer, pool->d.layers);
  if (window < 0) return fail(GDN_ERR_RANGE, "window < 0");
  if (!(fabsf(scale) * pool->d.k_scale <= 1e30f))
    return fail(GDN_ERR_ARG, "scale * k_scale must be a number of at most 1e30");
  if (batch == 0 || tokens == 0) return ok();
  if (!cu_seqlens || !slot_table || !kv_len || !q || !out) return fail(GDN_ERR_ARG, "a required pointer is NULL");
  if ((s = check_words({cu_seqlens, slot_table, kv_len, kv_begin, lse})) != GDN_OK) return s;
  const int64_t row = int64_t(q_heads) * pool->d.head_dim;
  if (q_stride < row) return fail(GDN_ERR_ARG, "q_stride below q_heads * head_dim");
  if (q_stride % 8 || !aligned(q, 16) || !aligned(out, 16))
    return fail(GDN_ERR_UNSUPPORTED, "q rows and out must be 16-byte aligned");
  const size_t need = gdn::chunk_workspace(pool, batch, tokens, q_heads, max_len, mass_tokens);
  if (need && (!workspace || workspace_bytes < need))
    return fail(GDN_ERR_ARG, "workspace of %zu bytes is below the needed %zu", workspace_bytes, need);
  if (need && !aligned(workspace, 256)) return fail(GDN_ERR_UNSUPPORTED, "workspace must be 256-byte aligned");
  const gdn::KvGeom g = gdn::kv_geom(pool, layer);
  const int64_t mass_bytes = mass_tokens ? int64_t(g.slots) * g.kv_heads * g.capacity * 4 : 0;
  s = check_apart({flat("out", out, tokens * row * 2), flat("lse", lse, int64_t(tokens) * q_heads * 4),
                   flat("workspace", workspace, int64_t(need)), flat("mass", g.mass, mass_bytes),
                   flat("err_word", g.err, 4)},
                  {{"q", {q, tokens, row * 2, q_stride * 2}}, flat("cu_seqlens", cu_seqlens, batch * 4 + 4),
                   flat("slot_table", slot_table, batch * 4), flat("kv_len", kv_len, batch * 4),
                   flat("kv_begin", kv_begin, batch * 4),
                   flat("page_table", g.page_table, int64_t(g.slots) * g.max_pages * 4)});
  if (s != GDN_OK) return s;
  gdn::ChunkArgs a{batch, tokens, q_heads, max_len, window, mass_tokens, cu_seqlens, slot_table, kv_len, kv_begin,
                   q, q_stride, scale, out, lse, workspace};
  return launched(gdn::launch_attn_prefill(pool, layer, a, static_cast<hipStream_t>(stream)),
                  "attn_prefill_paged launch");
}

GDN_API gdn_status block_norm(int64_t tokens, int32_t groups, int32_t dim, const uint16_t *y,
                              int64_t y_stride, const void *w_post, const uint16_t *gate,
                              int64_t gate_stride, int32_t act, float scale, const void *residual,
                              void *residual_out, int32_t res_dtype, const void *w_pre,
                              int32_t w_dtype, float eps, uint32_t flags, uint16_t *out,
                              void *stream) {
  if (tokens < 0) return fail(GDN_ERR_RANGE, "tokens < 0");
  if (groups <= 0 || dim <= 0) return fail(GDN_ERR_ARG, "need groups and dim >= 1");
  if (dim % 8 || dim > 32768)
    return fail(GDN_ERR_UNSUPPORTED, "dim %d is not a multiple of 8 up to 32768", dim);
  if (tokens > (int64_t(1) << 31) / groups)
    return fail(GDN_ERR_RANGE, "tokens * groups must be at most 2^31");
  if (act != GDN_ACT_NONE && act != GDN_ACT_SILU && act != GDN_ACT_SIGMOID)
    return fail(GDN_ERR_ARG, "act %d unknown", act);
  if (act != GDN_ACT_NONE && !gate) return fail(GDN_ERR_ARG, "act without a gate");
  if (res_dtype != GDN_F32 && res_dtype != GDN_BF16)
    return fail(GDN_ERR_ARG, "res_dtype must be GDN_F32 or GDN_BF16");
  if (w_dtype != GDN_F32 && w_dtype != GDN_BF16)
    return fail(GDN_ERR_ARG, "w_dtype must be GDN_F32 or GDN_BF16");
  if (flags & ~uint32_t(GDN_F_NORM_PLUS_ONE)) return fail(GDN_ERR_ARG, "unknown flag bits 0x%x", flags);
  if (!(eps > 0) || !isfinite(eps) || !isfinite(scale))
    return fail(GDN_ERR_ARG, "eps must be finite and positive, scale finite");
  if ((residual == nullptr) != (residual_out == nullptr))
    return fail(GDN_ERR_ARG, "residual and residual_out are given together");
  if (tokens == 0) return ok();
  if (!y || !out) return fail(GDN_ERR_ARG, "y or out is NULL");
  const int64_t row = int64_t(groups) * dim;
  if (y_stride < row || (gate && gate_stride < row))
    return fail(GDN_ERR_ARG, "a stride is below groups * dim");
  if (y_stride % 8 || (gate && gate_stride % 8))
    return fail(GDN_ERR_UNSUPPORTED, "strides must be multiples of 8 elements");
  for (const void *p : {static_cast<const void *>(y), w_post, static_cast<const void *>(gate), residual,
                        static_cast<const void *>(residual_out), w_pre, static_cast<const void *>(out)})
    if (!aligned(p, 16)) return fail(GDN_ERR_UNSUPPORTED, "pointers must be 16-byte aligned");
  // a thread reads its own elements before it writes them: the same memory works where the
  // header says so, a shifted one does not
  const Rows yr{y, tokens, row * 2, y_stride * 2}, gr{gate, tokens, row * 2, gate_stride * 2};
  const int64_t out_bytes = tokens * row * 2, res_bytes = tokens * row * (res_dtype == GDN_F32 ? 4 : 2);
  const int64_t w_bytes = int64_t(dim) * (w_dtype == GDN_F32 ? 4 : 2);
  const Rows wr[2] = {{w_post, 1, w_bytes, w_bytes}, {w_pre, 1, w_bytes, w_bytes}};
  const Rows rr{residual, 1, res_bytes, res_bytes};
  if (!(out == y && (y_stride == row || tokens == 1)) && overlap(yr, out, out_bytes))
    return fail(GDN_ERR_ARG, "out overlaps y (only out = y with y_stride = groups * dim may)");
  if (overlap(gr, out, out_bytes) || overlap(rr, out, out_bytes) || overlap(wr[0], out, out_bytes) ||
      overlap(wr[1], out, out_bytes) || overlap({residual_out, 1, res_bytes, res_bytes}, out, out_bytes))
    return fail(GDN_ERR_ARG, "out overlaps gate, a weight, residual or residual_out");
  if (overlap(yr, residual_out, res_bytes) || overlap(gr, residual_out, res_bytes) ||
      overlap(wr[0], residual_out, res_bytes) || overlap(wr[1], residual_out, res_bytes) ||
      (residual_out != residual && overlap(rr, residual_out, res_bytes)))
    return fail(GDN_ERR_ARG, "residual_out overlaps y, gate, a weight or part of residual");
  gdn::NormArgs a{tokens, groups, dim, y, y_stride, w_post, gate, gate_stride, act, scale, residual,
                  residual_out, res_dtype, w_pre, w_dtype, eps, flags, out};
  return launched(gdn::launch_block_norm(a, static_cast<hipStream_t>(stream)), "block_norm launch");
}
