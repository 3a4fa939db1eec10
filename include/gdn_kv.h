/*
 * gdn_kv.h -- C ABI of the full-attention half of a hybrid model's decode step on
 * MI355X (gfx950), beside the linear-attention half of gdn_slot.h.
 *
 * Hybrid models interleave their recurrent layers with full-attention layers, whose
 * keys and values live in a paged cache that the same request slots address (page
 * "SGLang之MambaRadixCache机制", sections 1.2 and 1.4: a KV pool per layer and a
 * request -> token-location table).  This header has
 *
 *   kv_append          store new tokens' keys and values (bf16, or e4m3 with a scale)
 *   attn_decode_paged  attention of one new token per request over its pages, split
 *                      over the cache's length and joined; optionally adds each
 *                      cached token's attention weight to a running sum
 *   kv_evict_plan      choose, per layer and key-value head, the tokens that a cache
 *                      over its budget keeps, by accumulated weight
 *   kv_evict_apply     move the kept tokens into the freed places
 *   block_norm         norm after a block, gate, residual scale and sum, norm before
 *                      the next block, in one pass (also the recurrence's gated norm)
 *
 * Formulas, with t over the visible tokens begin <= t < len of the request, h a query
 * head and g = h / (q_heads / kv_heads) its key-value head:
 *
 *   s_ht = scale q_h . k_gt       p_h = softmax_t(s_h)       out_h = sum_t p_ht v_gt
 *   lse_h = ln sum_t exp(s_ht)    mass_gt += sum over the heads h of g of p_ht
 *
 * Memory.  The caller owns every buffer; the library allocates no device memory.
 *
 *   k, v        [layers][pages][kv_heads][page_size][head_dim]  bf16 or e4m3;
 *               a key is k_scale * (stored value), a value v_scale * (stored value)
 *   page_table  int32 [slots][max_pages]: token index i of slot s lies in page
 *               page_table[s][i / page_size], row i % page_size
 *   mass        fp32  [layers][slots][kv_heads][max_pages * page_size], or NULL
 *   pos         int32, same shape: the token's position in the request, or NULL
 *
 * Slot 0 and page 0 are reserved (padding).  A slot id <= 0 skips its request or
 * token; one >= slots does too and sets GDN_ERRW_BAD_SLOT.  A page id outside
 * [1, pages) where a token is to be read or written sets GDN_ERRW_BAD_PAGE: an
 * attention treats that page's tokens as not visible, the other calls skip the token.
 * The bits go to the pool's error word (sticky; the caller clears it).
 *
 * int32 and fp32 arrays are 4-byte aligned, others as stated.
 *
 * Streams, errors and host-side checks are those of gdn_slot.h: asynchronous on the
 * given stream, everything the host can check is checked before any launch.  Every call
 * can be captured into a graph; replays read the device arrays anew.  Calls that share
 * a workspace, or of which one writes what another reads, must be ordered by the caller.
 */
#ifndef GDN_KV_H
#define GDN_KV_H

#include "gdn_slot.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct gdn_kv_pool *gdn_kv_pool_t;

/* storage type of a cache, beside GDN_BF16: OCP e4m3 (finite, largest 448) */
enum { GDN_F8_E4M3 = 2 };

/* a page id in a request's table is outside [1, pages) */
enum { GDN_ERRW_BAD_PAGE = 16 };

typedef struct {
  int32_t layers, pages, kv_heads, page_size, head_dim;
  int32_t slots, max_pages;
  int32_t kv_dtype;          /* GDN_BF16 | GDN_F8_E4M3 */
  float k_scale, v_scale;    /* finite, > 0; 1 for GDN_BF16 */
  void *k_base, *v_base;     /* device, 16-byte aligned, kv_pool_bytes() bytes each */
  const int32_t *page_table; /* device */
  float *mass;               /* device or NULL */
  int32_t *pos;              /* device or NULL */
  int32_t *err_word;         /* device int32 or NULL */
} gdn_kv_desc;

/* Bytes of k (and of v) and element count of mass (and of pos) for a descriptor's shape
 * (pointers and scales are ignored).  Pure host arithmetic. */
gdn_status kv_pool_bytes(const gdn_kv_desc *desc, size_t *kv_bytes, size_t *mass_elements);

/* Validate a descriptor and wrap it in a handle (host memory only; the buffers stay the
 * caller's).  Supported: head_dim in {64, 128, 256}, page_size a power of two in
 * [1, 1024], pages >= 2, slots >= 2, kv_heads <= 65535, max_pages * page_size < 2^30,
 * pages * kv_heads * page_size < 2^31, and k, v, mass and pos below 2^63 bytes each.  Thread-safe; the handle is immutable. */
gdn_status kv_pool_create(const gdn_kv_desc *desc, gdn_kv_pool_t *out);

/* Free a handle (not the buffers).  NULL is ignored. */
void kv_pool_destroy(gdn_kv_pool_t pool);

/* Store n new tokens of one layer.
 * slot_ids    device int32 [n], index device int32 [n]: token i goes to place index[i]
 *             of slot slot_ids[i] (index outside [0, max_pages * page_size) sets
 *             GDN_ERRW_BAD_SEQLENS and skips the token); the (slot, index) pairs of a
 *             call must be distinct.  No input may lie where the call writes
 * k, v        device bf16, token i at k + i * k_stride (elements, a multiple of 8, at
 *             least kv_heads * head_dim; 16-byte aligned), [kv_heads][head_dim] there
 * position    device int32 [n], stored to pos; required iff the pool has pos
 * A GDN_BF16 pool takes the rows bit for bit.  A GDN_F8_E4M3 pool takes x / k_scale (x /
 * v_scale), divided in fp32, limited to +-448 and rounded to nearest even; NaN stays NaN.
 * If the pool has mass, the token's weights are set to 0. */
gdn_status kv_append(gdn_kv_pool_t pool, int32_t layer, int32_t n, const int32_t *slot_ids,
                     const int32_t *index, const int32_t *position, const uint16_t *k,
                     int64_t k_stride, const uint16_t *v, int64_t v_stride, void *stream);

/* attention flags */
enum { GDN_F_ACCUM_MASS = 1u };

/* Workspace of attn_decode_paged for `batch` requests of up to max_len tokens.  Pure
 * host arithmetic.  With GDN_F_ACCUM_MASS it holds every score, 4 * batch * q_heads *
 * max_len bytes by the bound, not the lengths (128 requests of 32 heads, 131072 tokens:
 * 2.1 GB), so a close bound is smaller too. */
gdn_status attn_workspace_bytes(gdn_kv_pool_t pool, int32_t batch, int32_t q_heads,
                                int32_t max_len, uint32_t flags, size_t *bytes);

/* Attention of one new token per request over one layer's cache (its own key and value
 * are appended before).
 * q_heads     a multiple of kv_heads, at most 64 per key-value head
 * max_len     host int: no request has more tokens (one that has, or a negative length
 *             or begin, sets GDN_ERRW_BAD_SEQLENS and is skipped).  It decides how the
 *             length is split, so a close bound is faster; at most
 *             max_pages * page_size
 * slot_table  device int32 [batch]
 * kv_len      device int32 [batch]: tokens in the cache
 * kv_begin    device int32 [batch] or NULL (= 0): first visible place of the cache.  Places
 *             are the order of the tokens, and so a sliding window, only in a slot that no
 *             kv_evict_apply has cut: its moves put late tokens into early places, and the
 *             pool's pos is not looked at here.  A slot that was cut is attended to whole
 * q           device bf16, request b at q + b * q_stride (elements, a multiple of 8, at
 *             least q_heads * head_dim; 16-byte aligned), [q_heads][head_dim] there
 * scale       |scale * k_scale| at most 1e30
 * flags       GDN_F_ACCUM_MASS: add the weights to the pool's mass (which it must have;
 *             live slots must be distinct then).  Only visible tokens' entries change
 * out         device bf16 [batch][q_heads][head_dim], 16-byte aligned
 * lse         device fp32 [batch][q_heads] or NULL
 * workspace   attn_workspace_bytes(...) bytes, 256-byte aligned; its contents are not
 *             read across calls
 * What the call writes (out, lse, workspace, with the flag the layer's mass, and the error
 * word) must not overlap what it reads (q, slot_table, kv_len, kv_begin, page_table) or each
 * other.
 * A request that sees no token (skipped, begin >= len, or every score -inf) gets out = 0
 * and lse = -inf and adds no weight.  Tokens outside [begin, len) are not read into the
 * result whatever their rows hold.  A visible token's infinite value makes that column of out
 * infinite (NaN beside one of the other sign; NaN or infinite where the token's weight is below
 * 2^-100 of the largest).  A score of +inf or NaN has no softmax: that head's out and lse are
 * NaN, and so are the weights that it adds.  The values' sum before the division by l is
 * held in fp32: the number of visible tokens times the largest stored |value| stays below
 * 3.4e38.  The result does not depend on the order in which the workgroups run. */
gdn_status attn_decode_paged(gdn_kv_pool_t pool, int32_t layer, int32_t batch, int32_t q_heads,
                             int32_t max_len, const int32_t *slot_table, const int32_t *kv_len,
                             const int32_t *kv_begin, const uint16_t *q, int64_t q_stride,
                             float scale, uint32_t flags, uint16_t *out, float *lse,
                             void *workspace, size_t workspace_bytes, void *stream);

/* Plan an eviction in layers [layer_begin, layer_end).  Per request, layer and key-value
 * head, a cache of n = kv_len[b] > budget tokens keeps `budget` of them: those with
 * pos < sink or pos >= next_pos[b] - recent first, then those of the largest mass; ties
 * (among the protected too, if they alone exceed the budget) go to the lowest index.  A
 * NaN or negative mass counts as 0.  The kept tokens at index >= budget, in order, move to
 * the freed places below budget, in order; attention over all places does not depend on
 * their order (attn_decode_paged's kv_begin does, and does not go with a slot that was cut).
 * Nothing is moved by this call.
 * max_len     no request has more tokens (more, or fewer than 0: GDN_ERRW_BAD_SEQLENS,
 *             skipped); at most max_pages * page_size.  It chooses how a list is
 *             worked on (up to 2048, up to 36864, longer), so a close bound is faster
 * budget      >= 1;  sink, recent >= 0 with sink + recent <= budget
 * n_moves     device int32 [layer_end - layer_begin][batch][kv_heads]: 0 where nothing
 *             moves
 * moves       device int32 [layer_end - layer_begin][batch][kv_heads][max_moves][2]:
 *             (source, destination) indices, the first n_moves entries written, the
 *             others left as they are; max_moves >= min(budget, max_len - budget), and
 *             layers * batch * kv_heads * max_moves below 2^40
 * kv_len_out  device int32 [batch]: min(n, budget); a skipped request's length is
 *             copied
 * What the call writes (n_moves, moves, kv_len_out and the error word) must not overlap
 * what it reads (slot_table, kv_len, next_pos, the layers' mass and pos) or each other.
 * Where layer_begin = layer_end nothing is planned and nothing written, kv_len_out
 * neither.  The pool must have mass and pos. */
gdn_status kv_evict_plan(gdn_kv_pool_t pool, int32_t layer_begin, int32_t layer_end,
                         int32_t batch, int32_t max_len, const int32_t *slot_table,
                         const int32_t *kv_len, const int32_t *next_pos, int32_t budget,
                         int32_t sink, int32_t recent, int32_t max_moves, int32_t *n_moves,
                         int32_t *moves, int32_t *kv_len_out, void *stream);

/* Carry out moves: for every layer, request, head and entry, the rows of k and v and, if
 * the pool has them, the entries of mass and pos at the source index are copied to the
 * destination index.  Byte-exact.  No destination of a (layer, request, head) may be a
 * source or another destination of it (a plan's never are), live slots must be distinct, and
 * the pages written must belong to their request alone.  A count outside
 * [0, max_moves] sets GDN_ERRW_BAD_SEQLENS and skips that list; an index outside
 * [0, max_pages * page_size) does and skips the entry.  layers * batch * kv_heads *
 * max_moves is below 2^40. */
gdn_status kv_evict_apply(gdn_kv_pool_t pool, int32_t layer_begin, int32_t layer_end,
                          int32_t batch, int32_t max_moves, const int32_t *slot_table,
                          const int32_t *n_moves, const int32_t *moves, void *stream);

/* gate activations of block_norm */
enum { GDN_ACT_NONE = 0, GDN_ACT_SILU = 1, GDN_ACT_SIGMOID = 2 };

/* block_norm flags: weights are stored as w - 1 (the factor is 1 + w) */
enum { GDN_F_NORM_PLUS_ONE = 1u };

/* Between two blocks, per row x of `dim` values (rms(x) = x / sqrt(mean(x^2) + eps)):
 *
 *   u = y;  u = rms(u) * w_post         (w_post given)
 *   u = u * act(gate)                   (gate given: gate, silu(gate) or sigmoid(gate))
 *   u = scale * u;  r = residual + u    (residual given, else r = u)
 *   residual_out = r                    (residual given; may be the same memory)
 *   out = rms(r) * w_pre  (w_pre given), else out = r
 *
 * There are tokens * groups rows; a token's groups are adjacent and share the weights
 * [dim] (the recurrence's output norm: groups = heads, dim = head_v, gate = z).  y and
 * gate are bf16 with a stride per token (elements, a multiple of 8, at least
 * groups * dim); residual, residual_out (res_dtype GDN_BF16 or GDN_F32) and out (bf16) are
 * contiguous.  w_dtype (GDN_BF16 or GDN_F32) is the weights' type.  dim is a multiple of
 * 8, at most 32768; every pointer 16-byte aligned.  Everything is computed in fp32 (a row
 * whose squares sum past 3.4e38 has rms(x) = 0 there, a gate below -87 sigmoid 0) and
 * each output is rounded once, r for the second norm not at all.  residual_out may be
 * residual and out may be y (with y_stride = groups * dim); otherwise outputs must not
 * overlap inputs.  eps > 0. */
gdn_status block_norm(int64_t tokens, int32_t groups, int32_t dim, const uint16_t *y,
                      int64_t y_stride, const void *w_post, const uint16_t *gate,
                      int64_t gate_stride, int32_t act, float scale, const void *residual,
                      void *residual_out, int32_t res_dtype, const void *w_pre, int32_t w_dtype,
                      float eps, uint32_t flags, uint16_t *out, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* GDN_KV_H */
