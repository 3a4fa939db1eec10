// kv.hpp -- internal declarations of the paged key-value cache, its attention and its
// eviction, and of the norm between blocks.  Not installed; the public interface is
// include/gdn_kv.h.
#pragma once

#include <algorithm>

#include "common.hpp"
#include "gdn_kv.h"

struct gdn_kv_pool {
  gdn_kv_desc d;
  int32_t capacity;     // max_pages * page_size: token places of a slot
  int32_t page_shift;   // log2(page_size)
  int64_t layer_rows;   // pages * kv_heads * page_size, < 2^31
  int32_t row_bytes;    // head_dim * element size
};

namespace gdn {

// What the device code of every cache kernel needs of a pool, passed by value.
struct KvGeom {
  char *k, *v;                // first row of the layer (or of layer 0)
  const int32_t *page_table;
  float *mass;                // entries of the layer (or of layer 0), or NULL
  int32_t *pos;
  int32_t *err;
  int64_t layer_rows;
  float k_scale, v_scale;
  int32_t pages, kv_heads, slots, max_pages, capacity, page_shift;
};

inline KvGeom kv_geom(const gdn_kv_pool *p, int layer) {
  KvGeom g;
  const int64_t off = int64_t(layer) * p->layer_rows * p->row_bytes;
  const int64_t moff = int64_t(layer) * p->d.slots * p->d.kv_heads * p->capacity;
  g.k = static_cast<char *>(p->d.k_base) + off;
  g.v = static_cast<char *>(p->d.v_base) + off;
  g.page_table = p->d.page_table;
  g.mass = p->d.mass ? p->d.mass + moff : nullptr;
  g.pos = p->d.pos ? p->d.pos + moff : nullptr;
  g.err = p->d.err_word;
  g.layer_rows = p->layer_rows;
  g.k_scale = p->d.k_scale;
  g.v_scale = p->d.v_scale;
  g.pages = p->d.pages;
  g.kv_heads = p->d.kv_heads;
  g.slots = p->d.slots;
  g.max_pages = p->d.max_pages;
  g.capacity = p->capacity;
  g.page_shift = p->page_shift;
  return g;
}

// Row (of the layer's [pages][kv_heads][page_size] rows) of token place i of a slot for
// head h, or -1 where the page id is not a page.  i is in [0, capacity).
__device__ __forceinline__ int kv_row(const KvGeom &g, int slot, int h, int i) {
  const int page = g.page_table[int64_t(slot) * g.max_pages + (i >> g.page_shift)];
  if (page <= 0 || page >= g.pages) return -1;
  return ((page * g.kv_heads + h) << g.page_shift) + (i & ((1 << g.page_shift) - 1));
}

// A grid of any number of workgroups as two dimensions (a launch holds fewer than 2^32
// threads in one), and a workgroup's number in it, which may pass the last one.
inline dim3 flat_grid(int64_t blocks) {
  const int64_t x = std::min<int64_t>(blocks, 1 << 21);
  return dim3(unsigned(x), unsigned((blocks + x - 1) / x));
}
__device__ __forceinline__ int64_t flat_block() { return int64_t(blockIdx.y) * gridDim.x + blockIdx.x; }

// Inclusive sum over the wave's lanes in order.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  v += uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x111, 0xF, 0xF, false));  // row_shr 1
  v += uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x112, 0xF, 0xF, false));
  v += uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x114, 0xF, 0xF, false));
  v += uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x118, 0xF, 0xF, false));
  v += uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x142, 0xA, 0xF, false));  // row_bcast 15
  v += uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x143, 0xC, 0xF, false));  // row_bcast 31
  return v;
}

__device__ __forceinline__ void set_err(int32_t *err, int bit) {
  if (err) atomicOr(err, bit);
}

struct AppendArgs {
  int n;
  const int32_t *slot_ids, *index, *position;
  const uint16_t *k, *v;
  int64_t k_stride, v_stride;
};
hipError_t launch_kv_append(const gdn_kv_pool *p, int layer, const AppendArgs &a, hipStream_t s);

struct EvictArgs {
  int layers, batch, max_len, budget, sink, recent, max_moves;
  const int32_t *slot_table, *kv_len, *next_pos;
  int32_t *n_moves, *moves, *kv_len_out;
};
hipError_t launch_kv_evict_plan(const gdn_kv_pool *p, int layer, const EvictArgs &a, hipStream_t s);
hipError_t launch_kv_evict_apply(const gdn_kv_pool *p, int layer, const EvictArgs &a, hipStream_t s);

// whether the call's blocks of 128 tokens can be counted in 31 bits
bool attn_fits(const gdn_kv_pool *p, int batch, int q_heads, int max_len);
size_t attn_workspace(const gdn_kv_pool *p, int batch, int q_heads, int max_len, uint32_t flags);

struct AttnArgs {
  int batch, q_heads, max_len;
  const int32_t *slot_table, *kv_len, *kv_begin;
  const uint16_t *q;
  int64_t q_stride;
  float scale;
  uint32_t flags;
  uint16_t *out;
  float *lse;
  void *workspace;
};
hipError_t launch_attn_decode(const gdn_kv_pool *p, int layer, const AttnArgs &a, hipStream_t s);

struct NormArgs {
  int64_t tokens;
  int groups, dim;
  const uint16_t *y;
  int64_t y_stride;
  const void *w_post;
  const uint16_t *gate;
  int64_t gate_stride;
  int act;
  float scale;
  const void *residual;
  void *residual_out;
  int res_dtype;
  const void *w_pre;
  int w_dtype;
  float eps;
  uint32_t flags;
  uint16_t *out;
};
hipError_t launch_block_norm(const NormArgs &a, hipStream_t s);

}  // namespace gdn
