// kv_cache.hip -- the paged key-value cache's own kernels: append, eviction plan and
// the moves of an eviction (formulas and rules: include/gdn_kv.h).
#include "kv.hpp"
#include "lanes.hpp"

namespace gdn {
namespace {

// ------------------------------------------------------------------ append --
// One thread per 8 consecutive values of a token's key and of its value: two 16-byte
// loads, one store each.  Bound by the bytes (and by the launch for one decode step).
constexpr int kAppendThreads = 256;

// 8 bf16 values / scale, limited to e4m3's largest value, rounded once to nearest even
// (the limits keep NaN: both comparisons are false)
__device__ __forceinline__ u32x2 quantise8(const u32x4 &x, float scale) {
  u32x2 r;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    float f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t w = x[2 * p + (e >> 1)];
      float t = __uint_as_float((e & 1) ? (w & 0xffff0000u) : (w << 16)) / scale;
      t = t > 448.f ? 448.f : t;
      f[e] = t < -448.f ? -448.f : t;
    }
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
    r[p] = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], w, true));
  }
  return r;
}

template <bool kF8>
__global__ __launch_bounds__(kAppendThreads) void kv_append_kernel(KvGeom g, int head_dim, AppendArgs a) {
  const int vecs = head_dim >> 3;       // 16-byte pieces of a head's row
  const int per = g.kv_heads * vecs;
  const int64_t item = int64_t(blockIdx.x) * kAppendThreads + threadIdx.x;
  const int token = int(item / per);
  if (token >= a.n) return;
  const int j = int(item - int64_t(token) * per);
  const int h = j / vecs, piece = j - h * vecs;
  const int slot = a.slot_ids[token], i = a.index[token];
  const bool first = j == 0;
  if (slot <= 0 || slot >= g.slots) {
    if (first && slot >= g.slots) set_err(g.err, GDN_ERRW_BAD_SLOT);
    return;
  }
  if (i < 0 || i >= g.capacity) {
    if (first) set_err(g.err, GDN_ERRW_BAD_SEQLENS);
    return;
  }
  const u32x4 kx = *reinterpret_cast<const u32x4 *>(a.k + token * a.k_stride + 8 * j);
  const u32x4 vx = *reinterpret_cast<const u32x4 *>(a.v + token * a.v_stride + 8 * j);
  const int row = kv_row(g, slot, h, i);
  if (row < 0) {
    if (first) set_err(g.err, GDN_ERRW_BAD_PAGE);
    return;
  }
  if (kF8) {
    const int64_t off = int64_t(row) * head_dim + 8 * piece;
    *reinterpret_cast<u32x2 *>(g.k + off) = quantise8(kx, g.k_scale);
    *reinterpret_cast<u32x2 *>(g.v + off) = quantise8(vx, g.v_scale);
  } else {
    const int64_t off = (int64_t(row) * head_dim + 8 * piece) * 2;
    *reinterpret_cast<u32x4 *>(g.k + off) = kx;
    *reinterpret_cast<u32x4 *>(g.v + off) = vx;
  }
  if (piece == 0) {
    const int64_t m = (int64_t(slot) * g.kv_heads + h) * g.capacity + i;
    if (g.mass) g.mass[m] = 0.f;
    if (g.pos) g.pos[m] = a.position[token];
  }
}

// ----------------------------------------------------------- eviction plan --
// One workgroup per (layer, request, head).  A token's key is its weight's bits (weights
// are >= 0, so the bits order as the values do), or all ones where it is protected; the
// kept tokens are the `budget` largest keys, ties to the lowest index.
//
// The threshold key is found by narrowing a key range [lo, hi]: each round counts the
// range's keys in up to 2048 equal bins (shared memory), finds the bin that holds the
// k-th largest and takes it as the next range.  The first range is the smallest and
// largest unprotected key, so the bins spread over the exponents that occur, and three
// rounds settle 32 bits.  Then one pass in index order numbers the freed places and the
// tokens to move by ballots and a scan of the waves' counts.
//
// Bound by reading mass and pos once: up to kPlanThreads * 32 tokens the keys stay in
// registers; longer caches read both again in each round (from the caches).
constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kBins = 2048;
constexpr uint32_t kProtected = 0xffffffffu;

struct PlanShared {
  uint32_t bins[kBins];
  uint32_t wave[2][kPlanWaves];
  uint32_t lo, hi, need, exact;
};

__device__ __forceinline__ uint32_t wave_add(uint32_t v) {
  for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

// exclusive sum of v over the workgroup's threads in thread order, total in *all
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *wave, uint32_t *all) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  uint32_t inc = v;
  for (int m = 1; m < 64; m <<= 1) {
    const uint32_t o = __shfl_up(inc, m);
    if (lane >= m) inc += o;
  }
  __syncthreads();  // the previous use of `wave` is over
  if (lane == 63) wave[w] = inc;
  __syncthreads();
  uint32_t before = 0, total = 0;
  for (int i = 0; i < kPlanWaves; ++i) {
    const uint32_t c = wave[i];
    before += i < w ? c : 0;
    total += c;
  }
  *all = total;
  return before + inc - v;
}

// R > 0: up to R * kPlanThreads tokens, keys in registers; R == 0: any number
template <int R>
__global__ __launch_bounds__(kPlanThreads) void kv_evict_plan_kernel(KvGeom g, EvictArgs a) {
  __shared__ PlanShared sh;
  const int unit = blockIdx.x;
  const int h = unit % g.kv_heads, lb = unit / g.kv_heads;
  const int b = lb % a.batch, layer = lb / a.batch;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int slot = a.slot_table[b], n = a.kv_len[b];
  const bool teller = layer == 0 && h == 0 && tid == 0;
  const bool bad_slot = slot <= 0 || slot >= g.slots;
  const bool bad_len = n < 0 || n > a.max_len;
  if (teller) {
    if (slot >= g.slots) set_err(g.err, GDN_ERRW_BAD_SLOT);
    else if (slot > 0 && bad_len) set_err(g.err, GDN_ERRW_BAD_SEQLENS);
    a.kv_len_out[b] = bad_slot || bad_len || n < a.budget ? n : a.budget;
  }
  if (bad_slot || bad_len || n <= a.budget) {
    if (tid == 0) a.n_moves[unit] = 0;
    return;
  }
  const int64_t base = ((int64_t(layer) * g.slots + slot) * g.kv_heads + h) * g.capacity;
  const float *mass = g.mass + base;
  const int32_t *pos = g.pos + base;
  // next_pos - recent may pass the 32-bit range
  const int64_t from = int64_t(a.next_pos[b]) - a.recent;
  const int rounds = R > 0 ? R : (n + kPlanThreads - 1) / kPlanThreads;

  auto load_key = [&](int i) -> uint32_t {
    const float m = mass[i];
    const int32_t p = pos[i];
    const uint32_t key = m > 0.f ? __float_as_uint(m) : 0u;
    return p < a.sink || int64_t(p) >= from ? kProtected : key;
  };
  uint32_t keys[R > 0 ? R : 1];
  if (R > 0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = r * kPlanThreads + tid;
      keys[r] = i < n ? load_key(i) : 0u;
    }
  }
  // f(index, key) for this thread's tokens
  auto each = [&](auto f) {
    if constexpr (R > 0) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int i = r * kPlanThreads + tid;
        if (i < n) f(i, keys[r]);
      }
    } else {
      for (int i = tid; i < n; i += kPlanThreads) f(i, load_key(i));
    }
  };

  // ---- range of the unprotected keys, count of the protected ------------------
  uint32_t kmin = kProtected, kmax = 0, prot = 0;
  each([&](int, uint32_t key) {
    if (key == kProtected) {
      ++prot;
    } else {
      kmin = min(kmin, key);
      kmax = max(kmax, key);
    }
  });
  for (int m = 32; m; m >>= 1) {
    kmin = min(kmin, __shfl_xor(kmin, m));
    kmax = max(kmax, __shfl_xor(kmax, m));
  }
  prot = wave_add(prot);
  if (tid == 0) {
    sh.lo = kProtected;
    sh.hi = 0;
    sh.need = 0;
  }
  __syncthreads();
  if (lane == 0) {
    atomicMin(&sh.lo, kmin);
    atomicMax(&sh.hi, kmax);
    atomicAdd(&sh.need, prot);
  }
  __syncthreads();
  uint32_t lo = sh.lo, hi = sh.hi;
  prot = sh.need;
  // keep every key above `lo` at the end, and the first `need` of those equal to it;
  // with `exact` every key >= lo
  uint32_t need;
  bool exact = false;
  if (prot >= uint32_t(a.budget)) {  // the protected alone fill the budget
    lo = hi = kProtected;
    need = a.budget;
  } else {
    need = a.budget - prot;
  }
  while (lo < hi && !exact) {  // ends: each round leaves at most 1/1024 of the range
    const uint32_t width = hi - lo;
    const int top = 32 - __clz(width);
    const int shift = top > 11 ? top - 11 : 0;
    __syncthreads();
    for (int i = tid; i < kBins; i += kPlanThreads) sh.bins[i] = 0;
    __syncthreads();
    each([&](int, uint32_t key) {
      if (key >= lo && key <= hi) atomicAdd(&sh.bins[(key - lo) >> shift], 1u);
    });
    __syncthreads();
    // thread t looks at bins 2047 - 2t and 2046 - 2t: sums from the top
    const int b1 = kBins - 1 - 2 * tid, b0 = b1 - 1;
    const uint32_t c1 = sh.bins[b1], c0 = sh.bins[b0];
    uint32_t all;
    const uint32_t above = block_scan(c1 + c0, sh.wave[0], &all);
    if (above < need && above + c1 + c0 >= need) {
      const bool second = above + c1 < need;
      const uint32_t bin = second ? b0 : b1, over = second ? above + c1 : above;
      const uint32_t in_bin = second ? c0 : c1;
      sh.lo = lo + (bin << shift);
      sh.hi = min(hi, sh.lo + ((1u << shift) - 1u));
      sh.need = need - over;
      sh.exact = need - over == in_bin;  // the whole bin is kept
    }
    __syncthreads();
    lo = sh.lo;
    hi = sh.hi;
    need = sh.need;
    exact = sh.exact != 0;
  }

  // ---- number the ties, then the freed places and the tokens to move ----------
  const int64_t list = int64_t(unit) * a.max_moves;
  uint32_t tie_base = 0, free_base = 0, move_base = 0;
  for (int r = 0; r < rounds; ++r) {
    const int i = r * kPlanThreads + tid;
    uint32_t key = 0;
    if constexpr (R > 0) {
#pragma unroll
      for (int q = 0; q < R; ++q) key = q == r ? keys[q] : key;
    } else {
      if (i < n) key = load_key(i);
    }
    const bool on = i < n;
    bool keep = on && (exact ? key >= lo : key > lo);
    uint32_t all;
    if (!exact) {
      const bool tie = on && key == lo;
      const uint32_t before = block_scan(tie ? 1u : 0u, sh.wave[0], &all);
      if (tie && tie_base + before < need) keep = true;
      tie_base += all;
    }
    const bool freed = on && !keep && i < a.budget;
    const bool moved = on && keep && i >= a.budget;
    const uint32_t before = block_scan((freed ? 1u : 0u) | (moved ? 0x10000u : 0u), sh.wave[1], &all);
    if (freed) a.moves[2 * (list + free_base + (before & 0xffffu)) + 1] = i;
    if (moved) a.moves[2 * (list + move_base + (before >> 16))] = i;
    free_base += all & 0xffffu;
    move_base += all >> 16;
  }
  if (tid == 0) a.n_moves[unit] = int(move_base);
}

// ---------------------------------------------------------- eviction moves --
// x: blocks of kMovesPerBlock entries of a list, y: (layer, request, head).  A row is
// spread over row_bytes / 16 lanes; a thread carries 16 bytes of the key and of the value
// of each of its entries.  Sources and destinations are disjoint, so there is no order.
constexpr int kMoveThreads = 256;
constexpr int kMovesPerBlock = 64;

__global__ __launch_bounds__(kMoveThreads) void kv_evict_apply_kernel(KvGeom g, int row_bytes, int units,
                                                                      EvictArgs a) {
  const int unit = blockIdx.x % units, block = blockIdx.x / units;
  const int h = unit % g.kv_heads, lb = unit / g.kv_heads;
  const int b = lb % a.batch, layer = lb / a.batch;
  const int count = a.n_moves[unit];
  const bool teller = block == 0 && threadIdx.x == 0;
  if (count < 0 || count > a.max_moves) {
    if (teller) set_err(g.err, GDN_ERRW_BAD_SEQLENS);
    return;
  }
  const int first = block * kMovesPerBlock;
  if (first >= count) return;
  const int slot = a.slot_table[b];
  if (slot <= 0 || slot >= g.slots) {
    if (teller && slot >= g.slots) set_err(g.err, GDN_ERRW_BAD_SLOT);
    return;
  }
  const int last = min(count, first + kMovesPerBlock);
  const int lanes = row_bytes >> 4;  // per row
  const int piece = threadIdx.x % lanes;
  char *const k = g.k + int64_t(layer) * g.layer_rows * row_bytes + 16 * piece;
  char *const v = g.v + int64_t(layer) * g.layer_rows * row_bytes + 16 * piece;
  const int64_t mrow = ((int64_t(layer) * g.slots + slot) * g.kv_heads + h) * g.capacity;
  for (int j = first + threadIdx.x / lanes; j < last; j += kMoveThreads / lanes) {
    const int64_t e = 2 * (int64_t(unit) * a.max_moves + j);
    const int src = a.moves[e], dst = a.moves[e + 1];
    if (src < 0 || src >= g.capacity || dst < 0 || dst >= g.capacity) {
      if (piece == 0) set_err(g.err, GDN_ERRW_BAD_SEQLENS);
      continue;
    }
    const int rs = kv_row(g, slot, h, src), rd = kv_row(g, slot, h, dst);
    if (rs < 0 || rd < 0) {
      if (piece == 0) set_err(g.err, GDN_ERRW_BAD_PAGE);
      continue;
    }
    const u32x4 kx = *reinterpret_cast<const u32x4 *>(k + int64_t(rs) * row_bytes);
    const u32x4 vx = *reinterpret_cast<const u32x4 *>(v + int64_t(rs) * row_bytes);
    *reinterpret_cast<u32x4 *>(k + int64_t(rd) * row_bytes) = kx;
    *reinterpret_cast<u32x4 *>(v + int64_t(rd) * row_bytes) = vx;
    if (piece == 0) {
      if (g.mass) g.mass[mrow + dst] = g.mass[mrow + src];
      if (g.pos) g.pos[mrow + dst] = g.pos[mrow + src];
    }
  }
}

}  // namespace

hipError_t launch_kv_append(const gdn_kv_pool *p, int layer, const AppendArgs &a, hipStream_t s) {
  const int64_t items = int64_t(a.n) * p->d.kv_heads * (p->d.head_dim >> 3);
  const dim3 grid(unsigned((items + kAppendThreads - 1) / kAppendThreads));
  const KvGeom g = kv_geom(p, layer);
  if (p->d.kv_dtype == GDN_BF16)
    hipLaunchKernelGGL((kv_append_kernel<false>), grid, dim3(kAppendThreads), 0, s, g, p->d.head_dim, a);
  else
    hipLaunchKernelGGL((kv_append_kernel<true>), grid, dim3(kAppendThreads), 0, s, g, p->d.head_dim, a);
  return hipGetLastError();
}

hipError_t launch_kv_evict_plan(const gdn_kv_pool *p, int layer, const EvictArgs &a, hipStream_t s) {
  const dim3 grid(unsigned(a.layers * a.batch * p->d.kv_heads)), block(kPlanThreads);
  const KvGeom g = kv_geom(p, layer);
  if (a.max_len <= 2 * kPlanThreads)
    hipLaunchKernelGGL((kv_evict_plan_kernel<2>), grid, block, 0, s, g, a);
  else if (a.max_len <= 8 * kPlanThreads)
    hipLaunchKernelGGL((kv_evict_plan_kernel<8>), grid, block, 0, s, g, a);
  else if (a.max_len <= 32 * kPlanThreads)
    hipLaunchKernelGGL((kv_evict_plan_kernel<32>), grid, block, 0, s, g, a);
  else
    hipLaunchKernelGGL((kv_evict_plan_kernel<0>), grid, block, 0, s, g, a);
  return hipGetLastError();
}

hipError_t launch_kv_evict_apply(const gdn_kv_pool *p, int layer, const EvictArgs &a, hipStream_t s) {
  const int units = a.layers * a.batch * p->d.kv_heads;
  const int64_t blocks = (a.max_moves + kMovesPerBlock - 1) / kMovesPerBlock;
  if (blocks * units >= (int64_t(1) << 31)) return hipErrorInvalidValue;
  hipLaunchKernelGGL(kv_evict_apply_kernel, dim3(unsigned(blocks * units)), dim3(kMoveThreads), 0, s,
                     kv_geom(p, layer), p->row_bytes, units, a);
  return hipGetLastError();
}

}  // namespace gdn
