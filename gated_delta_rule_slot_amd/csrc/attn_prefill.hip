// attn_prefill.hip -- attention of chunks of new tokens over a paged key-value cache
// (formulas: include/gdn_kv.h).
//
// The query heads of one key-value head read the same keys, so a request's rows of one
// key-value head are (new token, head of the group), token by token, and a workgroup takes
// kRows of them over tiles of KT places.  4 D flops for every (row, place): bound by the
// matrix units, or, for few rows, by the reading of the cache.
//
//   S^T = K Q^T   A = keys (rows = places), B = queries (columns = rows of the call).  A lane
//                 gets, for row c = lane % 32 and half h = lane / 32, the scores of places
//                 8 i + 4 h + j of 32 (i, j < 4).
//   O^T = V^T P^T takes P^T as B with exactly those places as the lane's eight k indices:
//                 16 s + 4 h + j and 16 s + 8 + 4 h + j.  A is read from rows of values by the
//                 transposing read of shared memory, in the same order.
// The row is the lane's column in both products, so the softmax's m and l are lane-local and
// only the maximum crosses the halves.  Queries stay in registers.  Keys and values go from
// memory to shared memory without passing registers (bf16; e4m3 is converted on its way), one
// tile ahead, with one barrier a tile.
//
// The exponent's reference m follows the running maximum only where that has grown by more
// than 2^8 (a wave's common decision), so O is rarely rescaled: weights are at most 2^8 then,
// and fp32 sums and bf16 weights lose nothing by that.  The weights are rounded to bf16 once for
// the product (their sum l is not): an error of at most 2^-8 of a weighted mean of |v|, about as
// large as the output's own rounding.  Two bf16 parts would take half as many matrix
// instructions again.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "kv.hpp"
#include "lanes.hpp"
#include "mfma.hpp"

namespace gdn {
namespace {

#ifndef GDN_NQ
#define GDN_NQ 1
#endif
constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kCUs = 256;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;
constexpr float kNegInf = -__builtin_inff();
constexpr float kGrowth = 8.f;  // log2 of how far the maximum may pass the reference

constexpr int kRows = 32 * kWaves;  // rows of a workgroup, for each block of its waves

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4t __attribute__((ext_vector_type(4)));
// (constant address space: these arrays do not change during the call, so wave-uniform reads
// are scalar loads)
typedef const int32_t __attribute__((address_space(4))) *table_t;

struct ChunkDev {
  ChunkArgs a;
  int group, tiles, parts;
  float c;          // |scale * k_scale| in log2 units
  uint32_t flip, keep;  // for two bf16 queries: the scale's sign, and 0 if it is 0 (c is 1 then)
  int rows;         // of a tile
  float *o, *ml;    // parts > 1: [tile][kv head][part][rows] rows of O, and of m and l
  float *lse;       // [tokens][q_heads], or NULL
};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ float ref(float m) { return m == kNegInf ? 0.f : m; }
// the larger / the sum of a value and its counterpart in the other half
__device__ __forceinline__ float halves_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float halves_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ f32x16 mfma32(const bf16x8 &a, const bf16x8 &b, const f32x16 &c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// ---- values that are not finite ---------------------------------------------
// 0 * NaN is NaN, so a row whose weight of a place is 0 because it does not see it would take that
// place's NaN or infinite values.  Where a workgroup's result is not finite, its tile is walked
// again with every such value as 0, which gives the finite part of the sums, then with 1 in the
// place of inf and NaN and 0 elsewhere, then with 1 in the place of -inf and NaN: a sum above 0
// says that the row sees one with a weight above 0.
enum { kAsIs, kFinite, kUp, kDown };
__device__ __forceinline__ u32x4 sorted(u32x4 x, int kind) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t r = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t v = (x[i] >> (16 * e)) & 0xffffu, a = v & 0x7fffu;
      const bool mark = a > 0x7f80u || v == (kind == kUp ? 0x7f80u : 0xff80u);
      r |= (kind == kFinite ? (a < 0x7f80u ? v : 0u) : mark ? 0x3f80u : 0u) << (16 * e);
    }
    x[i] = r;
  }
  return x;
}
// a sum with an infinite (or NaN) value added
__device__ __forceinline__ float beyond(float sum, int kind) { return sum + (kind == kUp ? -kNegInf : kNegInf); }

// ---- which rows a tile has -------------------------------------------------
// The tiles of request b begin at cu[b] * group / rows + b: at least as many as it needs, and
// found from cu alone, so that no list of tiles has to be made first.
struct Chunk {
  int b, bos, n, rows0;  // request, its first token and number of tokens, the tile's first row
  int slot, len, begin;
  bool any, live;        // whether the tile has rows, whether they see anything at all
};
__device__ __forceinline__ Chunk chunk_of(const KvGeom &g, const ChunkDev &p, int tile, bool tell) {
  const table_t cu = (table_t)p.a.cu_seqlens;
  auto first = [&](int b) { return int64_t(cu[b]) * p.group / p.rows + b; };
  int lo = 0, hi = p.a.batch;  // the last request whose tiles begin at `tile` or before
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first(mid) <= tile) lo = mid;
    else hi = mid;
  }
  Chunk r;
  r.b = lo;
  r.bos = cu[lo];
  const int eos = cu[lo + 1];
  const int64_t at = (tile - first(lo)) * p.rows;
  const bool ok = r.bos >= 0 && eos >= r.bos && eos <= p.a.tokens;
  r.n = ok ? eos - r.bos : 0;
  r.any = ok && at >= 0 && at < int64_t(r.n) * p.group;
  r.rows0 = r.any ? int(at) : 0;
  r.slot = ((table_t)p.a.slot_table)[lo];
  r.len = ((table_t)p.a.kv_len)[lo];
  r.begin = p.a.kv_begin ? ((table_t)p.a.kv_begin)[lo] : 0;
  const bool lens = r.len >= r.n && r.len <= p.a.max_len && r.begin >= 0;
  r.live = r.any && r.slot > 0 && r.slot < g.slots && lens;
  if (tell) {
    if (!ok) set_err(g.err, GDN_ERRW_BAD_SEQLENS);
    else if (r.any && r.slot >= g.slots) set_err(g.err, GDN_ERRW_BAD_SLOT);
    else if (r.any && r.slot > 0 && !lens) set_err(g.err, GDN_ERRW_BAD_SEQLENS);
  }
  return r;
}
// first place that the query at `place` sees
__device__ __forceinline__ int seen_from(const ChunkDev &p, int begin, int place) {
  return p.a.window ? max(begin, place - p.a.window + 1) : begin;
}

// ---- shared memory ---------------------------------------------------------
// A tile has KT rows of D bf16 values; 16-byte piece c of row r lies at piece c ^ twist(r).
// Keys are read 32 rows at the same piece, values 4 rows of 64 adjacent bytes: both meet every
// bank equally often.
template <int D>
__device__ __forceinline__ int twist(int r) {
  return D == 64 ? (((r >> 1) & 1) << 2 | ((r >> 2) & 3)) : ((r & 3) << 2 | ((r >> 2) & 3));
}

template <int D, bool kF8>
struct Tile {
  static constexpr int KT = D == 256 ? 32 : 64;  // places
  static constexpr int RB = 2 * D;               // bytes of a row in shared memory
  static constexpr int SB = kF8 ? D : RB;        // and in the cache
  static constexpr int kBytes = KT * RB;
  static constexpr int kLanes = SB / 16;         // lanes that load a row
  static constexpr int kLoadRows = 64 / kLanes;  // rows of a wave's load
  static constexpr int kLoads = KT / (kWaves * kLoadRows);
  static constexpr int kShared = 4 * kBytes + 16;
};

// kWide: pages hold 16 tokens or more, so that the rows of a wave's load lie in one page.
// NQ: blocks of 32 rows of a wave.
template <int D, bool kF8, bool kWide, int NQ>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(NQ == 1 ? 2 : 1)))
void attn_prefill_kernel(KvGeom g, ChunkDev p) {
  using T = Tile<D, kF8>;
  constexpr int KT = T::KT, KB = KT / 32, KS = D / 16, DB = D / 32, NL = T::kLoads, ROWS = kRows * NQ;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  // a tile (by its number's parity) that has a page outside the pool
  int *const sbad = reinterpret_cast<int *>(lds + 4 * T::kBytes);

  const int lane = threadIdx.x & 63, c = lane & 31, half = lane >> 5;
  const int wave = uniform(threadIdx.x >> 6);
  const int64_t item = flat_block();
  const int h = int(item % g.kv_heads);
  const int64_t rest = item / g.kv_heads;
  const int part = int(rest % p.parts);
  const int tile = p.tiles - 1 - int(rest / p.parts);  // the last tiles see the most places
  if (tile < 0) return;
  const Chunk ch = chunk_of(g, p, tile, h == 0 && part == 0 && threadIdx.x == 0);
  if (!ch.any) return;

  const int G = p.group, all = ch.n * G;
  const int row0 = ch.rows0 + 32 * NQ * wave;
  const bool wlive = ch.live && row0 < all;
  const int place0 = ch.len - ch.n;  // of the first new token
  int place[NQ], from[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    // (rows behind the last repeat it and are not stored)
    place[n] = place0 + min(row0 + 32 * n + c, all - 1) / G;
    from[n] = seen_from(p, ch.begin, place[n]);
  }
  const int wfirst = place0 + min(row0, all - 1) / G, wlast = place0 + min(row0 + 32 * NQ - 1, all - 1) / G;
  const int wfrom = seen_from(p, ch.begin, wfirst), wfrom_last = seen_from(p, ch.begin, wlast);

  // tiles of the workgroup: what its rows see, and this part of it
  int t0 = 0, t1 = 0;
  if (ch.live) {
    const int gfirst = place0 + ch.rows0 / G, glast = place0 + min(ch.rows0 + ROWS - 1, all - 1) / G;
    const int lo = seen_from(p, ch.begin, gfirst) / KT, hi = glast / KT + 1;
    const int per = (max(hi - lo, 0) + p.parts - 1) / p.parts;
    t0 = lo + part * per;
    t1 = min(hi, t0 + per);
  }

  bf16x8 q[NQ][KS];
  if (wlive && t0 < t1) {
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int row = min(row0 + 32 * n + c, all - 1), token = row / G, head = h * G + (row - token * G);
      const uint16_t *src = p.a.q + (ch.bos + token) * p.a.q_stride + int64_t(head) * D + 8 * half;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        u32x4 w = *reinterpret_cast<const u32x4 *>(src + 16 * s);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = (w[i] ^ p.flip) & p.keep;
        q[n][s] = __builtin_bit_cast(bf16x8, w);
      }
    }
  }

  // ---- loads ----
  const int lrow = lane / T::kLanes, lpiece = lane % T::kLanes;
  auto load_row = [&](int j) { return (j * kWaves + wave) * T::kLoadRows; };  // first row of load j
  const table_t table = (table_t)(g.page_table + int64_t(max(ch.slot, 0)) * g.max_pages);
  const int page_mask = (1 << g.page_shift) - 1;
  const int loff = (kWide ? lrow * T::RB : 0) + ((lpiece ^ twist<D>(wave * T::kLoadRows + lrow)) << 4);
  int ids[kWide ? NL : 1];
  auto load_ids = [&](int t) {
    if constexpr (kWide) {
#pragma unroll
      for (int j = 0; j < NL; ++j) ids[j] = table[min(t * KT + load_row(j), ch.len - 1) >> g.page_shift];
    }
  };
  uint32_t hidden;       // loads (bits j) of the tile to come whose lane's row is no place of the request
  bool clear;            // whether any of the wave has one
  int64_t src[NL];       // byte offsets of the tile to come in the layer's keys and values
  auto locate = [&](int t) {
    hidden = 0;
    bool bad = false;
#pragma unroll
    for (int j = 0; j < NL; ++j) {
      const int first = t * KT + load_row(j), at = first + lrow;
      int id;
      if constexpr (kWide) id = ids[j];
      else id = g.page_table[int64_t(ch.slot) * g.max_pages + (min(at, ch.len - 1) >> g.page_shift)];
      const bool wrong = id <= 0 || id >= g.pages;
      id = wrong ? 0 : id;
      bad = bad || wrong;
      hidden |= (wrong || at >= ch.len || at < ch.begin) ? 1u << j : 0u;
      if constexpr (kWide)
        src[j] = (int64_t((id * g.kv_heads + h) << g.page_shift) + (first & page_mask)) * T::SB;
      else
        src[j] = (int64_t((id * g.kv_heads + h) << g.page_shift) + (at & page_mask)) * T::SB;
    }
    if (__any(bad)) {
      if (lane == 0) {
        sbad[t & 1] = t;
        set_err(g.err, GDN_ERRW_BAD_PAGE);
      }
    }
    clear = __any(hidden != 0);
  };
  // bf16: from memory to shared memory; a lane's 16 bytes land at its place in the wave's 1 KB,
  // so it asks for the piece that belongs there
  auto ask = [&](int t) {
    if constexpr (!kF8) {
      char *to = lds + (t & 1) * 2 * T::kBytes;
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        // (the twist of the rows of load j differs from load 0's in one bit at most)
        constexpr int kStep = kWaves * T::kLoadRows;
        static_assert(kStep % 16 == 0 || kStep == 8, "twist");
        const uint32_t off = uint32_t(loff) ^ (kStep == 8 ? (j & 1) * 32 : 0);
        char *dst = to + load_row(j) * T::RB;
        typedef __attribute__((address_space(1))) const void *gp;
        typedef __attribute__((address_space(3))) void *lp;
        __builtin_amdgcn_global_load_lds((gp)(g.k + src[j] + off), (lp)dst, 16, 0, 0);
        __builtin_amdgcn_global_load_lds((gp)(g.v + src[j] + off), (lp)(dst + T::kBytes), 16, 0, 0);
      }
    }
  };
  // rows that are no places of the request hold anything: zeros keep 0 * NaN out of the product
  auto clear_rows = [&](int t) {
    if constexpr (!kF8) {
      char *to = lds + (t & 1) * 2 * T::kBytes + T::kBytes;
#pragma unroll
      for (int j = 0; j < NL; ++j)
        if (hidden >> j & 1) *reinterpret_cast<u32x4 *>(to + load_row(j) * T::RB + lane * 16) = u32x4{0, 0, 0, 0};
    }
  };
  // the wave's values of the tile replaced as the walk asks for
  auto sort_rows = [&](int t, int kind) {
    if constexpr (!kF8) {
      char *to = lds + (t & 1) * 2 * T::kBytes + T::kBytes;
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        u32x4 *at = reinterpret_cast<u32x4 *>(to + load_row(j) * T::RB + lane * 16);
        *at = sorted(*at, kind);
      }
    }
  };
  // e4m3: through registers, 16 values a lane
  u32x4 kraw[kF8 ? NL : 1], vraw[kF8 ? NL : 1];
  auto fetch = [&](u32x4 *raw, const char *base) {
    if constexpr (kF8) {
#pragma unroll
      for (int j = 0; j < NL; ++j)
        raw[j] = *reinterpret_cast<const u32x4 *>(base + src[j] + (kWide ? lrow * T::SB : 0) + 16 * lpiece);
    }
  };
  auto put = [&](const u32x4 *raw, char *to, bool zero, int kind) {
    if constexpr (kF8) {
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        const int r = load_row(j) + lrow;
        u32x4 x = raw[j];
        if (zero && (hidden >> j & 1)) x = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          u32x4 w;
          uint32_t a, b;
          f8_to_bf16(x[2 * e], &a, &b);
          w[0] = a; w[1] = b;
          f8_to_bf16(x[2 * e + 1], &a, &b);
          w[2] = a; w[3] = b;
          if (kind != kAsIs) w = sorted(w, kind);
          *reinterpret_cast<u32x4 *>(to + r * T::RB + (((2 * lpiece + e) ^ twist<D>(r)) << 4)) = w;
        }
      }
    }
  };

  // ---- the walk ----
  // keys: row c of a block of 32, piece half of step 0; step s is 2 s further, which the twist
  // turns into an exclusive or.  Values: row vrow of the half's four, 4 adjacent values of the
  // block of 32 columns
  const int vrow = 4 * half + ((lane >> 2) & 3), vpair = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
  const int kaddr = c * T::RB + ((half ^ twist<D>(c)) << 4);
  const int vaddr = vrow * T::RB + ((vpair ^ twist<D>(vrow)) << 4) + 8 * (lane & 1);
  constexpr int kAhead = 4;

  f32x16 o[NQ][DB];
  float m[NQ], l[NQ];
  auto walk = [&](int kind) {
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
#pragma unroll
      for (int b = 0; b < DB; ++b) o[n][b] = f32x16{};
      m[n] = kNegInf;
      l[n] = 0.f;
    }
    if (threadIdx.x < 2) sbad[threadIdx.x] = -1;
    __syncthreads();
    if (t0 >= t1) return;
    load_ids(t0);
    locate(t0);
    ask(t0);
    if constexpr (kF8) {
      char *to = lds + (t0 & 1) * 2 * T::kBytes;
      fetch(kraw, g.k);
      fetch(vraw, g.v);
      put(kraw, to, false, kAsIs);
      put(vraw, to + T::kBytes, clear, kind);
    }
    load_ids(t0 + 1);
    // tile t is there, and the next one on its way
    auto stage = [&](int t) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      if (!kF8 && clear) clear_rows(t);
      if (!kF8 && kind != kAsIs) sort_rows(t, kind);
      __syncthreads();
      const bool more = t + 1 < t1;
      if (more) {
        locate(t + 1);
        ask(t + 1);
        if constexpr (kF8) {
          fetch(kraw, g.k);
          fetch(vraw, g.v);
        }
        load_ids(t + 2);
      }
    };
    auto finish = [&](int t) {
      if (kF8 && t + 1 < t1) {
        char *to = lds + ((t + 1) & 1) * 2 * T::kBytes;
        put(kraw, to, false, kAsIs);
        put(vraw, to + T::kBytes, clear, kind);
      }
    };
    auto skip = [&](int a, int b) {
#pragma unroll 1
      for (int t = a; t < b; ++t) {
        stage(t);
        finish(t);
      }
    };
    // the tiles that the wave's rows see
    const int w0 = wlive ? min(t1, max(t0, wfrom / KT)) : t1, w1 = wlive ? max(w0, min(t1, wlast / KT + 1)) : t1;
    skip(t0, w0);
#pragma unroll 1
    for (int t = w0; t < w1; ++t) {
      stage(t);
            const int p0 = t * KT;
      {
        f32x16 s[NQ][KB];
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int kb = 0; kb < KB; ++kb) s[n][kb] = f32x16{};
        int ka = kaddr + (t & 1) * 2 * T::kBytes, va = vaddr + (t & 1) * 2 * T::kBytes + T::kBytes;
        asm volatile("" : "+v"(ka), "+v"(va));  // (addresses are worked out here, not kept over the walk)
        auto kread = [&](int i) {
          return *reinterpret_cast<const bf16x8 *>(lds + (ka ^ (32 * (i / KB))) + 32 * (i % KB) * T::RB);
        };
        auto vread = [&](int i) {
          s16x4t v[2];
#pragma unroll
          for (int e = 0; e < 2; ++e)
            v[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4t *)(
                lds + (va ^ (64 * (i % DB) + 32 * e)) + (16 * (i / DB) + 8 * e) * T::RB));
          return __builtin_bit_cast(bf16x8, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
        };
        bf16x8 ring[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) ring[i] = kread(i);
#pragma unroll
        for (int i = 0; i < KS * KB; ++i) {
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int n = 0; n < NQ; ++n) s[n][i % KB] = mfma32(ring[i % kAhead], q[n][i / KB], s[n][i % KB]);
          if (i + kAhead < KS * KB) ring[i % kAhead] = kread(i + kAhead);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) ring[i] = vread(i);
        __builtin_amdgcn_sched_barrier(0);
        const bool flagged = sbad[t & 1] == t;
        const bool partial = p0 < wfrom_last || p0 + KT - 1 > wfirst || flagged;
        if (partial) {
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const int at = p0 + 32 * kb + 8 * (e >> 2) + 4 * half + (e & 3);
                if (at > place[n] || at < from[n]) s[n][kb][e] = kNegInf;
              }
          if (flagged) {
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const int at = p0 + 32 * kb + 8 * (e >> 2) + 4 * half + (e & 3);
                const int id = g.page_table[int64_t(ch.slot) * g.max_pages + (min(at, ch.len - 1) >> g.page_shift)];
                if (id <= 0 || id >= g.pages)
#pragma unroll
                  for (int n = 0; n < NQ; ++n) s[n][kb][e] = kNegInf;
              }
          }
        }
        float mr[NQ];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          float top = s[n][0][0];
#pragma unroll
          for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int e = 0; e < 16; ++e) top = fmaxf(top, s[n][kb][e]);
          top = halves_max(top) * p.c;
          if (__any(top > m[n] + kGrowth)) {
            const float to = fmaxf(m[n], top), f = fexp2(m[n] - ref(to));
            l[n] *= f;
#pragma unroll
            for (int b = 0; b < DB; ++b)
#pragma unroll
              for (int e = 0; e < 16; ++e) o[n][b][e] *= f;
            m[n] = to;
          }
          mr[n] = ref(m[n]);
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              s[n][kb][e] = fexp2(fmaf(s[n][kb][e], p.c, -mr[n]));
              sum[e & 3] += s[n][kb][e];
            }
          l[n] += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        }
#pragma unroll
          for (int ks = 0; ks < 2 * KB; ++ks) {
            bf16x8 pf[NQ];
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
              u32x4 w;
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[i] = cvt_pk_bf16(s[n][ks >> 1][8 * (ks & 1) + 2 * i], s[n][ks >> 1][8 * (ks & 1) + 2 * i + 1]);
              pf[n] = __builtin_bit_cast(bf16x8, w);
            }
#pragma unroll
            for (int b = 0; b < DB; ++b) {
              constexpr int all_v = 2 * KB * DB;
              const int i = ks * DB + b;
              __builtin_amdgcn_sched_barrier(0);
#pragma unroll
              for (int n = 0; n < NQ; ++n) o[n][b] = mfma32(ring[i % kAhead], pf[n], o[n][b]);
              if (i + kAhead < all_v) ring[i % kAhead] = vread(i + kAhead);
            }
          }
      }
      finish(t);
    }
    skip(w1, t1);
  };
  // ---- results ----
  // (arguments and rows are read and worked out anew: they would take registers over the walk)
  auto store = [&](int kind) {
    const char __attribute__((address_space(4))) *args =
        (const char __attribute__((address_space(4))) *)__builtin_amdgcn_kernarg_segment_ptr();
    int first = row0 + c;
    asm volatile("" : "+s"(args), "+v"(first));
    static_assert(sizeof(KvGeom) % alignof(ChunkDev) == 0 && alignof(ChunkDev) == 8, "kernel arguments");
    const auto &p = *(const ChunkDev __attribute__((address_space(4))) *)(args + sizeof(KvGeom));
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const float ln = halves_sum(l[n]);
      const int row = first + 32 * n, mine = row - ch.rows0;  // row of the request, of the tile
      if (row < all) {
        if (p.parts > 1) {
          const int64_t at = (((int64_t(tile) * g.kv_heads + h) * p.parts + part) * ROWS) + mine;
          if (half == 0 && kind <= kFinite) {
            p.ml[2 * at] = ln == 0.f ? kNegInf : m[n];
            p.ml[2 * at + 1] = ln;
          }
          float *to = p.o + at * D + 4 * half;
          if (ln != 0.f)
#pragma unroll
            for (int b = 0; b < DB; ++b)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                f32x4 v = {o[n][b][4 * i], o[n][b][4 * i + 1], o[n][b][4 * i + 2], o[n][b][4 * i + 3]};
                if (kind > kFinite) {
                  const f32x4 old = ld4(to + 32 * b + 8 * i);
#pragma unroll
                  for (int e = 0; e < 4; ++e) v[e] = v[e] > 0.f ? beyond(old[e], kind) : old[e];
                }
                st4(to + 32 * b + 8 * i, v);
              }
          continue;
        }
        const int token = row / p.group;
        const int64_t orow = int64_t(ch.bos + token) * p.a.q_heads + h * p.group + (row - token * p.group);
        if (p.lse && half == 0 && kind <= kFinite)
          p.lse[orow] = ln == 0.f ? kNegInf : (m[n] + __builtin_amdgcn_logf(ln)) * kLn2;
        const float f = ln == 0.f ? 0.f : g.v_scale / ln;
        uint16_t *to = p.a.out + orow * D + 8 * half;
#pragma unroll
        for (int b = 0; b < DB; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            // columns 16 i + 8 h + 0..3 and + 4..7 of the block: the halves swap what the other stores
            u32x4 w;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t x = cvt_pk_bf16(o[n][b][8 * i + 2 * e] * f, o[n][b][8 * i + 2 * e + 1] * f);
              const uint32_t y = cvt_pk_bf16(o[n][b][8 * i + 4 + 2 * e] * f, o[n][b][8 * i + 5 + 2 * e] * f);
              const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
              w[e] = r[0];
              w[2 + e] = r[1];
            }
            u32x4 *at = reinterpret_cast<u32x4 *>(to + 32 * b + 16 * i);
            if (kind > kFinite) {
              const u32x4 old = *at;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float lo = __uint_as_float(w[e] << 16), hi = __uint_as_float(w[e] & 0xffff0000u);
                const float a = __uint_as_float(old[e] << 16), b = __uint_as_float(old[e] & 0xffff0000u);
                w[e] = pack_bf16x2(lo > 0.f ? beyond(a, kind) : a, hi > 0.f ? beyond(b, kind) : b);
              }
            }
            *at = w;
          }
      }
    }
  };

#pragma unroll 1
  for (int kind = kAsIs;;) {
    walk(kind);
    if (kind == kAsIs) {
      // a NaN may come from a value that the row does not see (0 * NaN)
      float bad = 0.f;
      if (wlive) {
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int b = 0; b < DB; ++b)
#pragma unroll
            for (int e = 0; e < 16; ++e) bad = fmaf(o[n][b][e], 0.f, bad);
      }
      if (__syncthreads_or(bad != 0.f)) {
        kind = kFinite;
        continue;
      }
    }
    store(kind);
    if (kind == kAsIs || kind == kDown) break;
    ++kind;
  }
}

// Rows whose places were divided: the parts' O, m and l joined.  One workgroup per tile and
// key-value head, a wave per row.
template <int D>
__global__ __launch_bounds__(kThreads) void attn_prefill_join_kernel(KvGeom g, ChunkDev p) {
  const int64_t item = flat_block();
  const int h = int(item % g.kv_heads), tile = int(item / g.kv_heads);
  if (tile >= p.tiles) return;
  const Chunk ch = chunk_of(g, p, tile, false);
  if (!ch.any) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int rows = min(p.rows, ch.n * p.group - ch.rows0);
  constexpr int N = D / 64;  // columns of a lane
  for (int i = wave; i < rows; i += kWaves) {
    const int64_t at = (int64_t(tile) * g.kv_heads + h) * p.parts * p.rows + i;
    float m = kNegInf;
    for (int part = 0; part < p.parts; ++part) m = fmaxf(m, p.ml[2 * (at + int64_t(part) * p.rows)]);
    float l = 0.f, o[N];
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = 0.f;
    for (int part = 0; part < p.parts; ++part) {
      const int64_t r = at + int64_t(part) * p.rows;
      const float pm = p.ml[2 * r], pl = p.ml[2 * r + 1];
      if (pl == 0.f) continue;
      const float f = fexp2(pm - m);
      l = fmaf(pl, f, l);
      const float *src = p.o + r * D + lane * N;
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = fmaf(src[e], f, o[e]);
    }
    const int row = ch.rows0 + i, token = row / p.group, head = h * p.group + (row - token * p.group);
    const int64_t orow = int64_t(ch.bos + token) * p.a.q_heads + head;
    if (p.lse && lane == 0) p.lse[orow] = l == 0.f ? kNegInf : (m + __builtin_amdgcn_logf(l)) * kLn2;
    const float f = l == 0.f ? 0.f : g.v_scale / l;
    uint16_t *to = p.a.out + orow * D + lane * N;
    if constexpr (N == 1) {
      to[0] = f32_to_bf16(o[0] * f);
    } else {
#pragma unroll
      for (int e = 0; e < N / 2; ++e) reinterpret_cast<uint32_t *>(to)[e] = cvt_pk_bf16(o[2 * e] * f, o[2 * e + 1] * f);
    }
  }
}

// ---- the last queries' weights, added to mass -------------------------------
// One workgroup per request, key-value head and 4 * KP places; a wave keeps the keys of its KP
// places in registers and walks the rows of the last queries 32 at a time, so every entry of
// mass has one owner and one order of summation.  A weight is exp(s - lse).
template <int D>
struct MassTile {
  static constexpr int KP = D == 256 ? 32 : 64;
  static constexpr int kPlaces = KP * kWaves;
};
template <int D, bool kF8>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2)))
void attn_prefill_mass_kernel(KvGeom g, ChunkDev p, int blocks) {
  constexpr int KP = MassTile<D>::KP, KB = KP / 32, KS = D / 16;
  const int64_t item = flat_block();
  const int h = int(item % g.kv_heads);
  const int64_t rest = item / g.kv_heads;
  const int b = int(rest / blocks);
  if (b >= p.a.batch) return;
  const table_t cu = (table_t)p.a.cu_seqlens;
  const int bos = cu[b], eos = cu[b + 1], slot = ((table_t)p.a.slot_table)[b], len = ((table_t)p.a.kv_len)[b];
  const int begin = p.a.kv_begin ? ((table_t)p.a.kv_begin)[b] : 0;
  const int n = eos - bos;
  if (bos < 0 || n <= 0 || eos > p.a.tokens || slot <= 0 || slot >= g.slots || len < n || len > p.a.max_len || begin < 0)
    return;
  const int late = min(n, p.a.mass_tokens);   // queries that count
  const int place0 = len - n, first = n - late;
  const int lane = threadIdx.x & 63, c = lane & 31, half = lane >> 5;
  const int wave = uniform(threadIdx.x >> 6);
  const int lowest = seen_from(p, begin, place0 + first) / MassTile<D>::kPlaces * MassTile<D>::kPlaces;
  const int p0 = lowest + int(rest % blocks) * MassTile<D>::kPlaces + wave * KP;
  if (p0 >= len) return;
  const int G = p.group;

  // a place's key: row c of block kb
  bf16x8 k[KB][KS];
  uint32_t there = 0;  // bits kb: the place is one of the request
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    const int at = p0 + 32 * kb + c, in = min(at, len - 1);
    const int row = kv_row(g, slot, h, in);
    there |= (at < len && at >= begin && row >= 0) ? 1u << kb : 0u;
    const char *src = g.k + int64_t(max(row, 0)) * (kF8 ? D : 2 * D);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      if constexpr (kF8) {
        const u32x2 x = *reinterpret_cast<const u32x2 *>(src + 16 * s + 8 * half);
        u32x4 w;
        uint32_t lo, hi;
        f8_to_bf16(x[0], &lo, &hi);
        w[0] = lo; w[1] = hi;
        f8_to_bf16(x[1], &lo, &hi);
        w[2] = lo; w[3] = hi;
        k[kb][s] = __builtin_bit_cast(bf16x8, w);
      } else {
        k[kb][s] = *reinterpret_cast<const bf16x8 *>(src + 32 * s + 16 * half);
      }
    }
  }

  f32x16 sum[KB];
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) sum[kb] = f32x16{};
  const int all = n * G;
  // the first row that sees the wave's first place, and the last that sees its last
  int r0 = max(first, p0 - place0) * G;
  int r1 = all;
  if (p.a.window) r1 = int(min(int64_t(all), max(int64_t(0), int64_t(p0) + KP - 1 + p.a.window - place0) * G));
#pragma unroll 1
  for (int r = r0; r < r1; r += 32) {
    const int row = min(r + c, all - 1), token = row / G, head = h * G + (row - token * G);
    const int place = place0 + token, from = seen_from(p, begin, place);
    const int64_t qrow = int64_t(bos + token);
    const uint16_t *src = p.a.q + qrow * p.a.q_stride + int64_t(head) * D + 8 * half;
    const float lse = p.lse[qrow * p.a.q_heads + head];
    f32x16 s[KB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) s[kb] = f32x16{};
#pragma unroll
    for (int st = 0; st < KS; ++st) {
      u32x4 w = *reinterpret_cast<const u32x4 *>(src + 16 * st);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = (w[i] ^ p.flip) & p.keep;
      const bf16x8 q = __builtin_bit_cast(bf16x8, w);
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) s[kb] = mfma32(k[kb][st], q, s[kb]);
    }
    const bool mine = r + c < r1 && lse != kNegInf;
    const float shift = lse * kLog2e;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int at = p0 + 32 * kb + 8 * (e >> 2) + 4 * half + (e & 3);
        const float w = fexp2(fmaf(s[kb][e], p.c, -shift));
        sum[kb][e] += mine && at <= place && at >= from ? w : 0.f;
      }
  }
  // over the 32 rows
  float *mass = g.mass + (int64_t(slot) * g.kv_heads + h) * g.capacity;
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    const uint64_t on = __ballot(there >> kb & 1);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float v = group_sum<32>(sum[kb][e]);
      const int i = 8 * (e >> 2) + 4 * half + (e & 3), at = p0 + 32 * kb + i;
      if (c == 0 && (on >> i & 1)) mass[at] += v;
    }
  }
}

size_t pad256(size_t n) { return (n + 255) & ~size_t(255); }

int64_t chunk_tiles(int batch, int tokens, int group, int rows) { return int64_t(tokens) * group / rows + batch; }
int chunk_rows() { return kRows * GDN_NQ; }

// Parts that a tile's places are divided into: workgroups for two on every compute unit, of 512
// places or more each (by the bound max_len).
int chunk_parts(const gdn_kv_pool *p, int64_t tiles, int max_len) {
  const int64_t groups = std::max<int64_t>(1, tiles * p->d.kv_heads);
  const int64_t want = (2 * kCUs + groups - 1) / groups;
  return int(std::max<int64_t>(1, std::min<int64_t>(want, max_len / 512)));
}

// Parts of the workspace, in order.
struct ChunkSpace {
  size_t o, ml, lse;
};
ChunkSpace chunk_space(const gdn_kv_pool *p, int batch, int tokens, int q_heads, int max_len, int mass_tokens) {
  ChunkSpace r{};
  const int64_t tiles = chunk_tiles(batch, tokens, q_heads / p->d.kv_heads, chunk_rows());
  const int parts = chunk_parts(p, tiles, max_len);
  if (parts > 1) {
    const size_t rows = size_t(tiles) * p->d.kv_heads * parts * chunk_rows();
    r.o = pad256(rows * p->d.head_dim * 4);
    r.ml = pad256(rows * 8);
  }
  if (mass_tokens > 0) r.lse = pad256(size_t(tokens) * q_heads * 4);
  return r;
}

template <int D, bool kF8>
hipError_t launch_dt(const KvGeom &g, const ChunkDev &p, hipStream_t s) {
  const bool wide = (1 << g.page_shift) >= 16;
  const int64_t units = int64_t(p.tiles) * g.kv_heads;
  const auto kernel = wide ? attn_prefill_kernel<D, kF8, true, GDN_NQ> : attn_prefill_kernel<D, kF8, false, GDN_NQ>;
  constexpr int shared = Tile<D, kF8>::kShared;
  hipLaunchKernelGGL(kernel, flat_grid(units * p.parts), dim3(kThreads), shared, s, g, p);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && p.parts > 1) {
    hipLaunchKernelGGL((attn_prefill_join_kernel<D>), flat_grid(units), dim3(kThreads), 0, s, g, p);
    e = hipGetLastError();
  }
  if (e == hipSuccess && p.a.mass_tokens > 0) {
    // the first block begins at or before the first place seen
    const int blocks = p.a.max_len / MassTile<D>::kPlaces + 1;
    hipLaunchKernelGGL((attn_prefill_mass_kernel<D, kF8>), flat_grid(int64_t(p.a.batch) * g.kv_heads * blocks),
                       dim3(kThreads), 0, s, g, p, blocks);
    e = hipGetLastError();
  }
  return e;
}

template <int D>
hipError_t launch_d(const KvGeom &g, const ChunkDev &p, bool f8, hipStream_t s) {
  return f8 ? launch_dt<D, true>(g, p, s) : launch_dt<D, false>(g, p, s);
}

}  // namespace

bool chunk_fits(const gdn_kv_pool *p, int batch, int tokens, int q_heads, int max_len) {
  const int64_t group = q_heads / p->d.kv_heads, limit = int64_t(1) << 31;
  const int64_t blocks = int64_t(max_len) / MassTile<256>::kPlaces + 1;
  // rows of a request and tiles are counted in 31 bits, workgroups in 40
  return int64_t(tokens) * group < limit - kRows && chunk_tiles(batch, tokens, int(group), kRows) < limit / p->d.kv_heads &&
         int64_t(batch) * p->d.kv_heads < (int64_t(1) << 40) / blocks;
}

size_t chunk_workspace(const gdn_kv_pool *p, int batch, int tokens, int q_heads, int max_len, int mass_tokens) {
  const ChunkSpace w = chunk_space(p, batch, tokens, q_heads, max_len, mass_tokens);
  return w.o + w.ml + w.lse;
}

hipError_t launch_attn_prefill(const gdn_kv_pool *pool, int layer, const ChunkArgs &a, hipStream_t s) {
  const KvGeom g = kv_geom(pool, layer);
  ChunkDev p{};
  p.a = a;
  p.group = a.q_heads / pool->d.kv_heads;
  p.rows = chunk_rows();
  p.tiles = int(chunk_tiles(a.batch, a.tokens, p.group, p.rows));
  p.parts = chunk_parts(pool, p.tiles, a.max_len);
  p.c = fabsf(a.scale) * pool->d.k_scale * kLog2e;
  p.flip = std::signbit(a.scale) ? 0x80008000u : 0u;
  p.keep = p.c == 0.f ? 0u : ~0u;  // (a score of -inf must stay -inf where it is multiplied by c)
  p.c = p.c == 0.f ? 1.f : p.c;
  const ChunkSpace w = chunk_space(pool, a.batch, a.tokens, a.q_heads, a.max_len, a.mass_tokens);
  char *at = static_cast<char *>(a.workspace);
  p.o = reinterpret_cast<float *>(at);
  p.ml = reinterpret_cast<float *>(at + w.o);
  p.lse = a.lse ? a.lse : a.mass_tokens > 0 ? reinterpret_cast<float *>(at + w.o + w.ml) : nullptr;
  const bool f8 = pool->d.kv_dtype == GDN_F8_E4M3;
  switch (pool->d.head_dim) {
    case 64: return launch_d<64>(g, p, f8, s);
    case 128: return launch_d<128>(g, p, f8, s);
    case 256: return launch_d<256>(g, p, f8, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace gdn
