// attn_prefill.hip -- attention of chunks of new tokens over a paged key-value cache
// (formulas: include/gdn_kv.h).
//
// The query heads of one key-value head read the same keys, so a request's rows of one
// key-value head are (new token, head of the group), token by token.  A tile has 128 of them, 32 of
// each wave of a workgroup, or twice as many, and walks over blocks of KT places.  4 D flops for every
// (row, place): bound by the matrix units, or, for few rows, by the reading of the cache.
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
// block ahead, with one barrier a block; their loads are issued between the products, and a wave in
// its products goes before one in its softmax.
//
// Two workgroups run on a compute unit (256 registers a lane, 64 KB; three with heads of 64), one in its
// products while the other is in its softmax: heads of 256 need O, the queries and 32 scores a row at once, which is why
// KT is 32 there.  A spilled register that is read again in the walk waits for all loads that were
// asked for after it, so what the walk does not need is worked out again behind it.
//
// The exponent's reference m is the maximum of some blocks before and stays as long as a lane's
// weights of a block sum to 2^8 at most (a wave's common decision): fp32 sums and bf16 weights lose
// nothing by that, and in most blocks neither is the maximum looked for nor O rescaled.  Where the sum is
// larger the block's scores are worked out again and m follows.  (Looking for the maximum in every
// block: 4.63 instead of 4.42 ms for 24576 tokens with heads of 128, 1006 instead of 1000 us for 512 tokens
// behind 131072 with heads of 256.  Scores that rise by 16 or more from block to block throughout
// pay for the second product: 8192 tokens 703 instead of 509 us.)
//
// m is a rounded product s c, and fma(s, c, -m) takes it from the unrounded one: all weights of a row have a
// factor of 2^(half a unit of m), at most 2^(2^-8) up to |m| = 2^16, which cancels.  Beyond, the product is
// rounded first: from |m| = 2^31 on the factor would be 2^128 and more, and the row's sum infinite or 0.
//
// The weights are rounded to bf16 once for the product (their sum l is not): an error of at most 2^-8
// of a weighted mean of |v|, about as large as the output's own rounding.  Two bf16 parts would take
// half as many matrix instructions again, which prompts would pay for in full.  Calls of a few rows a request are
// bound by reading and would not: they share the one form (attn_decode_paged, for single tokens, has two parts).
//
// Measured on MI355X (a matrix product of 8192^3 runs at 1325 TFLOP/s there): one prompt of 24576
// tokens 1105 TFLOP/s with heads of 256, 1059 of 128, 1007 of 64, from an e4m3 cache 1051, 1025 and 993; 512
// tokens behind 131072 1.04 ms, 1060 TFLOP/s; 6144 tokens 327 us, 947 (the last tiles run alone); 32 requests of
// 1 to 7 tokens over 500 to 8192: 76 us, 3.7 TB/s.  On other cards up to 7 % faster (305 us, 0.99 ms).
#include <algorithm>
#include <cmath>

#include "kv.hpp"
#include "lanes.hpp"
#include "mfma.hpp"

namespace gdn {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kCUs = 256;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;
constexpr float kNegInf = -__builtin_inff();
constexpr float kMost = 256.f;  // sum of a lane's weights of a block up to which the reference stays
constexpr float kFar = 65536.f;  // size of the reference up to which one fma takes it from the product s c

constexpr int kRowBits = 7;  // a tile has 2^7 rows, 32 of each wave, or 2^8, 64 of each

constexpr int kMostTiles = 32768;  // in one dimension of the grid

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4t __attribute__((ext_vector_type(4)));
// (constant address space: these arrays do not change during the call, so wave-uniform reads
// are scalar loads)
#ifdef __HIP_DEVICE_COMPILE__
#define GDN_CONSTANT __attribute__((address_space(4)))
#else
#define GDN_CONSTANT
#endif
typedef const int32_t GDN_CONSTANT *table_t;

struct ChunkDev {
  ChunkArgs a;
  int group, tiles;
  int bits;         // a tile has 2^bits rows
  int parts, piece; // a tile's blocks are divided into pieces of this many; at most `parts`
  int spread;       // whether a tile's pieces go to different XCDs
  float c;          // |scale * k_scale| in log2 units
  uint32_t flip, keep;  // for two bf16 queries: the scale's sign, and 0 if it is 0 (c is 1 then)
  uint32_t inverse;     // ceil(2^32 / group), for a group of 2 or more
  float *o, *ml;    // parts > 1: [part][token][q_heads] rows of O, and m and l
  float *lse;       // [tokens][q_heads], or NULL
  float *row_ml;    // [tokens][q_heads] rows' m and 1 / l for the weights' kernel (see row_factors), or NULL
};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ float ref(float m) { return m == kNegInf ? 0.f : m; }
// s c - m with the product rounded first, as it was for m: 0 for the score that m is of
__device__ __forceinline__ float rounded_apart(float s, float c, float m) {
  float x = s * c;
  asm("" : "+v"(x));  // (no fma)
  return x - m;
}
// What a row's weights 2^(s c - m) / l need; of a row that sees nothing, 2^-inf * 0
__device__ __forceinline__ void row_factors(float *to, float m, float l) {
  to[0] = l == 0.f ? -kNegInf : m;
  to[1] = l == 0.f ? 0.f : 1.f / l;
}
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
// says that the row sees one with a weight above 0.  Where the second walk's sums are not finite either, they may
// have outgrown fp32, as weights reach 2^4 and more where the reference stayed behind: it is done again with the
// reference following every block, so that no weight is above 1.
enum { kAsIs, kFinite, kClose, kUp, kDown };
__device__ __forceinline__ u32x4 sorted(u32x4 x, int kind) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t r = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t v = (x[i] >> (16 * e)) & 0xffffu, a = v & 0x7fffu;
      const bool mark = a > 0x7f80u || v == (kind == kUp ? 0x7f80u : 0xff80u);
      r |= (kind <= kClose ? (a < 0x7f80u ? v : 0u) : mark ? 0x3f80u : 0u) << (16 * e);
    }
    x[i] = r;
  }
  return x;
}
// the same for four e4m3 values: what is NaN becomes 0 or 1, other values themselves or 0
__device__ __forceinline__ uint32_t sorted_f8(uint32_t x, int kind) {
  uint32_t r = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t v = (x >> (8 * e)) & 0xffu;
    const bool nan = (v & 0x7fu) == 0x7fu;
    r |= (kind <= kClose ? (nan ? 0u : v) : nan ? 0x38u : 0u) << (8 * e);
  }
  return r;
}
// a sum with an infinite (or NaN) value added
__device__ __forceinline__ float beyond(float sum, int kind) { return sum + (kind == kUp ? -kNegInf : kNegInf); }

// ---- which rows a tile has -------------------------------------------------
// The tiles of request b begin at cu[b] * group / 2^bits + b: at least as many as it needs, and
// found from cu alone, so that no list of tiles has to be made first.
struct Chunk {
  int bos, n, rows0;     // the request's first token and number of tokens, the tile's first row
  int slot, len, begin;
  bool any, live;        // whether the tile has rows, whether they see anything at all
};
// The last request b for which begins(b, cu[b]) holds (it holds up to some request), or 0.  Called by
// whole waves: a lane looks at a request, so up to 64 requests take one step of reads and 4096
// two (a step costs a workgroup most of a microsecond).
template <typename F>
__device__ __forceinline__ int last_request(const ChunkDev &p, F begins) {
  const int lane = threadIdx.x & 63;
  int b = 0;  // it is one of n from here
  for (int n = p.a.batch; n > 1;) {
    const int step = (n + 63) >> 6, at = b + lane * step;
    const bool in = lane * step < n;
    const bool yes = begins(at, p.a.cu_seqlens[in ? at : b]);
    const int i = uniform(max(0, int(__builtin_popcountll(__ballot(in && yes))) - 1));
    n = min(step, n - i * step);
    b += i * step;
  }
  return b;
}
__device__ __forceinline__ Chunk chunk_of(const KvGeom &g, const ChunkDev &p, int tile, int b, bool tell) {
  const table_t cu = (table_t)p.a.cu_seqlens;
  Chunk r;
  r.bos = cu[b];
  const int eos = cu[b + 1];
  const int64_t at = (tile - ((int64_t(r.bos) * p.group) >> p.bits) - b) << p.bits;
  const bool ok = r.bos >= 0 && eos >= r.bos && eos <= p.a.tokens;
  r.n = ok ? eos - r.bos : 0;
  r.any = ok && at >= 0 && at < int64_t(r.n) * p.group;
  r.rows0 = r.any ? int(at) : 0;
  r.slot = ((table_t)p.a.slot_table)[b];
  r.len = ((table_t)p.a.kv_len)[b];
  r.begin = p.a.kv_begin ? ((table_t)p.a.kv_begin)[b] : 0;
  const bool lens = r.len >= r.n && r.len <= p.a.max_len && r.begin >= 0;
  r.live = r.any && r.slot > 0 && r.slot < g.slots && lens;
  if (tell) {
    const bool told = r.any || r.n == 0;  // (a request without rows has a tile too)
    if (!ok) set_err(g.err, GDN_ERRW_BAD_SEQLENS);
    else if (told && r.slot >= g.slots) set_err(g.err, GDN_ERRW_BAD_SLOT);
    else if (told && r.slot > 0 && !lens) set_err(g.err, GDN_ERRW_BAD_SEQLENS);
  }
  return r;
}
// a row's token: row / group (the product with the inverse is right or one too many below 2^31)
__device__ __forceinline__ int token_of(const ChunkDev &p, int row) {
  const int t = int(__umulhi(uint32_t(row), p.inverse));
  return p.group == 1 ? row : t - (t * p.group > row ? 1 : 0);
}
// first place that the query at `place` sees
__device__ __forceinline__ int seen_from(const ChunkDev &p, int begin, int place) {
  return p.a.window ? max(begin, place - p.a.window + 1) : begin;
}

// The blocks of KT places that a tile's rows see: lo and how many, and the first of these places.
struct Span {
  int lo, n, from;
};
template <int KT>
__device__ __forceinline__ Span span_of(const ChunkDev &p, const Chunk &ch) {
  if (!ch.live) return Span{0, 0, 0};
  const int all = ch.n * p.group, place0 = ch.len - ch.n;
  const int first = place0 + token_of(p, ch.rows0), last = place0 + token_of(p, min(ch.rows0 + (1 << p.bits) - 1, all - 1));
  const int from = seen_from(p, ch.begin, first), lo = from / KT;
  return Span{lo, from <= last ? last / KT + 1 - lo : 0, from};
}

// ---- shared memory ---------------------------------------------------------
// A tile has KT rows of D bf16 values; 16-byte piece c of row r lies at piece c ^ twist(r).
// Keys are read 32 rows at the same piece, values 4 rows of 64 adjacent bytes: both meet every
// bank equally often.
template <int D>
__device__ __forceinline__ int twist(int r) {
  return D == 64 ? (((r >> 1) & 1) << 2 | ((r >> 2) & 3)) : ((r & 3) << 2 | ((r >> 2) & 3));
}

// The order of a score's steps of 16 columns: a row of 512 bytes has twice the pieces that the twist
// permutes, so steps that differ by half of a row follow each other, and have their address in common.
template <int D>
constexpr int step_at(int i) {
  return D == 256 ? (i >> 1) + (i & 1) * (D / 32) : i;
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

// The kernel's arguments as they lie in memory: what a part of the kernel needs is read there, not
// held in registers through the others.
struct ChunkArgsAll {
  KvGeom g;
  ChunkDev p;
};
typedef const ChunkArgsAll GDN_CONSTANT *args_t;
__device__ __forceinline__ args_t fresh(args_t a) {
  asm volatile("" : "+s"(a));
  return a;
}

// kWide: pages hold 16 tokens or more, so that the rows of a wave's load lie in one page.
//
// A workgroup has one piece of one tile's blocks, for one key-value head.  The first pieces come
// first, and of them those of a request's last tiles, which see the most places: workgroups that
// run at the same time read the same keys, and the last ones to start are short.
// R: 32 R rows of each wave.
template <int D, bool kF8, bool kWide, int R>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2)))
void attn_prefill_kernel(ChunkArgsAll) {
  using T = Tile<D, kF8>;
  constexpr int KT = T::KT, KB = KT / 32, KS = D / 16, DB = D / 32, NL = T::kLoads;
  constexpr int kAhead = 3;  // fragments asked for before they are used (4 and 6 are the same where registers allow)
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const args_t args = (args_t)__builtin_amdgcn_kernarg_segment_ptr();
  // a block (by its number's parity) that has a page outside the pool
  int *const sbad = reinterpret_cast<int *>(lds + 4 * T::kBytes);
  const int lane = threadIdx.x & 63, c = lane & 31, half = lane >> 5;
  const int wave = uniform(threadIdx.x >> 6);

  const KvGeom g = args->g;
  const ChunkDev p = args->p;
  // (tiles in both of the grid's last two dimensions where none is divided)
  const int h = blockIdx.x, part = p.parts > 1 ? int(blockIdx.z) : 0;
  int order = int(blockIdx.y) + (p.parts > 1 ? (p.spread ? part : 0) : int(blockIdx.z) * kMostTiles);
  if (p.spread && order >= p.tiles) order %= p.tiles;
  const int tile = p.tiles - 1 - order;
  if (tile < 0) return;
  const int b = last_request(p, [&](int b, int cu) { return ((int64_t(cu) * p.group) >> p.bits) + b <= tile; });
  const Chunk ch = chunk_of(g, p, tile, b, h == 0 && part == 0 && threadIdx.x == 0);
  if (!ch.any) return;
  const Span span = span_of<KT>(p, ch);
  if (part > 0 && part * p.piece >= span.n) return;
  const bool whole = span.n <= p.piece;
  const int t0 = span.lo + part * p.piece, t1 = min(span.lo + span.n, t0 + p.piece);

  const int all = ch.n * p.group;
  const int row0 = ch.rows0 + 32 * R * wave;
  const bool wlive = ch.live && row0 < all;
  const int place0 = ch.len - ch.n;  // of the first new token
  int place[R];
  const int wfirst = place0 + token_of(p, min(row0, all - 1));
  const int wlast = place0 + token_of(p, min(row0 + 32 * R - 1, all - 1));
  const int wfrom = seen_from(p, ch.begin, wfirst), wfrom_last = seen_from(p, ch.begin, wlast);

  bf16x8 q[R][KS];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = min(row0 + 32 * r + c, all - 1);  // (rows behind the last repeat it and are not stored)
    const int token = token_of(p, row), head = h * p.group + (row - token * p.group);
    place[r] = place0 + token;
    if (!wlive || t0 >= t1) continue;
    const uint16_t *src = p.a.q + (ch.bos + token) * p.a.q_stride + int64_t(head) * D + 8 * half;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      u32x4 w = *reinterpret_cast<const u32x4 *>(src + 16 * s);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = (w[i] ^ p.flip) & p.keep;
      q[r][s] = __builtin_bit_cast(bf16x8, w);
    }
  }

  // ---- loads ----
  auto load_row = [&](int j) { return (j * kWaves + wave) * T::kLoadRows; };  // first row of load j
  const table_t table = (table_t)(g.page_table + int64_t(max(ch.slot, 0)) * g.max_pages);
  const int page_mask = (1 << g.page_shift) - 1;
  // a lane's place in a load: its row, and the piece of the row that belongs there
  auto lane_row = [&]() { return int(threadIdx.x & 63) / T::kLanes; };
  const int lpiece = lane % T::kLanes;
  const int loff = (kWide ? lane_row() * T::SB : 0) + ((kF8 ? lpiece : lpiece ^ twist<D>(wave * T::kLoadRows + lane_row())) << 4);
  // Pages in front of the first place that the tile's rows see need not be there: for rows of its first block
  // that lie before, those of that place are read (from: that place).
  constexpr int kAnywhere = INT32_MIN;
  int ids[kWide ? NL : 1];
  auto load_ids = [&](int t, int from = kAnywhere) {
    if constexpr (kWide) {
#pragma unroll
      for (int j = 0; j < NL; ++j)
        ids[j] = table[uint32_t(min(max(t * KT + load_row(j), from), ch.len - 1)) >> g.page_shift];
    }
  };
  bool edge;  // whether the block to come has rows that are no places of the request
  uint32_t src[NL];  // its rows in the layer's keys and values
  auto locate = [&](int t, int j, int from = kAnywhere) {
    const int at = max(t * KT + load_row(j) + (kWide ? 0 : lane_row()), kWide ? from & -T::kLoadRows : from);
    int id;
    if constexpr (kWide) id = ids[j];
    else id = g.page_table[int64_t(ch.slot) * g.max_pages + (min(at, ch.len - 1) >> g.page_shift)];
    const bool wrong = id <= 0 || id >= g.pages;
    id = wrong ? 0 : id;
    src[j] = uint32_t(((id * g.kv_heads + h) << g.page_shift) + (at & page_mask));
    return wrong;
  };
  auto locate_all = [&](int t, int from = kAnywhere) {
    bool bad = false;
#pragma unroll
    for (int j = 0; j < NL; ++j) bad |= locate(t, j, from);
    return bad;
  };
  // the block's rows have all been located; bad: one of the lane's is in no page
  auto located = [&](int t, bool bad) {
    if (kWide ? bad : __any(bad)) {
      bad = true;
      if ((threadIdx.x & 63) == 0) {
        sbad[t & 1] = t;
        set_err(g.err, GDN_ERRW_BAD_PAGE);
      }
    } else {
      bad = false;
    }
    edge = bad || t * KT < ch.begin || (t + 1) * KT > ch.len;
  };
  // whether the lane's row of load j of block t is no place of the request (the rare blocks)
  auto hidden = [&](int t, int j) {
    const int at = t * KT + load_row(j) + lane_row();
    const int id = g.page_table[int64_t(ch.slot) * g.max_pages + (min(at, ch.len - 1) >> g.page_shift)];
    return id <= 0 || id >= g.pages || at >= ch.len || at < ch.begin;
  };
  // bf16: from memory to shared memory; a lane's 16 bytes land at its place in the wave's 1 KB,
  // so it asks for the piece that belongs there
  auto ask = [&](int t, int j, bool values) {
    if constexpr (!kF8) {
      // (the twist of the rows of load j differs from load 0's in one bit at most)
      constexpr int kStep = kWaves * T::kLoadRows;
      static_assert(kStep % 16 == 0 || kStep == 8, "twist");
      const uint32_t off = uint32_t(loff) ^ (kStep == 8 ? (j & 1) * 32 : 0);
      char *dst = lds + (t & 1) * 2 * T::kBytes + load_row(j) * T::RB + (values ? T::kBytes : 0);
      const char *from = (values ? g.v : g.k) + uint64_t(src[j]) * T::SB;
      typedef __attribute__((address_space(3))) void *lp;
      if constexpr (kWide) {  // one page: a scalar base, and 32 bits of the lane's
        const auto rows = __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(from), 0, 1024, 0x00027000);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rows, (lp)dst, 16, int(off), 0, 0, 0);
      } else {
        __builtin_amdgcn_global_load_lds((__attribute__((address_space(1))) const char *)from + off, (lp)dst, 16, 0, 0);
      }
    }
  };
  auto ask_all = [&](int t) {
#pragma unroll
    for (int j = 0; j < NL; ++j) {
      ask(t, j, false);
      ask(t, j, true);
    }
  };
  // Rows that are no places of the request hold anything: zeros keep 0 * NaN out of the product.
  // Other walks than the first replace values.
  auto change_rows = [&](int t, int kind) {
    char *to = lds + (t & 1) * 2 * T::kBytes + T::kBytes;
#pragma unroll 1
    for (int j = 0; j < NL; ++j) {
      u32x4 *at = reinterpret_cast<u32x4 *>(to + load_row(j) * T::RB + int(threadIdx.x & 63) * 16);
      u32x4 x = *at;
      if (kind != kAsIs) x = sorted(x, kind);
      *at = hidden(t, j) ? u32x4{0, 0, 0, 0} : x;
    }
  };
  // e4m3: through registers, 16 values a lane; with heads of 256 the keys before the values, as there
  // are no registers for both
  constexpr bool kTwoSteps = kF8 && D == 256;
  u32x4 kraw[kF8 ? NL : 1], vraw[kF8 ? NL : 1];
  auto fetch = [&](u32x4 *raw, const char *base) {
    if constexpr (kF8) {
#pragma unroll
      for (int j = 0; j < NL; ++j) raw[j] = *reinterpret_cast<const u32x4 *>(base + uint64_t(src[j]) * T::SB + loff);
    }
  };
  auto put = [&](const u32x4 *raw, char *to) {
    if constexpr (kF8) {
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        const int r = load_row(j) + lane_row();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          u32x4 w;
          uint32_t a, b;
          f8_to_bf16(raw[j][2 * e], &a, &b);
          w[0] = a; w[1] = b;
          f8_to_bf16(raw[j][2 * e + 1], &a, &b);
          w[2] = a; w[3] = b;
          *reinterpret_cast<u32x4 *>(to + r * T::RB + (((2 * lpiece + e) ^ twist<D>(r)) << 4)) = w;
        }
      }
    }
  };
  auto change_raw = [&](int t, int kind) {  // what change_rows does, before the values are put
    if constexpr (kF8) {
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        const bool no = hidden(t, j);
#pragma unroll
        for (int i = 0; i < 4; ++i) vraw[j][i] = no ? 0u : kind == kAsIs ? vraw[j][i] : sorted_f8(vraw[j][i], kind);
      }
    }
  };

  // ---- the walk ----
  // keys: row c of a block of 32, piece half of step 0; step s is 2 s further, which the twist
  // turns into an exclusive or.  Values: row vrow of the half's four, 4 adjacent values of the
  // block of 32 columns
  const int vrow = 4 * half + ((lane >> 2) & 3), vpair = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
  const int kaddr = c * T::RB + ((half ^ twist<D>(c)) << 4);
  const int vaddr = vrow * T::RB + ((vpair ^ twist<D>(vrow)) << 4) + 8 * (lane & 1) + T::kBytes;
  // (the blocks of columns likewise)
  auto step_of = [](int i) { return step_at<D>(i); };
  auto block_of = [](int i) { return D == 256 ? (i >> 1) + (i & 1) * (DB / 2) : i; };

  f32x16 o[R][DB];
  float m[R], l[R];
  auto walk = [&](int kind) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int b = 0; b < DB; ++b) o[r][b] = f32x16{};
      m[r] = kNegInf;
      l[r] = 0.f;
    }
    __syncthreads();  // (the last walk's blocks have been read)
    if (threadIdx.x < 2) sbad[threadIdx.x] = -1;
    __syncthreads();
    if (t0 >= t1) return;
    auto convert = [&](int t) {
      if constexpr (kF8) {
        char *to = lds + (t & 1) * 2 * T::kBytes;
        put(kraw, to);
        if (edge || kind != kAsIs) change_raw(t, kind);
        put(vraw, to + T::kBytes);
      }
    };
    load_ids(t0, span.from);
    located(t0, locate_all(t0, span.from));
    ask_all(t0);
    fetch(kraw, g.k);
    fetch(vraw, g.v);
    convert(t0);
    load_ids(t0 + 1);
    // block t is there
    auto arrive = [&](int t) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      if (!kF8 && (edge || kind != kAsIs)) [[unlikely]] change_rows(t, kind);
      __syncthreads();
    };
    auto skip = [&](int a, int b) {
#pragma unroll 1
      for (int t = a; t < b; ++t) {
        arrive(t);
        if (t + 1 < t1) {
          located(t + 1, locate_all(t + 1));
          ask_all(t + 1);
          fetch(kraw, g.k);
          fetch(vraw, g.v);
          load_ids(t + 2);
          convert(t + 1);
        }
      }
    };
    // the blocks that the wave's rows see
    const int w0 = wlive ? min(t1, max(t0, wfrom / KT)) : t1, w1 = wlive ? max(w0, min(t1, wlast / KT + 1)) : t1;
    skip(t0, w0);
#pragma unroll 1
    for (int t = w0; t < w1; ++t) {
      arrive(t);
      const int p0 = t * KT;
      // (the last block is asked for again, as one that nobody reads: no branch among the products.  Pages are
      // those of the places behind it, or, small ones, its own, which have been looked at)
      const int next = min(t + 1, t1 - 1);
      f32x16 s[R][KB];
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) s[r][kb] = f32x16{};
      // (the blocks' base in shared memory is a multiple of a row's bytes, so the twist's bits can be changed
      // behind its addition)
      typedef __attribute__((address_space(3))) char *lp;
      uint32_t ka = uint32_t(uintptr_t((lp)lds)) + kaddr + (t & 1) * 2 * T::kBytes, va = ka - kaddr + vaddr;
      asm volatile("" : "+v"(ka), "+v"(va));  // (addresses are worked out here, not kept over the walk)
      auto kread = [&](int i) {
        const uint32_t at = 32 * step_of(i / KB), twisted = D == 256 ? at % 256 : at;
        return *(__attribute__((address_space(3))) const bf16x8 *)(uintptr_t)((ka ^ twisted) + (at - twisted) +
                                                                             32 * (i % KB) * T::RB);
      };
      auto vread = [&](int i) {
        s16x4t v[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t at = 64 * block_of(i % DB) + 32 * e, twisted = D == 256 ? at % 256 : at;
          v[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4t *)(uintptr_t)(
              (va ^ twisted) + (at - twisted) + (16 * (i / DB) + 8 * e) * T::RB));
        }
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
      };
      const int flag = sbad[t & 1];
      if constexpr (kTwoSteps) {
        located(t + 1, locate_all(next) && (kWide || next > t));
        load_ids(next + 1);
        fetch(kraw, g.k);
      }
      bf16x8 ring[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) ring[i] = kread(i);
      // a wave in its products goes before one in its softmax (2 to 3 % in all)
      __builtin_amdgcn_s_setprio(1);
      // the next block's loads go out between the products, whose issue they do not hold up
      constexpr int kEvery = KS * KB / (2 * NL);  // products between two loads
      bool bad = false;
#pragma unroll
      for (int i = 0; i < KS * KB; ++i) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int r = 0; r < R; ++r) s[r][i % KB] = mfma32(ring[i % kAhead], q[r][step_of(i / KB)], s[r][i % KB]);
        if (i + kAhead < KS * KB) ring[i % kAhead] = kread(i + kAhead);
        if (!kTwoSteps && i % kEvery == 0) {
          const int j = i / kEvery / 2;
          if (i / kEvery % 2 == 0) {
            bad |= locate(next, j);
            ask(t + 1, j, false);
          } else {
            ask(t + 1, j, true);
          }
        }
      }
      __builtin_amdgcn_s_setprio(0);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) ring[i] = vread(i);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (kTwoSteps) {
        put(kraw, lds + ((t + 1) & 1) * 2 * T::kBytes);
        fetch(vraw, g.v);
      } else {
        located(t + 1, bad && (kWide || next > t));
        fetch(kraw, g.k);
        fetch(vraw, g.v);
        load_ids(next + 1);
      }
      const bool flagged = uniform(flag) == t;
      const bool in_part = p0 < wfrom_last || p0 + KT - 1 > wfirst || flagged;
      auto hide = [&](int r) {  // what the rows do not see
        uint32_t no = 0;        // scores of places that are in no page
        if (flagged) [[unlikely]] {
#pragma unroll 1
          for (int e = 0; e < 16 * KB; ++e) {
            const int at = p0 + 32 * (e >> 4) + 8 * ((e >> 2) & 3) + 4 * half + (e & 3);
            const int id = g.page_table[int64_t(ch.slot) * g.max_pages + (min(at, ch.len - 1) >> g.page_shift)];
            no |= id <= 0 || id >= g.pages ? 1u << e : 0u;
          }
        }
        const int from = seen_from(p, ch.begin, place[r]);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int at = p0 + 32 * kb + 8 * (e >> 2) + 4 * half + (e & 3);
            if (at > place[r] || at < from || (no >> (16 * kb + e) & 1)) s[r][kb][e] = kNegInf;
          }
      };
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (in_part) [[unlikely]] hide(r);
        auto weigh = [&] {  // scores to weights, and their sum
          const float mr = ref(m[r]);
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              s[r][kb][e] = fexp2(fmaf(s[r][kb][e], p.c, -mr));
              sum[e & 3] += s[r][kb][e];
            }
          return (sum[0] + sum[1]) + (sum[2] + sum[3]);
        };
        float sum = 0.f;
        bool follow = in_part || kind == kClose || __any(!(fabsf(m[r]) <= kFar));  // (-inf: nothing seen so far)
        if (!follow) {
          sum = weigh();
          if (__any(!(sum <= kMost))) [[unlikely]] {
            follow = true;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) s[r][kb] = f32x16{};
#pragma unroll
            for (int i = 0; i < KS * KB; ++i) s[r][i % KB] = mfma32(kread(i), q[r][step_of(i / KB)], s[r][i % KB]);
          }
        }
        if (follow) [[unlikely]] {
          float top = s[r][0][0];
#pragma unroll
          for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int e = 0; e < 16; ++e) top = fmaxf(top, s[r][kb][e]);
          top = halves_max(top) * p.c;
          const float to = fmaxf(m[r], top), f = fexp2(m[r] - ref(to));
          l[r] *= f;
#pragma unroll
          for (int b = 0; b < DB; ++b)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[r][b][e] *= f;
          m[r] = to;
          if (fabsf(ref(to)) > kFar) [[unlikely]] {  // (divided by c, so that the code of the weights serves)
            const float back = 1.f / p.c;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
              for (int e = 0; e < 16; ++e) s[r][kb][e] = rounded_apart(s[r][kb][e], p.c, to) * back;
            m[r] = 0.f;
          }
          sum = weigh();
          m[r] = to;
        }
        l[r] += sum;
      }
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int ks = 0; ks < 2 * KB; ++ks) {
        bf16x8 pf[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          u32x4 w;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = cvt_pk_bf16(s[r][ks >> 1][8 * (ks & 1) + 2 * i], s[r][ks >> 1][8 * (ks & 1) + 2 * i + 1]);
          pf[r] = __builtin_bit_cast(bf16x8, w);
        }
#pragma unroll
        for (int b = 0; b < DB; ++b) {
          const int i = ks * DB + b;
          if (b == 0 && D == 256) asm volatile("" : "+v"(va));
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int r = 0; r < R; ++r) o[r][block_of(b)] = mfma32(ring[i % kAhead], pf[r], o[r][block_of(b)]);
          if (i + kAhead < 2 * KB * DB) ring[i % kAhead] = vread(i + kAhead);
        }
      }
      __builtin_amdgcn_s_setprio(0);
      if constexpr (kTwoSteps) {
        if (edge || kind != kAsIs) [[unlikely]] change_raw(next, kind);
        put(vraw, lds + ((t + 1) & 1) * 2 * T::kBytes + T::kBytes);
      } else {
        convert(t + 1);
      }
    }
    skip(w1, t1);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  };

  // ---- results ----
  auto store = [&](int kind, int r) {
    int row = row0 + 32 * r + c;
    asm volatile("" : "+v"(row));
    const args_t again = fresh(args);
    const auto &p = again->p;
    const float ln = halves_sum(l[r]);
    if (row >= ch.n * p.group) return;
    const int token = row / p.group;
    const int64_t orow = int64_t(ch.bos + token) * p.a.q_heads + h * p.group + (row - token * p.group);
    if (!whole) {
      const int64_t at = int64_t(part) * p.a.tokens * p.a.q_heads + orow;
      if (half == 0 && kind <= kClose) {
        p.ml[2 * at] = ln == 0.f ? kNegInf : m[r];
        p.ml[2 * at + 1] = ln;
      }
      if (ln == 0.f) return;
      float *to = p.o + at * D + 4 * half;
#pragma unroll
      for (int b = 0; b < DB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f32x4 v = {o[r][b][4 * i], o[r][b][4 * i + 1], o[r][b][4 * i + 2], o[r][b][4 * i + 3]};
          if (kind > kClose) {
            const f32x4 old = ld4(to + 32 * b + 8 * i);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = v[e] > 0.f ? beyond(old[e], kind) : old[e];
          }
          st4(to + 32 * b + 8 * i, v);
        }
      return;
    }
    if (p.lse && half == 0 && kind <= kClose)
      p.lse[orow] = ln == 0.f ? kNegInf : (m[r] + __builtin_amdgcn_logf(ln)) * kLn2;
    if (p.row_ml && half == 0 && kind <= kClose) row_factors(p.row_ml + 2 * orow, m[r], ln);
    const float f = ln == 0.f ? 0.f : again->g.v_scale / ln;
    uint16_t *to = p.a.out + orow * D + 8 * half;
#pragma unroll
    for (int b = 0; b < DB; ++b)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // columns 16 i + 8 h + 0..3 and + 4..7 of the block: the halves swap what the other stores
        u32x4 w;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t x = cvt_pk_bf16(o[r][b][8 * i + 2 * e] * f, o[r][b][8 * i + 2 * e + 1] * f);
          const uint32_t y = cvt_pk_bf16(o[r][b][8 * i + 4 + 2 * e] * f, o[r][b][8 * i + 5 + 2 * e] * f);
          const auto both = __builtin_amdgcn_permlane32_swap(x, y, false, false);
          w[e] = both[0];
          w[2 + e] = both[1];
        }
        u32x4 *at = reinterpret_cast<u32x4 *>(to + 32 * b + 16 * i);
        if (kind > kClose) {
          const u32x4 old = *at;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float lo = __uint_as_float(w[e] << 16), hi = __uint_as_float(w[e] & 0xffff0000u);
            const float x = __uint_as_float(old[e] << 16), y = __uint_as_float(old[e] & 0xffff0000u);
            w[e] = pack_bf16x2(lo > 0.f ? beyond(x, kind) : x, hi > 0.f ? beyond(y, kind) : y);
          }
        }
        *at = w;
      }
  };

#pragma unroll 1
  for (int kind = kAsIs;;) {
    walk(kind);
    if (kind <= kFinite) {
      // a NaN may come from a value that the row does not see (0 * NaN)
      float bad = 0.f;
      if (wlive) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int b = 0; b < DB; ++b)
#pragma unroll
            for (int e = 0; e < 16; ++e) bad = fmaf(o[r][b][e], 0.f, bad);
      }
      // (flags: static shared memory would move the blocks off address 0)
      const bool any = __any(bad != 0.f);
      if (threadIdx.x == 0) sbad[2] = 0;
      __syncthreads();
      if (any && lane == 0) sbad[2] = 1;
      __syncthreads();
      if (uniform(sbad[2])) {
        ++kind;
        continue;
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) store(kind, r);
    if (kind == kAsIs || kind == kDown) break;
    kind = kind == kUp ? kDown : kUp;
  }
}

// Rows of tiles that were divided: the pieces' O, m and l joined.  A wave has `heads` query heads of
// a token, one after the other; its lanes first have a piece's m and l each, then D / 64 columns of
// the row.
template <int D>
__global__ __launch_bounds__(kThreads) void attn_prefill_join_kernel(KvGeom g, ChunkDev p, int heads) {
  constexpr int N = D / 64, kPieces = 4;
  typedef float fN __attribute__((ext_vector_type(N)));
  const int groups = (p.a.q_heads + heads - 1) / heads;
  const int64_t item = flat_block() * kWaves + uniform(threadIdx.x >> 6);
  const int token = int(item / groups), first = int(item - int64_t(token) * groups) * heads;
  if (token >= p.a.tokens) return;
  const int b = last_request(p, [&](int, int cu) { return cu <= token; });
  const table_t cu = (table_t)p.a.cu_seqlens;
  const int bos = cu[b];
  if (token < bos || token >= cu[b + 1]) return;
  const int lane = threadIdx.x & 63;
  const int64_t stride = int64_t(p.a.tokens) * p.a.q_heads;  // rows of a part
#pragma unroll 1
  for (int head = first; head < min(first + heads, p.a.q_heads); ++head) {
    const int row = (token - bos) * p.group + head % p.group;
    const int tile = int((int64_t(bos) * p.group) >> p.bits) + b + (row >> p.bits);
    const Chunk ch = chunk_of(g, p, tile, b, false);
    if (!ch.any) return;
    const int pieces = (span_of<Tile<D, false>::KT>(p, ch).n + p.piece - 1) / p.piece;
    if (pieces < 2) continue;
    const int64_t orow = int64_t(token) * p.a.q_heads + head;
    float top = kNegInf, l = 0.f;
    fN o = {};
    for (int base = 0; base < pieces; base += 64) {
      const int n = min(64, pieces - base);
      const float *e = p.ml + 2 * (orow + (base + min(lane, n - 1)) * stride);
      const float m = lane < n ? e[0] : kNegInf, pl = lane < n ? e[1] : 0.f;
      float mm = fmaxf(m, top);  // (the sums so far have the maximum top)
#pragma unroll
      for (int d = 32; d; d >>= 1) mm = fmaxf(mm, __shfl_xor(mm, d));
      const float f = pl == 0.f ? 0.f : fexp2(m - mm), old = top == kNegInf ? 0.f : fexp2(top - mm);
      l = fmaf(l, old, wave_sum(pl * f));
      // (what has underflowed is left out, as in the walk: never 0 * inf)
#pragma unroll
      for (int c = 0; c < N; ++c) o[c] = old == 0.f ? 0.f : o[c] * old;
      top = mm;
      const float *src = p.o + (orow + base * stride) * D + lane * N;
      for (int k = 0; k < n; k += kPieces) {
        fN v[kPieces];
#pragma unroll
        for (int u = 0; u < kPieces; ++u) v[u] = *reinterpret_cast<const fN *>(src + min(k + u, n - 1) * stride * D);
#pragma unroll
        for (int u = 0; u < kPieces; ++u) {
          // (a lane past the last has l = 0; a piece of l = 0 has not written its O)
          const int at = min(k + u, 63);
          const float fk = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f), at));
          const float lk = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(pl), at));
#pragma unroll
          for (int c = 0; c < N; ++c) o[c] = lk == 0.f || fk == 0.f || k + u > 63 ? o[c] : fmaf(v[u][c], fk, o[c]);
        }
      }
    }
    if (p.lse && lane == 0) p.lse[orow] = l == 0.f ? kNegInf : (top + __builtin_amdgcn_logf(l)) * kLn2;
    if (p.row_ml && lane == 0) row_factors(p.row_ml + 2 * orow, top, l);
    const float f = l == 0.f ? 0.f : g.v_scale / l;
    uint16_t *to = p.a.out + orow * D + lane * N;
    if constexpr (N == 1) {
      to[0] = f32_to_bf16(o[0] * f);
    } else {
#pragma unroll
      for (int c = 0; c < N / 2; ++c) reinterpret_cast<uint32_t *>(to)[c] = cvt_pk_bf16(o[2 * c] * f, o[2 * c + 1] * f);
    }
  }
}

// ---- the last queries' weights, added to mass -------------------------------
// One workgroup per request, key-value head and 4 * kMassPlaces places; a wave keeps the keys of its
// places in registers and walks the rows of the last queries, kMassRows at a time, which the waves
// share in shared memory (in the layout of a block of keys), asked for one step ahead.  So every
// entry of mass has one owner and one order of summation.  A weight is 2^(s c - m) / l with the row's m and
// l, its score and exponent worked out as for l, bit for bit (against the logarithm lse a large score would lose
// |lse| 2^-23, and one whose columns are summed in another order as much).
//
// (512 queries over 131584 places, 16 heads of 256: 0.70 ms; two 4099-token prompts 57 us.  Reading the rows
// by each wave for itself: 2.25 ms for the former, bound by its scattered reads; 64 places a wave instead of 32:
// 83 against 65 us for the latter when that was tried, as there are too few waves.)
constexpr int kMassRows = 64, kMassPlaces = 32;

template <int D, bool kF8>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2)))
void attn_prefill_mass_kernel(KvGeom g, ChunkDev p, int blocks) {
  constexpr int KP = kMassPlaces, KB = KP / 32, KS = D / 16, NB = kMassRows / 32, RB = 2 * D, PLACES = KP * kWaves;
  constexpr int LANES = RB / 16, LROWS = 64 / LANES, LOADS = kMassRows / (kWaves * LROWS);
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int64_t item = flat_block();
  const int h = int(item % g.kv_heads);
  const int64_t rest = item / g.kv_heads;
  const int b = int(rest / blocks);
  if (b >= p.a.batch) return;
  const table_t cu = (table_t)p.a.cu_seqlens;
  const int bos = cu[b], eos = cu[b + 1], slot = ((table_t)p.a.slot_table)[b], len = ((table_t)p.a.kv_len)[b];
  const int begin = p.a.kv_begin ? ((table_t)p.a.kv_begin)[b] : 0;
  if (bos < 0 || eos <= bos || eos > p.a.tokens) return;
  const int n = eos - bos;
  if (slot <= 0 || slot >= g.slots || len < n || len > p.a.max_len || begin < 0)
    return;
  const int late = min(n, p.a.mass_tokens);   // queries that count
  const int place0 = len - n, first = n - late;
  const int lane = threadIdx.x & 63, c = lane & 31, half = lane >> 5;
  const int wave = uniform(threadIdx.x >> 6);
  const int lowest = seen_from(p, begin, place0 + first);
  if (lowest >= len) return;
  const int g0 = lowest / PLACES * PLACES + int(rest % blocks) * PLACES;
  if (g0 >= len) return;
  const int p0 = g0 + wave * KP;
  const int G = p.group, all = n * G;

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
      u32x4 w;
      if constexpr (kF8) {
        const u32x2 x = *reinterpret_cast<const u32x2 *>(src + 16 * s + 8 * half);
        uint32_t lo, hi;
        f8_to_bf16(x[0], &lo, &hi);
        w[0] = lo; w[1] = hi;
        f8_to_bf16(x[1], &lo, &hi);
        w[2] = lo; w[3] = hi;
      } else {
        w = *reinterpret_cast<const u32x4 *>(src + 32 * s + 16 * half);
      }
      // (the scale's sign and 0, on this side of the product)
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = (w[i] ^ p.flip) & p.keep;
      k[kb][s] = __builtin_bit_cast(bf16x8, w);
    }
  }

  // rows of the queries that see any of the workgroup's places
  const int r0 = max(first, g0 - place0) * G;
  int r1 = all;
  if (p.a.window) r1 = int(min(int64_t(all), max(int64_t(0), int64_t(g0) + PLACES - 1 + p.a.window - place0) * G));
  f32x2_t ml[NB];
  auto ask = [&](int r, int buffer) {
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const int at = (j * kWaves + wave) * LROWS, i = at + lane / LANES;
      const int row = min(r + i, all - 1), token = token_of(p, row), head = h * G + (row - token * G);
      const uint16_t *src = p.a.q + int64_t(bos + token) * p.a.q_stride + int64_t(head) * D;
      const int piece = (lane % LANES) ^ twist<D>(i);
      __builtin_amdgcn_global_load_lds((__attribute__((address_space(1))) const char *)src + 16 * piece,
                                       (__attribute__((address_space(3))) void *)(lds + buffer * kMassRows * RB + at * RB),
                                       16, 0, 0);
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int row = min(r + 32 * nb + c, all - 1), token = token_of(p, row);
      const int64_t orow = int64_t(bos + token) * p.a.q_heads + h * G + (row - token * G);
      ml[nb] = *reinterpret_cast<const f32x2_t *>(p.row_ml + 2 * orow);
    }
  };
  f32x16 sum[KB];
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) sum[kb] = f32x16{};
  const int qaddr = c * RB + ((half ^ twist<D>(c)) << 4);
  if (r0 < r1) ask(r0, 0);
  int buffer = 0;
#pragma unroll 1
  for (int r = r0; r < r1; r += kMassRows, buffer ^= 1) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    float m[NB], part[NB];
    bool far = false;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      m[nb] = ml[nb][0];
      part[nb] = ml[nb][1];
      far |= !(fabsf(m[nb]) <= kFar);
    }
    if (r + kMassRows < r1) ask(r + kMassRows, buffer ^ 1);
    const int first_place = place0 + token_of(p, r), last_place = place0 + token_of(p, min(r + kMassRows, r1) - 1);
    if (p0 > last_place || p0 + KP <= seen_from(p, begin, first_place)) continue;  // the wave's places are not seen
    int qa = qaddr + buffer * kMassRows * RB;
    asm volatile("" : "+v"(qa));
    f32x16 s[KB][NB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) s[kb][nb] = f32x16{};
    constexpr int kAhead = 4;
    auto qread = [&](int i) {
      return *reinterpret_cast<const bf16x8 *>(lds + (qa ^ (32 * step_at<D>(i / NB))) + 32 * (i % NB) * RB);
    };
    bf16x8 ring[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) ring[i] = qread(i);
#pragma unroll
    for (int i = 0; i < KS * NB; ++i) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
        s[kb][i % NB] = mfma32(k[kb][step_at<D>(i / NB)], ring[i % kAhead], s[kb][i % NB]);
      if (i + kAhead < KS * NB) ring[i % kAhead] = qread(i + kAhead);
    }
    __builtin_amdgcn_sched_barrier(0);
    if (__any(far)) [[unlikely]] {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        if (m[nb] != -kNegInf && !(fabsf(m[nb]) <= kFar)) {
          const float back = 1.f / p.c;
#pragma unroll
          for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int e = 0; e < 16; ++e) s[kb][nb][e] = rounded_apart(s[kb][nb][e], p.c, m[nb]) * back;
          m[nb] = 0.f;
        }
    }
    const bool whole = r + kMassRows <= r1 && p0 + KP - 1 <= first_place && p0 >= seen_from(p, begin, last_place);
    if (whole) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
          for (int e = 0; e < 16; ++e) sum[kb][e] = fmaf(fexp2(fmaf(s[kb][nb][e], p.c, -m[nb])), part[nb], sum[kb][e]);
    } else {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int row = r + 32 * nb + c, place = place0 + token_of(p, min(row, all - 1));
        const int from = seen_from(p, begin, place), to = row < r1 ? place : -1;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int at = p0 + 32 * kb + 8 * (e >> 2) + 4 * half + (e & 3);
            const float more = fmaf(fexp2(fmaf(s[kb][nb][e], p.c, -m[nb])), part[nb], sum[kb][e]);
            sum[kb][e] = at <= to && at >= from ? more : sum[kb][e];
          }
      }
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

int64_t chunk_tiles(int batch, int tokens, int group, int bits = kRowBits) {
  return ((int64_t(tokens) * group) >> bits) + batch;
}

// How a call's tiles are divided.
struct ChunkPlan {
  int64_t tiles;
  int bits, parts, piece, spread;
  size_t o, ml, row_ml;  // parts of the workspace, in order
};
ChunkPlan chunk_plan(const gdn_kv_pool *p, int batch, int tokens, int q_heads, int max_len, int mass_tokens) {
  ChunkPlan r{};
  if (batch == 0 || tokens == 0) return r;
  const int KT = p->d.head_dim == 256 ? 32 : 64, group = q_heads / p->d.kv_heads;
  const int most = max_len / KT + 1;  // blocks of a tile
  constexpr int64_t slots = 2 * kCUs;
  // What follows is as if all requests were alike (the host knows no more).  With as many tiles as
  // workgroups that run at once, none is divided: pieces gain nothing (6144 tokens, 8 by 2 heads of 256:
  // 347 us whole, 404 in pieces of up to 0.6 of the longest, 375 of 0.8).  Fewer are, so that the pieces
  // fill the compute units: once for one request whose tiles all see about as many places, half more
  // often where lengths differ or the first tiles see few places (1024 tokens: 52 us whole, 45 in six, 56 in nine), and more often yet where
  // pieces stay long (25 requests of up to 30000: 476 us in two, 254 in ten, 263 in twenty).  A piece
  // takes some 5 us more than its blocks and the join 5 to 10, so there are at least 4 blocks to a
  // piece, 7 of several requests, and short lists stay whole (4 requests of up to 333: 26 us, 37 in two).
  const int64_t each = (int64_t(tokens) + batch - 1) / batch, own = ((each * group - 1) >> kRowBits) + 1;
  const int64_t units = batch * own * p->d.kv_heads;
  // Tiles of twice the rows, where a wave has the registers for them, read shared memory half as often and
  // convert e4m3 half as often, but fewer of them run at once and end less evenly.  24576 tokens, 64 heads
  // of 64: 4.77 instead of 5.04 ms, from e4m3 4.95 instead of 5.20, 32 heads (6144 tiles of 128 rows) 2.41
  // instead of 2.53; 8 requests of 4096 by 12 heads (3072 tiles): 284 us instead of 272; 64 short requests
  // (8192 tiles, 16 of a head) 469 instead of 454.
  r.bits = kRowBits + (p->d.head_dim == 64 && units >= 12 * slots && own >= 32 ? 1 : 0);
  r.tiles = chunk_tiles(batch, tokens, group, r.bits);
  if (units < slots && most >= 16) {
    const int64_t half_more = (3 * slots / 2 + units - 1) / units;
    int64_t want = slots / units, limit = most / 4;
    if (2 * each > max_len) want = half_more;
    else if (batch > 1) want = std::max(half_more, std::min(4 * slots / units, int64_t(most / 48))), limit = most / 7;
    r.parts = int(std::min(want, limit));
  }
  r.parts = std::max(1, r.parts);
  // Pieces of one tile would all run on the XCDs that its number gives (of lists that differ in
  // length some XCDs would have the long ones: 110 against 77 us for 32 requests of up to 8192), which
  // is as well where a request has many tiles that read the same keys (1.1 against 1.7 ms for 32 tiles).
  r.spread = r.parts > 1 && own == 1;
  r.piece = (most + r.parts - 1) / r.parts;
  r.parts = (most + r.piece - 1) / r.piece;
  if (r.parts > 1) {
    const size_t rows = size_t(r.parts) * tokens * q_heads;
    r.o = pad256(rows * p->d.head_dim * 4);
    r.ml = pad256(rows * 8);
  }
  if (mass_tokens > 0) r.row_ml = pad256(size_t(tokens) * q_heads * 8);
  return r;
}

template <int D, bool kF8>
hipError_t launch_dt(const KvGeom &g, const ChunkDev &p, hipStream_t s) {
  const bool wide = (1 << g.page_shift) >= 16;
  auto kernel = wide ? attn_prefill_kernel<D, kF8, true, 1> : attn_prefill_kernel<D, kF8, false, 1>;
  if constexpr (D == 64)
    if (p.bits > kRowBits) kernel = wide ? attn_prefill_kernel<D, kF8, true, 2> : attn_prefill_kernel<D, kF8, false, 2>;
  constexpr int shared = Tile<D, kF8>::kShared;
  const dim3 grid(unsigned(g.kv_heads), unsigned(std::min(p.tiles, kMostTiles)),
                  unsigned(p.parts > 1 ? p.parts : (p.tiles + kMostTiles - 1) / kMostTiles));
  hipLaunchKernelGGL(kernel, grid, dim3(kThreads), shared, s, ChunkArgsAll{g, p});
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && p.parts > 1) {
    const int heads = std::max<int64_t>(1, std::min<int64_t>(p.a.q_heads, int64_t(p.a.tokens) * p.a.q_heads >> 13));
    const int64_t waves = int64_t(p.a.tokens) * ((p.a.q_heads + heads - 1) / heads);
    hipLaunchKernelGGL((attn_prefill_join_kernel<D>), flat_grid((waves + kWaves - 1) / kWaves), dim3(kThreads), 0, s, g, p,
                       heads);
    e = hipGetLastError();
  }
  if (e == hipSuccess && p.a.mass_tokens > 0) {
    // the first block begins at or before the first place seen
    const int blocks = p.a.max_len / (kMassPlaces * kWaves) + 1;
    hipLaunchKernelGGL((attn_prefill_mass_kernel<D, kF8>), flat_grid(int64_t(p.a.batch) * g.kv_heads * blocks),
                       dim3(kThreads), 2 * kMassRows * 2 * D, s, g, p, blocks);
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
  const int64_t blocks = int64_t(max_len) / (kMassPlaces * kWaves) + 1;
  // rows of a request and tiles are counted in 31 bits, workgroups in 40
  return int64_t(tokens) * group < limit - 256 && chunk_tiles(batch, tokens, int(group)) < limit / p->d.kv_heads &&
         int64_t(batch) * p->d.kv_heads < (int64_t(1) << 40) / blocks;
}

size_t chunk_workspace(const gdn_kv_pool *p, int batch, int tokens, int q_heads, int max_len, int mass_tokens) {
  const ChunkPlan w = chunk_plan(p, batch, tokens, q_heads, max_len, mass_tokens);
  return w.o + w.ml + w.row_ml;
}

hipError_t launch_attn_prefill(const gdn_kv_pool *pool, int layer, const ChunkArgs &a, hipStream_t s) {
  const KvGeom g = kv_geom(pool, layer);
  ChunkDev p{};
  p.a = a;
  p.group = a.q_heads / pool->d.kv_heads;
  const ChunkPlan w = chunk_plan(pool, a.batch, a.tokens, a.q_heads, a.max_len, a.mass_tokens);
  p.inverse = uint32_t(((uint64_t(1) << 32) + p.group - 1) / p.group);
  p.tiles = int(w.tiles);
  p.bits = w.bits;
  p.parts = w.parts;
  p.piece = w.piece;
  p.spread = w.spread;
  p.c = fabsf(a.scale) * pool->d.k_scale * kLog2e;
  p.flip = std::signbit(a.scale) ? 0x80008000u : 0u;
  p.keep = p.c == 0.f ? 0u : ~0u;  // (a score of -inf must stay -inf where it is multiplied by c)
  p.c = p.c == 0.f ? 1.f : p.c;
  char *at = static_cast<char *>(a.workspace);
  p.o = reinterpret_cast<float *>(at);
  p.ml = reinterpret_cast<float *>(at += w.o);
  p.lse = a.lse;
  p.row_ml = a.mass_tokens > 0 ? reinterpret_cast<float *>(at + w.ml) : nullptr;
  const bool f8 = pool->d.kv_dtype == GDN_F8_E4M3;
  switch (pool->d.head_dim) {
    case 64: return launch_d<64>(g, p, f8, s);
    case 128: return launch_d<128>(g, p, f8, s);
    case 256: return launch_d<256>(g, p, f8, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace gdn
