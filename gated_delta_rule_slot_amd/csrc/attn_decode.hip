// attn_decode.hip -- attention of one new token per request over a paged key-value cache
// (formulas: include/gdn_kv.h), split over the cache's length and joined.
//
// Every key and value row is read once and used for the up to 16 query heads that share
// it: 4 * group flops for every element read, so the reads from memory bound it.  One pass
// keeps the running maximum m and sum l of the softmax per query head.
//
// A wave takes tiles of 32 tokens and needs no shared memory for them.
//   S^T = K Q^T   A = keys (rows = tokens), B = queries (columns = heads).  A lane gets,
//                 for head c = lane % 16 and group g = lane / 16, the scores of tokens
//                 4g + j and 16 + 4g + j (j < 4).
//   O^T = V^T P^T takes P^T as B with exactly those tokens as the lane's eight k
//                 indices (both operands use the order, so the sum is unchanged).  For A,
//                 the lane reads, of its eight tokens, the columns that belong to
//                 c, and picks one column of all eight by byte permutes.  So the values
//                 are read in whole rows and transposed in registers.
// The head is the lane's column in both products: m, l and the rescaling of O are
// lane-local, and only the maximum crosses lanes.
//
// P is carried as two bf16 parts (hi + lo, 16 bits): rounded once to bf16 its error would
// be about as large as the output's own rounding.  Both parts are positive, so an infinite
// value meets neither 0 nor two signs.  Scores, m, l and O are fp32.
//
// The work is counted in blocks of 128 tokens (4 waves, a tile each), in the order
// (request, key-value head, 16 query heads, position), and every workgroup takes an equal
// run of blocks: as many workgroups as run at once, whatever the requests' lengths.  (Equal
// splits of the longest length, at the best number of them, took 138 us for a ragged batch
// where equal runs took 131.)  A workgroup finds its run from the lengths on the device, walks
// it unit by unit, and joins its waves in shared memory at the end of each unit.  A unit that
// lies in one workgroup is final there; of the others m, l and O go to the workspace, and a
// second kernel joins them (and adds up the weights, from stored scores).
//
// Measured on MI355X (both kernels; scaling 4 GiB in place runs at 5.9 TB/s there): 4 requests of
// 90001-131072 tokens, 2 heads of 256, 956 MB: 152 us, 6.3 TB/s; 128 of 150-4099 tokens with
// weights, 547 MB: 106-114 us, 4.8-5.2 TB/s (join and weights 8.7 us of it); e4m3 in 16-token
// pages, 64 of 1000-8192 tokens in a 4096-token window, 8 heads of 128, 460 MB: 80-87 us; one
// of 777 tokens: 10.6 + 3.8 us, a chain of dependent reads (lengths, page ids, keys).
#include <algorithm>
#include <type_traits>

#include "kv.hpp"
#include "lanes.hpp"
#include "mfma.hpp"

namespace gdn {
namespace {

constexpr int kTile = 32;
constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;
constexpr float kNegInf = -__builtin_inff();

constexpr int kBlock = kTile * kWaves;  // tokens of a block
constexpr int kCUs = 256;

struct AttnDev {
  AttnArgs a;
  int head_blocks, group, workers;
  int join;         // whether the joining kernel runs (else every unit is one block at most)
  int64_t lpad;     // row length of the score array
  int32_t *unit;    // [units][2]: first and last worker of a unit, 2 w + (its first unit: 0, later: 1)
  float *o;         // [workers][2][16][D]: O of a worker's first and of its last unit
  float *ml;        // [workers][2][16][2]: their m and l
  float *done;      // [batch][q_heads][2]: m and l of units within one worker; with weights
  float *scores;    // [batch][q_heads][lpad], log2 units; with weights
};

// The visible range of request b and its number of blocks, 0 if it sees nothing (the reason
// is told by one caller).
struct Seen {
  int slot, begin, len, blocks;
};
__device__ __forceinline__ int blocks_of(const KvGeom &g, const AttnArgs &a, const Seen &r) {
  const bool ok = r.slot > 0 && r.slot < g.slots && r.len <= a.max_len && r.begin >= 0 && r.begin < r.len;
  return ok ? (r.len - (r.begin & ~(kTile - 1)) + kBlock - 1) / kBlock : 0;
}
__device__ __forceinline__ Seen seen_by(const KvGeom &g, const AttnArgs &a, int b, bool tell) {
  Seen r;
  r.slot = a.slot_table[b];
  r.len = a.kv_len[b];
  r.begin = a.kv_begin ? a.kv_begin[b] : 0;
  r.blocks = blocks_of(g, a, r);
  if (tell) {
    if (r.slot >= g.slots) set_err(g.err, GDN_ERRW_BAD_SLOT);
    else if (r.slot > 0 && (r.len < 0 || r.len > a.max_len || r.begin < 0)) set_err(g.err, GDN_ERRW_BAD_SEQLENS);
  }
  return r;
}

// First block of worker w.  (The host keeps the number of blocks below 2^31.)
__device__ __forceinline__ int first_block(int w, int all, int workers) { return int(int64_t(w) * all / workers); }
// A value that is the same in every lane, as a scalar.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Workgroup barrier that orders shared memory only: global loads issued before it stay in
// flight.
__device__ __forceinline__ void local_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// max / sum over the four 16-lane groups (same head), left in every lane
__device__ __forceinline__ float rows_max(float v) {
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float rows_sum(float v) {
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// Exponent's reference: a maximum of -inf (nothing seen yet) must not meet -inf - -inf.
__device__ __forceinline__ float ref(float m) { return m == kNegInf ? 0.f : m; }
// What a sum taken under the maximum m is worth under the larger maximum to.
__device__ __forceinline__ float factor(float m, float to) { return m == kNegInf ? 0.f : fexp2(m - to); }

// p >= 0 as two bf16 parts: its upper 16 bits, and the rest rounded to nearest (half a step of
// at most 2^-16 p).  The rest is taken of p (1 + 2^-23), so that it is above 0 for every p from
// 2^-103 on.
__device__ __forceinline__ Split split_weights(const float *p) {
  u32x4 h, l;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float rest[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float x = p[2 * i + e], hi = __uint_as_float(__float_as_uint(x) & 0xffff0000u);
      rest[e] = fmaf(x, 1.f + 0x1p-23f, -hi);
    }
    h[i] = halves(__float_as_uint(p[2 * i]), __float_as_uint(p[2 * i + 1]), 1);
    l[i] = cvt_pk_bf16(rest[0], rest[1]);
  }
  return Split{__builtin_bit_cast(bf16x8, h), __builtin_bit_cast(bf16x8, l)};
}

// How a lane reads rows of D values.  Keys: kPieces times 16 bytes, those of the four lane
// groups side by side; a piece of bf16 is the k indices of one MFMA step, one of e4m3 of
// two.  Values: kVPieces times kVWords words, the lane's D / 16 columns.
typedef uint32_t u32;
template <int D, bool kF8>
struct Lay;
template <int D>
struct Lay<D, false> {
  static constexpr int kSize = 2;
  static constexpr int kPieces = D / 32;       // 16-byte pieces of a key row per lane
  static constexpr int kVPieces = D == 256 ? 2 : 1;
  static constexpr int kVWords = D == 64 ? 2 : 4;  // words of one value piece
  // first dimension of step s for lane group g, and of a lane's value column i
  static __device__ __forceinline__ int kdim(int s, int g) { return 32 * s + 8 * g; }
  static __device__ __forceinline__ int vdim(int i, int c) {
    return D == 64 ? 4 * c + i : 128 * (i >> 3) + 8 * c + (i & 7);
  }
};
template <int D>
struct Lay<D, true> {
  static constexpr int kSize = 1;
  static constexpr int kPieces = D / 64;
  static constexpr int kVPieces = 1;
  static constexpr int kVWords = D / 64;
  static __device__ __forceinline__ int kdim(int s, int g) { return 64 * (s >> 1) + 16 * g + 8 * (s & 1); }
  static __device__ __forceinline__ int vdim(int i, int c) { return (D / 16) * c + i; }
};

template <int W>
struct Words {
  u32 w[W];
};
template <int W>
__device__ __forceinline__ Words<W> load_words(const char *p) {
  Words<W> r;
  if constexpr (W == 4) {
    const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
    r.w[0] = v[0]; r.w[1] = v[1]; r.w[2] = v[2]; r.w[3] = v[3];
  } else if constexpr (W == 2) {
    const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(p));
    r.w[0] = v[0]; r.w[1] = v[1];
  } else {
    r.w[0] = __builtin_nontemporal_load(reinterpret_cast<const u32 *>(p));
  }
  return r;
}
// four e4m3 values as two words of bf16 pairs (exact)
__device__ __forceinline__ void f8_to_bf16(u32 x, u32 *lo, u32 *hi) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  const f2 a = __builtin_amdgcn_cvt_pk_f32_fp8(int(x), false);
  const f2 b = __builtin_amdgcn_cvt_pk_f32_fp8(int(x), true);
  // an e4m3 value has 4 significant bits, so its fp32 form's low half is zero
  *lo = __builtin_amdgcn_perm(__float_as_uint(a[1]), __float_as_uint(a[0]), 0x07060302u);
  *hi = __builtin_amdgcn_perm(__float_as_uint(b[1]), __float_as_uint(b[0]), 0x07060302u);
}

// kWide: pages hold 16 tokens or more, so each half of a tile has adjacent rows and one
// wave-uniform page id; otherwise each token's row is looked up (128 requests of 2048 tokens,
// 4 heads of 128: 4-token pages 96.8 us, 16-token pages 91.3 us).
//
// The keys and values of a wave's next tile are asked for while the present one is worked
// on, also over the end of a unit: under load a dependent read takes 5 us and more, so a
// unit that began with its own reads of queries, page ids and keys cost about 8 us each time.
// kMass: scores are stored for the weights, 1: of up to 8 heads, 2: of up to 16.
//
// Registers: up to 255 VGPRs at two waves a SIMD.  The two forms of bf16, head dim 256, pages
// below 16 tokens and weights spill 4 of them (20 bytes a lane); no other spills.
template <int D, bool kF8, bool kWide, int kMass>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2)))
void attn_decode_kernel(KvGeom g, AttnDev p) {
  using L = Lay<D, kF8>;
  constexpr int KS = D / 32;        // MFMA steps of a score
  constexpr int NO = D / 16;        // 16-column tiles of O
  constexpr int VW = D / 32;        // bf16 words of a lane's columns of one token
  constexpr int RB = D * L::kSize;  // bytes of a row
  // O in shared memory, per wave: 16 bytes (o[i]) of each lane, for each i; a step of 4 floats
  // between the lane groups and an odd one (in 16 bytes) between the i keep the banks apart
  constexpr int kOi = 69 * 4, kSlab = NO * kOi;
  // scores of a tile there, by head (36 floats apart for the banks), and how many tiles fit
  constexpr int kScoreRow = 36, kScoreTile = 8 * (kMass ? kMass : 1) * kScoreRow, kStaged = kSlab / kScoreTile;
  // head dim 256: the queries stay in shared memory (their 32 registers would spill)
  constexpr bool kQShared = D == 256;
  constexpr int kQLoads = kQShared ? KS / kWaves : KS;
  extern __shared__ __attribute__((aligned(16))) float lds[];
  __shared__ float sm[kWaves][16], sl[kWaves][16];
  __shared__ u32x4 sq[kQShared ? KS : 1][64];

  const int lane = threadIdx.x & 63, c = lane & 15, gr = lane >> 4;
  const int wave = uniform(threadIdx.x >> 6);
  const int worker = blockIdx.x;
  const int units = g.kv_heads * p.head_blocks;  // of a request

  // (constant address space: these arrays do not change during the call, so wave-uniform
  // reads are scalar loads, which the waits for keys and values do not count)
  typedef const int32_t __attribute__((address_space(4))) *table_t;
  auto request = [&](int r) -> Seen {
    Seen v;
    v.slot = ((table_t)p.a.slot_table)[r];
    v.len = ((table_t)p.a.kv_len)[r];
    v.begin = p.a.kv_begin ? ((table_t)p.a.kv_begin)[r] : 0;
    v.blocks = blocks_of(g, p.a, v);
    return v;
  };

  // ---- this worker's run of blocks, by each wave for itself: lane i has four requests ----
  Seen four[4];
  int inc = 0;
  auto scan = [&](int base) -> int {
    int mine = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = base + 4 * lane + i;
      four[i] = seen_by(g, p.a, min(r, p.a.batch - 1), false);
      if (r >= p.a.batch) four[i].blocks = 0;
      mine += four[i].blocks;
    }
    inc = int(wave_scan(uint32_t(mine)));
    const int sum = __builtin_amdgcn_readlane(inc, 63);
    inc -= mine;  // of the lanes before
    return sum;
  };
  int all = 0;
  for (int base = 0; base < p.a.batch; base += 256) all += scan(base);
  const int last_sum = all;  // of the only step, if the batch fits one
  all *= units;
  const int sharing = min(p.workers, all);  // so that no worker between two others has nothing
  const int run_first = worker < sharing ? first_block(worker, all, sharing) : 0;
  int left = worker < sharing ? first_block(worker + 1, all, sharing) - run_first : 0;

  // A unit's part of the run: request b, key-value head h, query heads q0 .. q0 + heads - 1,
  // tokens first .. last - 1.
  struct Part {
    int b, unit, blk, nblk;
    Seen rq;
    int h, heads, q0, first, last;
  };
  auto part = [&](int b, int unit, int blk, const Seen &rq, int most) -> Part {
    Part r;
    r.b = b;
    r.unit = unit;
    r.blk = blk;
    r.rq = rq;
    r.nblk = min(rq.blocks - blk, most);
    r.h = unit / p.head_blocks;
    const int hb = unit - r.h * p.head_blocks;
    r.heads = min(16, p.group - 16 * hb);
    r.q0 = r.h * p.group + 16 * hb;
    r.first = (rq.begin & ~(kTile - 1)) + blk * kBlock;
    r.last = min(rq.len, r.first + r.nblk * kBlock);
    return r;
  };

  // Rows of a tile.  A token that is not visible, or whose page id is not a page, reads
  // page 0's rows (always there) and is masked by its bit of `seen`; of a tile without visible
  // tokens (a wave's next one at the end of its run) all lanes read the same few bytes.
  struct Rows {
    int row[2];  // kWide: first row of each half; else row[0] of lane i < 32: row of token t0 + i
    u32 seen;
  };
  struct Pages {
    int id[2];   // kWide: of each half; else id[0] of lane i < 32: of token t0 + i
  };
  const int in_page = (1 << g.page_shift) - 1;
  // The page ids are asked for a tile before their rows are (and, where the reads are not
  // scalar, before that tile's keys: loads return in order).
  auto ask = [&](const Part &u, int t0) -> Pages {
    const table_t table = (table_t)(g.page_table + int64_t(u.rq.slot) * g.max_pages);
    if constexpr (kWide)
      return Pages{{table[max(0, min(t0, u.last - 1)) >> g.page_shift],
                    table[max(0, min(t0 + 16, u.last - 1)) >> g.page_shift]}};
    else return Pages{{table[max(0, max(u.rq.begin, min(t0 + (lane & 31), u.last - 1))) >> g.page_shift], 0}};
  };
  auto resolve = [&](int h, int begin, int last, int t0, const Pages &pages) -> Rows {
    Rows r;
    if constexpr (kWide) {
      u32 m = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int t = t0 + 16 * u, page = pages.id[u];
        const bool in = t < last && t + 16 > begin, ok = page > 0 && page < g.pages;
        if (in && !ok && lane == 0) set_err(g.err, GDN_ERRW_BAD_PAGE);
        r.row[u] = in && ok ? ((page * g.kv_heads + h) << g.page_shift) + (t & in_page) : 0;
        m |= in && ok ? 0xffffu << (16 * u) : 0u;
      }
      // bits from begin on, and below last
      if (begin > t0) m &= begin - t0 >= 32 ? 0u : 0xffffffffu << (begin - t0);
      if (last - t0 < 32) m &= last > t0 ? (1u << (last - t0)) - 1u : 0u;
      r.seen = m;
    } else {
      const int t = t0 + (lane & 31), page = pages.id[0];
      const bool in = t >= begin && t < last;
      const bool ok = in && page > 0 && page < g.pages;
      if (__any(in && !ok)) {
        if (lane == 0) set_err(g.err, GDN_ERRW_BAD_PAGE);
      }
      r.row[0] = ok ? ((page * g.kv_heads + h) << g.page_shift) + (t & in_page) : 0;
      r.row[1] = 0;
      r.seen = u32(__ballot(ok));  // lanes 32 up repeat the lower ones
    }
    return r;
  };

  Words<4> kw[2][L::kPieces];
  Words<L::kVWords> vw[8][L::kVPieces];
  // (lane offsets are made anew for each use: held, they cost the last registers of head dim
  // 256, and a spilled one is read back in order behind the keys that were just asked for)
  auto lane_anew = []() -> int {
    int v = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0));
    asm volatile("" : "+v"(v));
    return v;
  };
  auto load_k = [&](const Rows &r) {
    const int ln = lane_anew();
    const u32 k_off = r.seen ? u32((ln & 15) * RB + 16 * (ln >> 4)) : 0u;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const char *at;
      if constexpr (kWide) at = g.k + int64_t(r.row[u]) * RB + k_off;
      else at = g.k + int64_t(__shfl(r.row[0], 16 * u + (ln & 15))) * RB + 16 * (ln >> 4);
#pragma unroll
      for (int s = 0; s < L::kPieces; ++s) kw[u][s] = load_words<4>(at + 64 * s);
    }
  };
  auto load_v = [&](const Rows &r) {
    const int ln = lane_anew();
    const u32 v_off = r.seen ? u32(4 * (ln >> 4) * RB + 4 * L::kVWords * (ln & 15)) : 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const char *at;
      if constexpr (kWide) at = g.v + int64_t(r.row[e >> 2]) * RB + (e & 3) * RB + v_off;
      else at = g.v + int64_t(__shfl(r.row[0], pk(ln >> 4, e))) * RB + 4 * L::kVWords * (ln & 15);
#pragma unroll
      for (int s = 0; s < L::kVPieces; ++s) vw[e][s] = load_words<L::kVWords>(at + 256 * s);
    }
  };
  // queries as the B operand (columns past the group are zero)
  auto load_q = [&](const Part &u, bf16x8 *qf) {
    const uint16_t *q = p.a.q + int64_t(u.b) * p.a.q_stride + int64_t(u.q0 + min(c, u.heads - 1)) * D;
#pragma unroll
    for (int i = 0; i < kQLoads; ++i)
      qf[i] = *reinterpret_cast<const bf16x8 *>(q + L::kdim(kQShared ? wave * kQLoads + i : i, gr));
  };

  constexpr int kStep = kBlock;
  const float to_log2 = p.a.scale * g.k_scale * kLog2e;
  if (left > 0) {
    // ---- find the run's first block -----------------------------------------------
    const int x = run_first / units;
    int b = 0, lo = 0;
    Seen rq{0, 0, 0, 0};
    for (int base = 0; base < p.a.batch; base += 256) {
      const int sum = p.a.batch > 256 ? scan(base) : last_sum;
      if (x < lo + sum) {
        // the last lane whose requests begin at or before x, and of its four the holder
        const int at = 63 - __clzll(__ballot(lo + inc <= x));
        lo += __builtin_amdgcn_readlane(inc, at);
        bool found = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const Seen v{__builtin_amdgcn_readlane(four[i].slot, at), __builtin_amdgcn_readlane(four[i].begin, at),
                       __builtin_amdgcn_readlane(four[i].len, at), __builtin_amdgcn_readlane(four[i].blocks, at)};
          if (found) continue;
          if (x < lo + v.blocks) {
            found = true;
            b = base + 4 * at + i;
            rq = v;
          } else {
            lo += v.blocks;
          }
        }
        break;
      }
      lo += sum;
    }
    const int in_request = run_first - lo * units;
    const int unit0 = in_request / rq.blocks;
    Part cur = part(b, unit0, in_request - unit0 * rq.blocks, rq, left);

    bf16x8 qf[kQLoads];
    load_q(cur, qf);
    __builtin_amdgcn_sched_barrier(0);
    int t0 = cur.first + kTile * wave;
    Pages page1;
    Rows now;
    {
      const Pages page0 = ask(cur, t0);
      page1 = ask(cur, t0 + kStep);
      now = resolve(cur.h, cur.rq.begin, cur.last, t0, page0);
      load_k(now);
      load_v(now);
    }
    __builtin_amdgcn_sched_barrier(0);
    bool first_unit = true;
    while (true) {
      if constexpr (kQShared) {
#pragma unroll
        for (int i = 0; i < kQLoads; ++i) {
          if (c >= cur.heads) qf[i] = bf16x8{};
          sq[wave * kQLoads + i][lane] = __builtin_bit_cast(u32x4, qf[i]);
        }
        local_barrier();
      } else {
#pragma unroll
        for (int i = 0; i < kQLoads; ++i)
          if (c >= cur.heads) qf[i] = bf16x8{};
      }
      // ---- the part after this one (or this one again, unused), its queries and pages -------
      left -= cur.nblk;
      Part nx = cur;
      if (left > 0) {
        int nb = cur.b, nu = cur.unit + 1;
        Seen nr = cur.rq;
        if (nu == units) {
          nu = 0;
          nr.blocks = 0;
          while (nr.blocks == 0 && ++nb < p.a.batch) nr = request(nb);
        }
        // (there always is one, unless the lengths change under the call; then the run ends)
        if (nr.blocks > 0) nx = part(nb, nu, 0, nr, left);
        else left = 0;
      }
      const int nx_last = left > 0 ? nx.last : 0;
      const int nt0 = nx.first + kTile * wave;
      bf16x8 qn[kQLoads];
      load_q(nx, qn);
      const Pages npage0 = ask(nx, nt0), npage1 = ask(nx, nt0 + kStep);

      f32x4 o[NO];
#pragma unroll
      for (int i = 0; i < NO; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
      float m = kNegInf, l = 0.f;
      int staged = 0;  // tiles whose scores are in shared memory
      const int64_t qrow = int64_t(cur.b) * p.a.q_heads + cur.q0;

      // ---- tiles ------------------------------------------------------------------
      // (a wave without a tile in this part takes one in which no token is seen: one place
      // in the code asks for keys and values, so their registers are never copied)
      {
        bool inside;  // the wave's next tile is of this part
        do {
          inside = t0 + kStep < cur.last;
          const int lane = lane_anew(), c = lane & 15, gr = lane >> 4;
          const Rows next = resolve(inside ? cur.h : nx.h, inside ? cur.rq.begin : nx.rq.begin,
                                    inside ? cur.last : nx_last, inside ? t0 + kStep : nt0, inside ? page1 : npage0);
          // scores
          f32x4 s[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
          for (int st = 0; st < KS; ++st) {
            bf16x8 qv;
            if constexpr (kQShared) qv = __builtin_bit_cast(bf16x8, sq[st][lane]);
            else qv = qf[st];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              u32x4 w;
              if constexpr (kF8) {
                const u32 x0 = kw[u][st >> 1].w[2 * (st & 1)], x1 = kw[u][st >> 1].w[2 * (st & 1) + 1];
                u32 a0, a1, a2, a3;
                f8_to_bf16(x0, &a0, &a1);
                f8_to_bf16(x1, &a2, &a3);
                w = u32x4{a0, a1, a2, a3};
              } else {
                w = u32x4{kw[u][st].w[0], kw[u][st].w[1], kw[u][st].w[2], kw[u][st].w[3]};
              }
              s[u] = mfma_bf16(__builtin_bit_cast(bf16x8, w), qv, s[u]);
            }
          }
          // (the barriers keep the next tile's loads behind the last use of their registers)
          __builtin_amdgcn_sched_barrier(0);
          page1 = inside ? ask(cur, t0 + 2 * kStep) : npage1;
          load_k(next);
          __builtin_amdgcn_sched_barrier(0);

          // softmax
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = s[e >> 2][e & 3] * to_log2;
          const u32 seen = now.seen;
          const bool whole = seen == 0xffffffffu;
          if (!whole) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = (seen >> pk(gr, e)) & 1 ? x[e] : kNegInf;
          }
          float mx =
              fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
          mx = fmaxf(rows_max(mx), m);
          if (__any(mx > m)) {  // some head's maximum grew
            const float f = factor(m, mx);
            l *= f;
#pragma unroll
            for (int i = 0; i < NO; ++i) o[i] *= f;
            m = mx;
          }
          float pr[8];
          const float base = ref(m);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            pr[e] = fexp2(x[e] - base);
            l += pr[e];
          }
          const Split ps = split_weights(pr);

          // values: columns of eight tokens by byte permutes
          if (!whole) {  // never 0 * inf
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const bool on = (seen >> pk(gr, e)) & 1;
#pragma unroll
              for (int q = 0; q < L::kVPieces; ++q)
#pragma unroll
                for (int w = 0; w < L::kVWords; ++w) vw[e][q].w[w] = on ? vw[e][q].w[w] : 0u;
            }
          }
#pragma unroll
          for (int w = 0; w < VW; ++w) {
            u32 word[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              if constexpr (kF8) {
                u32 lo8, hi8;
                f8_to_bf16(vw[e][0].w[w >> 1], &lo8, &hi8);
                word[e] = (w & 1) ? hi8 : lo8;
              } else {
                word[e] = vw[e][w / L::kVWords].w[w % L::kVWords];
              }
            }
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const u32x4 col = {halves(word[0], word[1], hf), halves(word[2], word[3], hf),
                                 halves(word[4], word[5], hf), halves(word[6], word[7], hf)};
              const bf16x8 av = __builtin_bit_cast(bf16x8, col);
              o[2 * w + hf] = mfma_bf16(av, ps.lo, o[2 * w + hf]);
              o[2 * w + hf] = mfma_bf16(av, ps.hi, o[2 * w + hf]);
            }
          }
          __builtin_amdgcn_sched_barrier(0);
          load_v(next);
          __builtin_amdgcn_sched_barrier(0);
          // Scores for the weights: kept in the wave's part of the shared memory that O takes
          // at the end, and stored to memory some tiles at a time.  (Stores count in order with
          // the loads and take longer: one in every tile, wherever it stood, cost 15 of 120 us
          // for 128 requests of 2100 tokens.)
          if constexpr (kMass != 0) {
            f32x4 lo4 = {x[0], x[1], x[2], x[3]}, hi4 = {x[4], x[5], x[6], x[7]};
            const int head = kMass == 1 ? c & 7 : c;
            float *const own = lds + wave * kSlab + head * kScoreRow + 4 * gr + (kMass == 1 ? 2 * (c & 8) : 0);
            if constexpr (kMass == 1) {  // up to 8 heads: lanes 8 up of 16 take the second half
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float r = dpp_mov<0x128>(hi4[e]);  // row_ror 8
                lo4[e] = c < 8 ? lo4[e] : r;
              }
              st4(own + staged * kScoreTile, lo4);
            } else {
              st4(own + staged * kScoreTile, lo4);
              st4(own + staged * kScoreTile + 16, hi4);
            }
            ++staged;
            if (staged == kStaged || !inside) {
              if (head < cur.heads) {
                float *at = p.scores + (qrow + head) * p.lpad + (t0 - (staged - 1) * kStep) + 4 * gr +
                            (kMass == 1 ? 2 * (c & 8) : 0);
                // (the one tile of a wave without tokens in this part stays out)
                for (int k = 0; k < staged && t0 < cur.last; ++k) {
                  st4(at + k * kStep, ld4(own + k * kScoreTile));
                  if constexpr (kMass == 2) st4(at + k * kStep + 16, ld4(own + k * kScoreTile + 16));
                }
              }
              staged = 0;
            }
          }
          now = next;
          t0 += kStep;
        } while (inside);
      }

      // ---- join the waves: o[i][j] is column vdim(i, 4 gr + j) of head c ------------------
      const int lane = lane_anew(), c = lane & 15, gr = lane >> 4;
      l = rows_sum(l);
      if (gr == 0) {
        sm[wave][c] = m;
        sl[wave][c] = l;
      }
      {
        float *at = lds + wave * kSlab + 4 * (lane + gr);
#pragma unroll
        for (int i = 0; i < NO; ++i) st4(at + i * kOi, o[i]);
      }
      local_barrier();
      const bool whole_unit = cur.nblk == cur.rq.blocks;
      const int side = first_unit ? 0 : 1;
      // a thread takes kJ rows j0 up of four columns (4 q up) of its lane's head: 4 adjacent
      // values of O for each j
      if (c < cur.heads) {
        constexpr int kJ = NO / 4;
        typedef float vec_j __attribute__((ext_vector_type(kJ)));
        const int q = wave * kJ / 4, j0 = wave * kJ % 4;
        float mh = sm[0][c], lt = 0.f;
#pragma unroll
        for (int w = 1; w < kWaves; ++w) mh = fmaxf(mh, sm[w][c]);
        float sum[4][kJ];
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int r = 0; r < kJ; ++r) sum[e][r] = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          const float f = factor(sm[w][c], mh);
          lt = fmaf(sl[w][c], f, lt);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float *at = lds + w * kSlab + (4 * q + e) * kOi + 4 * (lane + gr) + j0;
            vec_j v;
            if constexpr (kJ == 1) v[0] = *at;
            else v = *reinterpret_cast<const vec_j *>(at);
#pragma unroll
            for (int r = 0; r < kJ; ++r) sum[e][r] = fmaf(v[r], f, sum[e][r]);
          }
        }
        const bool teller = wave == 0 && gr == 0;
        if (!whole_unit) {
          const int64_t row = (int64_t(worker) * 2 + side) * 16 + c;
#pragma unroll
          for (int r = 0; r < kJ; ++r)
            st4(p.o + row * D + L::vdim(4 * q, 4 * gr + j0 + r), f32x4{sum[0][r], sum[1][r], sum[2][r], sum[3][r]});
          if (teller) {
            p.ml[2 * row] = mh;
            p.ml[2 * row + 1] = lt;
          }
        } else {
          // (every score -inf: 0, where the sum may be 0 times a NaN or an infinity)
          const float inv = g.v_scale / lt;
          const u32 any = lt == 0.f ? 0u : ~0u;
#pragma unroll
          for (int r = 0; r < kJ; ++r)
            *reinterpret_cast<u32x2 *>(p.a.out + (qrow + c) * D + L::vdim(4 * q, 4 * gr + j0 + r)) =
                u32x2{any & cvt_pk_bf16(sum[0][r] * inv, sum[1][r] * inv),
                      any & cvt_pk_bf16(sum[2][r] * inv, sum[3][r] * inv)};
          if (teller) {
            if (p.a.lse) p.a.lse[qrow + c] = lt == 0.f ? kNegInf : (mh + log2f(lt)) * kLn2;
            if (kMass) {
              p.done[2 * (qrow + c)] = mh;
              p.done[2 * (qrow + c) + 1] = lt;
            }
          }
        }
      }
      if (p.join && threadIdx.x == 0) {  // where the parts of a unit lie, for the joining kernel
        int32_t *at = p.unit + 2 * (int64_t(cur.b) * units + cur.unit);
        if (cur.blk == 0) at[0] = 2 * worker + side;
        if (cur.blk + cur.nblk == cur.rq.blocks) at[1] = 2 * worker + side;
      }
      if (left <= 0) break;
      local_barrier();  // the shared arrays are free again
      cur = nx;
      t0 = nt0;
      first_unit = false;
#pragma unroll
      for (int i = 0; i < kQLoads; ++i) qf[i] = qn[i];
    }
  }

  // ---- requests that see nothing, dealt out to the workers ------------------------
  for (int e = worker; e < p.a.batch; e += p.workers) {
    if (seen_by(g, p.a, e, threadIdx.x == 0).blocks) continue;
    const int64_t row = int64_t(e) * p.a.q_heads;
    for (int i = threadIdx.x; i < p.a.q_heads * (D / 8); i += kThreads)
      reinterpret_cast<u32x4 *>(p.a.out + row * D)[i] = u32x4{0, 0, 0, 0};
    for (int i = threadIdx.x; p.a.lse && i < p.a.q_heads; i += kThreads) p.a.lse[row + i] = kNegInf;
    for (int i = threadIdx.x; p.join && i < 2 * units; i += kThreads) p.unit[2 * int64_t(e) * units + i] = 0;
  }
}

// Joins the parts of each (request, query head) that more than one worker had, and adds
// the weights
//   mass[t] += sum over the group's heads of 2^(score - m) / l.
// Workgroups: with weights first one per kMassTokens tokens of each (request, key-value
// head), then one per (request, query head).
constexpr int kMassTokens = 1024;

// The workers w0 .. w1 of a unit.  Only w0's part may be a later unit of its run: a worker
// that goes on with a unit begins with it.
struct Parts {
  int w0, w1, side;
  __device__ __forceinline__ int64_t row(int w, int head) const {
    return (int64_t(w) * 2 + (w == w0 ? side : 0)) * 16 + head;
  }
};
__device__ __forceinline__ Parts parts_of(const KvGeom &g, const AttnDev &p, int b, int unit) {
  const int32_t *at = p.unit + 2 * (int64_t(b) * g.kv_heads * p.head_blocks + unit);
  return Parts{at[0] >> 1, at[1] >> 1, at[0] & 1};
}
// m and l of a head over the parts, by the lanes of a wave
__device__ __forceinline__ void join_ml(const float *ml, const Parts &pt, int head, int lane, float *m, float *l) {
  float mm = kNegInf, ll = 0.f;
  for (int w = pt.w0 + lane; w <= pt.w1; w += 64) mm = fmaxf(mm, ml[2 * pt.row(w, head)]);
  for (int x = 32; x; x >>= 1) mm = fmaxf(mm, __shfl_xor(mm, x));
  for (int w = pt.w0 + lane; w <= pt.w1; w += 64) {
    const float *e = ml + 2 * pt.row(w, head);
    ll = fmaf(e[1], factor(e[0], mm), ll);
  }
  *m = mm;
  *l = wave_sum(ll);
}

template <int D>
__global__ __launch_bounds__(kThreads) void attn_join_kernel(KvGeom g, AttnDev p, int mass_blocks) {
  __shared__ __attribute__((aligned(16))) float acc[kWaves][D];
  __shared__ float hm[64], hl[64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // (the weights' workgroups come first: they take longer)
  const int64_t id = flat_block(), masses = int64_t(p.a.batch) * g.kv_heads * mass_blocks;
  if (id >= masses) {
    if (id - masses >= int64_t(p.a.batch) * p.a.q_heads) return;
    const int qr = int(id - masses), b = qr / p.a.q_heads, qh = qr - b * p.a.q_heads;
    const int h = qh / p.group, j = qh - h * p.group;  // head j of the group
    const Parts pt = parts_of(g, p, b, h * p.head_blocks + (j >> 4));
    if (pt.w1 <= pt.w0) return;  // nothing, or final already
    // every wave takes each fourth part, four of them at a time under their common maximum
    constexpr int C = D / 64;  // columns of a lane
    typedef float vec_c __attribute__((ext_vector_type(C)));
    float m = kNegInf, l = 0.f, sum[C];
#pragma unroll
    for (int i = 0; i < C; ++i) sum[i] = 0.f;
    for (int w = pt.w0 + wave; w <= pt.w1; w += 4 * kWaves) {
      float mw[4], lw[4];
      vec_c ow[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t r = pt.row(min(w + k * kWaves, pt.w1), j & 15);
        mw[k] = p.ml[2 * r];
        lw[k] = p.ml[2 * r + 1];
        ow[k] = *reinterpret_cast<const vec_c *>(p.o + r * D + C * lane);
      }
      float mt = m;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (w + k * kWaves > pt.w1) mw[k] = kNegInf, lw[k] = 0.f, ow[k] = vec_c(0.f);
        mt = fmaxf(mt, mw[k]);
      }
      const float f0 = factor(m, mt);
      l *= f0;
#pragma unroll
      for (int i = 0; i < C; ++i) sum[i] *= f0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float f = factor(mw[k], mt);
        l = fmaf(lw[k], f, l);
#pragma unroll
        for (int i = 0; i < C; ++i) sum[i] = fmaf(ow[k][i], f, sum[i]);
      }
      m = mt;
    }
#pragma unroll
    for (int i = 0; i < C; ++i) acc[wave][C * lane + i] = sum[i];
    if (lane == 0) {
      hm[wave] = m;
      hl[wave] = l;
    }
    local_barrier();
    m = hm[0];
    l = 0.f;
#pragma unroll
    for (int w = 1; w < kWaves; ++w) m = fmaxf(m, hm[w]);
    float f[kWaves];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      f[w] = factor(hm[w], m);
      l = fmaf(hl[w], f[w], l);
    }
    const float inv = g.v_scale / l;
    if (int(threadIdx.x) < D / 2) {  // two columns a thread
      float t0 = 0.f, t1 = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        t0 = fmaf(acc[w][2 * threadIdx.x], f[w], t0);
        t1 = fmaf(acc[w][2 * threadIdx.x + 1], f[w], t1);
      }
      reinterpret_cast<u32 *>(p.a.out + int64_t(qr) * D)[threadIdx.x] = l == 0.f ? 0u : cvt_pk_bf16(t0 * inv, t1 * inv);
    }
    if (p.a.lse && threadIdx.x == 0) p.a.lse[qr] = l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
    return;
  }
  const int block = int(id % mass_blocks), bh = int(id / mass_blocks);
  const int h = bh % g.kv_heads, b = bh / g.kv_heads;
  const Seen rq = seen_by(g, p.a, b, false);
  const int64_t from = int64_t(rq.begin & ~3) + int64_t(block) * kMassTokens;
  if (rq.blocks == 0 || from >= rq.len) return;
  const int64_t qr0 = int64_t(b) * p.a.q_heads + h * p.group;
  // the scores of the first heads and the weights so far are asked for before the heads' m
  // and l are known
  constexpr int kAhead = 8;
  const int64_t t = from + 4 * threadIdx.x;
  const bool on = t < rq.len;
  const float *sc = p.scores + qr0 * p.lpad + (on ? t : from);
  float *mass = g.mass + (int64_t(rq.slot) * g.kv_heads + h) * g.capacity;
  f32x4 x[kAhead];
#pragma unroll
  for (int j = 0; j < kAhead; ++j) x[j] = ld4(sc + min(j, p.group - 1) * p.lpad);
  float sum[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) sum[e] = mass[min(t + e, int64_t(rq.len) - 1)];
  const Parts whole = parts_of(g, p, b, h * p.head_blocks);
  if (p.head_blocks == 1 && whole.w1 - whole.w0 < 8) {  // the usual case: 8 lanes a head
    const int j = threadIdx.x >> 3, w = whole.w0 + (threadIdx.x & 7);
    float m = kNegInf, l = 0.f;
    if (j < p.group && w <= whole.w1) {
      const float *e = whole.w1 > whole.w0 ? p.ml + 2 * whole.row(w, j) : p.done + 2 * (qr0 + j);
      m = e[0];
      l = e[1];
    }
    float mm = fmaxf(m, dpp_mov<0xB1>(m));
    mm = fmaxf(mm, dpp_mov<0x4E>(mm));
    mm = fmaxf(mm, dpp_mov<0x141>(mm));
    l = group_sum<8>(l * factor(m, mm));
    if (j < p.group && (threadIdx.x & 7) == 0) {
      hm[j] = ref(mm);
      hl[j] = l == 0.f ? 0.f : 1.f / l;
    }
  } else for (int j = wave; j < p.group; j += kWaves) {
    const Parts pt = parts_of(g, p, b, h * p.head_blocks + (j >> 4));
    float m, l;
    if (pt.w1 > pt.w0) {
      join_ml(p.ml, pt, j & 15, lane, &m, &l);
    } else {
      m = p.done[2 * (qr0 + j)];
      l = p.done[2 * (qr0 + j) + 1];
    }
    if (lane == 0) {
      hm[j] = ref(m);
      hl[j] = l == 0.f ? 0.f : 1.f / l;
    }
  }
  local_barrier();
  f32x4 add = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < kAhead; ++j)
    if (j < p.group)
#pragma unroll
      for (int e = 0; e < 4; ++e) add[e] = fmaf(fexp2(x[j][e] - hm[j]), hl[j], add[e]);
#pragma unroll 4
  for (int j = kAhead; j < p.group; ++j) {
    const f32x4 y = ld4(sc + j * p.lpad);
#pragma unroll
    for (int e = 0; e < 4; ++e) add[e] = fmaf(fexp2(y[e] - hm[j]), hl[j], add[e]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (on && t + e >= rq.begin && t + e < rq.len) mass[t + e] = sum[e] + add[e];
}

size_t pad256(size_t n) { return (n + 255) & ~size_t(255); }
int64_t score_row(int max_len) { return (int64_t(max_len) + kTile - 1) / kTile * kTile; }

template <int D, bool kF8>
hipError_t launch_dt(const KvGeom &g, const AttnDev &p, hipStream_t s) {
  const size_t lds = size_t(kWaves) * (D / 16) * 69 * 16;
  const bool wide = (1 << g.page_shift) >= 16;
  const int mass = !p.scores ? 0 : p.group <= 8 ? 1 : 2;
  typedef void (*kernel_t)(KvGeom, AttnDev);
  static const kernel_t kernels[2][3] = {
      {attn_decode_kernel<D, kF8, false, 0>, attn_decode_kernel<D, kF8, false, 1>, attn_decode_kernel<D, kF8, false, 2>},
      {attn_decode_kernel<D, kF8, true, 0>, attn_decode_kernel<D, kF8, true, 1>, attn_decode_kernel<D, kF8, true, 2>}};
  const kernel_t kernel = kernels[wide][mass];
  hipLaunchKernelGGL(kernel, dim3(unsigned(p.workers)), dim3(kThreads), lds, s, g, p);
  return hipGetLastError();
}

template <int D>
hipError_t launch_d(const KvGeom &g, const AttnDev &p, bool f8, hipStream_t s) {
  const int mass_blocks = p.scores ? (p.a.max_len + 3 + kMassTokens - 1) / kMassTokens : 0;
  const int64_t joins = int64_t(p.a.batch) * p.a.q_heads + int64_t(p.a.batch) * g.kv_heads * mass_blocks;
  hipError_t e = f8 ? launch_dt<D, true>(g, p, s) : launch_dt<D, false>(g, p, s);
  if (e != hipSuccess || !p.join) return e;
  hipLaunchKernelGGL((attn_join_kernel<D>), flat_grid(joins), dim3(kThreads), 0, s, g, p, mass_blocks);
  return hipGetLastError();
}

// Blocks of a unit of max_len tokens (its first tile may begin before the first one seen).
int64_t unit_blocks(int max_len) { return std::max<int64_t>(1, (int64_t(max_len) + kTile - 1 + kBlock - 1) / kBlock); }

// Workers of a call: one per compute unit, or fewer where there are not that many blocks.  Its
// 4 waves keep a tile of keys and values each in flight: 128 KB with rows of 512 bytes (bf16,
// head dim 256), 16 KB with rows of 64 (e4m3, head dim 64).  Measured with one and two per
// compute unit, us, in pages of 4, 16, 32, 64 and 128 tokens:
//   rows of 64 bytes      two gain wherever there is work for both: 64 requests of 4096 tokens, 8
//                         heads (66 blocks per compute unit): 93 / 61, 63 / 49, 69 / 49, 62 / 48,
//                         62 / 48; 17 blocks: 21 / 19.5, 8: 16.3 / 14.7; 4 blocks: 14.4 / 16.7
//   rows of 128 bytes     the same call in e4m3: 122 / 98, 131 / 90, then 88 / 88; in bf16 108 / 100,
//                         101 / 88 (lengths of 4000 to 4096), then 86 / 86.  A head's run in a page
//                         is short there, and the workers meet on few memory channels at a time.
//                         At 17 blocks two gain in pages of 4 (33 / 29.4) and lose in others (28.6 /
//                         30.2, 27.3 / 30.0)
//   256 and 512 bytes     one is as good or better: 164 / 166, 320 / 320; at 17 blocks 45 / 48, 86 / 90;
//                         pages of 4 tokens of 256 bytes 190 / 179, at 8 blocks 31.1 / 32.5
int attn_workers(const gdn_kv_pool *p, int batch, int q_heads, int max_len) {
  const int group = q_heads / p->d.kv_heads;
  const int64_t units = int64_t(batch) * p->d.kv_heads * ((group + 15) / 16);
  const int64_t blocks = units * unit_blocks(max_len);
  const bool small = p->row_bytes <= 64 || (p->d.page_size < 16 && p->row_bytes <= 128);
  const bool two = blocks >= 8 * kCUs && (small || (blocks >= 32 * kCUs && p->d.page_size * p->row_bytes <= 2048));
  return int(std::max<int64_t>(1, std::min<int64_t>(kCUs * (two ? 2 : 1), blocks)));
}

// One block per unit at most: no unit is ever divided.
bool attn_joins(int max_len, uint32_t flags) { return max_len > kBlock || (flags & GDN_F_ACCUM_MASS); }

// Parts of the workspace, in order.
struct AttnSpace {
  size_t unit, o, ml, done, scores;
};
AttnSpace attn_space(const gdn_kv_pool *p, int batch, int q_heads, int max_len, uint32_t flags) {
  AttnSpace r{};
  if (!attn_joins(max_len, flags)) return r;
  const size_t parts = size_t(attn_workers(p, batch, q_heads, max_len)) * 2 * 16, rows = size_t(batch) * q_heads;
  r.unit = pad256(size_t(batch) * p->d.kv_heads * ((q_heads / p->d.kv_heads + 15) / 16) * 8);
  r.o = pad256(parts * p->d.head_dim * 4);
  r.ml = pad256(parts * 8);
  if (flags & GDN_F_ACCUM_MASS) {
    r.done = pad256(rows * 8);
    r.scores = rows * size_t(score_row(max_len)) * 4;
  }
  return r;
}

}  // namespace

bool attn_fits(const gdn_kv_pool *p, int batch, int q_heads, int max_len) {
  const int64_t head_blocks = (q_heads / p->d.kv_heads + 15) / 16;
  return int64_t(batch) * p->d.kv_heads * head_blocks < (int64_t(1) << 31) / unit_blocks(max_len);
}

size_t attn_workspace(const gdn_kv_pool *p, int batch, int q_heads, int max_len, uint32_t flags) {
  const AttnSpace w = attn_space(p, batch, q_heads, max_len, flags);
  return w.unit + w.o + w.ml + w.done + w.scores;
}

hipError_t launch_attn_decode(const gdn_kv_pool *pool, int layer, const AttnArgs &a, hipStream_t s) {
  const KvGeom g = kv_geom(pool, layer);
  AttnDev p{};
  p.a = a;
  p.group = a.q_heads / pool->d.kv_heads;
  p.head_blocks = (p.group + 15) / 16;
  p.workers = attn_workers(pool, a.batch, a.q_heads, a.max_len);
  p.join = attn_joins(a.max_len, a.flags);
  p.lpad = score_row(a.max_len);
  if (p.join) {
    const AttnSpace w = attn_space(pool, a.batch, a.q_heads, a.max_len, a.flags);
    char *at = static_cast<char *>(a.workspace);
    p.unit = reinterpret_cast<int32_t *>(at);
    p.o = reinterpret_cast<float *>(at += w.unit);
    p.ml = reinterpret_cast<float *>(at += w.o);
    if (a.flags & GDN_F_ACCUM_MASS) {
      p.done = reinterpret_cast<float *>(at += w.ml);
      p.scores = reinterpret_cast<float *>(at += w.done);
    }
  }
  const bool f8 = pool->d.kv_dtype == GDN_F8_E4M3;
  switch (pool->d.head_dim) {
    case 64: return launch_d<64>(g, p, f8, s);
    case 128: return launch_d<128>(g, p, f8, s);
    case 256: return launch_d<256>(g, p, f8, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace gdn
