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
// be about as large as the output's own rounding.  Scores, m, l and O are fp32.
//
// The work is counted in blocks of 128 tokens (4 waves, a tile each), in the order
// (request, key-value head, 16 query heads, position), and every workgroup takes an equal
// run of blocks: as many workgroups as run at once, whatever the requests' lengths.  (Equal
// splits of the longest length left a third of the chip waiting for a ragged batch.)  A
// workgroup finds its run from the lengths on the device, walks it unit by unit, and
// joins its waves in shared memory at the end of each unit.  A unit that lies in
// one workgroup is final there; of the others m, l and O go to the workspace, and a second
// kernel joins them (and adds up the weights, from stored scores).
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
  int32_t *pre;     // [batch + 1] blocks of the requests before each, per head and head block
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
__device__ __forceinline__ Seen seen_by(const KvGeom &g, const AttnArgs &a, int b, bool tell) {
  Seen r;
  r.slot = a.slot_table[b];
  r.len = a.kv_len[b];
  r.begin = a.kv_begin ? a.kv_begin[b] : 0;
  r.blocks = 0;
  if (r.slot <= 0 || r.slot >= g.slots) {
    if (tell && r.slot >= g.slots) set_err(g.err, GDN_ERRW_BAD_SLOT);
  } else if (r.len < 0 || r.len > a.max_len || r.begin < 0) {
    if (tell) set_err(g.err, GDN_ERRW_BAD_SEQLENS);
  } else if (r.begin < r.len) {
    r.blocks = (r.len - (r.begin & ~(kTile - 1)) + kBlock - 1) / kBlock;
  }
  return r;
}

// First block of worker w, and the worker that holds block x: floor(w all / workers) is the
// first, so the holder is the largest w with w all < (x + 1) workers.
// (The host keeps the number of blocks below 2^31.)
__device__ __forceinline__ int first_block(int w, int all, int workers) { return int(int64_t(w) * all / workers); }
__device__ __forceinline__ int worker_of(int x, int all, int workers) {
  return int(((int64_t(x) + 1) * workers - 1) / all);
}
// A value that is the same in every lane, as a scalar.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

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

// Element types.  kWords: 32-bit words of one lane's piece of a row.
//   K: piece s of a row (4 lanes of different g side by side): the k indices of kSteps
//      MFMA steps.  V: the D / 16 columns of a lane, as bf16 words after conversion.
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

// kWide: pages hold whole tiles (page_size >= 32), so a tile's rows are adjacent and its
// one page id is wave-uniform; otherwise each token's row is looked up.
template <int D, bool kF8, bool kWide, bool kMass>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2)))
void attn_decode_kernel(KvGeom g, AttnDev p) {
  using L = Lay<D, kF8>;
  constexpr int KS = D / 32;        // MFMA steps of a score
  constexpr int NO = D / 16;        // 16-column tiles of O
  constexpr int VW = D / 32;        // bf16 words of a lane's columns of one token
  constexpr int RB = D * L::kSize;  // bytes of a row
  // head dim 256: the queries stay in shared memory (their 32 registers would spill)
  constexpr bool kQShared = D == 256;
  extern __shared__ __attribute__((aligned(16))) float lds[];
  __shared__ float sm[kWaves][16], sl[kWaves][16];
  __shared__ u32x4 sq[kQShared ? KS : 1][64];

  __shared__ int spre[kThreads];
  __shared__ int sfound[2 + kWaves];

  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  const int worker = blockIdx.x;
  const int units = g.kv_heads * p.head_blocks;  // of a request

  // ---- this worker's run of blocks ---------------------------------------------
  // scan(base): spre[i] = blocks of requests base .. base + i, returns their sum
  auto scan = [&](int base) -> int {
    const int r = base + int(threadIdx.x);
    int inc = r < p.a.batch ? seen_by(g, p.a, r, false).blocks : 0;
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(inc, d);
      if (lane >= d) inc += o;
    }
    __syncthreads();  // the previous use of the shared sums is over
    if (lane == 63) sfound[2 + wave] = inc;
    __syncthreads();
    for (int w = 0; w < wave; ++w) inc += sfound[2 + w];
    spre[threadIdx.x] = inc;
    __syncthreads();
    return uniform(spre[kThreads - 1]);
  };
  int all = 0;
  for (int base = 0; base < p.a.batch; base += kThreads) {
    const int sum = scan(base);
    if (p.join && worker == 0 && base + int(threadIdx.x) < p.a.batch)
      p.pre[base + threadIdx.x + 1] = all + spre[threadIdx.x];
    all += sum;
  }
  if (p.join && worker == 0 && threadIdx.x == 0) p.pre[0] = 0;
  all *= units;
  const int sharing = min(p.workers, all);  // so that no worker between two others has nothing
  const int run_first = worker < sharing ? first_block(worker, all, sharing) : 0;
  int left = worker < sharing ? first_block(worker + 1, all, sharing) - run_first : 0;
  int b = 0;       // request, unit within it and block within the unit
  int unit = 0, blk = 0;
  Seen rq{0, 0, 0, 0};
  auto request = [&](int r) -> Seen {
    const Seen v = seen_by(g, p.a, r, false);
    return Seen{uniform(v.slot), uniform(v.begin), uniform(v.len), uniform(v.blocks)};
  };
  if (left > 0) {
    const int x = run_first / units;
    int before = 0;
    for (int base = 0; base < p.a.batch; base += kThreads) {
      const int sum = p.a.batch > kThreads ? scan(base) : uniform(spre[kThreads - 1]);
      if (x < before + sum) {
        const int lo = before + (threadIdx.x ? spre[threadIdx.x - 1] : 0), hi = before + spre[threadIdx.x];
        if (lo <= x && x < hi) {
          sfound[0] = base + threadIdx.x;
          sfound[1] = lo;
        }
        break;
      }
      before += sum;
    }
    __syncthreads();
    b = uniform(sfound[0]);
    rq = request(b);
    const int in_request = run_first - uniform(sfound[1]) * units;
    unit = in_request / rq.blocks;
    blk = in_request - unit * rq.blocks;
  }

  bool first_unit = true;
  while (left > 0) {
    // (made anew for each unit: addresses that depend on the lane alone would otherwise be
    // kept in registers across all units, 20 of them)
    int lane_now = threadIdx.x & 63;
    asm volatile("" : "+v"(lane_now));
    const int lane = lane_now, c = lane & 15, gr = lane >> 4;
    const int nblk = min(rq.blocks - blk, left);
    const int h = unit / p.head_blocks, hb = unit - h * p.head_blocks;
    const int slot = rq.slot, begin = rq.begin;
    const int first = (begin & ~(kTile - 1)) + blk * kBlock;
    const int last = min(rq.len, first + nblk * kBlock);
    const bool whole_unit = nblk == rq.blocks;
    const int heads = min(16, p.group - 16 * hb);           // query heads of this unit
    const int q0 = h * p.group + 16 * hb;                   // the first of them
    const int64_t qrow = int64_t(b) * p.a.q_heads + q0;

  // (constant address space: the table does not change during the call, so a wave-uniform
  // read of it is a scalar load, which the waits for keys and values do not count)
  typedef const int32_t __attribute__((address_space(4))) *table_t;
  const table_t table = (table_t)(g.page_table + int64_t(slot) * g.max_pages);
  const int in_page = (1 << g.page_shift) - 1;

  // Rows of a tile.  A token that is not visible, or whose page id is not a page, reads
  // page 0's rows (always there) and is masked by its bit of `seen`.
  struct Rows {
    int row;   // kWide: first row of the tile; else lane i < 32: row of token t0 + i
    u32 seen;
  };
  // The page ids are loaded two tiles ahead, before the keys and values of the next tile:
  // loads return in order, so waiting for an id that was asked for after them would wait for
  // them too.
  auto ask = [&](int t0) -> int {
    if constexpr (kWide) return table[min(t0, last - 1) >> g.page_shift];
    else return table[max(begin, min(t0 + (lane & 31), last - 1)) >> g.page_shift];
  };
  auto resolve = [&](int t0, int page) -> Rows {
    Rows r;
    if constexpr (kWide) {
      const bool ok = page > 0 && page < g.pages;
      if (!ok && t0 < last) {
        if (lane == 0) set_err(g.err, GDN_ERRW_BAD_PAGE);
      }
      r.row = ok ? ((page * g.kv_heads + h) << g.page_shift) + (t0 & in_page) : 0;
      // bits from begin on, and below last
      u32 m = ok ? 0xffffffffu : 0u;
      if (begin > t0) m &= begin - t0 >= 32 ? 0u : 0xffffffffu << (begin - t0);
      if (last - t0 < 32) m &= last > t0 ? (1u << (last - t0)) - 1u : 0u;
      r.seen = m;
    } else {
      const int t = t0 + (lane & 31);
      const bool in = t >= begin && t < last;
      const bool ok = in && page > 0 && page < g.pages;
      if (__any(in && !ok)) {
        if (lane == 0) set_err(g.err, GDN_ERRW_BAD_PAGE);
      }
      r.row = ok ? ((page * g.kv_heads + h) << g.page_shift) + (t & in_page) : 0;
      r.seen = u32(__ballot(ok));  // lanes 32 up repeat the lower ones
    }
    return r;
  };

  Words<4> kw[2][L::kPieces];
  Words<L::kVWords> vw[8][L::kVPieces];
  const u32 k_off = u32(c * RB + 16 * gr), v_off = u32(4 * gr * RB + 4 * L::kVWords * c);
  auto load_k = [&](const Rows &r) {
    const char *tile = g.k + int64_t(r.row) * RB;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const char *at;
      if constexpr (kWide) at = tile + 16 * u * RB + k_off;
      else at = g.k + int64_t(__shfl(r.row, 16 * u + c)) * RB + 16 * gr;
#pragma unroll
      for (int s = 0; s < L::kPieces; ++s) kw[u][s] = load_words<4>(at + 64 * s);
    }
  };
  auto load_v = [&](const Rows &r) {
    const char *tile = g.v + int64_t(r.row) * RB;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const char *at;
      if constexpr (kWide) at = tile + pk(0, e) * RB + v_off;
      else at = g.v + int64_t(__shfl(r.row, pk(gr, e))) * RB + 4 * L::kVWords * c;
#pragma unroll
      for (int s = 0; s < L::kVPieces; ++s) vw[e][s] = load_words<L::kVWords>(at + 256 * s);
    }
  };

  // Queries as the B operand (columns past the group are zero), asked for before the first
  // keys for the same reason.
  constexpr int kQLoads = kQShared ? KS / kWaves : KS;
  bf16x8 qf[kQLoads];
  {
    const uint16_t *q = p.a.q + int64_t(b) * p.a.q_stride + int64_t(q0 + min(c, heads - 1)) * D;
#pragma unroll
    for (int i = 0; i < kQLoads; ++i)
      qf[i] = *reinterpret_cast<const bf16x8 *>(q + L::kdim(kQShared ? wave * kQLoads + i : i, gr));
  }
  __builtin_amdgcn_sched_barrier(0);

  constexpr int kStep = kTile * kWaves;
  int t0 = first + kTile * wave;
  Rows now{0, 0}, next{0, 0};
  {
    const int p0 = ask(t0), p1 = ask(t0 + kStep);
    now = resolve(t0, p0);
    if (t0 < last) {
      load_k(now);
      load_v(now);
    }
    next = resolve(t0 + kStep, p1);
  }

  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < kQLoads; ++i) {
    if (c >= heads) qf[i] = bf16x8{};
    if constexpr (kQShared) sq[wave * kQLoads + i][lane] = __builtin_bit_cast(u32x4, qf[i]);
  }
  if constexpr (kQShared) __syncthreads();
  const float to_log2 = p.a.scale * g.k_scale * kLog2e;

  f32x4 o[NO];
#pragma unroll
  for (int i = 0; i < NO; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = kNegInf, l = 0.f;

  // One tile.  The last one of a wave is a body of its own: loads under a condition would
  // make every wait of the loop assume that they were not issued, and wait for all.
  auto tile = [&](auto more_c) {
    constexpr bool more = decltype(more_c)::value;
    const int page2 = more ? ask(t0 + 2 * kStep) : 0;

    // ---- scores ----------------------------------------------------------
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
    if constexpr (more) load_k(next);
    __builtin_amdgcn_sched_barrier(0);

    // ---- softmax ---------------------------------------------------------
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = s[e >> 2][e & 3] * to_log2;
    const u32 seen = now.seen;
    const bool whole = seen == 0xffffffffu;
    if (!whole) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = (seen >> pk(gr, e)) & 1 ? x[e] : kNegInf;
    }
    if (kMass && c < heads) {
      float *at = p.scores + (qrow + c) * p.lpad + t0 + 4 * gr;
      st4(at, f32x4{x[0], x[1], x[2], x[3]});
      st4(at + 16, f32x4{x[4], x[5], x[6], x[7]});
    }
    float mx = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
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
    const Split ps = split8(pr);

    // ---- values: columns of eight tokens by byte permutes --------------------
#pragma unroll
    for (int w = 0; w < VW; ++w) {
      u32 word[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (kF8) {
          u32 lo, hi;
          f8_to_bf16(vw[e][0].w[w >> 1], &lo, &hi);
          word[e] = (w & 1) ? hi : lo;
        } else {
          word[e] = vw[e][w / L::kVWords].w[w % L::kVWords];
        }
        if (!whole) word[e] = (seen >> pk(gr, e)) & 1 ? word[e] : 0u;  // never 0 * inf
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
    if constexpr (more) {
      load_v(next);
      __builtin_amdgcn_sched_barrier(0);
      now = next;
      next = resolve(t0 + 2 * kStep, page2);
    }
  };
  if (t0 < last) {
    for (; t0 + kStep < last; t0 += kStep) tile(std::true_type{});
    tile(std::false_type{});
  }

  // ---- join the waves: o[i][j] is column vdim(i, 4 gr + j) of head c ---------
  // Two slabs of shared memory: waves 2 and 3 store, waves 0 and 1 add.  Four i make 16
  // adjacent bytes; rows are padded by 16 bytes, so eight lanes cover all banks.
  constexpr int DS = D + 4;
  l = rows_sum(l);
  if (gr == 0) {
    sm[wave][c] = m;
    sl[wave][c] = l;
  }
  __syncthreads();
  float mt = sm[0][c];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) mt = fmaxf(mt, sm[w][c]);
  const float f = factor(m, mt);
  float *slab = lds + ((wave & 1) * heads + c) * DS;
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    if ((wave >> 1) != pass && c < heads) {
#pragma unroll
      for (int q = 0; q < NO / 4; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float *at = slab + L::vdim(4 * q, 4 * gr + j);
          f32x4 x = {o[4 * q][j], o[4 * q + 1][j], o[4 * q + 2][j], o[4 * q + 3][j]};
          x *= f;
          if (pass) x += ld4(at);
          st4(at, x);
        }
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < heads * (D / 4); i += kThreads) {
    const int hd = i / (D / 4), d = 4 * (i % (D / 4));
    float mh = sm[0][hd], lt = 0.f;
#pragma unroll
    for (int w = 1; w < kWaves; ++w) mh = fmaxf(mh, sm[w][hd]);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) lt = fmaf(sl[w][hd], factor(sm[w][hd], mh), lt);
    f32x4 sum = ld4(lds + hd * DS + d) + ld4(lds + (heads + hd) * DS + d);
    if (!whole_unit) {
      const int64_t r = (int64_t(worker) * 2 + (first_unit ? 0 : 1)) * 16 + hd;
      st4(p.o + r * D + d, sum);
      if (d == 0) {
        p.ml[2 * r] = mh;
        p.ml[2 * r + 1] = lt;
      }
    } else {
      sum *= lt == 0.f ? 0.f : g.v_scale / lt;
      *reinterpret_cast<u32x2 *>(p.a.out + (qrow + hd) * D + d) =
          u32x2{cvt_pk_bf16(sum[0], sum[1]), cvt_pk_bf16(sum[2], sum[3])};
      if (d == 0) {
        if (p.a.lse) p.a.lse[qrow + hd] = lt == 0.f ? kNegInf : (mh + log2f(lt)) * kLn2;
        if (kMass) {
          p.done[2 * (qrow + hd)] = mh;
          p.done[2 * (qrow + hd) + 1] = lt;
        }
      }
    }
  }
  __syncthreads();  // the shared arrays are free again

    // ---- the next unit -------------------------------------------------------------
    left -= nblk;
    blk = 0;
    first_unit = false;
    if (left > 0 && ++unit == units) {
      unit = 0;
      do rq = request(++b);
      while (rq.blocks == 0 && b + 1 < p.a.batch);
      if (rq.blocks == 0) break;
    }
  }

  // ---- requests that see nothing, dealt out to the workers ------------------------
  for (int e = worker; e < p.a.batch; e += p.workers) {
    if (seen_by(g, p.a, e, threadIdx.x == 0).blocks) continue;
    const int64_t row = int64_t(e) * p.a.q_heads;
    for (int i = threadIdx.x; i < p.a.q_heads * (D / 8); i += kThreads)
      reinterpret_cast<u32x4 *>(p.a.out + row * D)[i] = u32x4{0, 0, 0, 0};
    if (p.a.lse && int(threadIdx.x) < p.a.q_heads)
      for (int i = threadIdx.x; i < p.a.q_heads; i += kThreads) p.a.lse[row + i] = kNegInf;
  }
}

// Joins the parts of each (request, query head) that more than one worker had, and adds
// the weights
//   mass[t] += sum over the group's heads of 2^(score - m) / l.
// Workgroups: first one per (request, query head), then, with weights, one per
// kMassTokens tokens of each (request, key-value head).
constexpr int kMassTokens = 1024;

// The workers w0 .. w1 of a unit; the part of w0 is its first unit's where its run begins
// with the unit, else its last; the others' is their first.
struct Parts {
  int w0, w1;
  bool begins;
  __device__ __forceinline__ int64_t row(int w, int head) const {
    return (int64_t(w) * 2 + (w == w0 && !begins ? 1 : 0)) * 16 + head;
  }
};
__device__ __forceinline__ Parts parts_of(const KvGeom &g, const AttnDev &p, int b, int unit) {
  const int units = g.kv_heads * p.head_blocks;
  const int n = p.pre[b + 1] - p.pre[b], all = p.pre[p.a.batch] * units;
  const int first = p.pre[b] * units + unit * n, sharing = min(p.workers, all);
  Parts r{0, -1, true};
  if (n > 0) {
    r.w0 = worker_of(first, all, sharing);
    r.w1 = worker_of(first + n - 1, all, sharing);
    r.begins = first_block(r.w0, all, sharing) == first;
  }
  return r;
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
  const int joins = p.a.batch * p.a.q_heads;
  if (int(blockIdx.x) < joins) {
    const int qr = blockIdx.x, b = qr / p.a.q_heads, qh = qr - b * p.a.q_heads;
    const int h = qh / p.group, j = qh - h * p.group;  // head j of the group
    const Parts pt = parts_of(g, p, b, h * p.head_blocks + (j >> 4));
    if (pt.w1 <= pt.w0) return;  // nothing, or final already
    float m, l;
    join_ml(p.ml, pt, j & 15, lane, &m, &l);  // every wave for itself
    constexpr int C = D / 64;  // columns of a lane
    float sum[C];
#pragma unroll
    for (int i = 0; i < C; ++i) sum[i] = 0.f;
#pragma unroll 4
    for (int w = pt.w0 + wave; w <= pt.w1; w += kWaves) {
      const int64_t r = pt.row(w, j & 15);
      const float f = factor(p.ml[2 * r], m);
#pragma unroll
      for (int i = 0; i < C; ++i) sum[i] = fmaf(f, p.o[r * D + C * lane + i], sum[i]);
    }
#pragma unroll
    for (int i = 0; i < C; ++i) acc[wave][C * lane + i] = sum[i];
    __syncthreads();
    const float inv = l == 0.f ? 0.f : g.v_scale / l;
    for (int i = threadIdx.x; i < D; i += kThreads) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) t += acc[w][i];
      p.a.out[int64_t(qr) * D + i] = f32_to_bf16(t * inv);
    }
    if (p.a.lse && threadIdx.x == 0) p.a.lse[qr] = l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
    return;
  }
  const int64_t id = int64_t(blockIdx.x) - joins;
  const int block = int(id % mass_blocks), bh = int(id / mass_blocks);
  const int h = bh % g.kv_heads, b = bh / g.kv_heads;
  const Seen rq = seen_by(g, p.a, b, false);
  const int64_t from = int64_t(rq.begin & ~3) + int64_t(block) * kMassTokens;
  if (rq.blocks == 0 || from >= rq.len) return;
  const int64_t qr0 = int64_t(b) * p.a.q_heads + h * p.group;
  for (int j = wave; j < p.group; j += kWaves) {
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
  __syncthreads();
  const int64_t t = from + 4 * threadIdx.x;
  if (t >= rq.len) return;
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  const float *sc = p.scores + qr0 * p.lpad + t;
#pragma unroll 4
  for (int j = 0; j < p.group; ++j) {
    const f32x4 x = ld4(sc + j * p.lpad);
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] = fmaf(fexp2(x[e] - hm[j]), hl[j], sum[e]);
  }
  float *mass = g.mass + (int64_t(rq.slot) * g.kv_heads + h) * g.capacity + t;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (t + e >= rq.begin && t + e < rq.len) mass[e] += sum[e];
}

size_t pad256(size_t n) { return (n + 255) & ~size_t(255); }
int64_t score_row(int max_len) { return (int64_t(max_len) + kTile - 1) / kTile * kTile; }

template <int D, bool kF8>
hipError_t launch_dt(const KvGeom &g, const AttnDev &p, hipStream_t s) {
  const size_t lds = size_t(2) * std::min(16, p.group) * (D + 4) * 4;
  const bool wide = (1 << g.page_shift) >= kTile;
  const auto kernel = wide ? (p.scores ? attn_decode_kernel<D, kF8, true, true> : attn_decode_kernel<D, kF8, true, false>)
                           : (p.scores ? attn_decode_kernel<D, kF8, false, true> : attn_decode_kernel<D, kF8, false, false>);
  hipLaunchKernelGGL(kernel, dim3(unsigned(p.workers)), dim3(kThreads), lds, s, g, p);
  return hipGetLastError();
}

template <int D>
hipError_t launch_d(const KvGeom &g, const AttnDev &p, bool f8, hipStream_t s) {
  const int mass_blocks = p.scores ? (p.a.max_len + 3 + kMassTokens - 1) / kMassTokens : 0;
  const int64_t joins = int64_t(p.a.batch) * p.a.q_heads + int64_t(p.a.batch) * g.kv_heads * mass_blocks;
  if (joins >= (int64_t(1) << 31)) return hipErrorInvalidValue;
  hipError_t e = f8 ? launch_dt<D, true>(g, p, s) : launch_dt<D, false>(g, p, s);
  if (e != hipSuccess || !p.join) return e;
  hipLaunchKernelGGL((attn_join_kernel<D>), dim3(unsigned(joins)), dim3(kThreads), 0, s, g, p, mass_blocks);
  return hipGetLastError();
}

// Blocks of a unit of max_len tokens (its first tile may begin before the first one seen).
int64_t unit_blocks(int max_len) { return std::max<int64_t>(1, (int64_t(max_len) + kTile - 1 + kBlock - 1) / kBlock); }

// Workers of a call: what runs at once, or fewer where there are not that many blocks.
int attn_workers(const gdn_kv_pool *p, int batch, int q_heads, int max_len) {
  const int group = q_heads / p->d.kv_heads;
  const int64_t units = int64_t(batch) * p->d.kv_heads * ((group + 15) / 16);
  return int(std::max<int64_t>(1, std::min<int64_t>(kCUs * 2, units * unit_blocks(max_len))));
}

// One block per unit at most: no unit is ever divided.
bool attn_joins(int max_len, uint32_t flags) { return max_len > kBlock || (flags & GDN_F_ACCUM_MASS); }

// Parts of the workspace, in order.
struct AttnSpace {
  size_t pre, o, ml, done, scores;
};
AttnSpace attn_space(const gdn_kv_pool *p, int batch, int q_heads, int max_len, uint32_t flags) {
  AttnSpace r{};
  if (!attn_joins(max_len, flags)) return r;
  const size_t parts = size_t(attn_workers(p, batch, q_heads, max_len)) * 2 * 16, rows = size_t(batch) * q_heads;
  r.pre = pad256((size_t(batch) + 1) * 4);
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
  return w.pre + w.o + w.ml + w.done + w.scores;
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
    p.pre = reinterpret_cast<int32_t *>(at);
    p.o = reinterpret_cast<float *>(at += w.pre);
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
