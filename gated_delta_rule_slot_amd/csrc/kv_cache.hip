// kv_cache.hip -- the paged key-value cache's own kernels: append, eviction plan and
// the moves of an eviction (formulas and rules: include/gdn_kv.h).
#include <type_traits>

#include "kv.hpp"
#include "lanes.hpp"

namespace gdn {
namespace {

// ------------------------------------------------------------------ append --
// One thread per 8 consecutive values of a token's key and of its value: two 16-byte
// loads, one store each.  Bound by the bytes (and by the launch for one decode step):
// 6144 tokens of 8 heads of 128 into e4m3, 38 MB, 10.7 us (8.1 us at a copy's rate); 128
// tokens of 2 heads of 256, 2.9 us.  Two or four tokens a thread (12.2, 14.1 us) and
// non-temporal loads (16.1 us) were slower, non-temporal stores the same.
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
  const int64_t item = flat_block() * kAppendThreads + threadIdx.x;
  if (item >= int64_t(a.n) * per) return;
  const int token = int(item / per);
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
// range's keys in up to BINS equal bins (shared memory), finds the bin that holds the
// k-th largest and takes it as the next range, and stops early where a whole bin is kept.
// The first round's range is all weights above 0 (8 bins, or 4, an octave), so it counts
// while the keys are loaded; a threshold among the weights of 0 is seen at once.
//
// Every wave owns a run of adjacent tokens, so the order of the lists needs no barrier per
// 64 tokens: a wave puts the places that it takes, the freed ones and then the tokens to
// move, side by side over its own keys, one sum over the waves gives each its start, and it
// writes its places out 64 at a time.
//
// Measured: 512 lists of 1020-1088 tokens 6.8 us (4 MB: latency); 128 lists of 32769
// tokens and fewer 21 us (39 MB, 6.6 us at the rate of reads).  Of the 21 some 7.5 are the
// loading, 1 the choice of the range, 2.5 a second round, 4 the taking and 3 the writing, on
// the half of the compute units that have a list.  A range pass before the first round,
// counts by ballots in a pass of their own and a store a round took 27 us; keys in registers
// with unrolled passes 31.7 us, reading them again 61 us.  Equal weights throughout (which a
// softmax does not leave) are the slow case, 35 us.
//
// The keys lie in shared memory (up to 36 * 1024 tokens), so mass and pos are read once; a
// longer cache reads both again in each pass.  A pass takes U times 64 tokens in a step,
// all of their keys read before the first is used (the compiler does not unroll loops with
// ballots by itself); the loads of mass and pos go out kLoads at a time, with no condition
// between them.
constexpr uint32_t kProtected = 0xffffffffu;

template <int THREADS, int BINS>
struct PlanShared {
  uint32_t bins[BINS];
  uint32_t wave[5][THREADS / 64];
  uint32_t lo, hi, need, exact, held;
};

// Sum over the waves before this one of what each wrote before the last barrier.
template <int WAVES>
__device__ __forceinline__ uint32_t before(const uint32_t *wave) {
  const int w = threadIdx.x >> 6;
  uint32_t sum = 0;
#pragma unroll
  for (int i = 0; i < WAVES; ++i) sum += i < w ? wave[i] : 0;
  return sum;
}
// The same with v written here (wave-uniform); the caller's arrays differ between uses that
// no barrier parts.
template <int WAVES>
__device__ __forceinline__ uint32_t before_wave(uint32_t v, uint32_t *wave) {
  if ((threadIdx.x & 63) == 0) wave[threadIdx.x >> 6] = v;
  __syncthreads();
  return before<WAVES>(wave);
}

// from + the mask's bits of the lanes below
__device__ __forceinline__ uint32_t lanes_below(uint64_t mask, uint32_t from) {
  return __builtin_amdgcn_mbcnt_hi(uint32_t(mask >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(mask), from));
}

// kHeld: the keys of all tokens in dynamic shared memory, a whole number of U * THREADS
template <int THREADS, bool kHeld, int BINS, int U>
__global__ __launch_bounds__(THREADS) void kv_evict_plan_kernel(KvGeom g, EvictArgs a) {
  constexpr int WAVES = THREADS / 64;
  constexpr int PER = BINS / THREADS;  // bins of a thread
  constexpr int kBits = BINS == 2048 ? 11 : 10;
  constexpr int kLoads = THREADS == 256 ? 8 : 16;
  static_assert(BINS == 1 << kBits, "bins");
  __shared__ PlanShared<THREADS, BINS> sh;
  extern __shared__ __align__(16) uint32_t held[];
  using Keys = uint32_t __attribute__((ext_vector_type(kHeld ? U : 2)));
  const int64_t block = flat_block();
  if (block >= int64_t(a.layers) * a.batch * g.kv_heads) return;
  const int unit = int(block);
  const int h = unit % g.kv_heads, lb = unit / g.kv_heads;
  const int b = lb % a.batch, layer = lb / a.batch;
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
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
  // (next_pos - recent may pass the 32-bit range, downwards)
  const int32_t from = int32_t(max(int64_t(a.next_pos[b]) - a.recent, int64_t(INT32_MIN)));
  const int rounds = (n + U * THREADS - 1) / (U * THREADS) * U;  // of 64 tokens, per wave
  const int first = w * rounds * 64;               // of this wave

  // Key of place i.  One behind the last token has key 0 and needs no test in the passes:
  // it is not below budget, so not freed; it comes after all ties; and a key of 0 is only
  // ever kept as a tie.
  const char *mass_bytes = reinterpret_cast<const char *>(mass), *pos_bytes = reinterpret_cast<const char *>(pos);
  auto load_some = [&](int i0, auto count, auto inside, uint32_t *out) {
    constexpr int N = decltype(count)::value;
    constexpr bool kInside = decltype(inside)::value;  // all of these places are in the cache
    float m[N];
    int32_t p[N];
#pragma unroll
    for (int q = 0; q < N; ++q) {  // (a 32-bit offset to a scalar base; capacity < 2^30)
      const int i = i0 + 64 * q + lane;
      const uint32_t at = 4u * uint32_t(kInside ? i : min(i, n - 1));
      m[q] = *reinterpret_cast<const float *>(mass_bytes + at);
      p[q] = *reinterpret_cast<const int32_t *>(pos_bytes + at);
    }
#pragma unroll
    for (int q = 0; q < N; ++q) {
      const uint32_t key = m[q] > 0.f ? __float_as_uint(m[q]) : 0u;
      const bool safe = (p[q] < a.sink) | (p[q] >= from);
      out[q] = !kInside && i0 + 64 * q + lane >= n ? 0u : safe ? kProtected : key;
    }
  };
  auto load_keys = [&](int i0, auto count, uint32_t *out) {
    if (THREADS > 256 && i0 + 64 * decltype(count)::value <= n) load_some(i0, count, std::true_type{}, out);
    else load_some(i0, count, std::false_type{}, out);
  };
  // f(first token, keys of N rounds), or f(first token, key), for this wave's rounds in order
  constexpr int N = kHeld ? U : kLoads;
  auto each_step = [&](auto f) {
    for (int r = 0; r < rounds; r += N) {
      uint32_t k[N];
      if constexpr (kHeld) {
#pragma unroll
        for (int q = 0; q < N; ++q) k[q] = held[first + 64 * (r + q) + lane];
      } else {
        load_keys(first + 64 * r, std::integral_constant<int, N>{}, k);
      }
      f(first + 64 * r, k);
    }
  };
  auto each = [&](auto f) {
    each_step([&](int i0, const uint32_t (&k)[N]) {
#pragma unroll
      for (int q = 0; q < N; ++q)
        if (kHeld || i0 + 64 * q < first + 64 * rounds) f(i0 + 64 * q, k[q]);
    });
  };
  // f(key) for this wave's keys in any order: U adjacent ones a lane, the next read ahead
  auto each_key = [&](auto f) {
    if constexpr (kHeld) {
      const Keys *mine = reinterpret_cast<const Keys *>(held + first) + lane;
      Keys x = mine[0];
      for (int r = 0; r < rounds; r += U) {
        const Keys next = mine[64 * min(r / U + 1, rounds / U - 1)];
#pragma unroll
        for (int q = 0; q < U; ++q) f(x[q]);
        x = next;
      }
    } else {
      each([&](int, uint32_t key) { f(key); });
    }
  };

  // ---- first round: the weights above 0 by the bits below the sign; the protected ----
  // thread t has bins BINS - 1 - PER t downwards: sums from the top
  const int top_bin = BINS - 1 - PER * tid;
  auto clear = [&] {
#pragma unroll
    for (int q = 0; q < PER; ++q) sh.bins[top_bin - q] = 0;
    __syncthreads();
  };
  // One more in `bin` where `in`.  kAlike: lanes that all have one bin add once (32769 equal
  // weights: 97 us without)
  auto count = [&](bool in, uint32_t bin, auto alike) {
    if constexpr (decltype(alike)::value) {
      const uint64_t who = __ballot(in);
      const int one = who ? __ffsll(static_cast<unsigned long long>(who)) - 1 : 0;
      if (__ballot(in & (bin != uint32_t(__builtin_amdgcn_readlane(bin, one)))) == 0) {
        if (in & (lane == one)) atomicAdd(&sh.bins[bin], uint32_t(__popcll(who)));
        return;
      }
    }
    if (in) atomicAdd(&sh.bins[bin], 1u);
  };
  // (tested on a step's first round for all of them: a test in every round took 3 us)
  auto one_bin = [&](bool in, uint32_t bin) -> bool {
    const uint64_t who = __ballot(in);
    return who && __ballot(in & (bin != uint32_t(__builtin_amdgcn_readlane(
                                           bin, __ffsll(static_cast<unsigned long long>(who)) - 1)))) == 0;
  };
  uint32_t prot = 0;
  auto look = [&](int r, const uint32_t (&k)[kLoads]) {
    auto all = [&](auto alike) {
#pragma unroll
      for (int q = 0; q < kLoads; ++q) {
        if (r + q < rounds) {
          if (kHeld) held[first + 64 * (r + q) + lane] = k[q];  // read again by this wave only
          prot += __popcll(__ballot(k[q] == kProtected));
          count(k[q] - 1u < kProtected - 1u, k[q] >> (31 - kBits), alike);
        }
      }
    };
    if (one_bin(k[0] - 1u < kProtected - 1u, k[0] >> (31 - kBits))) all(std::true_type{});
    else all(std::false_type{});
  };
  clear();
  for (int r = 0; r < rounds; r += kLoads) {
    uint32_t k[kLoads];
    load_keys(first + 64 * r, std::integral_constant<int, kLoads>{}, k);
    look(r, k);
  }
  if (lane == 0) sh.wave[4][w] = prot;
  __syncthreads();
  prot = 0;
#pragma unroll
  for (int i = 0; i < WAVES; ++i) prot += sh.wave[4][i];

  // keep every key above `lo` at the end, and the first `need` of those equal to it;
  // with `exact` every key >= lo
  uint32_t lo = 0, hi = 0x7fffffffu, need = uint32_t(a.budget) - prot;
  bool exact = false;
  // the bin of the range from lo on that holds the need-th largest key becomes the range;
  // returns the count of all bins
  auto choose = [&](int shift) -> uint32_t {
    uint32_t mine = 0, c[PER];
#pragma unroll
    for (int q = 0; q < PER; ++q) mine += c[q] = sh.bins[top_bin - q];
    const uint32_t inc = wave_scan(mine);
    uint32_t above = before_wave<WAVES>(__builtin_amdgcn_readlane(inc, 63), sh.wave[0]) + inc - mine;
    uint32_t all = 0;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) all += sh.wave[0][i];
    if (above < need && above + mine >= need) {
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        if (above < need && above + c[q] >= need) {
          const uint32_t l = lo + (uint32_t(top_bin - q) << shift);
          sh.lo = max(l, 1u);  // (a weight of 0 is in no bin)
          sh.hi = min(hi, l + ((1u << shift) - 1u));
          sh.need = need - above;
          sh.exact = need - above == c[q];  // the whole bin is kept
          sh.held = c[q];
        }
        above += c[q];
      }
    }
    __syncthreads();
    return all;
  };
  auto chosen = [&] {
    lo = sh.lo;
    hi = sh.hi;
    need = sh.need;
    exact = sh.exact != 0;
  };
  if (prot >= uint32_t(a.budget)) {  // the protected alone fill the budget
    lo = hi = kProtected;
    need = a.budget;
  } else {
    const uint32_t some = choose(31 - kBits);
    if (some < need) {  // some weights of 0 are kept
      lo = hi = 0;
      need -= some;
    } else {
      chosen();
    }
  }
  while (lo < hi && !exact) {  // ends: each round leaves at most 2 / BINS of the range
    const uint32_t width = hi - lo;
    const int top = 32 - __clz(width);
    const int shift = top > kBits ? top - kBits : 0;
    clear();
    auto narrow = [&](auto alike) {
      each_key([&](uint32_t key) { count(key - lo <= width, (key - lo) >> shift, alike); });
    };
    // (the test costs more than it saves while other bins hold most keys: weights within one
    // octave 28 us with it, 24 without)
    if (sh.held > uint32_t(n) / 2) narrow(std::true_type{});
    else narrow(std::false_type{});
    __syncthreads();
    choose(shift);
    chosen();
  }

  // ---- freed places and tokens to move -----------------------------------------
  // Taken are the places below budget that are not kept and those from budget on that are:
  // in a wave's order all its freed places come before all its tokens to move.
  const int budget = a.budget;
  // kept are keys above `over` and, unless `exact`, ties while they are needed
  const uint32_t over = exact ? lo - 1u : lo;  // (`exact` only with lo above 0)
  // n_places into a list, four reads of the wave before the first store
  auto put = [&](int32_t *column, const uint32_t *from_lds, uint32_t n_places) {
    for (uint32_t e0 = lane; e0 < n_places + lane; e0 += 256) {
      uint32_t x[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) x[q] = from_lds[min(e0 + 64 * q, n_places - 1)];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (e0 + 64 * q < n_places) column[2 * (e0 + 64 * q)] = x[q];
    }
  };
  auto finish = [&](auto with_ties) {
    constexpr bool kTies = decltype(with_ties)::value;
    uint32_t tie0 = 0;
    if constexpr (kTies) {
      each([&](int, uint32_t key) { tie0 += __popcll(__ballot(key == lo)); });
      tie0 = before_wave<WAVES>(tie0, sh.wave[1]);
    }
    uint32_t ties = tie0;  // (how many came before)
    auto kept = [&](uint32_t key) -> bool {
      if constexpr (!kTies) {
        return key > over;
      } else {
        const uint64_t equal = __ballot(key == lo);
        const bool tie = key == lo && lanes_below(equal, ties) < need;
        ties += __popcll(equal);
        return key > over || tie;
      }
    };
    uint32_t all = 0, freed = 0;
    if constexpr (kHeld) {
      // The rounds of a step side by side and with no branch between them (a round at a time
      // took half as long again): lanes that take nothing write to the bins, which are over.
      uint32_t *const unused = sh.bins + lane;
      each_step([&](int i0, const uint32_t (&k)[N]) {
        auto take = [&](auto is_taken) {
          uint64_t mask[N];
          uint32_t *to[N];
#pragma unroll
          for (int q = 0; q < N; ++q) {
            const bool t = is_taken(q);
            mask[q] = __ballot(t);
            uint32_t *const at = held + first + lanes_below(mask[q], all);
            to[q] = t ? at : unused;
            all += __popcll(mask[q]);
          }
#pragma unroll
          for (int q = 0; q < N; ++q) *to[q] = i0 + 64 * q + lane;  // (keys that were read already)
        };
        if (i0 + 64 * N <= budget) {
          take([&](int q) { return !kept(k[q]); });
          freed = all;
        } else if (i0 >= budget) {
          take([&](int q) { return kept(k[q]); });
        } else {
          take([&](int q) {
            const bool below = i0 + 64 * q + lane < budget, t = kept(k[q]) != below;
            freed += __popcll(__ballot(t & below));
            return t;
          });
        }
      });
    } else {
      each([&](int i0, uint32_t key) {
        const bool below = i0 + lane < budget, t = kept(key) != below;
        all += __popcll(__ballot(t));
        freed += __popcll(__ballot(t & below));
      });
    }
    const uint32_t moved = all - freed;
    if (lane == 0) {
      sh.wave[2][w] = freed;
      sh.wave[3][w] = moved;
    }
    __syncthreads();
    const uint32_t free_at = __builtin_amdgcn_readfirstlane(before<WAVES>(sh.wave[2]));
    const uint32_t move_at = __builtin_amdgcn_readfirstlane(before<WAVES>(sh.wave[3]));
    if (tid == THREADS - 1) a.n_moves[unit] = int(move_at + moved);
    int32_t *list = a.moves + 2 * int64_t(unit) * a.max_moves;
    int32_t *to = list + 2 * free_at + 1, *src = list + 2 * move_at;
    if constexpr (kHeld) {
      put(to, held + first, freed);
      put(src, held + first + freed, moved);
    } else {
      ties = tie0;
      uint32_t at = 0;
      each([&](int i0, uint32_t key) {
        const bool t = kept(key) != (i0 + lane < budget);
        const uint64_t mask = __ballot(t);
        const uint32_t e = lanes_below(mask, at);
        if (t) (e < freed ? to + 2 * e : src + 2 * (e - freed))[0] = i0 + lane;
        at += __popcll(mask);
      });
    }
  };
  if (exact) finish(std::false_type{});
  else finish(std::true_type{});
}

// ---------------------------------------------------------- eviction moves --
// x: blocks of entries of a (layer, request, head)'s list.  A row is spread over
// row_bytes / 16 lanes; a thread carries 16 bytes of the key and of the value of kMoveRows
// entries, all loads issued before the first store.  The rows are looked up once per
// entry, by one thread each.  Sources and destinations are disjoint, so there is no order.
// Loads and stores are non-temporal: 128 lists of 6200 rows of 128 bytes, 88.4 us; with
// plain stores 101 us.
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 4;

__global__ __launch_bounds__(kMoveThreads) void kv_evict_apply_kernel(KvGeom g, int row_bytes, int units,
                                                                      EvictArgs a) {
  __shared__ int srow[kMoveThreads], drow[kMoveThreads];
  const int64_t id = flat_block();
  const int unit = int(id % units), lanes = row_bytes >> 4;  // per row: 4 .. 32
  const int entries = kMoveRows * kMoveThreads / lanes;      // of this block: 32 .. 256
  if (id / units * entries >= a.max_moves) return;
  const int block = int(id / units);
  const int h = unit % g.kv_heads, lb = unit / g.kv_heads;
  const int b = lb % a.batch, layer = lb / a.batch;
  const int first = block * entries;
  // (the entry is read beside the count, not after it: max_moves of them are there)
  const int j = first + threadIdx.x;
  const int64_t e = 2 * (int64_t(unit) * a.max_moves + min(j, a.max_moves - 1));
  const int src = a.moves[e], dst = a.moves[e + 1];
  const int count = a.n_moves[unit], slot = a.slot_table[b];
  const bool teller = block == 0 && threadIdx.x == 0;
  if (slot <= 0 || slot >= g.slots) {
    if (teller && slot >= g.slots) set_err(g.err, GDN_ERRW_BAD_SLOT);
    return;
  }
  if (count < 0 || count > a.max_moves) {
    if (teller) set_err(g.err, GDN_ERRW_BAD_SEQLENS);
    return;
  }
  if (first >= count) return;
  if (int(threadIdx.x) < entries) {
    int rs = -1, rd = -1;
    if (j < count) {
      if (src < 0 || src >= g.capacity || dst < 0 || dst >= g.capacity) {
        set_err(g.err, GDN_ERRW_BAD_SEQLENS);
      } else {
        rs = kv_row(g, slot, h, src);
        rd = kv_row(g, slot, h, dst);
        if (rs < 0 || rd < 0) {
          set_err(g.err, GDN_ERRW_BAD_PAGE);
          rs = -1;
        } else {
          const int64_t m = ((int64_t(layer) * g.slots + slot) * g.kv_heads + h) * g.capacity;
          if (g.mass) g.mass[m + dst] = g.mass[m + src];
          if (g.pos) g.pos[m + dst] = g.pos[m + src];
        }
      }
    }
    srow[threadIdx.x] = rs;
    drow[threadIdx.x] = rd;
  }
  __syncthreads();
  const int piece = threadIdx.x % lanes, mine = threadIdx.x / lanes, step = kMoveThreads / lanes;
  char *const k = g.k + int64_t(layer) * g.layer_rows * row_bytes + 16 * piece;
  char *const v = g.v + int64_t(layer) * g.layer_rows * row_bytes + 16 * piece;
  u32x4 kx[kMoveRows], vx[kMoveRows];
#pragma unroll
  for (int u = 0; u < kMoveRows; ++u) {
    const int rs = srow[mine + u * step];
    if (rs >= 0) {
      kx[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(k + int64_t(rs) * row_bytes));
      vx[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(v + int64_t(rs) * row_bytes));
    }
  }
#pragma unroll
  for (int u = 0; u < kMoveRows; ++u) {
    if (srow[mine + u * step] >= 0) {
      const int64_t rd = drow[mine + u * step];
      __builtin_nontemporal_store(kx[u], reinterpret_cast<u32x4 *>(k + rd * row_bytes));
      __builtin_nontemporal_store(vx[u], reinterpret_cast<u32x4 *>(v + rd * row_bytes));
    }
  }
}

}  // namespace

hipError_t launch_kv_append(const gdn_kv_pool *p, int layer, const AppendArgs &a, hipStream_t s) {
  const int64_t items = int64_t(a.n) * p->d.kv_heads * (p->d.head_dim >> 3);
  const dim3 grid = flat_grid((items + kAppendThreads - 1) / kAppendThreads);
  const KvGeom g = kv_geom(p, layer);
  if (p->d.kv_dtype == GDN_BF16)
    hipLaunchKernelGGL((kv_append_kernel<false>), grid, dim3(kAppendThreads), 0, s, g, p->d.head_dim, a);
  else
    hipLaunchKernelGGL((kv_append_kernel<true>), grid, dim3(kAppendThreads), 0, s, g, p->d.head_dim, a);
  return hipGetLastError();
}

namespace {
template <int THREADS, bool kHeld, int BINS, int U>
hipError_t launch_plan(const KvGeom &g, const EvictArgs &a, hipStream_t s) {
  constexpr int step = U * THREADS;
  const size_t held = kHeld ? size_t((a.max_len + step - 1) / step) * step * 4 : 0;
  hipLaunchKernelGGL((kv_evict_plan_kernel<THREADS, kHeld, BINS, U>), flat_grid(int64_t(a.layers) * a.batch * g.kv_heads),
                     dim3(THREADS), held, s, g, a);
  return hipGetLastError();
}
}  // namespace

// Which form runs goes by the bound max_len, the only length that the host knows.
//   256 against 1024 threads a list, us: 512 lists of 1088 tokens 7.1 / 12.1, of 2048 7.7 / 11.9,
//   of 4096 10.9 / 12.5, of 8192 17.6 / 15.7; 128 lists of 2048 6.9 / 8.4, of 4096 8.7 / 8.8, of
//   6000 10.8 / 9.4; 16 lists of 2048 7.1 / 7.7, of 4096 8.3 / 8.1.  (They meet near 4096: the
//   border could lie higher.)
//   keys held against read again in each pass: 128 lists of 20000 15.4 / 27.2, 16 of 36864
//   18.0 / 32.5; 36 * 1024 keys and the bins are what shared memory takes.
// A bound far above the lengths costs: 128 lists of 2000 tokens 6.9 with max_len 2048, 8.3 up to
// 36864, 13.6 past it; 512 lists 7.4, 12.1 (15.2 at 36864, one workgroup per compute unit), 25.0.
hipError_t launch_kv_evict_plan(const gdn_kv_pool *p, int layer, const EvictArgs &a, hipStream_t s) {
  const KvGeom g = kv_geom(p, layer);
  if (a.max_len <= 2048) return launch_plan<256, true, 1024, 2>(g, a, s);
  if (a.max_len <= 36 * 1024) return launch_plan<1024, true, 2048, 4>(g, a, s);
  return launch_plan<1024, false, 2048, 1>(g, a, s);
}

hipError_t launch_kv_evict_apply(const gdn_kv_pool *p, int layer, const EvictArgs &a, hipStream_t s) {
  const int units = a.layers * a.batch * p->d.kv_heads;
  const int entries = kMoveRows * kMoveThreads / (p->row_bytes >> 4);
  const int64_t blocks = (int64_t(a.max_moves) + entries - 1) / entries;
  hipLaunchKernelGGL(kv_evict_apply_kernel, flat_grid(blocks * units), dim3(kMoveThreads), 0, s,
                     kv_geom(p, layer), p->row_bytes, units, a);
  return hipGetLastError();
}

}  // namespace gdn
