// kv_pages.hip -- page tables and token maps from request lengths, and pages given back
// (rules: include/gdn_kv.h).
#include "kv.hpp"
#include "lanes.hpp"

namespace gdn {
namespace {

// from + the mask's bits of the lanes below
__device__ __forceinline__ uint32_t lanes_below(uint64_t mask, uint32_t from) {
  return __builtin_amdgcn_mbcnt_hi(uint32_t(mask >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(mask), from));
}

// Sum over the threads of the workgroup before this one, and over all of them.  wave is shared
// memory that no other use touches until a barrier has passed.
template <int THREADS>
__device__ __forceinline__ uint64_t block_scan(uint32_t v, uint32_t *wave, uint64_t *all) {
  constexpr int WAVES = THREADS / 64;
  const uint32_t inc = wave_scan(v);
  const int w = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 63) wave[w] = inc;
  __syncthreads();
  uint64_t before = 0, sum = 0;
#pragma unroll
  for (int i = 0; i < WAVES; ++i) {
    const uint32_t x = wave[i];
    before += i < w ? x : 0;
    sum += x;
  }
  *all = sum;
  return before + inc - v;
}

// ------------------------------------------------------------- batch map --
// Requests are taken THREADS at a time, one a thread: a sum over their tokens gives cu_seqlens,
// one over the pages that they lack the place of each in the free list.  Then every thread
// makes four adjacent tokens' entries: it finds the first one's request among the ends in shared
// memory, and a token at the start of a page takes that page from the list.  A new page always
// has a new token at its start, so no pass over pages is needed.
//
// kTokens: the tokens' entries (of the workgroup's part), cu_seqlens and slot_out.  kCounts: the
// lengths, positions and the list's count, which may be the arrays that both forms read.  One
// workgroup does both where there are few tokens; else the tokens have their own workgroups,
// each of which makes the sums for itself, and a second launch of one workgroup writes the
// counts behind them.
//
// Measured: 128 requests of one token 4.7 us on the device, latency (lengths, then the list, two sums
// over the waves); 64 requests of up to 1500 tokens, 48 000 in all, 5.1 + 2.6 us.
constexpr int kTokensPer = 4;

template <int THREADS>
struct MapShared {
  uint32_t waves[2][THREADS / 64];
  int end[THREADS], slot[THREADS], place[THREADS], pos[THREADS], rank[THREADS];
};

template <int THREADS, bool kTokens, bool kCounts>
__global__ __launch_bounds__(THREADS) void kv_batch_map_kernel(KvGeom g, MapArgs a, int part) {
  __shared__ MapShared<THREADS> sh;
  const int tid = threadIdx.x;
  const int page = 1 << g.page_shift;
  const int have = a.n_free[0], nf = max(0, min(have, a.free_capacity));
  const bool first = kCounts && tid == 0;
  if (first && have != nf) set_err(g.err, GDN_ERRW_BAD_SEQLENS);
  const bool lead = blockIdx.x == 0;
  if (kTokens && lead && tid == 0) a.cu_seqlens[0] = 0;
  // tokens of this workgroup
  const int64_t from64 = kTokens && !kCounts ? int64_t(blockIdx.x) * part : 0;
  const int from = int(min(from64, int64_t(a.max_tokens)));
  const int to = kTokens && !kCounts ? int(min(from64 + part, int64_t(a.max_tokens))) : a.max_tokens;

  uint64_t sum = 0;  // tokens of the requests before
  int pages = 0;    // pages that they lack
  int taken = 0;    // pages that they were given
  for (int b0 = 0; b0 < a.batch; b0 += THREADS) {
    const int b = b0 + tid;
    const bool on = b < a.batch;
    int slot = 0, len = 0, n = 0, pos = 0;
    if (on) {
      slot = a.slot_table[b];
      len = a.kv_len[b];
      n = a.new_len ? a.new_len[b] : 1;
      pos = a.next_pos ? a.next_pos[b] : len;
    }
    uint64_t all;
    // (counts stay below 2^26, so a wave's sum fits 32 bits)
    const uint32_t count = uint32_t(max(0, min(n, a.max_tokens + 1)));
    const uint64_t before = block_scan<THREADS>(on ? count : 0, sh.waves[0], &all);
    const uint64_t limit = uint64_t(a.max_tokens);
    const int start = int(min(limit, sum + before)), end = int(min(limit, sum + before + count));
    const bool live = on && slot > 0 && slot < g.slots;
    const bool fits = sum + before + count <= limit;
    const bool valid = live && n >= 0 && len >= 0 && int64_t(len) + n <= g.capacity && fits &&
                       int64_t(pos) + n <= INT32_MAX;
    const int held = valid ? (len + page - 1) >> g.page_shift : 0;
    const int need = valid ? ((len + n + page - 1) >> g.page_shift) - held : 0;
    uint64_t lacked;
    const int rank = pages + int(block_scan<THREADS>(uint32_t(need), sh.waves[1], &lacked));
    const bool served = valid && (need == 0 || rank + need <= nf);
    if (kCounts && on) {
      if (slot >= g.slots) set_err(g.err, GDN_ERRW_BAD_SLOT);
      else if (live && !valid) set_err(g.err, GDN_ERRW_BAD_SEQLENS);
      else if (live && !served) set_err(g.err, GDN_ERRW_NO_PAGES);
      a.kv_len_out[b] = len + (served ? n : 0);
      if (a.next_pos_out) a.next_pos_out[b] = pos + (served ? n : 0);
    }
    if (kTokens && lead && on) {
      a.cu_seqlens[b + 1] = end;
      a.slot_out[b] = served ? slot : 0;
    }
    if (kTokens) {
      sh.end[tid] = end;
      sh.slot[tid] = served ? slot : 0;
      sh.place[tid] = len - start;
      sh.pos[tid] = pos - start;
      sh.rank[tid] = rank - held;
    }
    if (kCounts) {  // served requests that lack pages come before the refused ones
      uint32_t last = served && need > 0 ? uint32_t(rank + need) : 0;
#pragma unroll
      for (int d = 32; d; d >>= 1) last = max(last, uint32_t(__shfl_xor(int(last), d)));
      taken = max(taken, int(last));
    }
    const int begin = int(min(limit, sum)), chunk_end = int(min(limit, sum + all));
    __syncthreads();
    if (kTokens) {
      const int requests = min(THREADS, a.batch - b0);
      const int t0 = max(from, begin), t1 = min(to, chunk_end);
      for (int t = (t0 & ~(kTokensPer - 1)) + tid * kTokensPer; t < t1; t += THREADS * kTokensPer) {
        const int mine0 = max(t, t0), mine1 = min(t + kTokensPer, t1);
        int lo = 0, hi = requests - 1;  // the first request that ends behind the first token
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (sh.end[mid] > mine0) hi = mid;
          else lo = mid + 1;
        }
        int vs[kTokensPer], vi[kTokensPer], vp[kTokensPer];
#pragma unroll
        for (int e = 0; e < kTokensPer; ++e) {
          const int u = t + e;
          vs[e] = vi[e] = vp[e] = 0;
          if (u < mine0 || u >= mine1) continue;
          while (sh.end[lo] <= u) ++lo;
          const int s = sh.slot[lo];
          if (s <= 0) continue;
          const int place = sh.place[lo] + u;
          vs[e] = s;
          vi[e] = place;
          vp[e] = sh.pos[lo] + u;
          if ((place & (page - 1)) == 0) {
            const int entry = place >> g.page_shift;
            a.page_table[int64_t(s) * g.max_pages + entry] = a.free_pages[nf - 1 - (sh.rank[lo] + entry)];
          }
        }
        for (int u = mine0; u < mine1; ++u) {
          const int e = u - t;
          a.token_slot[u] = e == 0 ? vs[0] : e == 1 ? vs[1] : e == 2 ? vs[2] : vs[3];
          a.token_index[u] = e == 0 ? vi[0] : e == 1 ? vi[1] : e == 2 ? vi[2] : vi[3];
          if (a.token_pos) a.token_pos[u] = e == 0 ? vp[0] : e == 1 ? vp[1] : e == 2 ? vp[2] : vp[3];
        }
      }
    }
    sum += all;
    pages += int(lacked);
    __syncthreads();
  }
  if (kTokens) {  // behind the last request: padding
    for (int t = max(from, int(min(sum, uint64_t(a.max_tokens)))) + tid; t < to; t += THREADS) {
      a.token_slot[t] = 0;
      a.token_index[t] = 0;
      if (a.token_pos) a.token_pos[t] = 0;
    }
  }
  if (kCounts) {
    if ((tid & 63) == 0) sh.waves[0][tid >> 6] = uint32_t(taken);
    __syncthreads();
    if (tid == 0) {
      uint32_t most = 0;
      for (int i = 0; i < THREADS / 64; ++i) most = max(most, sh.waves[0][i]);
      a.n_free_out[0] = nf - int(most);
    }
  }
}

// --------------------------------------------------------------- release --
// One workgroup; requests THREADS at a time.  A wave counts the pages of its requests, a sum
// over the requests gives each its place in the list, and the wave moves them there.  Entries are
// read kEach * 64 at a time, and those of a wave's next request before the present one's are used:
// 64 requests of some 260 pages were a chain of 64 reads (17.6 us) and are one of 8 (12.2 us).
// Where no request has more than kFew (a page or two behind a budget), a thread reads its own (32
// requests that free one page each 3.4 us, by waves 3.7).
constexpr int kReleaseThreads = 1024, kFew = 4;

__global__ __launch_bounds__(kReleaseThreads) void kv_release_kernel(KvGeom g, ReleaseArgs a) {
  constexpr int THREADS = kReleaseThreads, WAVES = THREADS / 64, kEach = 8, kStep = 64 * kEach;
  __shared__ uint32_t waves[WAVES];
  __shared__ int count[THREADS], row[THREADS], e0[THREADS], e1[THREADS];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int page = 1 << g.page_shift;
  const int have = a.n_free[0], nf = max(0, min(have, a.free_capacity));
  if (tid == 0 && have != nf) set_err(g.err, GDN_ERRW_BAD_SEQLENS);
  int64_t held = nf;  // the list's length so far
  for (int b0 = 0; b0 < a.batch; b0 += THREADS) {
    const int b = b0 + tid, requests = min(THREADS, a.batch - b0);
    auto given = [&](int id) { return id > 0 && id < g.pages; };
    int n = 0;  // entries of the thread's request
    if (b < a.batch) {
      const int slot = a.slot_table[b], len = a.kv_len[b], keep = a.keep ? a.keep[b] : 0;
      const bool live = slot > 0 && slot < g.slots, ok = len >= 0 && len <= g.capacity && keep >= 0;
      if (slot >= g.slots) set_err(g.err, GDN_ERRW_BAD_SLOT);
      else if (live && !ok) set_err(g.err, GDN_ERRW_BAD_SEQLENS);
      const bool on = live && ok && keep < len;
      row[tid] = on ? slot : 0;
      e0[tid] = on ? (keep + page - 1) >> g.page_shift : 0;
      e1[tid] = on ? (len + page - 1) >> g.page_shift : 0;
      n = e1[tid] - e0[tid];
    }
    uint64_t all;
    if (!__syncthreads_or(n > kFew)) {  // a thread has its request for itself
      int32_t *entries = a.page_table + (n > 0 ? int64_t(row[tid]) * g.max_pages + e0[tid] : 0);
      int id[kFew];
#pragma unroll
      for (int u = 0; u < kFew; ++u) id[u] = u < n ? entries[u] : 0;
      uint32_t mine = 0;
#pragma unroll
      for (int u = 0; u < kFew; ++u) mine += given(id[u]) ? 1 : 0;
      int64_t to = held + int64_t(block_scan<THREADS>(mine, waves, &all));
#pragma unroll
      for (int u = 0; u < kFew; ++u) {
        const bool on = given(id[u]);
        if (on && to < a.free_capacity) {
          a.free_pages[to] = id[u];
          entries[u] = 0;
        } else if (u < n) {
          set_err(g.err, GDN_ERRW_BAD_PAGE);
        }
        to += on ? 1 : 0;
      }
      held += int64_t(all);
      __syncthreads();
      continue;
    }
    // the entries of request r from `base` on; 0 behind its last
    auto read = [&](int r, int base, int *id) {
      const int32_t *entries = a.page_table + int64_t(row[r]) * g.max_pages;
#pragma unroll
      for (int u = 0; u < kEach; ++u) {
        const int e = base + 64 * u + lane;
        id[u] = e < e1[r] ? entries[e] : 0;
      }
    };
    // f(r, base, id) for all of the wave's requests and entries, in order
    auto each = [&](auto f) {
      int id[kEach], next[kEach];
      if (w < requests) read(w, e0[w], id);
      for (int r = w; r < requests; r += WAVES) {
        if (r + WAVES < requests) read(r + WAVES, e0[r + WAVES], next);
        for (int base = e0[r];;) {
          f(r, base, id);
          if ((base += kStep) >= e1[r]) break;
          read(r, base, id);
        }
#pragma unroll
        for (int u = 0; u < kEach; ++u) id[u] = next[u];
      }
    };
    each([&](int r, int base, const int *id) {
      uint32_t n = 0;
#pragma unroll
      for (int u = 0; u < kEach; ++u) n += uint32_t(__builtin_popcountll(__ballot(given(id[u]))));
      if (lane == 0) count[r] = int(n) + (base == e0[r] ? 0 : count[r]);
    });
    __syncthreads();
    const uint64_t before = block_scan<THREADS>(tid < requests ? uint32_t(count[tid]) : 0, waves, &all);
    if (tid < requests) count[tid] = int(before);
    __syncthreads();
    int64_t at = 0;
    each([&](int r, int base, const int *id) {
      int32_t *entries = a.page_table + int64_t(row[r]) * g.max_pages;
      if (base == e0[r]) at = held + count[r];
#pragma unroll
      for (int u = 0; u < kEach; ++u) {
        const int e = base + 64 * u + lane;
        const bool on = given(id[u]);
        const uint64_t mask = __ballot(on);
        const int64_t to = at + lanes_below(mask, 0);
        if (on && to < a.free_capacity) {
          a.free_pages[to] = id[u];
          entries[e] = 0;
        } else if (e < e1[r]) {
          set_err(g.err, GDN_ERRW_BAD_PAGE);
        }
        at += __builtin_popcountll(mask);
      }
    });
    held += int64_t(all);
    __syncthreads();
  }
  if (tid == 0) a.n_free_out[0] = int(min(held, int64_t(a.free_capacity)));
}

}  // namespace

hipError_t launch_kv_batch_map(const gdn_kv_pool *p, const MapArgs &a, hipStream_t s) {
  const KvGeom g = kv_geom(p, 0);
  // one workgroup up to 2048 tokens: 16 requests of 128 tokens 6.3 us (6.7 in two launches), one of 512
  // 4.1 (5.9), but 16 of 256 9.5 (6.6) and 64 of 125 19.5 (7.0)
  constexpr int T = 256, kOne = 2048, kPart = T * kTokensPer;
  if (a.max_tokens <= kOne) {
    hipLaunchKernelGGL((kv_batch_map_kernel<T, true, true>), dim3(1), dim3(T), 0, s, g, a, 0);
    return hipGetLastError();
  }
  const unsigned groups = unsigned((a.max_tokens + kPart - 1) / kPart);
  hipLaunchKernelGGL((kv_batch_map_kernel<T, true, false>), dim3(groups), dim3(T), 0, s, g, a, kPart);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((kv_batch_map_kernel<T, false, true>), dim3(1), dim3(T), 0, s, g, a, 0);
  return hipGetLastError();
}

hipError_t launch_kv_release(const gdn_kv_pool *p, const ReleaseArgs &a, hipStream_t s) {
  hipLaunchKernelGGL(kv_release_kernel, dim3(1), dim3(kReleaseThreads), 0, s, kv_geom(p, 0), a);
  return hipGetLastError();
}

}  // namespace gdn
