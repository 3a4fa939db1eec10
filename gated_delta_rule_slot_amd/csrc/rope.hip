// rope.hip -- rotary positions of queries and keys, and the append of keys and values to the
// paged cache (formulas: include/gdn_kv.h).
//
// A pair (x, y) of a head's row is turned by the angle position * freq_i.  A thread has 16
// values of a row: 8 pairs of the turned part (two runs of 8 rot_dim / 2 apart, or 16 adjacent
// ones where the pairs are adjacent), or 16 values that are passed on.  It has the same place
// in every row that it takes, so the 8 angles of its token are worked out once, and a wave goes
// over a token's heads, D / 16 lanes a head.  Bound by the bytes.
//
// The angle is worked out in turns in fp64 and brought to [-1/2, 1/2] before it is rounded to
// fp32: its error is 2^-24 of a turn at most however far the position (fp32 would be wrong by
// whole radians at position 10^7).  Everything else is fp32, and each output is rounded once.
//
// Measured: 6144 tokens of 32 + 2 * 8 heads of 128 into e4m3, 139 MB, 34-36 us (29 at a copy's rate);
// 128 tokens of 16 + 2 * 2 heads of 256 4.5 us, latency.
#include <algorithm>
#include <cmath>

#include "kv.hpp"
#include "lanes.hpp"

namespace gdn {
namespace {

constexpr int kThreads = 256;
typedef const int32_t __attribute__((address_space(4))) *table_t;

__device__ __forceinline__ void widen8(const u32x4 &x, float *f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(x[i] << 16);
    f[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ u32x4 narrow8(const float *f) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  return r;
}

// waves a token's rows are divided over: split
template <int D, bool kF8, bool kAdjacent>
__global__ __launch_bounds__(kThreads) void rope_append_kernel(KvGeom g, RopeArgs a, int split) {
  constexpr int PIECES = D / 16, ROWS = 64 / PIECES;  // lanes of a row, rows of a wave
  const int lane = threadIdx.x & 63;
  const int64_t unit = flat_block() * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (unit >= int64_t(a.n) * split) return;
  const int token = int(unit / split), part = int(unit - int64_t(token) * split);
  const int slot = ((table_t)a.slot_ids)[token], place = ((table_t)a.index)[token];
  const bool teller = part == 0 && lane == 0;
  if (slot <= 0 || slot >= g.slots) {
    if (teller && slot >= g.slots) set_err(g.err, GDN_ERRW_BAD_SLOT);
    return;
  }
  int64_t base = -1;  // the token's row of key-value head 0; a head is page_size rows further
  if (place < 0 || place >= g.capacity) {
    if (teller) set_err(g.err, GDN_ERRW_BAD_SEQLENS);
  } else {
    base = kv_row(g, slot, 0, place);
    if (base < 0 && teller) set_err(g.err, GDN_ERRW_BAD_PAGE);
  }
  const int position = ((table_t)a.position)[token];
  const int piece = lane % PIECES;
  const bool turned = piece < a.rot_dim / 16;
  // the thread's two runs of 8 values
  const int d0 = !turned || kAdjacent ? 16 * piece : 8 * piece;
  const int d1 = !turned || kAdjacent ? d0 + 8 : d0 + a.rot_dim / 2;
  float cs[8], sn[8];
  if (turned) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double turns = double(position) * (a.freqs[8 * piece + i] * 0.15915494309189533577);
      const float x = float(turns - rint(turns));
      sincospif(2.f * x, &sn[i], &cs[i]);
      sn[i] *= a.amplitude;
      cs[i] *= a.amplitude;
    }
  }
  const int all = a.q_heads + 2 * g.kv_heads;
  const int64_t q0 = token * a.q_stride, k0 = token * a.k_stride, v0 = token * a.v_stride;
#pragma unroll 2
  for (int r = part * ROWS + lane / PIECES; r < all; r += split * ROWS) {
    const bool query = r < a.q_heads, value = r >= a.q_heads + g.kv_heads;
    const int h = query ? r : value ? r - a.q_heads - g.kv_heads : r - a.q_heads;
    if (!query && base < 0) continue;
    const uint16_t *src = (query ? a.q + q0 : value ? a.v + v0 : a.k + k0) + int64_t(h) * D;
    u32x4 x = *reinterpret_cast<const u32x4 *>(src + d0), y = *reinterpret_cast<const u32x4 *>(src + d1);
    float f[16];
    widen8(x, f);
    widen8(y, f + 8);
    if (turned && !value) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float &u = kAdjacent ? f[2 * i] : f[i], &w = kAdjacent ? f[2 * i + 1] : f[8 + i];
        const float re = fmaf(u, cs[i], -(w * sn[i])), im = fmaf(w, cs[i], u * sn[i]);
        u = re;
        w = im;
      }
      x = narrow8(f);
      y = narrow8(f + 8);
    }
    if (query) {
      uint16_t *to = a.q_out + token * a.q_out_stride + int64_t(h) * D;
      *reinterpret_cast<u32x4 *>(to + d0) = x;
      *reinterpret_cast<u32x4 *>(to + d1) = y;
      continue;
    }
    const int64_t row = base + (int64_t(h) << g.page_shift);
    char *to = (value ? g.v : g.k) + row * D * (kF8 ? 1 : 2);
    if constexpr (kF8) {
      const float scale = value ? g.v_scale : g.k_scale;
      *reinterpret_cast<u32x2 *>(to + d0) = u32x2{f8_pack4(f, scale), f8_pack4(f + 4, scale)};
      *reinterpret_cast<u32x2 *>(to + d1) = u32x2{f8_pack4(f + 8, scale), f8_pack4(f + 12, scale)};
    } else {
      *reinterpret_cast<u32x4 *>(to + 2 * d0) = x;
      *reinterpret_cast<u32x4 *>(to + 2 * d1) = y;
    }
    if (!value && piece == 0) {
      const int64_t m = (int64_t(slot) * g.kv_heads + h) * g.capacity + place;
      if (g.mass) g.mass[m] = 0.f;
      if (g.pos) g.pos[m] = position;
    }
  }
}

template <int D>
hipError_t launch_d(const gdn_kv_pool *p, int layer, const RopeArgs &a, hipStream_t s) {
  const KvGeom g = kv_geom(p, layer);
  constexpr int ROWS = 64 / (D / 16);
  const int turns = (a.q_heads + 2 * g.kv_heads + ROWS - 1) / ROWS;  // of one wave over a token's rows
  // Few tokens: a wave for every turn, up to the waves that run at once.  128 tokens of 16 + 2 * 2 heads of
  // 256 4.4 us (one wave a token: 6.6), 512 6.1 (6.7), 2048 10.8 (11.0; all turns: 13.0); of 32 + 2 * 8 heads
  // of 128 into e4m3, 2048 tokens 12.1 (12.9; 17.0).
  const int split = int(std::max<int64_t>(1, std::min<int64_t>(turns, 4096 / a.n)));
  const int64_t units = int64_t(a.n) * split;
  const bool f8 = p->d.kv_dtype == GDN_F8_E4M3, adjacent = a.layout == GDN_ROPE_INTERLEAVED;
  const auto kernel = f8 ? (adjacent ? rope_append_kernel<D, true, true> : rope_append_kernel<D, true, false>)
                         : (adjacent ? rope_append_kernel<D, false, true> : rope_append_kernel<D, false, false>);
  hipLaunchKernelGGL(kernel, flat_grid((units + kThreads / 64 - 1) / (kThreads / 64)), dim3(kThreads), 0, s, g, a, split);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope_append(const gdn_kv_pool *p, int layer, const RopeArgs &a, hipStream_t s) {
  switch (p->d.head_dim) {
    case 64: return launch_d<64>(p, layer, a, s);
    case 128: return launch_d<128>(p, layer, a, s);
    case 256: return launch_d<256>(p, layer, a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace gdn
