// norm.hip -- block_norm: the norm after a block, its gate, the residual scale and sum,
// and the norm before the next block, in one pass over each row (formulas:
// include/gdn_kv.h).
//
// Every tensor is read or written once, so the call is bound by its bytes; a row stays in
// registers between the two reductions.  A row is spread over LANES threads, 8
// consecutive values (16 bytes of bf16) each, VPT such pieces a thread: few, wide rows get a
// thread per piece (256 rows of 4096: 512 threads 4.4 us, 256 threads of two pieces 5.0 us).
// Measured: 6144 x 32 rows of 128 with gate, 151 MB, 29.6-32.7 us (32 us at a copy's rate);
// 128 rows of 2048 with both norms, gate and residual 4.1 us, the launch and two sums.
#include "kv.hpp"
#include "lanes.hpp"

namespace gdn {
namespace {

constexpr int kNormThreads = 256;

__device__ __forceinline__ void widen8(const u32x4 &r, float *f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(r[i] << 16);
    f[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ u32x4 narrow8(const float *f) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  return r;
}
// kStream: the tensors do not fit the caches and are not kept there
template <bool kStream>
__device__ __forceinline__ u32x4 get16(const void *p) {
  const u32x4 *q = static_cast<const u32x4 *>(p);
  return kStream ? __builtin_nontemporal_load(q) : *q;
}
template <bool kStream>
__device__ __forceinline__ void put16(void *p, const u32x4 &v) {
  u32x4 *q = static_cast<u32x4 *>(p);
  if (kStream) __builtin_nontemporal_store(v, q);
  else *q = v;
}
// 8 values at element offset `at` of a bf16 or fp32 array
template <bool kStream>
__device__ __forceinline__ void load8(const void *p, int64_t at, bool f32, float *f) {
  if (f32) {
    const float *q = static_cast<const float *>(p) + at;
    const u32x4 lo = get16<kStream>(q), hi = get16<kStream>(q + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = __uint_as_float(lo[i]);
      f[4 + i] = __uint_as_float(hi[i]);
    }
  } else {
    widen8(get16<kStream>(static_cast<const uint16_t *>(p) + at), f);
  }
}

// Sum over a row's LANES threads, the same bits in each of them.
template <int LANES>
__device__ __forceinline__ float row_sum(float v, float *red) {
  if constexpr (LANES <= 64) {
    return group_sum<LANES>(v);
  } else {
    v = wave_sum(v);
    __syncthreads();  // the previous use of `red` is over
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < LANES / 64; ++i) t += red[i];
    return t;
  }
}

template <int LANES, int VPT, bool kStream>
__global__ __launch_bounds__((LANES > kNormThreads ? LANES : kNormThreads)) void block_norm_kernel(
    NormArgs a, int64_t rows) {
  constexpr int THREADS = LANES > kNormThreads ? LANES : kNormThreads;
  __shared__ float red[LANES > 64 ? LANES / 64 : 1];
  const int64_t row = flat_block() * (THREADS / LANES) + threadIdx.x / LANES;
  const bool live = row < rows;  // uniform over a row's threads
  const int l = threadIdx.x % LANES;
  const int64_t r0 = live ? row : 0;
  const int64_t token = r0 / a.groups;
  const int64_t in_token = (r0 - token * a.groups) * a.dim;
  const uint16_t *y = a.y + token * a.y_stride + in_token;
  const uint16_t *gate = a.gate ? a.gate + token * a.gate_stride + in_token : nullptr;
  const int64_t flat = r0 * a.dim;
  const bool wf32 = a.w_dtype == GDN_F32, rf32 = a.res_dtype == GDN_F32;
  const float one = (a.flags & GDN_F_NORM_PLUS_ONE) ? 1.f : 0.f;
  const float inv_dim = 1.f / float(a.dim);

  // all loads of the row are issued before anything waits
  u32x4 yr[VPT], gr[VPT];
  float u[VPT][8], res[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int d = 8 * (l + i * LANES);
    const bool on = live && d < a.dim;
    yr[i] = gr[i] = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) res[i][e] = 0.f;
    if (on) {
      yr[i] = get16<kStream>(y + d);
      if (gate) gr[i] = get16<kStream>(gate + d);
      if (a.residual) load8<kStream>(a.residual, flat + d, rf32, res[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) widen8(yr[i], u[i]);

  float inv = 1.f;
  if (a.w_post) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(u[i][e], u[i][e], ss);
    inv = 1.f / sqrtf(fmaf(row_sum<LANES>(ss, red), inv_dim, a.eps));
  }
  float s2 = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int d = 8 * (l + i * LANES);
    const bool on = live && d < a.dim;
    if (on) {
      if (a.w_post) {
        float w[8];
        load8<false>(a.w_post, d, wf32, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[i][e] = u[i][e] * inv * (one + w[e]);
      }
      if (gate) {
        float z[8];
        widen8(gr[i], z);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float sg = __builtin_amdgcn_rcpf(1.f + __expf(-z[e]));  // (within one unit)
          u[i][e] *= a.act == GDN_ACT_NONE ? z[e] : a.act == GDN_ACT_SILU ? z[e] * sg : sg;
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        u[i][e] = a.residual ? fmaf(a.scale, u[i][e], res[i][e]) : a.scale * u[i][e];
        s2 = fmaf(u[i][e], u[i][e], s2);
      }
      if (a.residual) {
        if (rf32) {
          u32x4 lo, hi;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            lo[e] = __float_as_uint(u[i][e]);
            hi[e] = __float_as_uint(u[i][4 + e]);
          }
          float *q = static_cast<float *>(a.residual_out) + flat + d;
          put16<kStream>(q, lo);
          put16<kStream>(q + 4, hi);
        } else {
          put16<kStream>(static_cast<uint16_t *>(a.residual_out) + flat + d, narrow8(u[i]));
        }
      }
    }
  }
  float inv2 = 1.f;
  if (a.w_pre) inv2 = 1.f / sqrtf(fmaf(row_sum<LANES>(s2, red), inv_dim, a.eps));
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int d = 8 * (l + i * LANES);
    if (live && d < a.dim) {
      if (a.w_pre) {
        float w[8];
        load8<false>(a.w_pre, d, wf32, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[i][e] = u[i][e] * inv2 * (one + w[e]);
      }
      put16<kStream>(a.out + flat + d, narrow8(u[i]));
    }
  }
}

template <int LANES, int VPT>
hipError_t launch_rows(const NormArgs &a, hipStream_t s) {
  constexpr int THREADS = LANES > kNormThreads ? LANES : kNormThreads;
  const int64_t rows = a.tokens * a.groups, per = THREADS / LANES;
  const dim3 grid = flat_grid((rows + per - 1) / per);
  // From 24 MB a tensor on: 4096 rows of 4096 (33 MB) 27.5 against 30.2 us, 8192 of 2048 32.5
  // against 36.9 us; below, the next kernel finds the rows in the caches (19 MB: no gain,
  // 128 rows of 2048: 4.4 against 4.1 us).
  if (rows * a.dim >= 12 << 20)
    hipLaunchKernelGGL((block_norm_kernel<LANES, VPT, true>), grid, dim3(THREADS), 0, s, a, rows);
  else
    hipLaunchKernelGGL((block_norm_kernel<LANES, VPT, false>), grid, dim3(THREADS), 0, s, a, rows);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_block_norm(const NormArgs &a, hipStream_t s) {
  const int vecs = a.dim / 8;
  if (vecs <= 8) return launch_rows<8, 1>(a, s);
  if (vecs <= 16) return launch_rows<16, 1>(a, s);
  if (vecs <= 32) return launch_rows<32, 1>(a, s);
  if (vecs <= 64) return launch_rows<64, 1>(a, s);
  if (vecs <= 256) return launch_rows<256, 1>(a, s);
  if (vecs <= 512) return launch_rows<512, 1>(a, s);
  if (vecs <= 1024) return launch_rows<512, 2>(a, s);
  if (vecs <= 2048) return launch_rows<1024, 2>(a, s);
  return launch_rows<1024, 4>(a, s);
}

}  // namespace gdn
