// Writing new K and V rows into a paged cache (quantising them on the way) and reading
// cached rows back into contiguous bf16.
//
// Both are one pass over the rows: their floor is the rows read and written once at the
// copy rate. A row's d values belong to d/8 neighbouring lanes (d/16 where it is quantised),
// so that the row's largest magnitude is a few shuffles and nothing is staged.
#include <algorithm>
#include <type_traits>

#include "paged.cuh"

namespace sa {
namespace {

constexpr int kThreads = 256;
// Rows of K and of V in flight per thread of a read, and blocks of one that has work for them:
// 4 x 16 heads x 63,960 e4m3 rows 507 us; two rows 511, with twice the blocks 508 (1,560 bf16
// rows a head 20.7, 21.0 and 20.6).
constexpr int kReadUnroll = 4;
constexpr int kReadBlocks = 148 * 16;

SA_DEVI uint32_t max_abs2(uint32_t a, uint32_t b) {   // of bf16 pairs; NaN stays NaN
  const __nv_bfloat162 m = __hmax2_nan(__habs2(*reinterpret_cast<const __nv_bfloat162*>(&a)),
                                       __habs2(*reinterpret_cast<const __nv_bfloat162*>(&b)));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// A lane's largest magnitude of 16 values.
SA_DEVI uint32_t lane_top(const uint4 (&x)[2]) {
  return max_abs2(max_abs2(max_abs2(x[0].x, x[0].y), max_abs2(x[0].z, x[0].w)),
                  max_abs2(max_abs2(x[1].x, x[1].y), max_abs2(x[1].z, x[1].w)));
}
// The largest magnitudes of a K row (low half) and a V row (high half) as bf16 bits, over the
// LPR lanes that share the rows.
template <int LPR>
SA_DEVI uint32_t row_tops(const uint4 (&k)[2], const uint4 (&v)[2]) {
  const uint32_t a = lane_top(k), b = lane_top(v);
  uint32_t top = max_abs2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) top = max_abs2(top, __shfl_xor_sync(~0u, top, o));
  return top;
}

constexpr uint32_t kInf = 0x7F80u;

// A row with infinities or NaN (rare): zeros in their places for the scale (NANS false), or
// NaN in the places of infinities for the codes.
template <bool NANS>
SA_DEVI uint4 without_inf(uint4 x) {
  uint32_t* w = &x.x;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if ((w[i] >> (16 * j) & 0x7FFFu) >= kInf)
        w[i] = NANS ? w[i] | 0x7FFFu << (16 * j) : w[i] & ~(0xFFFFu << (16 * j));
  return x;
}

// E8M0 of the smallest power of two s with top / s <= 448 = 1.75 * 2^8: the exponent of
// top less 8, one more when its significand is above 1.75; 1 for a row of zeros, never
// below 2^-126 (so that s and 1/s are normal fp32).
SA_DEVI uint32_t row_scale(uint32_t top) {
  if (top == 0) return 127u;
  const int e = (int)(top >> 7) - 8 + ((top & 0x7Fu) > 0x60u);
  return (uint32_t)max(e, 1);
}

// Four bf16 pairs * 2^(127 - s) -> eight e4m3 codes. The product is exact in bf16 (what would
// fall below bf16's smallest normal value is far below e4m3's).
SA_DEVI uint2 row_codes(const uint4& x, uint32_t s) {
  const uint32_t inv = (254u - s) * 0x00800080u;
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]),
                                     *reinterpret_cast<const __nv_bfloat162*>(&inv));
    const uint32_t v = *reinterpret_cast<const uint32_t*>(&y);
    c[i] = __nv_cvt_float2_to_fp8x2(make_float2(bf16_lo(v), bf16_hi(v)), __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
}

// Scales of a K row (low half) and a V row (high half); their values ready for row_codes().
// Every lane of the warp calls.
template <int LPR>
SA_DEVI uint32_t quantise(uint4 (&k)[2], uint4 (&v)[2]) {
  uint32_t top = row_tops<LPR>(k, v);
  if (__any_sync(~0u, (top & 0xFFFFu) >= kInf || (top >> 16) >= kInf)) {
    const uint4 kf[2] = {without_inf<false>(k[0]), without_inf<false>(k[1])};
    const uint4 vf[2] = {without_inf<false>(v[0]), without_inf<false>(v[1])};
    top = row_tops<LPR>(kf, vf);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      k[i] = without_inf<true>(k[i]);
      v[i] = without_inf<true>(v[i]);
    }
  }
  return row_scale(top & 0xFFFFu) | row_scale(top >> 16) << 16;
}

// A thread brings two 16-byte pieces of K and of V: of one row (8-bit rows: half the shuffles
// and scales a row, 18.4 -> 16.4 us for 64 heads x 1,560 rows against one piece), or of a row
// each. A block takes the rows of one head's tokens, or (FLAT: few tokens) of all heads' in
// (head, token) order.
template <int D, bool E4M3>
struct Append {
  static constexpr int kLanes = E4M3 ? D / 16 : D / 8;      // of a row
  static constexpr int kRows = kThreads / kLanes;           // of a pass
  static constexpr int kPasses = E4M3 ? 1 : 2;
};

template <int D, bool E4M3, bool FLAT>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(CacheAppendArgs p) {
  using A = Append<D, E4M3>;
  constexpr int LPR = A::kLanes, PASSES = FLAT ? 1 : A::kPasses;
  const int b = FLAT ? blockIdx.y : blockIdx.z;
  const int start = p.start[b];
  int n = p.count ? p.count[b] : p.T;
  if (n < 0 || n > p.T || start < 0) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && p.c.err_flag)
      atomicOr(p.c.err_flag, SA_FLAG_INDEX_BIT);
    n = start < 0 || n < 0 ? 0 : p.T;
  }
  const int in_page = (1 << p.c.page_log2) - 1, lane = threadIdx.x % LPR;
  const uint32_t r0 = blockIdx.x * (A::kRows * PASSES) + threadIdx.x / LPR;
  uint32_t h = FLAT ? r0 / (uint32_t)p.T : blockIdx.y, t0 = FLAT ? r0 - h * (uint32_t)p.T : r0;
  if (FLAT && h >= (uint32_t)p.c.H) {
    h = 0;
    t0 = (uint32_t)p.T;
  }
  const uint16_t* kp = p.k + b * p.ks.b + h * p.ks.h + lane * 8;
  const uint16_t* vp = p.v + b * p.vs.b + h * p.vs.h + lane * 8;
  const int32_t* table = p.c.table + b * p.c.table_stride;
  uint4 kx[2], vx[2];
  int pg[PASSES];
  const uint4 zero = make_uint4(0, 0, 0, 0);
  kx[0] = kx[1] = vx[0] = vx[1] = zero;
#pragma unroll
  for (int u = 0; u < PASSES; ++u) {
    const uint32_t t = t0 + u * A::kRows;
    pg[u] = -1;
    if (t < (uint32_t)n) {
      const uint32_t lp = ((uint32_t)start + t) >> p.c.page_log2;     // both below 2^31
      if (lp < (uint32_t)p.c.table_width) pg[u] = table[lp];
      kx[u] = __ldg(reinterpret_cast<const uint4*>(kp + t * p.ks.t));
      vx[u] = __ldg(reinterpret_cast<const uint4*>(vp + t * p.vs.t));
      if constexpr (E4M3) {
        kx[1] = __ldg(reinterpret_cast<const uint4*>(kp + t * p.ks.t) + LPR);
        vx[1] = __ldg(reinterpret_cast<const uint4*>(vp + t * p.vs.t) + LPR);
      }
    }
  }
  uint32_t scale = 0;
  if constexpr (E4M3) scale = quantise<LPR>(kx, vx);
#pragma unroll
  for (int u = 0; u < PASSES; ++u) {
    const uint32_t t = t0 + u * A::kRows;
    if ((unsigned)pg[u] >= (unsigned)p.c.num_pages) {
      if (t < (uint32_t)n && p.c.err_flag) atomicOr(p.c.err_flag, SA_FLAG_INDEX_BIT);
      continue;
    }
    const int64_t dst = (((int64_t)pg[u] * p.c.H + h) << p.c.page_log2) + (((uint32_t)start + t) & in_page);
    if constexpr (E4M3) {
      uint2* kd = reinterpret_cast<uint2*>(p.c.k) + dst * (D / 8) + lane;
      uint2* vd = reinterpret_cast<uint2*>(p.c.v) + dst * (D / 8) + lane;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        kd[i * LPR] = row_codes(kx[i], scale & 0xFFFFu);
        vd[i * LPR] = row_codes(vx[i], scale >> 16);
      }
      if (lane == 0) {
        p.c.k_scale[dst] = (uint8_t)scale;
        p.c.v_scale[dst] = (uint8_t)(scale >> 16);
      }
    } else {
      reinterpret_cast<uint4*>(p.c.k)[dst * LPR + lane] = kx[u];
      reinterpret_cast<uint4*>(p.c.v)[dst * LPR + lane] = vx[u];
    }
  }
}

// Eight e4m3 codes times the row's scale -> eight bf16.
SA_DEVI uint4 row_values(const uint2& x, float s) {
  const uint32_t w[2] = {x.x, x.y};
  uint32_t y[4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t h = e4m3x2_to_f16x2(w[i] >> (16 * j));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      y[2 * i + j] = pack_bf16(f.x * s, f.y * s);
    }
  return make_uint4(y[0], y[1], y[2], y[3]);
}

// A block takes every gridDim.x-th tile of a sequence's rows, counted from its first one: how
// many rows there are is known on the device only.
template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(CacheReadArgs p) {
  constexpr int LPR = D / 8, RPP = kThreads / LPR;
  using Word = std::conditional_t<E4M3, uint2, uint4>;    // a lane's eight values as they are held
  const int h = blockIdx.y, b = blockIdx.z;
  int n = seq_len(p.c, p.lens, b), f = p.first ? p.first[b] : 0;
  if (n > p.N || f < 0) {
    if (threadIdx.x == 0 && p.c.err_flag) atomicOr(p.c.err_flag, SA_FLAG_INDEX_BIT);
    n = min(n, p.N);
    f = max(f, 0);
  }
  const int in_page = (1 << p.c.page_log2) - 1, lane = threadIdx.x % LPR;
  uint16_t* kd = p.k + b * p.ks.b + h * p.ks.h + lane * 8;
  uint16_t* vd = p.v + b * p.vs.b + h * p.vs.h + lane * 8;
  for (int64_t t0 = f + (int64_t)blockIdx.x * (RPP * kReadUnroll) + threadIdx.x / LPR; t0 < n;
       t0 += (int64_t)gridDim.x * (RPP * kReadUnroll)) {
    Word kx[kReadUnroll], vx[kReadUnroll];
    float ks[kReadUnroll], vs[kReadUnroll];
    int pg[kReadUnroll];
#pragma unroll
    for (int u = 0; u < kReadUnroll; ++u) {
      const int64_t t = t0 + u * RPP;
      pg[u] = t < n ? pool_page(p.c, b, (int)(t >> p.c.page_log2)) : -1;
    }
#pragma unroll
    for (int u = 0; u < kReadUnroll; ++u) {
      if (pg[u] < 0) continue;
      const int64_t src = (((int64_t)pg[u] * p.c.H + h) << p.c.page_log2) + ((t0 + u * RPP) & in_page);
      kx[u] = __ldg(reinterpret_cast<const Word*>(p.c.k) + src * LPR + lane);
      vx[u] = __ldg(reinterpret_cast<const Word*>(p.c.v) + src * LPR + lane);
      if constexpr (E4M3) {
        ks[u] = e8m0_value(p.c.k_scale[src]);
        vs[u] = e8m0_value(p.c.v_scale[src]);
      }
    }
#pragma unroll
    for (int u = 0; u < kReadUnroll; ++u) {
      if (pg[u] < 0) continue;
      const int64_t t = t0 + u * RPP;
      if constexpr (E4M3) {
        *reinterpret_cast<uint4*>(kd + t * p.ks.t) = row_values(kx[u], ks[u]);
        *reinterpret_cast<uint4*>(vd + t * p.vs.t) = row_values(vx[u], vs[u]);
      } else {
        *reinterpret_cast<uint4*>(kd + t * p.ks.t) = kx[u];
        *reinterpret_cast<uint4*>(vd + t * p.vs.t) = vx[u];
      }
    }
  }
}

// A head's tokens fill a block's rows, or the rows of all heads are dealt out in one.
template <int D, bool E4M3>
cudaError_t append_t(const CacheAppendArgs& p, cudaStream_t st) {
  using A = Append<D, E4M3>;
  constexpr int per = A::kRows * A::kPasses;
  if (p.T >= per) {
    const dim3 grid((unsigned)(((long long)p.T + per - 1) / per), (unsigned)p.c.H, (unsigned)p.B);
    cache_append_kernel<D, E4M3, false><<<grid, kThreads, 0, st>>>(p);
  } else {
    const dim3 grid((unsigned)(((long long)p.c.H * p.T + A::kRows - 1) / A::kRows), (unsigned)p.B);
    cache_append_kernel<D, E4M3, true><<<grid, kThreads, 0, st>>>(p);
  }
  return cudaGetLastError();
}

template <int D, bool E4M3>
cudaError_t read_t(const CacheReadArgs& p, cudaStream_t st) {
  constexpr int per = kThreads / (D / 8) * kReadUnroll;
  const long long bh = (long long)p.B * p.c.H, tiles = ((long long)p.N + per - 1) / per;
  const long long share = (kReadBlocks + bh - 1) / bh;
  const dim3 grid((unsigned)std::min(tiles, share), (unsigned)p.c.H, (unsigned)p.B);
  cache_read_kernel<D, E4M3><<<grid, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_append(const CacheAppendArgs& p, cudaStream_t st) {
  if (p.c.d == 64) return p.c.e4m3 ? append_t<64, true>(p, st) : append_t<64, false>(p, st);
  return p.c.e4m3 ? append_t<128, true>(p, st) : append_t<128, false>(p, st);
}

cudaError_t launch_cache_read(const CacheReadArgs& p, cudaStream_t st) {
  if (p.c.d == 64) return p.c.e4m3 ? read_t<64, true>(p, st) : read_t<64, false>(p, st);
  return p.c.e4m3 ? read_t<128, true>(p, st) : read_t<128, false>(p, st);
}

}  // namespace sa
