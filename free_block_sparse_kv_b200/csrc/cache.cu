// Writing new K and V rows into a paged cache (quantising them on the way) and reading
// cached rows back into contiguous bf16.
//
// Both are one pass over the rows: their floor is the rows read and written once at the
// copy rate. A row's d values belong to d/8 neighbouring lanes (append) or d/16 (8-bit
// read), so that the row's largest magnitude is a few shuffles and nothing is staged.
#include "paged.cuh"

namespace sa {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;  // rows of K and of V in flight per thread

// The row's largest finite magnitude as bf16 bits, over the LPR lanes that share the row.
template <int LPR>
SA_DEVI uint32_t row_top(const uint4& x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = w[i] & 0x7FFF7FFFu;
    top = __vmaxu2(top, a & ~__vcmpgeu2(a, 0x7F807F80u));  // infinities and NaN left out
  }
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(~0u, top, o));
  return max(top & 0xFFFFu, top >> 16);
}

// E8M0 of the smallest power of two s with top / s <= 448 = 1.75 * 2^8: the exponent of
// top less 8, one more when its significand is above 1.75; 1 for a row of zeros, never
// below 2^-126 (so that s and 1/s are normal fp32).
SA_DEVI uint32_t row_scale(uint32_t top) {
  if (top == 0) return 127u;
  const int e = (int)(top >> 7) - 8 + ((top & 0x7Fu) > 0x60u);
  return (uint32_t)max(e, 1);
}

// Four bf16 pairs * 2^(127 - s) -> eight e4m3 codes; infinities become NaN codes.
SA_DEVI uint2 row_codes(const uint4& x, uint32_t s) {
  const float inv = __uint_as_float((254u - s) << 23);
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t bad = __vcmpgeu2(w[i] & 0x7FFF7FFFu, 0x7F807F80u);
    const uint32_t v = w[i] | (bad & 0x7FFF7FFFu);
    c[i] = __nv_cvt_float2_to_fp8x2(make_float2(bf16_lo(v) * inv, bf16_hi(v) * inv),
                                    __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(CacheAppendArgs p) {
  constexpr int LPR = D / 8, RPP = kThreads / LPR;
  const int b = blockIdx.y;
  const int start = p.start[b];
  int n = p.count ? p.count[b] : p.T;
  if (n < 0 || n > p.T || start < 0) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && p.c.err_flag)
      atomicOr(p.c.err_flag, SA_FLAG_INDEX_BIT);
    n = start < 0 || n < 0 ? 0 : p.T;
  }
  const int page = 1 << p.c.page_log2, lane = threadIdx.x % LPR;
  const long long rows = (long long)p.c.H * p.T;
  const long long r0 = (long long)blockIdx.x * (RPP * kUnroll) + threadIdx.x / LPR;
  uint4 kx[kUnroll], vx[kUnroll];
  int64_t dst[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long r = r0 + u * RPP;
    dst[u] = -1;
    kx[u] = vx[u] = make_uint4(0, 0, 0, 0);
    if (r >= rows) continue;
    const int h = (int)((uint32_t)r / (uint32_t)p.T), t = (int)((uint32_t)r % (uint32_t)p.T);
    if (t >= n) continue;
    const int64_t pos = (int64_t)start + t;
    const int64_t lp = pos >> p.c.page_log2;
    if (lp >= p.c.table_width) {
      if (p.c.err_flag) atomicOr(p.c.err_flag, SA_FLAG_INDEX_BIT);
      continue;
    }
    const int pg = pool_page(p.c, b, (int)lp);
    if (pg < 0) continue;
    dst[u] = (((int64_t)pg * p.c.H + h) << p.c.page_log2) + (pos & (page - 1));
    kx[u] = __ldg(reinterpret_cast<const uint4*>(p.k + b * p.ks.b + h * p.ks.h + t * p.ks.t) + lane);
    vx[u] = __ldg(reinterpret_cast<const uint4*>(p.v + b * p.vs.b + h * p.vs.h + t * p.vs.t) + lane);
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    if constexpr (E4M3) {
      const uint32_t ks = row_scale(row_top<LPR>(kx[u])), vs = row_scale(row_top<LPR>(vx[u]));
      if (dst[u] < 0) continue;
      reinterpret_cast<uint2*>(p.c.k)[dst[u] * LPR + lane] = row_codes(kx[u], ks);
      reinterpret_cast<uint2*>(p.c.v)[dst[u] * LPR + lane] = row_codes(vx[u], vs);
      if (lane == 0) {
        p.c.k_scale[dst[u]] = (uint8_t)ks;
        p.c.v_scale[dst[u]] = (uint8_t)vs;
      }
    } else {
      if (dst[u] < 0) continue;
      reinterpret_cast<uint4*>(p.c.k)[dst[u] * LPR + lane] = kx[u];
      reinterpret_cast<uint4*>(p.c.v)[dst[u] * LPR + lane] = vx[u];
    }
  }
}

// Sixteen e4m3 codes times the row's scale -> sixteen bf16 (two 16-byte words).
SA_DEVI void row_values(const uint4& x, float s, uint4 out[2]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t h = e4m3x2_to_f16x2(w[i] >> (16 * j));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      y[2 * i + j] = pack_bf16(f.x * s, f.y * s);
    }
  out[0] = make_uint4(y[0], y[1], y[2], y[3]);
  out[1] = make_uint4(y[4], y[5], y[6], y[7]);
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(CacheReadArgs p) {
  constexpr int LPR = E4M3 ? D / 16 : D / 8, RPP = kThreads / LPR;
  const int h = blockIdx.y, b = blockIdx.z;
  int n = seq_len(p.c, p.lens, b), f = p.first ? p.first[b] : 0;
  if (n > p.N || f < 0) {
    if (threadIdx.x == 0 && p.c.err_flag) atomicOr(p.c.err_flag, SA_FLAG_INDEX_BIT);
    n = min(n, p.N);
    f = max(f, 0);
  }
  const int page = 1 << p.c.page_log2, lane = threadIdx.x % LPR;
  const int64_t t0 = (int64_t)blockIdx.x * (RPP * kUnroll) + threadIdx.x / LPR;
  uint4 kx[kUnroll], vx[kUnroll];
  float ks[kUnroll], vs[kUnroll];
  bool live[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t t = t0 + u * RPP;
    live[u] = false;
    if (t < f || t >= n) continue;
    const int pg = pool_page(p.c, b, (int)(t >> p.c.page_log2));
    if (pg < 0) continue;
    live[u] = true;
    const int64_t src = (((int64_t)pg * p.c.H + h) << p.c.page_log2) + (t & (page - 1));
    kx[u] = __ldg(reinterpret_cast<const uint4*>(p.c.k) + src * LPR + lane);
    vx[u] = __ldg(reinterpret_cast<const uint4*>(p.c.v) + src * LPR + lane);
    if (E4M3) {
      ks[u] = e8m0_value(p.c.k_scale[src]);
      vs[u] = e8m0_value(p.c.v_scale[src]);
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    if (!live[u]) continue;
    const int64_t t = t0 + u * RPP;
    uint4* kd = reinterpret_cast<uint4*>(p.k + b * p.ks.b + h * p.ks.h + t * p.ks.t);
    uint4* vd = reinterpret_cast<uint4*>(p.v + b * p.vs.b + h * p.vs.h + t * p.vs.t);
    if constexpr (E4M3) {
      uint4 y[2];
      row_values(kx[u], ks[u], y);
      kd[2 * lane] = y[0];
      kd[2 * lane + 1] = y[1];
      row_values(vx[u], vs[u], y);
      vd[2 * lane] = y[0];
      vd[2 * lane + 1] = y[1];
    } else {
      kd[lane] = kx[u];
      vd[lane] = vx[u];
    }
  }
}

template <int D, bool E4M3>
cudaError_t append_t(const CacheAppendArgs& p, cudaStream_t st) {
  constexpr int per = kThreads / (D / 8) * kUnroll;
  const long long rows = (long long)p.c.H * p.T;
  const dim3 grid((unsigned)((rows + per - 1) / per), (unsigned)p.B);
  cache_append_kernel<D, E4M3><<<grid, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <int D, bool E4M3>
cudaError_t read_t(const CacheReadArgs& p, cudaStream_t st) {
  constexpr int per = kThreads / (E4M3 ? D / 16 : D / 8) * kUnroll;
  const dim3 grid((unsigned)(((long long)p.N + per - 1) / per), (unsigned)p.c.H, (unsigned)p.B);
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
