// Attention of the last T tokens of every sequence over its paged cache.
//
// Per (b, kv head h) and query row (g, t):  l_p = scale * q . k_p over the positions
// p < len - (T - 1 - t) of the listed pages,  o = sum e^(l_p - m) v_p / sum e^(l_p - m),
// lse = m + ln sum e^(l_p - m), with the running maximum m and sum kept in fp32 over one
// pass (online softmax). One block per query row: the simplest form.
#include "../../include/sparse_attn.h"
#include "paged.cuh"

namespace sa {
namespace {

constexpr int kT = 128;  // threads, and keys per tile

template <int D, bool E4M3>
SA_DEVI float cached(const void* base, const uint8_t* scale, int64_t row, int c) {
  if constexpr (E4M3) {
    const uint32_t h = e4m3x2_to_f16x2(static_cast<const uint8_t*>(base)[row * D + c]);
    return __low2float(*reinterpret_cast<const __half2*>(&h)) * e8m0_value(scale[row]);
  } else {
    return bf16_lo(static_cast<const uint16_t*>(base)[row * D + c]);
  }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kT) decode_kernel(DecodeArgs p) {
  __shared__ float sq[D], sp[kT], red[4];
  __shared__ int64_t srow[kT];
  __shared__ float so[kT];
  const int t = blockIdx.x % p.T, hq = blockIdx.x / p.T, b = blockIdx.y;
  const int h = hq / (p.Hq / p.c.H), tid = threadIdx.x;
  const int page = 1 << p.c.page_log2;
  const int len = seq_len(p.c, p.lens, b), sees = len - (p.T - 1 - t);
  int64_t keys = len;
  const int32_t* list = nullptr;
  if (p.kv_idx) {
    const int64_t seg = (int64_t)b * p.c.H + h;
    keys = (int64_t)min(max(p.kv_cnt[seg], 0), p.cap) << p.c.page_log2;
    list = p.kv_idx + seg * p.cap;
  }
  if (tid < D) sq[tid] = bf16_lo(p.q[b * p.qs.b + hq * p.qs.h + t * p.qs.t + tid]);
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int64_t v0 = 0; v0 < keys; v0 += kT) {
    __syncthreads();
    int64_t row = -1;
    float s = -INFINITY;
    const int64_t vi = v0 + tid;
    if (vi < keys) {
      int64_t lp = vi >> p.c.page_log2;
      if (list) lp = list[lp];
      const int64_t pos = (lp << p.c.page_log2) + (vi & (page - 1));
      if (lp >= 0 && lp < p.c.table_width && pos < sees) {
        const int pg = pool_page(p.c, b, (int)lp);
        if (pg >= 0) {
          row = (((int64_t)pg * p.c.H + h) << p.c.page_log2) + (vi & (page - 1));
          float acc = 0.f;
          for (int c = 0; c < D; ++c) acc += sq[c] * cached<D, E4M3>(p.c.k, p.c.k_scale, row, c);
          s = acc * p.scale;
        }
      }
    }
    srow[tid] = row;
    float top = s;
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, x));
    if (tid % 32 == 0) red[tid / 32] = top;
    __syncthreads();
    const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float ref = mn == -INFINITY ? 0.f : mn;
    const float w = expf(m - ref);
    sp[tid] = row < 0 ? 0.f : expf(s - ref);
    __syncthreads();
    l *= w;
    o *= w;
    m = mn;
    const int n = (int)min((int64_t)kT, keys - v0);
    for (int j = 0; j < n; ++j) l += sp[j];
    // d = 64: the two halves of the block take every other key
    for (int j = tid / D; j < n; j += kT / D)
      if (srow[j] >= 0) o += sp[j] * cached<D, E4M3>(p.c.v, p.c.v_scale, srow[j], tid % D);
  }
  so[tid] = o;
  __syncthreads();
  if (tid < D) {
    for (int j = tid + D; j < kT; j += D) o += so[j];
    const float y = l == 0.f ? 0.f : o / l;
    const int64_t row = ((int64_t)b * p.Hq + hq) * p.T + t;
    if (p.out_dtype == SA_OUT_F32)
      static_cast<float*>(p.out)[row * D + tid] = y;
    else
      static_cast<__nv_bfloat16*>(p.out)[row * D + tid] = __float2bfloat16(y);
    if (p.lse && tid == 0) p.lse[row] = l == 0.f ? -INFINITY : m + logf(l);
  }
}

template <int D, bool E4M3>
cudaError_t run(const DecodeArgs& p, cudaStream_t st) {
  decode_kernel<D, E4M3><<<dim3((unsigned)(p.Hq * p.T), (unsigned)p.B), kT, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

size_t decode_work_bytes(int, int, int, int, int, int) { return 0; }

cudaError_t launch_decode(const DecodeArgs& p, cudaStream_t st) {
  if (p.c.d == 64) return p.c.e4m3 ? run<64, true>(p, st) : run<64, false>(p, st);
  return p.c.e4m3 ? run<128, true>(p, st) : run<128, false>(p, st);
}

}  // namespace sa
