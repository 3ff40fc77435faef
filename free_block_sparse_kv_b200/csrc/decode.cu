// Attention of the last T tokens of every sequence over its paged cache.
//
// Per (b, kv head h) the R = (Hq / Hkv) * T query rows (g, t) that share the head's keys:
//   l_p = scale * q . k_p over the positions p < len - (T - 1 - t) of the listed pages,
//   o = sum e^(l_p - m) v_p / sum e^(l_p - m),   lse = m + ln sum e^(l_p - m),
// in one pass over K and V with a running maximum m and sum in fp32 (base 2). Every cached
// row is read once for all R rows, at 4 R d operations per 4 d (bf16) or 2 d + 2 (e4m3)
// bytes: HBM bounds it up to R of about 32, so the design is about keeping loads in flight
// and every SM equally loaded:
//  - The work is cut into steps of 4 KB of K and 4 KB of V (16 to 64 keys). All steps of all
//    (sequence, kv head, group of rows) segments form one line, in which every warp of a
//    grid of one CTA per SM takes an equal, contiguous share, whatever the lengths. Shares
//    are found on the device from the lengths (a scan of one weight per sequence), so a
//    captured graph follows the lengths.
//  - A warp streams its steps through its own ring of cp.async stages, 16 bytes a lane, with
//    no barrier between warps; it looks page numbers up one step ahead.
//  - A segment that ends inside the share it began in is written out at once; the others
//    leave (m, l, numerator) partials, joined first inside the CTA and then, for segments
//    that span CTAs, by a second small kernel. Orders are fixed: same bits every run.
//  - Products run on mma.sync with the keys as the M dimension (S^T = K Q^T, O^T = V^T P^T):
//    one query row wastes 7/8 of a tile, not 15/16, and the tensor work stays far below the
//    time of the loads. Larger tensor instructions would leave the bound where it is.
// Roundings below fp32: P enters its product as two 16-bit pieces (high and rest, 2^-17 of
// each weight for bf16, 2^-23 for f16), because one bf16 piece (2^-9) would show in an fp32
// output. e4m3 codes enter as f16, exactly; the query then enters as f16 times a power of
// two per row that brings its largest value to 2^14 (what f16 drops is below 2^-38 of that
// value). The scale of a V row is folded into its weight: numerator weights carry their own
// running maximum of l_p + log2(scale_p), so that no scale can overflow or starve them.
#include <algorithm>
#include <atomic>

#include "../../include/sparse_attn.h"
#include "paged.cuh"

namespace sa {
namespace {

constexpr int kWarps = 8;
constexpr int kStages = 3;
constexpr int kThreads = kWarps * 32;
constexpr int kBuckets = kThreads;     // scan entries kept in shared memory
constexpr int kNoPos = 0x7FFFFF00;     // position of keys that nothing attends
constexpr float kPvShift = 14.f;       // f16 weights are at most 2^14 (fp16 ends at 2^16)

// CTA c leaves its record for the joining kernel: the segment that starts in its share and
// runs past it (seg < 0: none), where that segment starts, and how the line was cut.
struct Record {
  long long seg, s0, n, total;
  int ctas, pad[3];
};

template <int D, bool E4M3, int NT>
struct Cfg {
  static constexpr int kRow = D * (E4M3 ? 1 : 2);     // bytes of a cached row
  static constexpr int kKeys = 4096 / kRow;           // keys per step
  static constexpr int kSub = kKeys / 16;             // 16-key tiles per step
  static constexpr int kChunks = kRow / 16;
  static constexpr int kRows = 8 * NT;                // query rows of a segment
  static constexpr int kPad = D + 4;                  // floats between staged rows
  static constexpr int kMeta = 160;                   // scales (2 x kKeys), tile positions
  static constexpr int kMt = D / 16;
  static constexpr size_t kSlot = (size_t)kRows * (D + 2);  // floats of a global partial
  static constexpr size_t kSmem = (size_t)kWarps * kStages * (8192 + kMeta);
};

// Rows of 64 bytes: two to a 128-byte line, so the XOR takes the row's second and third bit.
template <int ROW>
SA_DEVI uint32_t swz_row(int row, int chunk) {
  if constexpr (ROW == 64) return row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
  return swz(row, chunk, ROW);
}

SA_DEVI uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(d) : "r"(a));
  return d;
}
SA_DEVI float ex2a(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
SA_DEVI float col_max(float x) {   // over the eight lanes that hold one column's keys
  x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
  x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
  return fmaxf(x, __shfl_xor_sync(~0u, x, 16));
}
SA_DEVI float col_sum(float x) {
  x += __shfl_xor_sync(~0u, x, 4);
  x += __shfl_xor_sync(~0u, x, 8);
  return x + __shfl_xor_sync(~0u, x, 16);
}
// A maximum to subtract: 0 while nothing was attended (-inf - -inf would be NaN).
SA_DEVI float ref_of(float m) { return m == -INFINITY ? 0.f : m; }

// What the steps of one unit (a sequence, or with kept lists a sequence's kv head) look like.
struct Unit {
  int len, n;                 // attended length, steps of each of its segments
  long long keys;             // keys in list order
};

template <class CF>
SA_DEVI Unit unit_of(const DecodeArgs& p, int u) {
  Unit x;
  const int b = p.kv_idx ? u / p.c.H : u;
  x.len = seq_len(p.c, p.lens, b);
  x.keys = x.len;
  if (p.kv_idx)
    x.keys = x.len == 0 ? 0 : (long long)min(max(p.kv_cnt[u], 0), p.cap) << p.c.page_log2;
  x.n = (int)((x.keys + CF::kKeys - 1) / CF::kKeys);
  return x;
}

// A place on the line of steps.
struct Cursor {
  int u, j, s;   // unit, segment of the unit, step of the segment
  Unit x;
};

template <class CF>
SA_DEVI void next_step(const DecodeArgs& p, Cursor& c, int segs, int units) {
  if (++c.s < c.x.n) return;
  c.s = 0;
  if (++c.j < segs) return;
  c.j = 0;
  do c.x = unit_of<CF>(p, ++c.u);
  while (c.x.n == 0 && c.u + 1 < units);
}

// (b, h, row group) of a cursor's segment.
struct Seg {
  int b, h, r0;
};
SA_DEVI Seg seg_of(const DecodeArgs& p, int u, int j, int groups, int rows) {
  Seg s;
  if (p.kv_idx) {
    s.b = u / p.c.H;
    s.h = u - s.b * p.c.H;
    s.r0 = j * rows;
  } else {
    s.b = u;
    s.h = j / groups;
    s.r0 = (j - s.h * groups) * rows;
  }
  return s;
}

// Four consecutive output values of one row.
SA_DEVI void put4(const DecodeArgs& p, int64_t row, int D, int c, float4 v) {
  if (p.out_dtype == SA_OUT_F32)
    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + row * D + c) = v;
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + row * D + c) =
        make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
}
SA_DEVI void put_lse(const DecodeArgs& p, int64_t row, float m, float l) {
  if (p.lse) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

template <int D, bool E4M3, int NT>
__global__ void __launch_bounds__(kThreads, 1) decode_kernel(DecodeArgs p, int units, int groups) {
  using CF = Cfg<D, E4M3, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_prefix[kBuckets + 1], s_warp[kWarps];
  __shared__ long long e_seg[2 * kWarps], e_s0[2 * kWarps];
  __shared__ int e_n[2 * kWarps];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, q4 = lane & 3, r8 = lane >> 2;
  const int G = p.Hq / p.c.H, R = G * p.T;
  const int segs = (p.kv_idx ? 1 : p.c.H) * groups;   // segments of a unit

  // ---- the line of steps: a scan over the units' weights
  const int per = (units + kBuckets - 1) / kBuckets;
  long long sum = 0;
  for (int u = tid * per; u < min(units, (tid + 1) * per); ++u)
    sum += (long long)unit_of<CF>(p, u).n * segs;
  long long incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(~0u, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_warp[w] = incl;
  if (tid < 2 * kWarps) e_seg[tid] = -1;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < w) before += s_warp[i];
    total += s_warp[i];
  }
  s_prefix[tid] = before + incl - sum;
  if (tid == 0) s_prefix[kBuckets] = total;
  __syncthreads();

  // rows of units without a key
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    if (unit_of<CF>(p, u).n) continue;
    const int b = p.kv_idx ? u / p.c.H : u, h = p.kv_idx ? u - b * p.c.H : 0;
    const int64_t row0 = ((int64_t)b * p.Hq + h * G) * p.T;
    const int64_t rows = p.kv_idx ? R : (int64_t)p.Hq * p.T;
    for (int64_t i = tid; i < rows * (D / 4); i += kThreads)
      put4(p, row0 + i / (D / 4), D, (int)(i % (D / 4)) * 4, make_float4(0.f, 0.f, 0.f, 0.f));
    for (int64_t i = tid; i < rows; i += kThreads) put_lse(p, row0 + i, 0.f, 0.f);
  }

  // ---- this CTA's and this warp's share
  const int ctas = (int)min((long long)gridDim.x, (total + kWarps - 1) / kWarps);
  Record* rec = static_cast<Record*>(p.work) + blockIdx.x;
  const bool active = (int)blockIdx.x < ctas;
  const long long lo_c = active ? blockIdx.x * total / ctas : 0;
  const long long hi_c = active ? (blockIdx.x + 1) * total / ctas : 0;
  const long long lo = lo_c + w * (hi_c - lo_c) / kWarps;
  const int steps = (int)(lo_c + (w + 1) * (hi_c - lo_c) / kWarps - lo);
  float* heads = reinterpret_cast<float*>(static_cast<Record*>(p.work) + gridDim.x);
  float* head = heads + ((size_t)blockIdx.x * kWarps + w) * CF::kSlot;
  float* cta_slots = heads + (size_t)gridDim.x * kWarps * CF::kSlot;

  uint8_t* ring = smem + (size_t)w * kStages * 8192;
  uint8_t* metas = smem + (size_t)kWarps * kStages * 8192 + (size_t)w * kStages * CF::kMeta;

  if (steps > 0) {
    Cursor cc;
    {
      int a = 0, z = kBuckets;   // the last bucket that starts at or before lo
      while (z - a > 1) {
        const int mid = (a + z) / 2;
        if (s_prefix[mid] <= lo) a = mid; else z = mid;
      }
      long long at = s_prefix[a];
      cc.u = a * per;
      cc.x = unit_of<CF>(p, cc.u);
      while (at + (long long)cc.x.n * segs <= lo && cc.u + 1 < units) {
        at += (long long)cc.x.n * segs;
        cc.x = unit_of<CF>(p, ++cc.u);
      }
      const long long in = lo - at;
      cc.j = (int)(in / cc.x.n);
      cc.s = (int)(in - (long long)cc.j * cc.x.n);
    }
    Cursor ic = cc;

    // Page and first position of the 16-key tile `lane` of the issue cursor's step.
    int pg = -1, pos = kNoPos;
    auto look_up = [&]() {
      pg = -1;
      pos = kNoPos;
      if (lane < CF::kSub) {
        const long long vi = (long long)ic.s * CF::kKeys + lane * 16;
        const Seg s = seg_of(p, ic.u, ic.j, groups, CF::kRows);
        if (vi < ic.x.keys) {
          int lp = (int)(vi >> p.c.page_log2);
          if (p.kv_idx) lp = p.kv_idx[(int64_t)ic.u * p.cap + lp];
          if ((unsigned)lp < (unsigned)p.c.table_width) {
            const int at = (lp << p.c.page_log2) + ((int)vi & ((1 << p.c.page_log2) - 1));
            if (at < ic.x.len) {
              pg = pool_page(p.c, s.b, lp);
              if (pg >= 0) pos = at;
            }
          }
        }
      }
    };
    int to_issue = steps;
    auto issue = [&](int st) {
      if (to_issue > 0) {
        const uint32_t kdst = smem_u32(ring + st * 8192), vdst = kdst + 4096;
        uint8_t* meta = metas + st * CF::kMeta;
        const int h = seg_of(p, ic.u, ic.j, groups, CF::kRows).h;
        const int mask = (1 << p.c.page_log2) - 1;
        if (lane < CF::kSub) reinterpret_cast<int*>(meta + 128)[lane] = pos;
#pragma unroll
        for (int t = 0; t < CF::kSub; ++t) {
          const int tpg = __shfl_sync(~0u, pg, t), tpos = __shfl_sync(~0u, pos, t);
          const int64_t row = tpg < 0 ? 0 : (((int64_t)tpg * p.c.H + h) << p.c.page_log2) + (tpos & mask);
          const uint8_t* ks = static_cast<const uint8_t*>(p.c.k) + row * CF::kRow;
          const uint8_t* vs = static_cast<const uint8_t*>(p.c.v) + row * CF::kRow;
          const int live = ic.x.len - tpos;      // rows of the tile that exist
#pragma unroll
          for (int i = 0; i < CF::kChunks / 2; ++i) {
            const int at = i * 32 + lane, r = at / CF::kChunks, c = at % CF::kChunks;
            const uint32_t off = swz_row<CF::kRow>(t * 16 + r, c);
            const int bytes = r < live ? 16 : 0;
            cp_async16(kdst + off, bytes ? ks + at * 16 : ks, bytes);
            cp_async16(vdst + off, bytes ? vs + at * 16 : vs, bytes);
          }
          if constexpr (E4M3) {
            if (lane < 2 && tpg >= 0)
              cp_async16(smem_u32(meta) + lane * CF::kKeys + t * 16,
                         (lane ? p.c.v_scale : p.c.k_scale) + row, 16);
          }
        }
        if (--to_issue > 0) {
          next_step<CF>(p, ic, segs, units);
          look_up();
        }
      }
      cp_async_commit();
    };
    look_up();
#pragma unroll 1
    for (int st = 0; st < kStages; ++st) issue(st);

    // ---- per segment state
    uint32_t qf[NT][D / 16][2];
    float m[NT][2], l[NT][2], mv[NT][2], f[NT][2];
    int lim[NT][2];
    float o[CF::kMt][NT][4];
    Seg sg;
    auto begin_segment = [&]() {
      sg = seg_of(p, cc.u, cc.j, groups, CF::kRows);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = sg.r0 + nt * 8 + r8;
        const int g = r / p.T, t = r - g * p.T;
        const uint16_t* qp = p.q + sg.b * p.qs.b + (int64_t)(sg.h * G + g) * p.qs.h + t * p.qs.t;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          qf[nt][ks][0] = qf[nt][ks][1] = 0;
          if (r < R) {
            if constexpr (E4M3) {   // the order in which a lane gets its K codes (see below)
              const uint2 y = __ldg(reinterpret_cast<const uint2*>(qp + ks * 16 + 4 * q4));
              qf[nt][ks][0] = y.x;
              qf[nt][ks][1] = y.y;
            } else {
              qf[nt][ks][0] = __ldg(reinterpret_cast<const uint32_t*>(qp + ks * 16 + 2 * q4));
              qf[nt][ks][1] = __ldg(reinterpret_cast<const uint32_t*>(qp + ks * 16 + 8 + 2 * q4));
            }
          }
        }
        float back = 1.f;
        if constexpr (E4M3) {
          uint32_t top = 0;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            top = __vmaxu2(top, __vmaxu2(qf[nt][ks][0] & 0x7FFF7FFFu, qf[nt][ks][1] & 0x7FFF7FFFu));
          top = __vmaxu2(top, __shfl_xor_sync(~0u, top, 1));
          top = __vmaxu2(top, __shfl_xor_sync(~0u, top, 2));
          // exponent field of the row's largest value; 2^(141 - e) brings it to 2^14
          const uint32_t e = max(max(top & 0xFFFFu, top >> 16) >> 7, 15u);
          const float to = __uint_as_float((268u - e) << 23);
          back = __uint_as_float((e - 14u) << 23);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              qf[nt][ks][i] = pack_f16(bf16_lo(qf[nt][ks][i]) * to, bf16_hi(qf[nt][ks][i]) * to);
        }
        back *= p.scale * kLog2e;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          f[nt][i] = __shfl_sync(~0u, back, (2 * q4 + i) * 4);
          const int rc = sg.r0 + nt * 8 + 2 * q4 + i;
          lim[nt][i] = cc.x.len - (rc < R ? p.T - 1 - rc % p.T : 0);
          m[nt][i] = mv[nt][i] = -INFINITY;
          l[nt][i] = 0.f;
        }
#pragma unroll
        for (int mt = 0; mt < CF::kMt; ++mt)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[mt][nt][i] = 0.f;
      }
    };

    // ---- one step: kSub tiles of 16 keys against the segment's rows
    auto compute = [&](int st) {
      const uint32_t kb = smem_u32(ring + st * 8192), vb = kb + 4096;
      const uint8_t* meta = metas + st * CF::kMeta;
      const int* tile_pos = reinterpret_cast<const int*>(meta + 128);
      float s[CF::kSub][NT][4];
      float sv[E4M3 ? CF::kSub : 1][NT][4];   // s + log2 of the key's V scale
      const int mi = lane >> 3, mr = lane & 7;
#pragma unroll
      for (int t = 0; t < CF::kSub; ++t) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[t][nt][i] = 0.f;
        // A = K: 16 keys x 16 values. For e4m3 a 16-byte chunk holds 16 values and a lane
        // gets four neighbours, which stand for columns 2q, 2q+1, 2q+8, 2q+9 of the product;
        // the query was loaded in the same order.
#pragma unroll
        for (int x = 0; x < CF::kChunks / 2; ++x) {
          uint32_t a[4];
          ldsm_x4(kb + swz_row<CF::kRow>(t * 16 + mr + (mi & 1) * 8, 2 * x + (mi >> 1)), a[0], a[1],
                  a[2], a[3]);
          if constexpr (E4M3) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t af[4] = {e4m3x2_to_f16x2(a[2 * y]), e4m3x2_to_f16x2(a[2 * y + 1]),
                                      e4m3x2_to_f16x2(a[2 * y] >> 16),
                                      e4m3x2_to_f16x2(a[2 * y + 1] >> 16)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16(s[t][nt], af, qf[nt][2 * x + y][0], qf[nt][2 * x + y][1]);
            }
          } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_bf16(s[t][nt], a, qf[nt][x][0], qf[nt][x][1]);
          }
        }
        // scale to base 2 and mask
        const int pos0 = tile_pos[t];
        const bool all = pos0 + 16 <= cc.x.len - p.T + 1;
        float ks[2] = {1.f, 1.f}, vl[2] = {0.f, 0.f};
        if constexpr (E4M3) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            ks[i] = e8m0_value(meta[t * 16 + r8 + 8 * i]);
            const uint32_t e = meta[CF::kKeys + t * 16 + r8 + 8 * i];
            vl[i] = e == 255u ? __uint_as_float(0x7FC00000u) : (float)e - 127.f;
          }
          // A row of zeros is stored with scale 1. It adds nothing to the numerator, and
          // must not set the level that the other rows' weights are held at.
          if (__any_sync(~0u, vl[0] == 0.f || vl[1] == 0.f)) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int row = t * 16 + r8 + 8 * i;
              uint32_t any = 0;
#pragma unroll
              for (int c = q4; c < CF::kChunks; c += 4) {
                const uint4 y = *reinterpret_cast<const uint4*>(ring + st * 8192 + 4096 +
                                                                swz_row<CF::kRow>(row, c));
                any |= (y.x | y.y | y.z | y.w) & 0x7F7F7F7Fu;
              }
              any |= __shfl_xor_sync(~0u, any, 1);
              any |= __shfl_xor_sync(~0u, any, 2);
              if (any == 0) vl[i] = -INFINITY;
            }
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float x = s[t][nt][i] * f[nt][i & 1];
            if constexpr (E4M3) x *= ks[i >> 1];
            const bool seen = all || pos0 + r8 + 8 * (i >> 1) < lim[nt][i & 1];
            s[t][nt][i] = seen ? x : -INFINITY;
            if constexpr (E4M3) sv[t][nt][i] = seen ? x + vl[i >> 1] : -INFINITY;
          }
      }
      // running maxima; accumulators are rescaled only when one of the warp's columns moved
      float nm[NT][2], nv[NT][2];
      bool moved = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x = m[nt][i], y = mv[nt][i];
#pragma unroll
          for (int t = 0; t < CF::kSub; ++t) {
            x = fmaxf(x, fmaxf(s[t][nt][i], s[t][nt][i + 2]));
            if constexpr (E4M3) y = fmaxf(y, fmaxf(sv[t][nt][i], sv[t][nt][i + 2]));
          }
          nm[nt][i] = col_max(x);
          if constexpr (E4M3) nv[nt][i] = col_max(y);
          moved |= nm[nt][i] != m[nt][i];
          if constexpr (E4M3) moved |= nv[nt][i] != mv[nt][i];
        }
      if (__any_sync(~0u, moved)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float a = ex2a(m[nt][i] - ref_of(nm[nt][i]));
            float c = a;
            if constexpr (E4M3) c = ex2a(mv[nt][i] - ref_of(nv[nt][i]));
            l[nt][i] *= a;
#pragma unroll
            for (int mt = 0; mt < CF::kMt; ++mt) {
              o[mt][nt][i] *= c;
              o[mt][nt][i + 2] *= c;
            }
            m[nt][i] = nm[nt][i];
            if constexpr (E4M3) mv[nt][i] = nv[nt][i];
          }
      }
#pragma unroll
      for (int t = 0; t < CF::kSub; ++t) {
        // B = P^T in two pieces, by transposing each 8x8 block of S^T
        uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            float e[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              e[i] = ex2a(s[t][nt][2 * hf + i] - ref_of(m[nt][i]));
              l[nt][i] += e[i];
              if constexpr (E4M3)
                e[i] = ex2a(sv[t][nt][2 * hf + i] - (ref_of(mv[nt][i]) - kPvShift));
            }
            if constexpr (E4M3) {
              const uint32_t hi = pack_f16(e[0], e[1]);
              const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
              ph[nt][hf] = movmatrix(hi);
              pl[nt][hf] = movmatrix(pack_f16(e[0] - b.x, e[1] - b.y));
            } else {
              const uint32_t hi = pack_bf16(e[0], e[1]);
              ph[nt][hf] = movmatrix(hi);
              pl[nt][hf] = movmatrix(pack_bf16(e[0] - bf16_lo(hi), e[1] - bf16_hi(hi)));
            }
          }
        // A = V^T. For e4m3 the transposed load moves pairs of neighbouring values; even
        // ones make one tile of 16 output columns and odd ones the next.
        const int pos0 = tile_pos[t];
        const bool part = p.T > 1 && pos0 < cc.x.len && pos0 + 16 > cc.x.len - p.T + 1;
        auto load_v = [&](int x, uint32_t (&a)[2][4]) {
          uint32_t y[4];
          ldsm_x4_t(vb + swz_row<CF::kRow>(t * 16 + mr + (mi >> 1) * 8, 2 * x + (mi & 1)), y[0], y[1],
                    y[2], y[3]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (E4M3) {
              a[0][i] = e4m3x2_to_f16x2(__byte_perm(y[i], 0, 0x4420));
              a[1][i] = e4m3x2_to_f16x2(__byte_perm(y[i], 0, 0x4431));
            } else {
              a[0][i] = y[i];
            }
          }
        };
        constexpr int PER = E4M3 ? 2 : 1;    // output tiles of a load
        if (!part) {
#pragma unroll
          for (int x = 0; x < CF::kChunks / 2; ++x) {
            uint32_t a[2][4];
            load_v(x, a);
#pragma unroll
            for (int y = 0; y < PER; ++y)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                if constexpr (E4M3) {
                  mma_f16(o[x * PER + y][nt], a[y], ph[nt][0], ph[nt][1]);
                  mma_f16(o[x * PER + y][nt], a[y], pl[nt][0], pl[nt][1]);
                } else {
                  mma_bf16(o[x * PER + y][nt], a[y], ph[nt][0], ph[nt][1]);
                  mma_bf16(o[x * PER + y][nt], a[y], pl[nt][0], pl[nt][1]);
                }
              }
          }
        } else {
          // New tokens that some rows attend and others do not: a zero weight times a
          // non-finite value would reach the others, so each token's rows take a product
          // of their own in which the values that they do not attend are zeros.
#pragma unroll 1
          for (int tok = 0; tok < p.T; ++tok) {
            const int mine = cc.x.len - (p.T - 1 - tok);
            uint32_t keep[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int k0 = pos0 + 2 * q4 + 8 * i;
              keep[i] = (k0 < mine ? 0xFFFFu : 0u) | (k0 + 1 < mine ? 0xFFFF0000u : 0u);
            }
#pragma unroll
            for (int x = 0; x < CF::kChunks / 2; ++x) {
              uint32_t a[2][4];
              load_v(x, a);
#pragma unroll
              for (int y = 0; y < PER; ++y) {
#pragma unroll
                for (int i = 0; i < 4; ++i) a[y][i] &= keep[i >> 1];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  float z[4] = {0.f, 0.f, 0.f, 0.f};
                  if constexpr (E4M3) {
                    mma_f16(z, a[y], ph[nt][0], ph[nt][1]);
                    mma_f16(z, a[y], pl[nt][0], pl[nt][1]);
                  } else {
                    mma_bf16(z, a[y], ph[nt][0], ph[nt][1]);
                    mma_bf16(z, a[y], pl[nt][0], pl[nt][1]);
                  }
#pragma unroll
                  for (int i = 0; i < 4; ++i)
                    if (lim[nt][i & 1] == mine) o[x * PER + y][nt][i] += z[i];
                }
              }
            }
          }
        }
      }
    };

    // Eight rows of accumulators into rows of kPad floats, each column times fac.
    auto stage_rows = [&](float* to, int nt, float f0, float f1) {
#pragma unroll
      for (int mt = 0; mt < CF::kMt; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = E4M3 ? 32 * (mt >> 1) + 2 * r8 + (mt & 1) + 16 * (i >> 1)
                             : 16 * mt + r8 + 8 * (i >> 1);
          to[(2 * q4 + (i & 1)) * CF::kPad + c] = o[mt][nt][i] * ((i & 1) ? f1 : f0);
        }
    };

    long long seg0 = lo - cc.s;      // first step of the current segment
    begin_segment();
#pragma unroll 1
    for (int i = 0; i < steps; ++i) {
      const int st = i % kStages;
      cp_async_wait<kStages - 1>();
      __syncwarp();
      compute(st);
      __syncwarp();
      const bool ends = cc.s + 1 == cc.x.n, last = i + 1 == steps;
      if (ends || last) {
        const bool whole = ends && seg0 >= lo;
        const int rows = min(CF::kRows, R - sg.r0);
        const int64_t row0 = ((int64_t)sg.b * p.Hq + sg.h * G) * p.T + sg.r0;
        float* slot = reinterpret_cast<float*>(ring);       // the partial at the share's end
        if (last) cp_async_wait<0>();
        __syncwarp();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float fac[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float lk = col_sum(l[nt][k]);
            fac[k] = 1.f;
            if constexpr (E4M3)
              fac[k] = mv[nt][k] == -INFINITY ? 0.f : ex2a(mv[nt][k] - kPvShift - ref_of(m[nt][k]));
            if (whole) fac[k] = lk == 0.f ? 0.f : fac[k] / lk;
            if (r8 == 0) {
              const int r = nt * 8 + 2 * q4 + k;
              if (whole) {
                if (r < rows) put_lse(p, row0 + r, m[nt][k], lk);
              } else {
                float* ml = last ? slot + CF::kRows * CF::kPad : head + CF::kRows * D;
                ml[r] = m[nt][k];
                ml[CF::kRows + r] = lk;
              }
            }
          }
          float* buf = !whole && last ? slot + nt * 8 * CF::kPad
                                      : reinterpret_cast<float*>(ring + st * 8192);
          stage_rows(buf, nt, fac[0], fac[1]);
          if (whole || !last) {
            __syncwarp();
            for (int x = lane; x < min(8, rows - nt * 8) * (D / 4); x += 32) {
              const int r = x / (D / 4), c = x % (D / 4) * 4;
              const float4 y = *reinterpret_cast<const float4*>(buf + r * CF::kPad + c);
              if (whole) put4(p, row0 + nt * 8 + r, D, c, y);
              else *reinterpret_cast<float4*>(head + (nt * 8 + r) * D + c) = y;
            }
            __syncwarp();
          }
        }
        if (!whole && lane == 0) {
          const int e = 2 * w + (last ? 1 : 0);
          e_seg[e] = (long long)cc.u * segs + cc.j;
          e_s0[e] = seg0;
          e_n[e] = cc.x.n;
        }
      }
      if (!last) {
        next_step<CF>(p, cc, segs, units);
        issue(st);
        if (ends) {
          seg0 = lo + i + 1;
          begin_segment();
        }
      }
    }
  }
  __syncthreads();

  // ---- join the partials of each segment that several warps of this CTA shared
  if (tid == 0) *rec = Record{-1, 0, 0, total, ctas, {0, 0, 0}};
  auto partial = [&](int e, int& stride) -> const float* {
    stride = (e & 1) ? CF::kPad : D;
    return (e & 1) ? reinterpret_cast<const float*>(smem + (size_t)(e >> 1) * kStages * 8192)
                   : heads + ((size_t)blockIdx.x * kWarps + (e >> 1)) * CF::kSlot;
  };
  for (int e0 = 0; e0 < 2 * kWarps;) {
    const long long seg = e_seg[e0];
    if (seg < 0) {
      ++e0;
      continue;
    }
    int e1 = e0 + 1;
    while (e1 < 2 * kWarps && (e_seg[e1] < 0 || e_seg[e1] == seg)) ++e1;
    const long long s0 = e_s0[e0], n = e_n[e0];
    const Seg sg = seg_of(p, (int)(seg / segs), (int)(seg % segs), groups, CF::kRows);
    const int rows = min(CF::kRows, R - sg.r0);
    const bool whole = s0 >= lo_c && s0 + n <= hi_c;
    const int64_t row0 = ((int64_t)sg.b * p.Hq + sg.h * G) * p.T + sg.r0;
    float* dst = cta_slots + ((size_t)blockIdx.x * 2 + (s0 < lo_c ? 0 : 1)) * CF::kSlot;
    for (int x = tid; x < rows * (D / 4); x += kThreads) {
      const int r = x / (D / 4), c = x % (D / 4) * 4;
      float M = -INFINITY;
      for (int e = e0; e < e1; ++e) {
        if (e_seg[e] < 0) continue;
        int sd;
        const float* s = partial(e, sd);
        M = fmaxf(M, s[CF::kRows * sd + r]);
      }
      float L = 0.f;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int e = e0; e < e1; ++e) {
        if (e_seg[e] < 0) continue;
        int sd;
        const float* s = partial(e, sd);
        const float a = ex2a(s[CF::kRows * sd + r] - ref_of(M));
        const float4 v = *reinterpret_cast<const float4*>(s + r * sd + c);
        L += a * s[CF::kRows * sd + CF::kRows + r];
        y.x += a * v.x;
        y.y += a * v.y;
        y.z += a * v.z;
        y.w += a * v.w;
      }
      if (whole) {
        const float inv = L == 0.f ? 0.f : 1.f / L;
        put4(p, row0 + r, D, c, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
        if (c == 0) put_lse(p, row0 + r, M, L);
      } else {
        *reinterpret_cast<float4*>(dst + r * D + c) = y;
        if (c == 0) {
          dst[CF::kRows * D + r] = M;
          dst[CF::kRows * D + CF::kRows + r] = L;
        }
      }
    }
    if (!whole && s0 >= lo_c && tid == 0) {
      rec->seg = seg;
      rec->s0 = s0;
      rec->n = n;
    }
    e0 = e1;
  }
}

// Joins the partials of the segment that starts in CTA blockIdx.x's share and spans CTAs:
// one block per row, its groups of D/4 threads take every eighth (or sixteenth) partial.
template <int D, int ROWS>
__global__ void __launch_bounds__(256) decode_join_kernel(DecodeArgs p, int groups, int ctas_max) {
  constexpr int LN = D / 4, GRP = 256 / LN;
  __shared__ float red[8];
  __shared__ float4 acc[256];
  __shared__ float accl[GRP];
  const Record rec = static_cast<const Record*>(p.work)[blockIdx.x];
  if (rec.seg < 0) return;
  const int G = p.Hq / p.c.H, R = G * p.T, row = blockIdx.y, tid = threadIdx.x;
  const int segs = (p.kv_idx ? 1 : p.c.H) * groups;
  const Seg sg = seg_of(p, (int)(rec.seg / segs), (int)(rec.seg % segs), groups, ROWS);
  if (row >= R - sg.r0) return;
  constexpr size_t kSlot = (size_t)ROWS * (D + 2);
  const float* slots = reinterpret_cast<const float*>(static_cast<const Record*>(p.work) + ctas_max) +
                       (size_t)ctas_max * kWarps * kSlot;
  // CTAs of the segment: blockIdx.x (slot 1), then those whose share starts inside it (slot 0)
  const long long end = rec.s0 + rec.n;
  int last = blockIdx.x + 1;
  while (last < rec.ctas && last * rec.total / rec.ctas < end) ++last;
  const int parts = last - blockIdx.x;
  auto slot = [&](int i) {
    return slots + ((size_t)(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * kSlot;
  };
  float M = -INFINITY;
  for (int i = tid; i < parts; i += 256) M = fmaxf(M, slot(i)[ROWS * D + row]);
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, o));
  if (tid % 32 == 0) red[tid / 32] = M;
  __syncthreads();
  for (int i = 0; i < 8; ++i) M = fmaxf(M, red[i]);
  const int c = tid % LN * 4, grp = tid / LN;
  float L = 0.f;
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = grp; i < parts; i += GRP) {
    const float* s = slot(i);
    const float a = ex2a(s[ROWS * D + row] - ref_of(M));
    const float4 v = *reinterpret_cast<const float4*>(s + row * D + c);
    L += a * s[ROWS * D + ROWS + row];
    y.x += a * v.x;
    y.y += a * v.y;
    y.z += a * v.z;
    y.w += a * v.w;
  }
  acc[tid] = y;
  if (c == 0) accl[grp] = L;
  __syncthreads();
  if (grp == 0) {
    L = 0.f;
    y = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int g = 0; g < GRP; ++g) {
      const float4 v = acc[g * LN + tid];
      L += accl[g];
      y.x += v.x;
      y.y += v.y;
      y.z += v.z;
      y.w += v.w;
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const int64_t orow = ((int64_t)sg.b * p.Hq + sg.h * G) * p.T + sg.r0 + row;
    put4(p, orow, D, c, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
    if (c == 0) put_lse(p, orow, M, L);
  }
}

// n-tiles of eight query rows per segment: the fewest that hold R rows, up to four (more
// rows take further segments, which read the keys again).
inline int tiles_for(int R) { return R <= 8 ? 1 : R <= 16 ? 2 : 4; }

template <int D, bool E4M3, int NT>
cudaError_t run(const DecodeArgs& p, cudaStream_t st) {
  using CF = Cfg<D, E4M3, NT>;
  const long long R = (long long)(p.Hq / p.c.H) * p.T;
  const int groups = (int)((R + CF::kRows - 1) / CF::kRows);
  const int units = p.kv_idx ? p.B * p.c.H : p.B;
  // never more CTAs than a table full of keys gives every warp a step
  const long long most = (long long)p.B * p.c.H * groups *
                         (((long long)(p.kv_idx ? p.cap : p.c.table_width) << p.c.page_log2) /
                              CF::kKeys + 1);
  const int ctas = (int)std::min<long long>(p.sms, (most + kWarps - 1) / kWarps);
  auto* kern = decode_kernel<D, E4M3, NT>;
  static std::atomic<bool> ready[64];   // per device: the shared-memory limit is raised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !ready[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)CF::kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) ready[dev].store(true, std::memory_order_relaxed);
  }
  kern<<<ctas, kThreads, CF::kSmem, st>>>(p, units, groups);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int rows = (int)std::min<long long>(R, CF::kRows);
  decode_join_kernel<D, CF::kRows><<<dim3(ctas, rows), 256, 0, st>>>(p, groups, ctas);
  return cudaGetLastError();
}

template <int D, bool E4M3>
cudaError_t run_rows(const DecodeArgs& p, cudaStream_t st) {
  const long long R = (long long)(p.Hq / p.c.H) * p.T;
  switch (tiles_for((int)std::min<long long>(R, 32))) {
    case 1: return run<D, E4M3, 1>(p, st);
    case 2: return run<D, E4M3, 2>(p, st);
    default: return run<D, E4M3, 4>(p, st);
  }
}

}  // namespace

size_t decode_work_bytes(int B, int Hq, int Hkv, int T, int d, int sms) {
  if (B == 0 || Hq == 0) return 0;
  const long long R = (long long)(Hq / Hkv) * T;
  const size_t slot = (size_t)8 * tiles_for((int)std::min<long long>(R, 32)) * (d + 2) * 4;
  return (size_t)sms * (sizeof(Record) + (kWarps + 2) * slot);
}

cudaError_t launch_decode(const DecodeArgs& p, cudaStream_t st) {
  if (p.c.d == 64) return p.c.e4m3 ? run_rows<64, true>(p, st) : run_rows<64, false>(p, st);
  return p.c.e4m3 ? run_rows<128, true>(p, st) : run_rows<128, false>(p, st);
}

}  // namespace sa
