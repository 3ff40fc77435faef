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
constexpr float kShift16 = 14.f;       // f16 weights are at most 2^14 (fp16 ends at 2^16)
constexpr float kShift8 = 8.f;         // e4m3 weights are at most 2^8 (e4m3 ends at 448)

// A segment: its sequence, kv head and first query row, its steps, and where it starts on the
// line (which tells segments apart).
struct Place {
  int b, h, r0, n;
  long long s0;
};

// What CTA c leaves for the joining kernel: the segment that starts in its share and runs
// past it (at.b < 0: none), and how the line was cut.
struct Record {
  Place at;
  long long total;
  int ctas, pad[3];
};
static_assert(sizeof(Record) == 48, "the partials behind the records start on 16 bytes");

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

// 16-byte async copy global -> shared.
SA_DEVI void cp_async16_whole(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src));
}
SA_DEVI uint16_t e4m3x2(float lo, float hi) {
  uint16_t y;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(y) : "f"(hi), "f"(lo));
  return y;
}
SA_DEVI float2 e4m3x2_values(uint16_t v) {
  const uint32_t h = e4m3x2_to_f16x2(v);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// D = A(16x32 e4m3, row) * B(32x8 e4m3, col) + D, fp32 accumulate.
SA_DEVI void mma_e4m3(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two transposed 16x16 blocks of bytes: a lane gets, of column lane/4 (and lane/4 + 8), the
// rows 4 (lane%4) .. + 3.
SA_DEVI void ldsm_t8(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
// log2 of an E8M0 scale.
SA_DEVI float e8m0_log2(uint32_t e) {
  return e == 255u ? __uint_as_float(0x7FC00000u) : (float)e - 127.f;
}

// What a step's tiles are and where: shared-memory addresses of its K and V rows, scales
// and tile positions, and the segment's length.
struct Step {
  uint32_t k, v;
  const uint8_t* vp;      // V rows, generic
  const uint8_t* meta;
  int len, T;
  bool all;               // every key of the step is attended by every row
  SA_DEVI int pos(int t) const { return reinterpret_cast<const int*>(meta + 128)[t]; }
  // Tile t holds new tokens that some rows attend and others do not.
  SA_DEVI bool part(int t) const { return T > 1 && pos(t) < len && pos(t) + 16 > len - T + 1; }
};

template <int D, bool E4M3, bool PAIRED>
struct Layout {
  static constexpr bool kE4M3 = E4M3;
  static constexpr int kRow = D * (E4M3 ? 1 : 2);     // bytes of a cached row
  static constexpr int kKeys = 4096 / kRow;           // keys per step
  static constexpr int kSub = kKeys / 16;             // 16-key tiles per step
  static constexpr int kChunks = kRow / 16;
  static constexpr int kPad = D + 4;                  // floats between staged rows
  static constexpr int kMeta = 160;                   // scales (2 x kKeys), tile positions
  static constexpr size_t kSmem = (size_t)kWarps * kStages * (8192 + kMeta) + 256;
  // Where key r of a 16-key tile lies: in order, or (PAIRED) the even keys, then the odd
  // ones, so that rows i and i + 8 of a product's 16-row operand are neighbouring keys.
  SA_DEVI static int place(int r) { return PAIRED ? (r & 1) * 8 + (r >> 1) : r; }
  // Shared-memory offset of the i-th 16-byte piece that a lane copies of a tile: the
  // lane's own part and a compile-time part.
  SA_DEVI static uint32_t lane_part(int lane) {
    const int r = lane / kChunks, c = lane % kChunks;
    return swz_row<kRow>(place(r), c);
  }
  SA_DEVI static uint32_t piece(uint32_t lane_off, int i) {
    constexpr int rows = 32 / kChunks;                // rows that one piece of a warp covers
    const int r = place(i * rows);                    // (a multiple of 2: no carry into place)
    const int x = kRow == 64 ? (r >> 1) & 3 : r & 7;
    return (lane_off ^ (uint32_t)(x << 4)) + r * kRow;
  }
};

// A row of zeros is stored with scale 1. It adds nothing to the numerator, and must not set
// the level that the other rows' weights are held at: its log2 scale becomes -inf. The four
// lanes of a row group look at keys k0 and k1 of tile t.
template <class L>
SA_DEVI void zero_rows(const Step& w, int t, int lane, int k0, int k1, float (&vl)[2]) {
  if (!__any_sync(~0u, vl[0] == 0.f || vl[1] == 0.f)) return;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = t * 16 + L::place(i ? k1 : k0);
    uint32_t any = 0;
#pragma unroll
    for (int c = 0; c < L::kChunks; c += 4) {
      const uint4 y = *reinterpret_cast<const uint4*>(w.vp + swz_row<L::kRow>(row, c + (lane & 3)));
      any |= (y.x | y.y | y.z | y.w) & 0x7F7F7F7Fu;
    }
    any |= __shfl_xor_sync(~0u, any, 1);
    any |= __shfl_xor_sync(~0u, any, 2);
    if (any == 0) vl[i] = -INFINITY;
  }
}

// ---------------------------------------------------------------------------------------
// 16-bit products: bf16 rows as they are, or (more than eight query rows) e4m3 codes as f16.
// A lane owns the columns (query rows) 2q and 2q + 1 of each n-tile.
// ---------------------------------------------------------------------------------------
template <int D, bool E4M3, int NT>
struct Math16 : Layout<D, E4M3, false> {
  using L = Layout<D, E4M3, false>;
  static constexpr int kRows = 8 * NT, kGroups = NT, kMt = D / 16;
  uint32_t qf[NT][D / 16][2];
  float m[NT][2], l[NT][2], mv[NT][2], f[NT][2];
  int lim[NT][2];
  float o[kMt][NT][4];
  int lane, q4, r8;

  SA_DEVI void begin(const DecodeArgs& p, int b, int h, int r0, int len) {
    const int G = p.Hq / p.c.H, R = G * p.T;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = r0 + nt * 8 + r8;
      const int g = r / p.T, t = r - g * p.T;
      const uint16_t* qp = p.q + b * p.qs.b + (int64_t)(h * G + g) * p.qs.h + t * p.qs.t;
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
        const int rc = r0 + nt * 8 + 2 * q4 + i;
        lim[nt][i] = len - (rc < R ? p.T - 1 - rc % p.T : 0);
        m[nt][i] = mv[nt][i] = -INFINITY;
        l[nt][i] = 0.f;
      }
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[mt][nt][i] = 0.f;
    }
  }

  SA_DEVI static void mma(float* d, const uint32_t* a, const uint32_t* b) {
    if constexpr (E4M3) mma_f16(d, a, b[0], b[1]); else mma_bf16(d, a, b[0], b[1]);
  }

  SA_DEVI void compute(const Step& w) {
    constexpr int SUB = L::kSub;
    float s[SUB][NT][4];
    float sv[E4M3 ? SUB : 1][NT][4];   // s + log2 of the key's V scale
    const int mi = lane >> 3, mr = lane & 7;
    const uint32_t ka = w.k + swz_row<L::kRow>(mr + (mi & 1) * 8, mi >> 1);
#pragma unroll
    for (int t = 0; t < SUB; ++t) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[t][nt][i] = 0.f;
      // A = K: 16 keys x 16 values. For e4m3 a 16-byte chunk holds 16 values and a lane
      // gets four neighbours, which stand for columns 2q, 2q+1, 2q+8, 2q+9 of the product;
      // the query was loaded in the same order.
#pragma unroll
      for (int x = 0; x < L::kChunks / 2; ++x) {
        uint32_t a[4];
        ldsm_x4((ka ^ (uint32_t)(2 * x << 4)) + t * 16 * L::kRow, a[0], a[1], a[2], a[3]);
        if constexpr (E4M3) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t af[4] = {e4m3x2_to_f16x2(a[2 * y]), e4m3x2_to_f16x2(a[2 * y + 1]),
                                    e4m3x2_to_f16x2(a[2 * y] >> 16),
                                    e4m3x2_to_f16x2(a[2 * y + 1] >> 16)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma(s[t][nt], af, qf[nt][2 * x + y]);
          }
        } else {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma(s[t][nt], a, qf[nt][x]);
        }
      }
      // scale to base 2 and mask
      float ks[2] = {1.f, 1.f}, vl[2] = {0.f, 0.f};
      if constexpr (E4M3) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          ks[i] = e8m0_value(w.meta[t * 16 + r8 + 8 * i]);
          vl[i] = e8m0_log2(w.meta[L::kKeys + t * 16 + r8 + 8 * i]);
        }
        zero_rows<L>(w, t, lane, r8, r8 + 8, vl);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x = s[t][nt][i] * f[nt][i & 1];
          if constexpr (E4M3) x *= ks[i >> 1];
          s[t][nt][i] = x;
          if constexpr (E4M3) sv[t][nt][i] = x + vl[i >> 1];
        }
      if (!w.all) {
        const int pos0 = w.pos(t);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (pos0 + r8 + 8 * (i >> 1) >= lim[nt][i & 1]) {
              s[t][nt][i] = -INFINITY;
              if constexpr (E4M3) sv[t][nt][i] = -INFINITY;
            }
      }
    }
    // running maxima: the warp looks across its lanes, and rescales, only when one of its
    // columns has a new one
    float nm[NT][2], nv[NT][2];
    bool moved = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = s[0][nt][i], y = E4M3 ? sv[0][nt][i] : 0.f;
#pragma unroll
        for (int t = 0; t < SUB; ++t) {
          x = fmaxf(x, fmaxf(s[t][nt][i], s[t][nt][i + 2]));
          if constexpr (E4M3) y = fmaxf(y, fmaxf(sv[t][nt][i], sv[t][nt][i + 2]));
        }
        nm[nt][i] = x;
        nv[nt][i] = y;
        moved |= x > m[nt][i];
        if constexpr (E4M3) moved |= y > mv[nt][i];
      }
    if (__any_sync(~0u, moved)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          nm[nt][i] = col_max(fmaxf(nm[nt][i], m[nt][i]));
          const float a = ex2a(m[nt][i] - ref_of(nm[nt][i]));
          float c = a;
          if constexpr (E4M3) {
            nv[nt][i] = col_max(fmaxf(nv[nt][i], mv[nt][i]));
            c = ex2a(mv[nt][i] - ref_of(nv[nt][i]));
            mv[nt][i] = nv[nt][i];
          }
          l[nt][i] *= a;
          m[nt][i] = nm[nt][i];
#pragma unroll
          for (int mt = 0; mt < kMt; ++mt) {
            o[mt][nt][i] *= c;
            o[mt][nt][i + 2] *= c;
          }
        }
    }
    const uint32_t va = w.v + swz_row<L::kRow>(mr + (mi >> 1) * 8, mi & 1);
#pragma unroll
    for (int t = 0; t < SUB; ++t) {
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
              e[i] = ex2a(sv[t][nt][2 * hf + i] - (ref_of(mv[nt][i]) - kShift16));
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
      auto load_v = [&](int x, uint32_t (&a)[2][4]) {
        uint32_t y[4];
        ldsm_x4_t((va ^ (uint32_t)(2 * x << 4)) + t * 16 * L::kRow, y[0], y[1], y[2], y[3]);
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
      if (w.all || !w.part(t)) {
#pragma unroll
        for (int x = 0; x < L::kChunks / 2; ++x) {
          uint32_t a[2][4];
          load_v(x, a);
#pragma unroll
          for (int y = 0; y < PER; ++y)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma(o[x * PER + y][nt], a[y], ph[nt]);
              mma(o[x * PER + y][nt], a[y], pl[nt]);
            }
        }
      } else {
        // New tokens that some rows attend and others do not: a zero weight times a
        // non-finite value would reach the others, so each token's rows take a product
        // of their own in which the values that they do not attend are zeros.
#pragma unroll 1
        for (int tok = 0; tok < w.T; ++tok) {
          const int mine = w.len - (w.T - 1 - tok);
          uint32_t keep[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int k0 = w.pos(t) + 2 * q4 + 8 * i;
            keep[i] = (k0 < mine ? 0xFFFFu : 0u) | (k0 + 1 < mine ? 0xFFFF0000u : 0u);
          }
#pragma unroll
          for (int x = 0; x < L::kChunks / 2; ++x) {
            uint32_t a[2][4];
            load_v(x, a);
#pragma unroll
            for (int y = 0; y < PER; ++y) {
#pragma unroll
              for (int i = 0; i < 4; ++i) a[y][i] &= keep[i >> 1];
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float z[4] = {0.f, 0.f, 0.f, 0.f};
                mma(z, a[y], ph[nt]);
                mma(z, a[y], pl[nt]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (lim[nt][i & 1] == mine) o[x * PER + y][nt][i] += z[i];
              }
            }
          }
        }
      }
    }
  }

  // Row sums across the lanes, and (f) the factor of each column's accumulators.
  SA_DEVI void close(bool whole) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        l[nt][k] = col_sum(l[nt][k]);
        float x = 1.f;
        if constexpr (E4M3)
          x = mv[nt][k] == -INFINITY ? 0.f : ex2a(mv[nt][k] - kShift16 - ref_of(m[nt][k]));
        if (whole) x = l[nt][k] == 0.f ? 0.f : x / l[nt][k];
        f[nt][k] = x;
      }
  }
  // fn(row, m, l) for the rows of 8-row group g.
  template <class F>
  SA_DEVI void stats(int g, F fn) {
    if (r8 == 0) {
      fn(g * 8 + 2 * q4, m[g][0], l[g][0]);
      fn(g * 8 + 2 * q4 + 1, m[g][1], l[g][1]);
    }
  }
  // The accumulators of 8-row group g as rows of kPad floats.
  SA_DEVI void stage(int g, float* to) {
#pragma unroll
    for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = E4M3 ? 32 * (mt >> 1) + 2 * r8 + (mt & 1) + 16 * (i >> 1)
                           : 16 * mt + r8 + 8 * (i >> 1);
        to[(2 * q4 + (i & 1)) * L::kPad + c] = o[mt][g][i] * f[g][i & 1];
      }
  }
};

// ---------------------------------------------------------------------------------------
// 8-bit products (up to eight query rows): the codes enter as they are, 32 to an instruction
// at twice the rate and without a conversion; the other operand is split into e4m3 pieces,
// each 2^-5 of the one before, that fill columns which few query rows would leave empty.
// A query row takes two pieces: bf16's eight significant bits are two times four (what is
// lost is below 2^-22 of the row's largest value). A weight takes four, 2^-16 of it. A tile
// of eight columns is four query rows times two pieces; a lane owns one row of each such
// quad, both its pieces, and the neighbouring keys 2i and 2i + 1 of a tile.
// ---------------------------------------------------------------------------------------
template <int D, int NQ>
struct Math8 : Layout<D, true, true> {
  using L = Layout<D, true, true>;
  static constexpr int kRows = 4 * NQ, kGroups = 1, kCh = D / 16;
  uint32_t qf[NQ][D / 32][2];
  float m[NQ], l[NQ], mv[NQ], f[NQ];
  int lim[NQ];
  float o[kCh][NQ][2][4];
  int lane, q4, r8;

  SA_DEVI void begin(const DecodeArgs& p, int b, int h, int r0, int len) {
    const int G = p.Hq / p.c.H, R = G * p.T;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int r = r0 + n * 4 + (r8 >> 1);
      const int g = r / p.T, t = r - g * p.T;
      const uint16_t* qp = p.q + b * p.qs.b + (int64_t)(h * G + g) * p.qs.h + t * p.qs.t;
      uint2 x[D / 32][2];
      uint32_t top = 0;
#pragma unroll
      for (int ks = 0; ks < D / 32; ++ks)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint2 y = make_uint2(0, 0);
          if (r < R) y = __ldg(reinterpret_cast<const uint2*>(qp + ks * 32 + i * 16 + 4 * q4));
          x[ks][i] = y;
          top = __vmaxu2(top, __vmaxu2(y.x & 0x7FFF7FFFu, y.y & 0x7FFF7FFFu));
        }
      top = __vmaxu2(top, __shfl_xor_sync(~0u, top, 1));
      top = __vmaxu2(top, __shfl_xor_sync(~0u, top, 2));
      // exponent field of the row's largest value; 2^(134 - e) brings it below 2^8
      const uint32_t e = max(max(top & 0xFFFFu, top >> 16) >> 7, 8u);
      const float to = __uint_as_float((261u - e) << 23);
      const float back = __uint_as_float((e - 7u) << 23) * (p.scale * kLog2e);
      auto codes = [&](uint32_t v) -> uint32_t {
        v |= __vcmpgeu2(v & 0x7FFF7FFFu, 0x7F807F80u) & 0x7FFF7FFFu;   // infinities as NaN
        const float a = bf16_lo(v) * to, c = bf16_hi(v) * to;
        const uint16_t y = e4m3x2(a, c);
        const float2 z = e4m3x2_values(y);
        return (r8 & 1) ? e4m3x2((a - z.x) * 32.f, (c - z.y) * 32.f) : y;
      };
#pragma unroll
      for (int ks = 0; ks < D / 32; ++ks)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          qf[n][ks][i] = codes(x[ks][i].x) | (codes(x[ks][i].y) << 16);
      f[n] = __shfl_sync(~0u, back, 8 * q4);
      const int rc = r0 + n * 4 + q4;
      lim[n] = len - (rc < R ? p.T - 1 - rc % p.T : 0);
      m[n] = mv[n] = -INFINITY;
      l[n] = 0.f;
#pragma unroll
      for (int c = 0; c < kCh; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) o[c][n][i >> 2][i & 3] = 0.f;
    }
  }

  SA_DEVI void compute(const Step& w) {
    constexpr int SUB = L::kSub;
    float s[SUB][NQ][2], sv[SUB][NQ][2];    // keys 2i, 2i + 1 of a tile; sv: + log2 of V's scale
    const int mi = lane >> 3, mr = lane & 7;
    const uint32_t ka = w.k + swz_row<L::kRow>(mr + (mi & 1) * 8, mi >> 1);
#pragma unroll
    for (int t = 0; t < SUB; ++t) {
      float c[NQ][4];
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[n][i] = 0.f;
#pragma unroll
      for (int ks = 0; ks < D / 32; ++ks) {
        uint32_t a[4];
        ldsm_x4((ka ^ (uint32_t)(2 * ks << 4)) + t * 16 * L::kRow, a[0], a[1], a[2], a[3]);
#pragma unroll
        for (int n = 0; n < NQ; ++n) mma_e4m3(c[n], a, qf[n][ks][0], qf[n][ks][1]);
      }
      const uint32_t kb = *reinterpret_cast<const uint16_t*>(w.meta + t * 16 + 2 * r8);
      const uint32_t vb = *reinterpret_cast<const uint16_t*>(w.meta + L::kKeys + t * 16 + 2 * r8);
      const float ks[2] = {e8m0_value(kb & 255u), e8m0_value(kb >> 8)};
      float vl[2] = {e8m0_log2(vb & 255u), e8m0_log2(vb >> 8)};
      zero_rows<L>(w, t, lane, 2 * r8, 2 * r8 + 1, vl);
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float x = fmaf(c[n][2 * i + 1], 1.f / 32.f, c[n][2 * i]) * (f[n] * ks[i]);
          s[t][n][i] = x;
          sv[t][n][i] = x + vl[i];
        }
      if (!w.all) {
        const int pos0 = w.pos(t) + 2 * r8;
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (pos0 + i >= lim[n]) s[t][n][i] = sv[t][n][i] = -INFINITY;
      }
    }
    float nm[NQ], nv[NQ];
    bool moved = false;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      nm[n] = s[0][n][0];
      nv[n] = sv[0][n][0];
#pragma unroll
      for (int t = 0; t < SUB; ++t) {
        nm[n] = fmaxf(nm[n], fmaxf(s[t][n][0], s[t][n][1]));
        nv[n] = fmaxf(nv[n], fmaxf(sv[t][n][0], sv[t][n][1]));
      }
      moved |= nm[n] > m[n] || nv[n] > mv[n];
    }
    if (__any_sync(~0u, moved)) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const float x = col_max(fmaxf(nm[n], m[n])), y = col_max(fmaxf(nv[n], mv[n]));
        l[n] *= ex2a(m[n] - ref_of(x));
        const float c = ex2a(mv[n] - ref_of(y));
        m[n] = x;
        mv[n] = y;
#pragma unroll
        for (int ch = 0; ch < kCh; ++ch)
#pragma unroll
          for (int i = 0; i < 8; ++i) o[ch][n][i >> 2][i & 3] *= c;
      }
    }
    const uint32_t va = w.v + (lane >> 4) * 16 * L::kRow + swz_row<L::kRow>(L::place(lane & 15), 0);
#pragma unroll
    for (int t = 0; t < SUB; t += 2) {
      uint32_t pb[NQ][2][2];     // [quad][pieces 1, 2 | 3, 4][tile]
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const float r = ref_of(m[n]), rv = ref_of(mv[n]) - kShift8;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          l[n] += ex2a(s[t + y][n][0] - r) + ex2a(s[t + y][n][1] - r);
          float a = ex2a(sv[t + y][n][0] - rv), b = ex2a(sv[t + y][n][1] - rv);
          uint32_t pc[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint16_t z = e4m3x2(a, b);
            pc[j] = z;
            if (j < 3) {
              const float2 v = e4m3x2_values(z);
              a = (a - v.x) * 32.f;
              b = (b - v.y) * 32.f;
            }
          }
          pb[n][0][y] = movmatrix(pc[0] | (pc[1] << 16));
          pb[n][1][y] = movmatrix(pc[2] | (pc[3] << 16));
        }
      }
      auto load_v = [&](int c, uint32_t* a) {
        ldsm_t8((va ^ (uint32_t)(c << 4)) + t * 16 * L::kRow, a);
      };
      if (w.all || !(w.part(t) || w.part(t + 1))) {
#pragma unroll
        for (int c = 0; c < kCh; ++c) {
          uint32_t a[4];
          load_v(c, a);
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            mma_e4m3(o[c][n][0], a, pb[n][0][0], pb[n][0][1]);
            mma_e4m3(o[c][n][1], a, pb[n][1][0], pb[n][1][1]);
          }
        }
      } else {   // see the 16-bit products
#pragma unroll 1
        for (int tok = 0; tok < w.T; ++tok) {
          const int mine = w.len - (w.T - 1 - tok);
          uint32_t keep[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            keep[y] = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (w.pos(t + y) + 4 * q4 + j < mine) keep[y] |= 0xFFu << (8 * j);
          }
#pragma unroll
          for (int c = 0; c < kCh; ++c) {
            uint32_t a[4];
            load_v(c, a);
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] &= keep[i >> 1];
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                float z[4] = {0.f, 0.f, 0.f, 0.f};
                mma_e4m3(z, a, pb[n][k][0], pb[n][k][1]);
                if (lim[n] == mine)
#pragma unroll
                  for (int i = 0; i < 4; ++i) o[c][n][k][i] += z[i];
              }
          }
        }
      }
    }
  }

  SA_DEVI void close(bool whole) {
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      l[n] = col_sum(l[n]);
      float x = mv[n] == -INFINITY ? 0.f : ex2a(mv[n] - kShift8 - ref_of(m[n]));
      if (whole) x = l[n] == 0.f ? 0.f : x / l[n];
      f[n] = x;
    }
  }
  template <class F>
  SA_DEVI void stats(int, F fn) {
    if (r8 == 0)
#pragma unroll
      for (int n = 0; n < NQ; ++n) fn(n * 4 + q4, m[n], l[n]);
  }
  SA_DEVI void stage(int, float* to) {
#pragma unroll
    for (int c = 0; c < kCh; ++c)
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float* x = o[c][n][0] + 2 * i;
          const float* y = o[c][n][1] + 2 * i;
          to[(n * 4 + q4) * L::kPad + c * 16 + r8 + 8 * i] =
              fmaf(fmaf(fmaf(y[1], 1.f / 32.f, y[0]), 1.f / 32.f, x[1]), 1.f / 32.f, x[0]) * f[n];
        }
  }
};

// What the steps of one unit (a sequence, or with kept lists a sequence's kv head) look like.
struct Unit {
  int len, n;                 // attended length, steps of each of its segments
  long long keys;             // keys in list order
};

template <class M>
SA_DEVI Unit unit_of(const DecodeArgs& p, int b, int h) {
  Unit x;
  x.len = seq_len(p.c, p.lens, b);
  x.keys = x.len;
  if (p.kv_idx && x.len)
    x.keys = (long long)min(max(p.kv_cnt[(int64_t)b * p.c.H + h], 0), p.cap) << p.c.page_log2;
  x.n = (int)((x.keys + M::kKeys - 1) / M::kKeys);
  return x;
}

// A place on the line of steps, which runs over b, h, row groups and steps of a segment.
struct Cursor {
  int b, h, r0, s;
  Unit x;
};

template <class M>
SA_DEVI void next_step(const DecodeArgs& p, Cursor& c, int R) {
  if (++c.s < c.x.n) return;
  c.s = 0;
  c.r0 += M::kRows;
  if (c.r0 < R) return;
  c.r0 = 0;
  if (++c.h < p.c.H && !p.kv_idx) return;
  do {
    if (c.h >= p.c.H) {
      c.h = 0;
      ++c.b;
    }
    if (c.b >= p.B) return;   // past the line: never taken
    c.x = unit_of<M>(p, c.b, c.h);
    if (c.x.n) return;
    c.h = p.kv_idx ? c.h + 1 : p.c.H;
  } while (true);
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

template <int D, class M>
__global__ void __launch_bounds__(kThreads, 1) decode_kernel(DecodeArgs p, int units, int groups) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ long long s_prefix[kBuckets + 1], s_warp[kWarps];
  __shared__ Place e_at[2 * kWarps];
  constexpr size_t kSlot = (size_t)M::kRows * (D + 2);   // floats of a global partial
  uint8_t* smem = smem_raw + ((256u - (smem_u32(smem_raw) & 255u)) & 255u);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int G = p.Hq / p.c.H, R = G * p.T;
  const int segs = (p.kv_idx ? 1 : p.c.H) * groups;   // segments of a unit
  auto unit_at = [&](int u) {
    return p.kv_idx ? unit_of<M>(p, u / p.c.H, u % p.c.H) : unit_of<M>(p, u, 0);
  };

  // ---- the line of steps: a scan over the units' weights
  const int per = (units + kBuckets - 1) / kBuckets;
  long long sum = 0;
  for (int u = tid * per; u < min(units, (tid + 1) * per); ++u)
    sum += (long long)unit_at(u).n * segs;
  long long incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(~0u, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_warp[w] = incl;
  if (tid < 2 * kWarps) e_at[tid].b = -1;
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
    if (unit_at(u).n) continue;
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
  float* head = heads + ((size_t)blockIdx.x * kWarps + w) * kSlot;
  float* cta_slots = heads + (size_t)gridDim.x * kWarps * kSlot;

  uint8_t* ring = smem + (size_t)w * kStages * 8192;
  uint8_t* metas = smem + (size_t)kWarps * kStages * 8192 + (size_t)w * kStages * M::kMeta;

  if (steps > 0) {
    Cursor cc;
    {
      int a = 0, z = kBuckets;   // the last bucket that starts at or before lo
      while (z - a > 1) {
        const int mid = (a + z) / 2;
        if (s_prefix[mid] <= lo) a = mid; else z = mid;
      }
      long long at = s_prefix[a];
      int u = a * per;
      cc.x = unit_at(u);
      while (at + (long long)cc.x.n * segs <= lo && u + 1 < units) {
        at += (long long)cc.x.n * segs;
        cc.x = unit_at(++u);
      }
      const long long in = lo - at;
      const int j = (int)(in / cc.x.n);
      cc.s = (int)(in - (long long)j * cc.x.n);
      cc.b = p.kv_idx ? u / p.c.H : u;
      cc.h = p.kv_idx ? u % p.c.H : j / groups;
      cc.r0 = (p.kv_idx ? j : j % groups) * M::kRows;
    }
    Cursor ic = cc;

    // Page and first position of the 16-key tile `lane` of the issue cursor's step.
    int pg = -1, pos = kNoPos;
    auto look_up = [&]() {
      pg = -1;
      pos = kNoPos;
      if (lane < M::kSub) {
        const long long vi = (long long)ic.s * M::kKeys + lane * 16;
        if (vi < ic.x.keys) {
          int lp = (int)(vi >> p.c.page_log2);
          if (p.kv_idx) lp = p.kv_idx[((int64_t)ic.b * p.c.H + ic.h) * p.cap + lp];
          if ((unsigned)lp < (unsigned)p.c.table_width) {
            const int at = (lp << p.c.page_log2) + ((int)vi & ((1 << p.c.page_log2) - 1));
            if (at < ic.x.len) {
              pg = pool_page(p.c, ic.b, lp);
              if (pg >= 0) pos = at;
            }
          }
        }
      }
    };
    const uint32_t lane_off = M::lane_part(lane);
    const int lane_row = lane / M::kChunks;
    int to_issue = steps;
    auto issue = [&](int st) {
      if (to_issue > 0) {
        const uint32_t kdst = smem_u32(ring + st * 8192);
        uint8_t* meta = metas + st * M::kMeta;
        if (lane < M::kSub) reinterpret_cast<int*>(meta + 128)[lane] = pos;
#pragma unroll
        for (int t = 0; t < M::kSub; ++t) {
          const int tpg = __shfl_sync(~0u, pg, t), tpos = __shfl_sync(~0u, pos, t);
          const int live = ic.x.len - tpos;      // rows of the tile that exist
          int64_t row = 0;
          if (tpg >= 0)
            row = (((int64_t)tpg * p.c.H + ic.h) << p.c.page_log2) + (tpos & ((1 << p.c.page_log2) - 1));
          const int64_t at = row * M::kRow + lane * 16;
          const uint8_t* ks = static_cast<const uint8_t*>(p.c.k) + at;
          const uint8_t* vs = static_cast<const uint8_t*>(p.c.v) + at;
          if (live >= 16) {
#pragma unroll
            for (int i = 0; i < M::kChunks / 2; ++i) {
              const uint32_t dst = kdst + t * 16 * M::kRow + M::piece(lane_off, i);
              cp_async16_whole(dst, ks + i * 512);
              cp_async16_whole(dst + 4096, vs + i * 512);
            }
          } else {
            // rows behind the last one are zeros here, whatever the page holds
#pragma unroll
            for (int i = 0; i < M::kChunks / 2; ++i) {
              const uint32_t dst = kdst + t * 16 * M::kRow + M::piece(lane_off, i);
              const bool in = i * (32 / M::kChunks) + lane_row < live;
              cp_async16(dst, in ? ks + i * 512 : static_cast<const uint8_t*>(p.c.k), in ? 16 : 0);
              cp_async16(dst + 4096, in ? vs + i * 512 : static_cast<const uint8_t*>(p.c.v), in ? 16 : 0);
            }
          }
          if constexpr (M::kE4M3) {
            if (lane < 2 && tpg >= 0)
              cp_async16_whole(smem_u32(meta) + lane * M::kKeys + t * 16,
                               (lane ? p.c.v_scale : p.c.k_scale) + row);
          }
        }
        if (--to_issue > 0) {
          next_step<M>(p, ic, R);
          look_up();
        }
      }
      cp_async_commit();
    };
    look_up();
#pragma unroll 1
    for (int st = 0; st < kStages; ++st) issue(st);

    M mth;
    mth.lane = lane;
    mth.q4 = lane & 3;
    mth.r8 = lane >> 2;
    long long seg0 = lo - cc.s;      // first step of the current segment
    mth.begin(p, cc.b, cc.h, cc.r0, cc.x.len);
    int st = 0;
#pragma unroll 1
    for (int i = 0; i < steps; ++i) {
      cp_async_wait<kStages - 1>();
      __syncwarp();
      {
        Step sp;
        sp.k = smem_u32(ring + st * 8192);
        sp.v = sp.k + 4096;
        sp.vp = ring + st * 8192 + 4096;
        sp.meta = metas + st * M::kMeta;
        sp.len = cc.x.len;
        sp.T = p.T;
        sp.all = true;
#pragma unroll
        for (int t = 0; t < M::kSub; ++t) sp.all &= sp.pos(t) + 16 <= cc.x.len - p.T + 1;
        mth.compute(sp);
      }
      __syncwarp();
      const bool ends = cc.s + 1 == cc.x.n, last = i + 1 == steps;
      if (ends || last) {
        const bool whole = ends && seg0 >= lo;
        const int rows = min(M::kRows, R - cc.r0);
        const int64_t row0 = ((int64_t)cc.b * p.Hq + cc.h * G) * p.T + cc.r0;
        float* slot = reinterpret_cast<float*>(ring);       // the partial at the share's end
        if (last) cp_async_wait<0>();
        __syncwarp();
        mth.close(whole);
#pragma unroll
        for (int g = 0; g < M::kGroups; ++g) {
          mth.stats(g, [&](int r, float m, float l) {
            if (whole) {
              if (r < rows) put_lse(p, row0 + r, m, l);
            } else {
              float* ml = last ? slot + M::kRows * M::kPad : head + M::kRows * D;
              ml[r] = m;
              ml[M::kRows + r] = l;
            }
          });
          float* buf = !whole && last ? slot + g * 8 * M::kPad
                                      : reinterpret_cast<float*>(ring + st * 8192);
          mth.stage(g, buf);
          if (whole || !last) {
            __syncwarp();
            for (int x = lane; x < min(8, rows - g * 8) * (D / 4); x += 32) {
              const int r = x / (D / 4), c = x % (D / 4) * 4;
              const float4 y = *reinterpret_cast<const float4*>(buf + r * M::kPad + c);
              if (whole) put4(p, row0 + g * 8 + r, D, c, y);
              else *reinterpret_cast<float4*>(head + (g * 8 + r) * D + c) = y;
            }
            __syncwarp();
          }
        }
        if (!whole && lane == 0)
          e_at[2 * w + (last ? 1 : 0)] = Place{cc.b, cc.h, cc.r0, cc.x.n, seg0};
      }
      if (!last) {
        next_step<M>(p, cc, R);
        issue(st);
        if (ends) {
          seg0 = lo + i + 1;
          mth.begin(p, cc.b, cc.h, cc.r0, cc.x.len);
        }
        st = st + 1 == kStages ? 0 : st + 1;
      }
    }
  }
  __syncthreads();

  // ---- join the partials of each segment that several warps of this CTA shared
  if (tid == 0) *rec = Record{Place{-1, 0, 0, 0, 0}, total, ctas, {0, 0, 0}};
  auto partial = [&](int e, int& stride) -> const float* {
    stride = (e & 1) ? M::kPad : D;
    return (e & 1) ? reinterpret_cast<const float*>(smem + (size_t)(e >> 1) * kStages * 8192)
                   : heads + ((size_t)blockIdx.x * kWarps + (e >> 1)) * kSlot;
  };
  for (int e0 = 0; e0 < 2 * kWarps;) {
    const Place at = e_at[e0];
    if (at.b < 0) {
      ++e0;
      continue;
    }
    int e1 = e0 + 1;
    while (e1 < 2 * kWarps && (e_at[e1].b < 0 || e_at[e1].s0 == at.s0)) ++e1;
    const int rows = min(M::kRows, R - at.r0);
    const bool whole = at.s0 >= lo_c && at.s0 + at.n <= hi_c;
    const int64_t row0 = ((int64_t)at.b * p.Hq + at.h * G) * p.T + at.r0;
    float* dst = cta_slots + ((size_t)blockIdx.x * 2 + (at.s0 < lo_c ? 0 : 1)) * kSlot;
    for (int x = tid; x < rows * (D / 4); x += kThreads) {
      const int r = x / (D / 4), c = x % (D / 4) * 4;
      float mx = -INFINITY;
      for (int e = e0; e < e1; ++e) {
        if (e_at[e].b < 0) continue;
        int sd;
        const float* s = partial(e, sd);
        mx = fmaxf(mx, s[M::kRows * sd + r]);
      }
      float ls = 0.f;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int e = e0; e < e1; ++e) {
        if (e_at[e].b < 0) continue;
        int sd;
        const float* s = partial(e, sd);
        const float a = ex2a(s[M::kRows * sd + r] - ref_of(mx));
        const float4 v = *reinterpret_cast<const float4*>(s + r * sd + c);
        ls += a * s[M::kRows * sd + M::kRows + r];
        y.x += a * v.x;
        y.y += a * v.y;
        y.z += a * v.z;
        y.w += a * v.w;
      }
      if (whole) {
        const float inv = ls == 0.f ? 0.f : 1.f / ls;
        put4(p, row0 + r, D, c, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
        if (c == 0) put_lse(p, row0 + r, mx, ls);
      } else {
        *reinterpret_cast<float4*>(dst + r * D + c) = y;
        if (c == 0) {
          dst[M::kRows * D + r] = mx;
          dst[M::kRows * D + M::kRows + r] = ls;
        }
      }
    }
    if (!whole && at.s0 >= lo_c && tid == 0) rec->at = at;
    e0 = e1;
  }
}

// Joins the partials of the segment that starts in CTA blockIdx.x's share and spans CTAs:
// one block per row, its groups of D/4 threads take every eighth (or sixteenth) partial.
template <int D, int ROWS>
__global__ void __launch_bounds__(256) decode_join_kernel(DecodeArgs p, int ctas_max) {
  constexpr int LN = D / 4, GRP = 256 / LN;
  __shared__ float red[8];
  __shared__ float4 acc[256];
  __shared__ float accl[GRP];
  const Record rec = static_cast<const Record*>(p.work)[blockIdx.x];
  if (rec.at.b < 0) return;
  const int G = p.Hq / p.c.H, R = G * p.T, row = blockIdx.y, tid = threadIdx.x;
  if (row >= R - rec.at.r0) return;
  constexpr size_t kSlot = (size_t)ROWS * (D + 2);
  const float* slots = reinterpret_cast<const float*>(static_cast<const Record*>(p.work) + ctas_max) +
                       (size_t)ctas_max * kWarps * kSlot;
  // CTAs of the segment: blockIdx.x (slot 1), then those whose share starts inside it (slot 0)
  const long long end = rec.at.s0 + rec.at.n;
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
    const int64_t orow = ((int64_t)rec.at.b * p.Hq + rec.at.h * G) * p.T + rec.at.r0 + row;
    put4(p, orow, D, c, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
    if (c == 0) put_lse(p, orow, M, L);
  }
}

template <int D, class M>
cudaError_t run(const DecodeArgs& p, cudaStream_t st) {
  const long long R = (long long)(p.Hq / p.c.H) * p.T;
  const int groups = (int)((R + M::kRows - 1) / M::kRows);
  const int units = p.kv_idx ? p.B * p.c.H : p.B;
  // never more CTAs than a table full of keys gives every warp a step
  const long long most = (long long)p.B * p.c.H * groups *
                         (((long long)(p.kv_idx ? p.cap : p.c.table_width) << p.c.page_log2) /
                              M::kKeys + 1);
  const int ctas = (int)std::min<long long>(p.sms, (most + kWarps - 1) / kWarps);
  auto* kern = decode_kernel<D, M>;
  static std::atomic<bool> ready[64];   // per device: the shared-memory limit is raised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !ready[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)M::kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) ready[dev].store(true, std::memory_order_relaxed);
  }
  kern<<<ctas, kThreads, M::kSmem, st>>>(p, units, groups);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int rows = (int)std::min<long long>(R, M::kRows);
  decode_join_kernel<D, M::kRows><<<dim3(ctas, rows), 256, 0, st>>>(p, ctas);
  return cudaGetLastError();
}

// The fewest rows per segment that hold the R rows of a kv head, up to 32 (more take further
// segments, which read the keys again).
template <int D>
cudaError_t run_rows(const DecodeArgs& p, cudaStream_t st) {
  const long long R = (long long)(p.Hq / p.c.H) * p.T;
  if (p.c.e4m3) {
    if (R <= 4) return run<D, Math8<D, 1>>(p, st);
    if (R <= 8) return run<D, Math8<D, 2>>(p, st);
    if (R <= 16) return run<D, Math16<D, true, 2>>(p, st);
    return run<D, Math16<D, true, 4>>(p, st);
  }
  if (R <= 8) return run<D, Math16<D, false, 1>>(p, st);
  if (R <= 16) return run<D, Math16<D, false, 2>>(p, st);
  return run<D, Math16<D, false, 4>>(p, st);
}

}  // namespace

size_t decode_work_bytes(int B, int Hq, int Hkv, int T, int d, int sms) {
  if (B == 0 || Hq == 0) return 0;
  const long long R = (long long)(Hq / Hkv) * T;
  const int rows = R <= 8 ? 8 : R <= 16 ? 16 : 32;
  return (size_t)sms * (sizeof(Record) + (kWarps + 2) * (size_t)rows * (d + 2) * 4);
}

cudaError_t launch_decode(const DecodeArgs& p, cudaStream_t st) {
  return p.c.d == 64 ? run_rows<64>(p, st) : run_rows<128>(p, st);
}

}  // namespace sa
