// Attention of the last T tokens of every sequence over its paged cache.
//
// Per (b, kv head h) the R = (Hq / Hkv) * T query rows (g, t) that share the head's keys:
//   l_p = scale * q . k_p over the positions p < len - (T - 1 - t) of the listed pages,
//   o = sum e^(l_p - m) v_p / sum e^(l_p - m),   lse = m + ln sum e^(l_p - m),
// in one pass over K and V with a running level m and a sum in fp32 (base 2). Every cached
// row is read once for all R rows, at 4 R d operations per 4 d (bf16) or 2 d + 2 (e4m3)
// bytes: HBM bounds it up to R of about 16, so the design is about keeping loads in flight
// and every SM equally loaded:
//  - The work is cut into steps of 4 KB of K and 4 KB of V (16 to 64 keys). All steps of all
//    (sequence, kv head, group of rows) segments form one line, in which every warp of a
//    grid of at most one CTA per SM takes an equal, contiguous share, whatever the lengths. Shares
//    are found on the device from the lengths (a scan of one weight per sequence), so a
//    captured graph follows the lengths.
//  - A warp streams its steps through its own ring of cp.async stages, 16 bytes a lane, with
//    no barrier between warps. Page numbers are looked up for up to 32 steps at a time, one
//    step ahead (a look-up at the copy it serves left the warp waiting 600 cycles a step).
//  - A segment that ends inside the share it began in is written out at once; the others
//    leave (m, l, numerator) partials, joined first inside the CTA and then, for segments
//    that span CTAs, by a second small kernel. Orders are fixed: same bits every run.
//  - Where one cluster per segment fills the GPU about as well (few, short segments), that
//    takes one launch and no scan: 16 heads of 1,560 rows 8.6 us against 10.5 on the line.
//  - Products run on mma.sync with the keys as the M dimension (S^T = K Q^T, O^T = V^T P^T):
//    one query row wastes 7/8 of a tile, not 15/16, and the tensor work (2 cycles of an SM a
//    product) stays below the time of the loads up to R = 16. At R = 32 it is about half of
//    what bounds the kernel; a tile of 128 keys on the larger tensor instructions is what
//    would move that.
//  - Twelve warps of two stages where eight rows suffice, eight of three or two otherwise
//    (registers): 64 ragged e4m3 sequences 108 us against 121 with eight warps of three.
// Measured on several B200s (calls back to back, inputs of three in turn): 4 x 16 heads x 63,960
// bf16 rows 298-325 us (7.0-6.4 TB/s); 40 heads x 75,600 e4m3 rows 125-133 us (6.2-5.9 TB/s),
// 130 with an fp32 output where it is 126; 64 e4m3 sequences of 0 to 8,191 rows, 8 kv heads of 4 query heads,
// pages of 16: 100-108 us (5.5-5.1 TB/s).
//
// Roundings below fp32. P enters its product as 16-bit pieces, each the rest of the one
// before: as many as keep the dropped rest below the output's own rounding (Math::PIECES).
// e4m3 codes enter as f16, exactly; the query then enters as f16 times a power of two per row
// that brings its largest value to 2^14 (what f16 drops is below 2^-38 of that value). A level
// that a running maximum passes is set 2^4 above it, so a weight is at most 1 (a larger one could
// overflow beside values near fp32's largest) and most steps rescale nothing.
// The scale of a V row, a power of two, multiplies its weight: exactly, relative to the largest
// scale so far, so that the largest weight lies between 2^11 and 2^15 of f16's range. f16 rounds
// to 2^-25 at least, which is 2^-36 of the largest weight for rows of that scale. Rows whose
// scale is far below it (a V row with an outlier raises it for every column) would fall out of
// that range: a step that holds one converts its codes and weights to bf16 pieces instead, whose
// range is fp32's (Math::kFar).
#pragma once

#include <algorithm>
#include <atomic>

#include "../../include/sparse_attn.h"
#include "paged.cuh"

namespace sa {
namespace {

constexpr int kLaneUnits = 8;          // units of a lane where a warp scans them by itself
// A cluster per segment saves the scan, the partials' way through memory and the second
// kernel: 2 to 5 us, the time of about this many steps of a warp. 100 kept pages of 64 rows in
// each of 64 heads: 38.6 us against 42.8 on the line. Equal lengths, 64 heads: 4,000
// bf16 rows 26.0 us against 29.9 on the line, 8,000 44.9 against 49.0; 48 heads (a third of the
// SMs idle) 8,000 rows 34.3 against 38.9, but 8-bit rows no faster from 16,000 on and 32 query
// rows slower from 4,000 on (37.6 against 35.3).
constexpr long long kClusterSlack = 4;
// Longer shares run on the line, which uneven lengths cannot unbalance: 64 heads of 1 to 16,000
// 8-bit rows 41.8 us in clusters, 33.9 on the line; 64 of 16,000 bf16 rows each 83.1 and 87.2.
constexpr long long kClusterSteps = 32;
constexpr int kNoPos = 0x7FFFFF00;     // position of keys that nothing attends
// The level that a column's weights are relative to is set this far (base 2) above the running
// maximum when that passes it: most steps then rescale nothing.
constexpr float kSlack = 4.f;
constexpr int kShift16 = 15;           // f16 weights are at most 2^15 (fp16 ends at 2^16)
constexpr int kNoLevel = -1000;        // no V row seen

// A segment: its sequence, kv head and first query row, its steps, and where it starts on the
// line (which tells segments apart).
struct Place {
  int b, h, r0, n;
  long long s0;
};

// What CTA c leaves for the joining kernel: the segment that starts in its share and runs
// past it (at.b < 0: none), and the last CTA that holds a part of it.
struct Record {
  Place at;
  int last, pad[5];
};
static_assert(sizeof(Record) == 48, "the partials behind the records start on 16 bytes");

SA_DEVI long long div_floor(long long a, int b) {   // a >= 0, b > 0
  return a < (1ll << 32) ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// The line cut into n shares that differ by one step at most.
struct Cut {
  long long q;
  int r;
  SA_DEVI Cut(long long total, int n) : q(n ? div_floor(total, n) : 0), r(n ? (int)(total - q * n) : 0) {}
  SA_DEVI long long lo(int c) const { return q * c + min(c, r); }
  SA_DEVI int share_of(long long x) const {   // x < total
    const long long big = (q + 1) * r;
    return (int)(x < big ? x / (q + 1) : r + (x - big) / q);
  }
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
SA_DEVI uint32_t f16x2_to_bf16x2(uint32_t v) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
  return pack_bf16(f.x, f.y);
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
// A column's level, given a step's maximum.
SA_DEVI float level(float x, float m) { return x > m ? x + kSlack : m; }
// A maximum to subtract: 0 while nothing was attended (-inf - -inf would be NaN).
SA_DEVI float ref_of(float m) { return m == -INFINITY ? 0.f : m; }

// 16-byte async copy global -> shared.
SA_DEVI void cp_async16_whole(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src));
}
// Two transposed 16x16 blocks of bytes: a lane gets, of column lane/4 (and lane/4 + 8), the
// rows 4 (lane%4) .. + 3.
SA_DEVI void ldsm_t8(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}

// What a step's tiles are and where: shared-memory addresses of its K and V rows, scales
// and tile positions, and the segment's length.
struct Step {
  uint32_t k, v;
  const uint8_t* vp;      // V rows, generic
  const uint8_t* meta;
  float2* sc;             // e4m3: (K scale, factor of the weight) of every key, made by scales()
  int len, T;
  bool all;               // every key of the step is attended by every row
  SA_DEVI int pos(int t) const { return reinterpret_cast<const int*>(meta + 128)[t]; }
  // Tile t holds new tokens that some rows attend and others do not.
  SA_DEVI bool part(int t) const { return T > 1 && pos(t) < len && pos(t) + 16 > len - T + 1; }
};

// Rows are copied as they are stored, 16 bytes a lane, into swizzled rows.
template <int D, bool E4M3, int WARPS, int STAGES>
struct Layout {
  static constexpr bool kE4M3 = E4M3;
  static constexpr int kWarps = WARPS, kStages = STAGES, kThreads = 32 * WARPS;
  static constexpr int kRow = D * (E4M3 ? 1 : 2);     // bytes of a cached row
  static constexpr int kKeys = 4096 / kRow;           // keys per step
  static constexpr int kSub = kKeys / 16;             // 16-key tiles per step
  static constexpr int kChunks = kRow / 16;
  static constexpr int kPad = D + 4;                  // floats between staged rows
  static constexpr int kMeta = 160;                   // scales (2 x kKeys), tile positions
  static constexpr int kScales = E4M3 ? kKeys * 8 : 0;
  // Where key r of a 16-key tile lies, which is its row of the S^T tile. bf16: in order.
  // e4m3: keys 4a, 4a+1 at 2a, 2a+1 and keys 4a+2, 4a+3 at 8+2a, 8+2a+1, the order in which
  // a transposing load of bytes hands a lane four neighbouring keys of V.
  SA_DEVI static int place(int r) {
    return E4M3 ? (r >> 2) * 2 + (r & 1) + ((r >> 1) & 1) * 8 : r;
  }
  // Key of row r < 8 of the tile, and how far the key of row r + 8 is from it.
  SA_DEVI static int key_of(int r) { return E4M3 ? (r >> 1) * 4 + (r & 1) : r; }
  static constexpr int kKeyStep = E4M3 ? 2 : 8;
  // Shared-memory offset of the i-th 16-byte piece that a lane copies of a tile: the
  // lane's own part and a compile-time part (place() and the swizzle add up without carries).
  SA_DEVI static uint32_t lane_part(int lane) {
    const int r = lane / kChunks, c = lane % kChunks;
    return swz_row<kRow>(place(r), c);
  }
  SA_DEVI static uint32_t piece(uint32_t lane_off, int i) {
    constexpr int rows = 32 / kChunks;                // rows that one piece of a warp covers
    const int r = place(i * rows);
    const int x = kRow == 64 ? (r >> 1) & 3 : r & 7;
    return (lane_off ^ (uint32_t)(x << 4)) + r * kRow;
  }
};

// 2^e; 0 below fp32's smallest normal value.
SA_DEVI float pow2(int e) { return __uint_as_float(e < -126 ? 0u : (uint32_t)(e + 127) << 23); }

// The arithmetic of a warp: 16-bit products of bf16 rows as they are, or of e4m3 codes as f16
// (mma.sync has no 8-bit form on this architecture that is not these conversions done again
// for every product). A lane owns the columns (query rows) 2q and 2q + 1 of each n-tile of
// eight, and two keys of each 16-key tile. F32: the output is fp32.
template <int D, bool E4M3, bool F32, int NT, int WARPS, int STAGES>
struct Math : Layout<D, E4M3, WARPS, STAGES> {
  using L = Layout<D, E4M3, WARPS, STAGES>;
  // 16-bit pieces of a weight: as many as keep what they drop below the output's own rounding
  // (half a step: 2^-8 of a bf16 value at most, 2^-24 of fp32): one f16 piece drops 2^-11 of a
  // weight at most and two bf16 pieces 2^-16; for fp32 outputs two f16 pieces drop 2^-22 and
  // three bf16 pieces 2^-24. One bf16 piece would drop as much as the bf16 output rounds. One
  // f16 piece leaves bf16 outputs 0.1610% from 64 bits in the mean where the rounding alone
  // leaves 0.1604%; a second would take 4 to 16% more time (4 to 32 rows).
  static constexpr int PIECES = (E4M3 ? 1 : 2) + F32;
  // The tensor cores cut the bits of a sum off where fp32 ends, which pulls a long chain
  // towards zero: 6e-5 of a sum of one sign after 1,900 steps, far below what a bf16 output
  // rounds. For fp32 outputs the products of a step (with 16 rows and more, a tile) are summed
  // there, and the steps added to nearest here: 4 x 16 heads x 63,960 bf16 rows 302 us against
  // 300, 40 heads x 75,600 e4m3 rows 131 against 125, 32 bf16 rows a segment 48.2 against 46.0.
  static constexpr bool kAdds = F32;
  static constexpr bool kF32 = F32;
  static constexpr int kRows = 8 * NT, kMt = D / 16;
  // With 32 rows the queries would take 64 registers of a lane: they stay in shared memory.
  static constexpr bool kQs = NT == 4;
  // With eight the next segment's are fetched there ahead of their use.
  static constexpr bool kAhead = NT == 1;
  static constexpr int kQueries = kQs || kAhead ? kRows * D * 2 + (kQs ? kRows * 4 : 0) : 0;
  // A warp's ring also takes its partial at the end of its share.
  static constexpr int kSlotBytes = kRows * L::kPad * 4;
  static constexpr int kRing = STAGES * 8192 > kSlotBytes ? STAGES * 8192 : (kSlotBytes + 255) / 256 * 256;
  static constexpr size_t smem(bool cluster) {   // a cluster's warps have one segment each
    return (size_t)WARPS * (kRing + STAGES * L::kMeta + L::kScales + (cluster && !kQs ? 0 : kQueries)) + 256;
  }
  uint32_t qf[kQs ? 1 : NT][D / 16][2];
  uint32_t qs;                     // this warp's queries in shared memory (kQs, kAhead)
  int r0, len, R;
  float m[NT][2], l[NT][2], f[NT][2];
  // e4m3: o is in units of 2^(top - kShift16). The largest scale of the V rows so far, as log2.
  int top;
  // Rows whose scale is more than 2^kFar below it take their step to bf16 pieces. Within it a
  // weight is rounded to 2^(kFar - 36) of the largest one or better; were 65,536 rows to err to
  // one side, that were 2^-16 of the sum for fp32 outputs and 2^-12 for bf16 ones. The scales of
  // rows of normally distributed values differ by 2^1. 40 heads x 75,600 rows, one row in 1,000
  // scaled up by 2^8: fp32 outputs 169 us against 130, bf16 outputs 146 against 127.
  static constexpr int kFar = F32 ? 4 : 8;
  float unit;                      // scale in base 2
  // How many positions a column's row attends; with 32 rows four bits a column hold how many
  // it does not (registers: 184 bytes spilled against 24).
  int lims[kQs ? 1 : NT][2];
  uint32_t before;
  SA_DEVI int lim(int nt, int i) const {
    return kQs ? len - (int)(before >> (8 * nt + 4 * i) & 15u) : lims[kQs ? 0 : nt][i];
  }
  float o[kMt][NT][4];
  int lane, q4, r8;

  SA_DEVI void fetch(const DecodeArgs& p, int b, int h, int nt, uint32_t (&x)[D / 16][2]) {
    const int G = p.Hq / p.c.H;
    const int r = r0 + nt * 8 + r8;
    const int g = r / p.T, t = r - g * p.T;
    const uint16_t* qp = p.q + b * p.qs.b + (int64_t)(h * G + g) * p.qs.h + t * p.qs.t;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      x[ks][0] = x[ks][1] = 0;
      if (r < R) {
        if constexpr (E4M3) {   // the order in which a lane gets its K codes (see below)
          const uint2 y = __ldg(reinterpret_cast<const uint2*>(qp + ks * 16 + 4 * q4));
          x[ks][0] = y.x;
          x[ks][1] = y.y;
        } else {
          x[ks][0] = __ldg(reinterpret_cast<const uint32_t*>(qp + ks * 16 + 2 * q4));
          x[ks][1] = __ldg(reinterpret_cast<const uint32_t*>(qp + ks * 16 + 8 + 2 * q4));
        }
      }
    }
  }
  // The lane's part of a bf16 query row as f16, times the power of two that brings the row's
  // largest value to 2^14; returns the way back.
  SA_DEVI static float to_f16(uint32_t (&x)[D / 16][2]) {
    uint32_t top = 0;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
      top = __vmaxu2(top, __vmaxu2(x[ks][0] & 0x7FFF7FFFu, x[ks][1] & 0x7FFF7FFFu));
    top = __vmaxu2(top, __shfl_xor_sync(~0u, top, 1));
    top = __vmaxu2(top, __shfl_xor_sync(~0u, top, 2));
    // exponent field of the row's largest value; 2^(141 - e) brings it to 2^14
    const uint32_t e = max(max(top & 0xFFFFu, top >> 16) >> 7, 15u);
    const float to = __uint_as_float((268u - e) << 23);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        x[ks][i] = pack_f16(bf16_lo(x[ks][i]) * to, bf16_hi(x[ks][i]) * to);
    return __uint_as_float((e - 14u) << 23);
  }

  // A segment's queries into this warp's buffer, 16 bytes a lane, zeros behind the last row;
  // part of the next group of copies.
  SA_DEVI void copy_queries(const DecodeArgs& p, int b, int h, int r0_) const {
    constexpr int CH = D / 8;
    const int G = p.Hq / p.c.H, rows = G * p.T - r0_;
#pragma unroll 4
    for (int i = lane; i < kRows * CH; i += 32) {
      const int k = i / CH, r = r0_ + k, g = r / p.T, t = r - g * p.T;
      const uint16_t* qp = p.q + b * p.qs.b + (int64_t)(h * G + g) * p.qs.h + t * p.qs.t + i % CH * 8;
      cp_async16(qs + swz(k, i % CH, 2 * D), k < rows ? qp : p.q, k < rows ? 16 : 0);
    }
  }
  SA_DEVI void load_prefetched(const DecodeArgs& p, int r0_, int len_) {
    R = p.Hq / p.c.H * p.T;
    r0 = r0_;
    len = len_;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // 4-byte word of the row: bf16 words 8 ks + q and + 4, e4m3 8 ks + 2q and + 1
        const int word = 8 * ks + (E4M3 ? 2 * q4 + i : q4 + 4 * i);
        asm volatile("ld.shared.b32 %0, [%1];\n"
                     : "=r"(qf[0][ks][i]) : "r"(qs + swz(r8, word >> 2, 2 * D) + (word & 3) * 4) : "memory");
      }
  }
  // The segment's queries are asked for, and (start) made operands once they are there.
  SA_DEVI void load(const DecodeArgs& p, int b, int h, int r0_, int len_) {
    R = p.Hq / p.c.H * p.T;
    r0 = r0_;
    len = len_;
    if constexpr (kQs) {
      copy_queries(p, b, h, r0);
    } else {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) fetch(p, b, h, nt, qf[nt]);
    }
  }
  // kQs: rows of 2 D bytes, 32-bit word q of a 16-column group the first of a lane's operand
  // pair and word 4 + q the second, so that a row-wise 8x8 load returns them. bf16 rows are
  // that as they are; with e4m3 keys they are turned into f16 in that order here.
  SA_DEVI void convert_queries(const DecodeArgs& p) {
#pragma unroll 1
    for (int nt = 0; nt < NT; ++nt) {
      uint32_t x[D / 16][2];
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];\n"
                     : "=r"(x[ks][0]), "=r"(x[ks][1])
                     : "r"(qs + swz(nt * 8 + r8, 2 * ks + (q4 >> 1), 2 * D) + (q4 & 1) * 8) : "memory");
      const float back = to_f16(x);
      __syncwarp();
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          asm volatile("st.shared.b32 [%0], %1;\n" ::"r"(qs + swz(nt * 8 + r8, 2 * ks + i, 2 * D) + 4 * q4),
                       "r"(x[ks][i]) : "memory");
      if (q4 == 0)
        asm volatile("st.shared.f32 [%0], %1;\n" ::"r"(qs + kRows * D * 2 + (nt * 8 + r8) * 4), "f"(back)
                     : "memory");
      __syncwarp();
    }
  }
  SA_DEVI void start(const DecodeArgs& p) {
    if constexpr (kQs && E4M3) convert_queries(p);
    before = 0;
    top = kNoLevel;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float back = 1.f;     // of row r8
      if constexpr (E4M3 && !kQs) back = to_f16(qf[nt]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f[nt][i] = 1.f;
        if constexpr (E4M3 && kQs)
          asm volatile("ld.shared.f32 %0, [%1];\n"
                       : "=f"(f[nt][i]) : "r"(qs + kRows * D * 2 + (nt * 8 + 2 * q4 + i) * 4) : "memory");
        else if constexpr (E4M3)
          f[nt][i] = __shfl_sync(~0u, back, (2 * q4 + i) * 4);
        unit = p.scale * kLog2e;
        f[nt][i] *= unit;
        const int rc = r0 + nt * 8 + 2 * q4 + i;
        const int unseen = rc < R ? p.T - 1 - rc % p.T : 0;
        before |= (uint32_t)unseen << (8 * nt + 4 * i);
        if constexpr (!kQs) lims[nt][i] = len - unseen;
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[nt][i] = -INFINITY;
        l[nt][i] = 0.f;
      }
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[mt][nt][i] = 0.f;
    }
  }

  template <bool F16>
  SA_DEVI static void mma_first(float* d, const uint32_t* a, const uint32_t* b) {   // on zeros
    if constexpr (F16)
      asm volatile(
          "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
          "{%10,%10,%10,%10};\n"
          : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
          : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(0.f));
    else
      asm volatile(
          "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
          "{%10,%10,%10,%10};\n"
          : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
          : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(0.f));
  }
  template <bool F16>
  SA_DEVI static void mma(float* d, const uint32_t* a, const uint32_t* b) {
    if constexpr (F16) mma_f16(d, a, b[0], b[1]); else mma_bf16(d, a, b[0], b[1]);
  }
  // The operands of 32 columns of n-tile nt: two per 16.
  SA_DEVI void queries(int nt, int pair, uint32_t (&b)[2][2]) {
    if constexpr (kQs) {
      ldsm_x4(qs + swz(nt * 8 + (lane & 7), 4 * pair + (lane >> 3), 2 * D), b[0][0], b[0][1], b[1][0],
              b[1][1]);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        b[i][0] = qf[nt][2 * pair + i][0];
        b[i][1] = qf[nt][2 * pair + i][1];
      }
    }
  }

  // No infinity or NaN among the V values of tile t.
  SA_DEVI bool finite_values(const Step& w, int t) const {
    uint32_t bad = 0;
#pragma unroll
    for (int i = 0; i < L::kChunks / 2; ++i) {
      const uint4 y = *reinterpret_cast<const uint4*>(w.vp + t * 16 * L::kRow + (i * 32 + lane) * 16);
      const uint32_t x[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)    // all ones in an exponent carry into the sign's place
        bad |= E4M3 ? (x[j] & 0x7F7F7F7Fu) + 0x01010101u : (x[j] & 0x7F807F80u) + 0x00800080u;
    }
    return !__any_sync(~0u, bad & (E4M3 ? 0x80808080u : 0x80008000u));
  }

  // The scales of a step's keys, a key to a lane: the K scale, and the V scale relative to the
  // largest so far. A row of zeros (append stores scale 1) adds nothing and is no reason for
  // another level; rows behind the last one hold anything. New tokens that some rows do not
  // attend leave the level alone as far as fp32's range allows, so that those rows keep their
  // bits: they belong to the last step of a sequence, which is held in bf16 pieces. Returns
  // whether the step is.
  SA_DEVI bool scales(const Step& w) {
    constexpr int PER = L::kKeys / 32;
    uint32_t kb[PER];
    int lv[PER], pos[PER];
    bool dead[PER], odd = !w.all && w.T > 1, wide = false;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int key = j * 32 + lane;
      kb[j] = w.meta[key];
      lv[j] = (int)w.meta[L::kKeys + key] - 127;
      pos[j] = w.all ? 0 : w.pos(key >> 4) + (key & 15);
      dead[j] = !w.all && pos[j] >= w.len;
      if (lv[j] == 0) {
        const int row = (key & ~15) + L::place(key & 15);
        uint32_t any = 0;
#pragma unroll 1
        for (int c = 0; c < L::kChunks; ++c) {
          const uint4 y = *reinterpret_cast<const uint4*>(w.vp + swz_row<L::kRow>(row, c));
          any |= (y.x | y.y | y.z | y.w) & 0x7F7F7F7Fu;
        }
        dead[j] |= any == 0;
      }
      odd |= !dead[j] && lv[j] != 128 && (uint32_t)(top - lv[j]) > (uint32_t)kFar;
    }
    if (__any_sync(~0u, odd)) {     // a scale above the level or far below it, or new tokens
      int most = kNoLevel, late = kNoLevel, least = -kNoLevel;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        if (dead[j] || lv[j] == 128) continue;
        if (w.all || pos[j] < w.len - w.T + 1) most = max(most, lv[j]);
        else late = max(late, lv[j]);
        least = min(least, lv[j]);
      }
      most = __reduce_max_sync(~0u, most);
      late = __reduce_max_sync(~0u, late);
      least = __reduce_min_sync(~0u, least);
      most = max(most, late - 96);
      if (most > top) {
        if (top != kNoLevel) {
          const int d = top - most, h = d >> 1;
          const float a = pow2(h), b = pow2(d - h);
#pragma unroll
          for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) o[mt][nt][i] = o[mt][nt][i] * a * b;
        }
        top = most;
      }
      wide = (!w.all && w.T > 1) || least < top - kFar;
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const float g = dead[j] ? 0.f : lv[j] == 128 ? __uint_as_float(0x7FC00000u)
                                                   : pow2(lv[j] - top + kShift16);
      w.sc[j * 32 + lane] = make_float2(e8m0_value(kb[j]), g);
    }
    __syncwarp();
    return wide;
  }

  SA_DEVI void compute(const Step& w) {
    bool wide = false;
    if constexpr (E4M3) wide = scales(w);
    // one n-tile: all tiles of the step together; more: one after the other, for the registers
    constexpr int AT_ONCE = NT == 1 ? L::kSub : 1;
#pragma unroll 1
    for (int t0 = 0; t0 < L::kSub; t0 += AT_ONCE) tiles<AT_ONCE>(w, t0, wide);
  }

  template <int SUB>
  SA_DEVI void tiles(const Step& w, int t0, bool wide) {
    float s[SUB][NT][4];
    float g[E4M3 ? SUB : 1][2];        // factor of the weights of the lane's keys
    const int mi = lane >> 3, mr = lane & 7, key = L::key_of(r8);
    const uint32_t ka = w.k + swz_row<L::kRow>(mr + (mi & 1) * 8, mi >> 1);
#pragma unroll
    for (int t = 0; t < SUB; ++t) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[t][nt][i] = 0.f;
      // A = K: 16 keys x 16 values, 32 values at a time. For e4m3 a 16-byte chunk holds 16
      // values and a lane gets four neighbours, which stand for columns 2q, 2q+1, 2q+8 and
      // 2q+9 of the product; the queries are in the same order.
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        uint32_t a[2][4];
        if constexpr (E4M3) {
          uint32_t y[4];
          ldsm_x4((ka ^ (uint32_t)(2 * x << 4)) + (t0 + t) * 16 * L::kRow, y[0], y[1], y[2], y[3]);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              a[i][j] = e4m3x2_to_f16x2(y[2 * i + j]);
              a[i][2 + j] = e4m3x2_to_f16x2(y[2 * i + j] >> 16);
            }
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            ldsm_x4((ka ^ (uint32_t)(2 * (2 * x + i) << 4)) + (t0 + t) * 16 * L::kRow, a[i][0], a[i][1],
                    a[i][2], a[i][3]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint32_t b[2][2];
          queries(nt, x, b);
          mma<E4M3>(s[t][nt], a[0], b[0]);
          mma<E4M3>(s[t][nt], a[1], b[1]);
        }
      }
      // scale to base 2 and mask
      float ks[2] = {1.f, 1.f};
      if constexpr (E4M3) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 sc = w.sc[(t0 + t) * 16 + key + L::kKeyStep * i];
          ks[i] = sc.x;
          g[t][i] = sc.y;
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x = s[t][nt][i] * (kQs && !E4M3 ? unit : f[nt][i & 1]);
          if constexpr (E4M3) x *= ks[i >> 1];
          s[t][nt][i] = x;
        }
      if (!w.all) {
        const int pos0 = w.pos(t0 + t) + key;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (pos0 + L::kKeyStep * (i >> 1) >= lim(nt, i & 1)) s[t][nt][i] = -INFINITY;
      }
    }
    // running maxima: the warp looks across its lanes, and rescales, only when one of its
    // columns has passed its level
    float nm[NT][2];
    bool moved = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = fmaxf(s[0][nt][i], s[0][nt][i + 2]);
#pragma unroll
        for (int t = 1; t < SUB; ++t) x = fmaxf(x, fmaxf(s[t][nt][i], s[t][nt][i + 2]));
        nm[nt][i] = x;
        moved |= x > m[nt][i];
      }
    if (__any_sync(~0u, moved)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          nm[nt][i] = level(col_max(nm[nt][i]), m[nt][i]);
          const float a = ex2a(m[nt][i] - ref_of(nm[nt][i]));
          l[nt][i] *= a;
          m[nt][i] = nm[nt][i];
#pragma unroll
          for (int mt = 0; mt < kMt; ++mt) {
            o[mt][nt][i] *= a;
            o[mt][nt][i + 2] *= a;
          }
        }
    }
    // weights, and what of them goes to the sum
#pragma unroll
    for (int t = 0; t < SUB; ++t)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = s[t][nt][i], e = ex2a(x - ref_of(m[nt][i & 1]));
          l[nt][i & 1] += e;
          // (a factor of NaN must not reach the rows that do not attend its key)
          s[t][nt][i] = !E4M3 ? e : w.all || x != -INFINITY ? e * g[E4M3 ? t : 0][i >> 1] : 0.f;
        }
    if (E4M3 && wide) {
#pragma unroll
      for (int t = 0; t < SUB; ++t) products<1, true>(w, t0 + t, s + t);
    } else {
      products<SUB, false>(w, t0, s);
    }
  }

  // o += P V over SUB tiles from t0 on. WIDE (e4m3): both in bf16, the weights in three pieces.
  template <int SUB, bool WIDE>
  SA_DEVI void products(const Step& w, int t0, float (*s)[NT][4]) {
    constexpr bool F16 = E4M3 && !WIDE;
    constexpr int PC = WIDE ? 3 : PIECES;
    const int mi = lane >> 3, mr = lane & 7;
    // V's addresses: bf16 as 8x8 blocks (keys mi>>1, values mi&1), e4m3 as two 16x16 blocks
    const uint32_t va = E4M3 ? w.v + swz_row<L::kRow>(L::place(lane & 15), lane >> 4)
                             : w.v + swz_row<L::kRow>(mr + (mi >> 1) * 8, mi & 1);
    // B = P^T in pieces, by transposing each 8x8 block of S^T
    uint32_t pw[SUB][PC][NT][2];
#pragma unroll
    for (int t = 0; t < SUB; ++t)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          float e[2] = {s[t][nt][2 * hf], s[t][nt][2 * hf + 1]};
#pragma unroll
          for (int k = 0; k < PC; ++k) {
            uint32_t hi;
            if constexpr (F16) {
              hi = pack_f16(e[0], e[1]);
              const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
              e[0] -= b.x;
              e[1] -= b.y;
            } else {
              hi = pack_bf16(e[0], e[1]);
              e[0] -= bf16_lo(hi);
              e[1] -= bf16_hi(hi);
            }
            pw[t][k][nt][hf] = movmatrix(hi);
          }
        }
    // A = V^T, 32 output columns at a time
    auto load_v = [&](int t, int x, uint32_t (&a)[2][4]) {
      if constexpr (E4M3) {
        uint32_t y[4];
        ldsm_t8((va ^ (uint32_t)(2 * x << 4)) + (t0 + t) * 16 * L::kRow, y);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            a[i][j] = e4m3x2_to_f16x2(y[2 * i + j]);
            a[i][2 + j] = e4m3x2_to_f16x2(y[2 * i + j] >> 16);
            if constexpr (WIDE) {
              a[i][j] = f16x2_to_bf16x2(a[i][j]);
              a[i][2 + j] = f16x2_to_bf16x2(a[i][2 + j]);
            }
          }
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          ldsm_x4_t((va ^ (uint32_t)(2 * (2 * x + i) << 4)) + (t0 + t) * 16 * L::kRow, a[i][0], a[i][1],
                    a[i][2], a[i][3]);
      }
    };
    bool clean = true;   // no tile that some rows attend and others do not has a non-finite value
    if (!F16 && !w.all)     // (e4m3: such tiles come here WIDE)
#pragma unroll 1
      for (int t = 0; t < SUB && clean; ++t) clean = !w.part(t0 + t) || finite_values(w, t0 + t);
    if (clean) {
      // (two columns' chains side by side for one n-tile, all n-tiles' for more)
      constexpr int Y = NT == 1 ? 2 : 1;
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        uint32_t a[SUB][2][4];
#pragma unroll
        for (int t = 0; t < SUB; ++t) load_v(t, x, a[t]);
#pragma unroll
        for (int y0 = 0; y0 < 2; y0 += Y) {
          float z[Y][NT][4];
#pragma unroll
          for (int t = 0; t < SUB; ++t)
#pragma unroll
            for (int k = 0; k < PC; ++k)
#pragma unroll
              for (int y = 0; y < Y; ++y)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  if (!kAdds) mma<F16>(o[x * 2 + y0 + y][nt], a[t][y0 + y], pw[t][k][nt]);
                  else if (t == 0 && k == 0) mma_first<F16>(z[y][nt], a[t][y0 + y], pw[t][k][nt]);
                  else mma<F16>(z[y][nt], a[t][y0 + y], pw[t][k][nt]);
                }
          if constexpr (kAdds) {
#pragma unroll
            for (int y = 0; y < Y; ++y)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[x * 2 + y0 + y][nt][i] += z[y][nt][i];
          }
        }
      }
    } else if constexpr (!F16) {
      // New tokens that some rows attend and others do not, with a non-finite value: a
      // zero weight times it would reach the others, so each token's rows take a product
      // of their own in which the values that they do not attend are zeros.
#pragma unroll
      for (int t = 0; t < SUB; ++t)
#pragma unroll 1
        for (int tok = 0; tok < w.T; ++tok) {
          const int mine = w.len - (w.T - 1 - tok);
          uint32_t keep[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int k0 = w.pos(t0 + t) + (E4M3 ? 4 * q4 + 2 * i : 2 * q4 + 8 * i);
            keep[i] = (k0 < mine ? 0xFFFFu : 0u) | (k0 + 1 < mine ? 0xFFFF0000u : 0u);
          }
#pragma unroll
          for (int x = 0; x < D / 32; ++x) {
            uint32_t a[2][4];
            load_v(t, x, a);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
#pragma unroll
              for (int i = 0; i < 4; ++i) a[y][i] &= keep[i >> 1];
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < PC; ++k) mma<F16>(z, a[y], pw[t][k][nt]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (lim(nt, i & 1) == mine) o[x * 2 + y][nt][i] += z[i];
              }
            }
          }
        }
    }
  }

  // Row sums across the lanes, and (f) the factor of each column's accumulators.
  SA_DEVI void close(bool whole) {
    float back = 1.f;
    if constexpr (E4M3) {
      // 2^(top - shift) as two factors: one would be below fp32's range for V rows near the
      // smallest scale (2^-126), though the values are not
      const int y = top == kNoLevel ? 0 : top - kShift16, h = y >> 1;
      const float a = pow2(h);
      back = pow2(y - h);
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[mt][nt][i] *= a;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        l[nt][k] = col_sum(l[nt][k]);
        f[nt][k] = !whole ? back : l[nt][k] == 0.f ? 0.f : back / l[nt][k];
      }
  }
  // fn(row, m, l) for the segment's rows.
  template <class F>
  SA_DEVI void stats(F fn) {
    if (r8 == 0)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        fn(nt * 8 + 2 * q4, m[nt][0], l[nt][0]);
        fn(nt * 8 + 2 * q4 + 1, m[nt][1], l[nt][1]);
      }
  }
  // fn(row, value column, numerator) for the lane's share: a warp's calls for one (mt, i) are
  // eight neighbouring columns of four rows, whole 32-byte sectors of fp32.
  template <class F>
  SA_DEVI void emit(F fn) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          fn(nt * 8 + 2 * q4 + (i & 1), 16 * mt + r8 + 8 * (i >> 1), o[mt][nt][i] * f[nt][i & 1]);
  }
};

// What the steps of one unit (a sequence, or with kept lists a sequence's kv head) look like.
struct Unit {
  int len, n;                 // attended length, steps of each of its segments
  int keys;                   // keys in list order
};

template <class M>
SA_DEVI Unit unit_of(const DecodeArgs& p, int b, int h) {
  Unit x;
  x.len = seq_len(p.c, p.lens, b);
  x.keys = x.len;
  if (p.kv_idx && x.len)
    x.keys = min(max(p.kv_cnt[(int64_t)b * p.c.H + h], 0), p.cap) << p.c.page_log2;
  x.n = (x.keys + M::kKeys - 1) / M::kKeys;
  return x;
}

// A place on the line of steps, which runs over b, h, row groups and steps of a segment.
struct Cursor {
  int b, h, r0, s;
  Unit x;
};

// On by k steps of the segment, and to the next segment with a key from its end.
template <class M>
SA_DEVI void advance(const DecodeArgs& p, Cursor& c, int k, int R) {
  c.s += k;
  if (c.s < c.x.n) return;
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

// Zeros and lse -inf for n rows from row0 on.
template <int D>
SA_DEVI void put_empty(const DecodeArgs& p, int64_t row0, int64_t n, int tid, int threads) {
  for (int64_t i = tid; i < n * (D / 4); i += threads)
    put4(p, row0 + i / (D / 4), D, (int)(i % (D / 4)) * 4, make_float4(0.f, 0.f, 0.f, 0.f));
  for (int64_t i = tid; i < n; i += threads) put_lse(p, row0 + i, 0.f, 0.f);
}

SA_DEVI uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}
SA_DEVI void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
SA_DEVI uint32_t peer_addr(const void* p, int rank) {   // the same shared variable of another CTA
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
SA_DEVI float peer_f32(uint32_t a) {
  float x;
  asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(x) : "r"(a) : "memory");
  return x;
}
SA_DEVI float4 peer_f32x4(uint32_t a) {
  float4 x;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(a) : "memory");
  return x;
}

// CLUSTER: cluster c of the grid takes segment c alone, its CTAs and their warps equal parts
// of the steps, and joins the partials over distributed shared memory: one launch, no scan
// of the lengths. Otherwise the line of all steps is cut as described at the top.
template <int D, class M, bool CLUSTER>
__global__ void __launch_bounds__(M::kThreads, 1) decode_kernel(DecodeArgs p, int units, int groups) {
  constexpr int kWarps = M::kWarps, kStages = M::kStages, kThreads = M::kThreads;
  constexpr int kBuckets = 128;          // scan entries kept in shared memory
  extern __shared__ uint8_t smem_raw[];
  __shared__ long long s_prefix[CLUSTER ? 1 : kBuckets + 1], s_warp[kWarps];
  // partials: of warp w, 2w at the head of its share, 2w + 1 at its end
  __shared__ Place e_at[2 * kWarps];
  __shared__ float s_ml[2 * kWarps][2][M::kRows];
  __shared__ __align__(16) float s_cta[CLUSTER ? M::kRows * (D + 2) : 4];
  constexpr size_t kSlot = (size_t)M::kRows * (D + 2);   // floats of a global partial
  uint8_t* smem = smem_raw + ((256u - (smem_u32(smem_raw) & 255u)) & 255u);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int G = p.Hq / p.c.H, R = G * p.T;
  const int segs = (p.kv_idx ? 1 : p.c.H) * groups;   // segments of a unit

  long long lo_c, hi_c, total = 0;      // this CTA's steps
  Cursor cc;                            // and (below) the warp's first one
  int ctas = 0, per = 1;
  int last_cta = -1;                    // of the CTAs that share this one's segment, if it has one only
  bool by_warp = true;
  long long incl = 0, mine = 0;         // steps up to and of this lane's (thread's) units
  if (lane < 2) e_at[2 * w + lane].b = -1;
  if constexpr (CLUSTER) {
    const int size = units;              // CTAs of a cluster
    const int seg = blockIdx.x / size, rank = blockIdx.x - seg * size;
    const int bh = groups > 1 ? seg / groups : seg;
    cc.b = bh / p.c.H;
    cc.h = bh - cc.b * p.c.H;
    cc.r0 = (seg - bh * groups) * M::kRows;
    cc.x = unit_of<M>(p, cc.b, cc.h);
    if (cc.x.n == 0) {                   // the whole cluster leaves
      if (rank == 0)
        put_empty<D>(p, ((int64_t)cc.b * p.Hq + cc.h * G) * p.T + cc.r0, min(M::kRows, R - cc.r0), tid,
                     kThreads);
      return;
    }
    const Cut cut(cc.x.n, size);
    lo_c = cut.lo(rank);
    hi_c = cut.lo(rank + 1);
  } else {
    asm volatile("griddepcontrol.launch_dependents;\n");   // the joining kernel may be set up
    // ---- the line of steps: a scan over the units' weights
    auto unit_at = [&](int u) {
      return p.kv_idx ? unit_of<M>(p, u / p.c.H, u % p.c.H) : unit_of<M>(p, u, 0);
    };
    // (up to 32 kLaneUnits units every warp scans them by itself, a run of them to a lane)
    by_warp = units <= 32 * kLaneUnits;
    per = by_warp ? (units + 31) / 32 : (units + kBuckets - 1) / kBuckets;
    const int first = (by_warp ? lane : tid) * per;
    bool none = false;
    for (int u = first; u < min(units, first + per) && (by_warp || tid < kBuckets); ++u) {
      const int n = unit_at(u).n;
      incl += (long long)n * segs;
      none |= n == 0;
    }
    mine = incl;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(~0u, incl, o);
      if (lane >= o) incl += y;
    }
    bool empty;
    if (by_warp) {
      total = __shfl_sync(~0u, incl, 31);
      empty = __any_sync(~0u, none);
    } else {
      if (lane == 31) s_warp[w] = incl;
      __syncthreads();
      long long before = 0;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        if (i < w) before += s_warp[i];
        total += s_warp[i];
      }
      if (tid < kBuckets) s_prefix[tid] = before + incl - mine;
      if (tid == 0) s_prefix[kBuckets] = total;
      empty = __syncthreads_or(none);
    }
    // rows of units without a key
    for (int u = blockIdx.x; empty && u < units; u += gridDim.x) {
      if (unit_at(u).n) continue;
      const int b = p.kv_idx ? u / p.c.H : u, h = p.kv_idx ? u - b * p.c.H : 0;
      put_empty<D>(p, ((int64_t)b * p.Hq + h * G) * p.T, p.kv_idx ? R : (int64_t)p.Hq * p.T, tid, kThreads);
    }
    ctas = (int)min((long long)gridDim.x, (total + kWarps - 1) / kWarps);
    // Few long segments: whole CTAs for each, where that lengthens no share by more than 1/32,
    // spares the CTAs that would hold the end of one segment and the start of another (they
    // took 15,000 cycles longer: four segments of 32 rows 53.2 us, so cut 48.7 us).
    bool aligned = per == 1 && by_warp && total > 0 && total < (1ll << 32) && ctas == (int)gridDim.x;
    int k = 0;                            // CTAs of each segment of this lane's unit
    if (aligned) {
      const long long n = mine / segs;    // its steps; 0: none
      k = (int)(n * ctas / total);
      aligned = __all_sync(~0u, n == 0 || (k > 0 && 32 * n * ctas <= 33 * k * total));
    }
    if (aligned) {
      int upto = k * segs;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(~0u, upto, o);
        if (lane >= o) upto += y;
      }
      const int c = blockIdx.x, u = __ffs(__ballot_sync(~0u, c < upto)) - 1;   // -1: CTAs left over
      lo_c = hi_c = 0;
      if (u >= 0) {
        const int ku = __shfl_sync(~0u, k, u), in = c - __shfl_sync(~0u, upto, u) + ku * segs;
        const long long nu = __shfl_sync(~0u, mine, u) / segs;
        const int j = in / ku, i = in - j * ku;
        const long long s0 = __shfl_sync(~0u, incl - mine, u) + j * nu;
        const Cut cut(nu, ku);
        lo_c = s0 + cut.lo(i);
        hi_c = s0 + cut.lo(i + 1);
        last_cta = c - i + ku - 1;
      }
    } else {
      const Cut cut(total, ctas);
      const bool active = (int)blockIdx.x < ctas;
      lo_c = active ? cut.lo(blockIdx.x) : 0;
      hi_c = active ? cut.lo(blockIdx.x + 1) : 0;
    }
  }
  // ---- this warp's share
  const int n_c = (int)(hi_c - lo_c), n_q = n_c / kWarps, n_r = n_c % kWarps;
  const long long lo = lo_c + n_q * w + min(w, n_r);
  const int steps = n_q + (w < n_r);
  Record* rec = static_cast<Record*>(p.work) + blockIdx.x;
  float* heads = reinterpret_cast<float*>(static_cast<Record*>(p.work) + gridDim.x);
  float* head = heads + ((size_t)blockIdx.x * kWarps + w) * kSlot;
  float* cta_slots = heads + (size_t)gridDim.x * kWarps * kSlot;

  uint8_t* ring = smem + (size_t)w * M::kRing;
  uint8_t* metas = smem + (size_t)kWarps * M::kRing + (size_t)w * kStages * M::kMeta;
  float2* scale_values = reinterpret_cast<float2*>(smem + (size_t)kWarps * (M::kRing + kStages * M::kMeta) +
                                                   (size_t)w * M::kScales);

  if (steps > 0) {
    if constexpr (CLUSTER) {
      cc.s = (int)lo;
    } else {
      int a = 0;                         // the last run of units that starts at or before lo
      long long at;
      if (by_warp) {
        a = 31 - __clz(__ballot_sync(~0u, incl - mine <= lo && mine > 0));
        at = __shfl_sync(~0u, incl - mine, a);
      } else {
        for (int z = kBuckets; z - a > 1;) {
          const int mid = (a + z) / 2;
          if (s_prefix[mid] <= lo) a = mid; else z = mid;
        }
        at = s_prefix[a];
      }
      int u = a * per;
      while (true) {
        cc.b = p.kv_idx ? u / p.c.H : u;
        cc.h = p.kv_idx ? u - cc.b * p.c.H : 0;
        cc.x = unit_of<M>(p, cc.b, cc.h);
        const long long n = (long long)cc.x.n * segs;
        if (at + n > lo || u + 1 >= units) break;
        at += n;
        ++u;
      }
      const long long in = lo - at;
      const int j = segs > 1 ? (int)div_floor(in, cc.x.n) : 0;
      cc.s = (int)(in - (long long)j * cc.x.n);
      if (!p.kv_idx) cc.h = groups > 1 ? j / groups : j;
      cc.r0 = (p.kv_idx ? j : j - cc.h * groups) * M::kRows;
    }
    M mth;
    mth.lane = lane;
    mth.q4 = lane & 3;
    mth.r8 = lane >> 2;
    mth.qs = smem_u32(smem) + kWarps * (M::kRing + kStages * M::kMeta + M::kScales) + w * M::kQueries;

    // Page numbers are looked up for a batch of steps of one segment at a time (lane = step of
    // the batch x tile of the step), one step ahead of their first use: no copy waits for a
    // table but the first.
    constexpr int kBatch = 32 / M::kSub;
    Cursor ac = cc;                      // first step of the batch
    int seg_looked = 0, seg_begun = 0, seg_fetched = 0;   // segments after the first: counts
    const int in_page = (1 << p.c.page_log2) - 1;
    int b_n = 0, b_i = 0, b_pos = 0, b_pg = 0, left = steps;   // left: steps from the batch's first on
    auto look_up = [&]() {
      b_n = min(min(kBatch, left), ac.x.n - ac.s);
      b_i = 0;
      b_pos = kNoPos;
      b_pg = 0;
      const int vi = ac.s * M::kKeys + lane * 16;
      if (lane < b_n * M::kSub && vi < ac.x.keys) {
        int lp = vi >> p.c.page_log2;
        if (p.kv_idx) lp = p.kv_idx[((int64_t)ac.b * p.c.H + ac.h) * p.cap + lp];
        if ((unsigned)lp < (unsigned)p.c.table_width) {
          const int at = (lp << p.c.page_log2) + (vi & in_page);
          if (at < ac.x.len) {
            b_pos = at;
            b_pg = p.c.table[ac.b * p.c.table_stride + lp];
          }
        }
      }
    };
    const uint32_t lane_off = M::lane_part(lane);
    const int lane_row = lane / M::kChunks;
    const uint32_t page_bytes = (uint32_t)p.c.H * M::kRow << p.c.page_log2;   // < 2^32
    const uint8_t* kbase = static_cast<const uint8_t*>(p.c.k) + lane * 16;
    const uint8_t* vbase = static_cast<const uint8_t*>(p.c.v) + lane * 16;
    auto issue = [&](int st) {
      if (left > 0) {
        const uint32_t kdst = smem_u32(ring + st * 8192);
        uint8_t* meta = metas + st * M::kMeta;
        if (b_i == 0 && b_pos != kNoPos && (unsigned)b_pg >= (unsigned)p.c.num_pages) {
          b_pos = kNoPos;
          if (p.c.err_flag) atomicOr(p.c.err_flag, SA_FLAG_INDEX_BIT);
        }
        const int first = b_i * M::kSub;
        if (M::kSub == 1 ? lane == first : lane - first >= 0 && lane - first < M::kSub)
          reinterpret_cast<int*>(meta + 128)[lane - first] = b_pos;
        const int pos0 = __shfl_sync(~0u, b_pos, first), pg0 = __shfl_sync(~0u, b_pg, first);
        const uint32_t hrow = (uint32_t)ac.h << p.c.page_log2;
        if (in_page + 1 >= M::kKeys && ac.x.len - pos0 >= M::kKeys) {
          // the whole step lies in one page
          const uint64_t at = (uint64_t)(uint32_t)pg0 * page_bytes +
                              (uint64_t)(hrow + (pos0 & in_page)) * M::kRow;
          const uint8_t* ks = kbase + at;
          const uint8_t* vs = vbase + at;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            constexpr int per_tile = M::kChunks / 2;
            const uint32_t dst = kdst + i / per_tile * 16 * M::kRow + M::piece(lane_off, i % per_tile);
            cp_async16_whole(dst, ks + i * 512);
            cp_async16_whole(dst + 4096, vs + i * 512);
          }
          if constexpr (M::kE4M3) {
            if (lane < 2 * M::kSub)
              cp_async16_whole(smem_u32(meta) + lane * 16,
                               (lane < M::kSub ? p.c.k_scale : p.c.v_scale - M::kKeys) +
                                   at / M::kRow + lane * 16);
          }
        } else {
#pragma unroll 1
          for (int t = 0; t < M::kSub; ++t) {
            const int pos = __shfl_sync(~0u, b_pos, first + t), pg = __shfl_sync(~0u, b_pg, first + t);
            const int live = ac.x.len - pos;     // rows of the tile that exist (< 0: no tile)
            const uint64_t at = live > 0 ? (uint64_t)(uint32_t)pg * page_bytes +
                                               (uint64_t)(hrow + (pos & in_page)) * M::kRow
                                         : 0;
            if (live >= 16) {
#pragma unroll
              for (int i = 0; i < M::kChunks / 2; ++i) {
                const uint32_t dst = kdst + t * 16 * M::kRow + M::piece(lane_off, i);
                cp_async16_whole(dst, kbase + at + i * 512);
                cp_async16_whole(dst + 4096, vbase + at + i * 512);
              }
            } else {
            // rows behind the last one are zeros here, whatever the page holds
#pragma unroll
            for (int i = 0; i < M::kChunks / 2; ++i) {
              const uint32_t dst = kdst + t * 16 * M::kRow + M::piece(lane_off, i);
              const bool in = i * (32 / M::kChunks) + lane_row < live;
              cp_async16(dst, in ? kbase + at + i * 512 : kbase, in ? 16 : 0);
              cp_async16(dst + 4096, in ? vbase + at + i * 512 : vbase, in ? 16 : 0);
            }
            }
            if constexpr (M::kE4M3) {
              if (lane < 2 && live > 0)
                cp_async16_whole(smem_u32(meta) + lane * M::kKeys + t * 16,
                                 (lane ? p.c.v_scale : p.c.k_scale) + at / M::kRow);
            }
          }
        }
        if (++b_i == b_n) {
          left -= b_n;
          if (left > 0) {
            advance<M>(p, ac, b_n, R);
            look_up();
            if constexpr (M::kAhead) {   // its buffer is free once the last segment asked for has begun
              if (ac.s == 0 && ++seg_looked == seg_begun + 1) {
                mth.copy_queries(p, ac.b, ac.h, ac.r0);
                seg_fetched = seg_looked;
              }
            }
          }
        }
      }
      cp_async_commit();
    };
    mth.load(p, cc.b, cc.h, cc.r0, cc.x.len);
    look_up();
#pragma unroll 1
    for (int st = 0; st < kStages; ++st) issue(st);

    long long seg0 = lo - cc.s;      // first step of the current segment
    if constexpr (M::kQs) {          // the queries came with the first step
      cp_async_wait<kStages - 1>();
      __syncwarp();
    }
    mth.start(p);
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
        sp.sc = scale_values;
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
        const bool whole = !CLUSTER && ends && seg0 >= lo;
        const int rows = min(M::kRows, R - cc.r0);
        const int64_t row0 = ((int64_t)cc.b * p.Hq + cc.h * G) * p.T + cc.r0;
        float* slot = reinterpret_cast<float*>(ring);       // the partial at the share's end
        if (last) cp_async_wait<0>();
        __syncwarp();
        mth.close(whole);
        mth.stats([&](int r, float m, float l) {
          if (whole) {
            if (r < rows) put_lse(p, row0 + r, m, l);
          } else {
            s_ml[2 * w + (last ? 1 : 0)][0][r] = m;
            s_ml[2 * w + (last ? 1 : 0)][1][r] = l;
          }
        });
        if (whole) {
          if (p.out_dtype == SA_OUT_F32) {
            float* dst = static_cast<float*>(p.out) + row0 * D;
            mth.emit([&](int r, int c, float y) { if (r < rows) dst[r * D + c] = y; });
          } else {
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + row0 * D;
            mth.emit([&](int r, int c, float y) { if (r < rows) dst[r * D + c] = __float2bfloat16(y); });
          }
        } else if (last) {
          mth.emit([&](int r, int c, float y) { slot[r * M::kPad + c] = y; });
        } else {
          mth.emit([&](int r, int c, float y) { if (r < rows) head[r * D + c] = y; });
        }
        if (!whole && lane == 0)
          e_at[2 * w + (last ? 1 : 0)] = Place{cc.b, cc.h, cc.r0, cc.x.n, seg0};
      }
      if (!last) {
        advance<M>(p, cc, 1, R);
        issue(st);
        if (ends) {
          seg0 = lo + i + 1;
          ++seg_begun;
          if (M::kAhead && seg_fetched == seg_begun) mth.load_prefetched(p, cc.r0, cc.x.len);
          else mth.load(p, cc.b, cc.h, cc.r0, cc.x.len);
          if constexpr (M::kQs) {
            cp_async_commit();
            cp_async_wait<0>();
            __syncwarp();
          }
          mth.start(p);
          __syncwarp();
        }
        st = st + 1 == kStages ? 0 : st + 1;
      }
    }
  }
  __syncthreads();

  // ---- join the partials of each segment that several warps of this CTA shared
  // Lane e of every warp looks at partial e. A segment's partials are neighbours: the end
  // partials of consecutive warps and at most one head partial, the last of them.
  const bool valid = lane < 2 * kWarps && e_at[lane < 2 * kWarps ? lane : 0].b >= 0;
  const int key = valid ? (int)(e_at[lane].s0 - lo_c) : 0;     // |s0 - lo_c| < 2^31: within a segment or share
  const uint32_t held = __ballot_sync(~0u, valid), below = held & ((1u << lane) - 1u);
  const int before = __shfl_sync(~0u, key, below ? 31 - __clz(below) : lane);
  const uint32_t first = __ballot_sync(~0u, valid && (!below || before != key));
  // The threads share out all segments' values, four of a row to a thread and round.
  const int per_seg = min(M::kRows, R) * (D / 4), total_items = __popc(first) * per_seg;
  uint32_t left = first;               // from the segment of the thread's item on
  int x = tid;                         // and the item in it
  for (int i0 = 0; i0 < total_items; i0 += kThreads, x += kThreads) {
    while (x >= per_seg && left) {
      x -= per_seg;
      left &= left - 1;
    }
    if (!left) break;
    const int e0 = __ffs(left) - 1;
    const uint32_t next = left & (left - 1);
    const uint32_t mask = held & (~0u << e0) & (next ? (1u << (__ffs(next) - 1)) - 1u : ~0u);
    const int r = x / (D / 4), c = x % (D / 4) * 4;
    const Place at = e_at[e0];
    if (r >= R - at.r0) continue;
    const int hd = __ffs(mask & 0x55555555u) - 1;      // the head partial, -1: none
    const bool whole = !CLUSTER && at.s0 >= lo_c && at.s0 + at.n <= hi_c;
    float wt[kWarps], mx = -INFINITY, ls = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    float mh = -INFINITY, lh = 0.f;
    if (hd >= 0) {
      mh = s_ml[hd][0][r];
      lh = s_ml[hd][1][r];
      y = *reinterpret_cast<const float4*>(heads + ((size_t)blockIdx.x * kWarps + (hd >> 1)) * kSlot +
                                           r * D + c);
    }
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      wt[i] = mask >> (2 * i + 1) & 1 ? s_ml[2 * i + 1][0][r] : -INFINITY;
      mx = fmaxf(mx, wt[i]);
    }
    mx = fmaxf(mx, mh);
    const float ah = ex2a(mh - ref_of(mx));
    ls = ah * lh;
    y = make_float4(ah * y.x, ah * y.y, ah * y.z, ah * y.w);
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const bool in = mask >> (2 * i + 1) & 1;
      // (loaded in any case, so that the loads do not wait for one another)
      const float4 v = *reinterpret_cast<const float4*>(
          reinterpret_cast<const float*>(smem + (size_t)i * M::kRing) + r * M::kPad + c);
      const float l = s_ml[2 * i + 1][1][r], a = ex2a(wt[i] - ref_of(mx));
      ls += in ? a * l : 0.f;
      y.x += in ? a * v.x : 0.f;
      y.y += in ? a * v.y : 0.f;
      y.z += in ? a * v.z : 0.f;
      y.w += in ? a * v.w : 0.f;
    }
    if (whole) {
      const int64_t row0 = ((int64_t)at.b * p.Hq + at.h * G) * p.T + at.r0;
      const float inv = ls == 0.f ? 0.f : 1.f / ls;
      put4(p, row0 + r, D, c, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
      if (c == 0) put_lse(p, row0 + r, mx, ls);
    } else {
      float* dst = CLUSTER ? s_cta : cta_slots + ((size_t)blockIdx.x * 2 + (at.s0 < lo_c ? 0 : 1)) * kSlot;
      *reinterpret_cast<float4*>(dst + r * D + c) = y;
      if (c == 0) {
        dst[M::kRows * D + r] = mx;
        dst[M::kRows * D + M::kRows + r] = ls;
        if (!CLUSTER && r == 0 && at.s0 >= lo_c) {
          rec->at = at;
          rec->last = last_cta >= 0 ? last_cta : Cut(total, ctas).share_of(at.s0 + at.n - 1);
        }
      }
    }
  }
  if (!CLUSTER && tid == 0) {   // no segment starts here and runs on: nothing to join
    const Place at = first ? e_at[31 - __clz(first)] : Place{0, 0, 0, 0, 0};
    if (!first || at.s0 < lo_c || at.s0 + at.n <= hi_c) rec->at.b = -1;
  }

  if constexpr (CLUSTER) {
    // ---- and of the cluster's CTAs: each joins its share of the rows
    const int size = units, rank = (int)cluster_rank(), used = min(size, cc.x.n);
    cluster_sync();
    const int rows = min(M::kRows, R - cc.r0);
    const int64_t row0 = ((int64_t)cc.b * p.Hq + cc.h * G) * p.T + cc.r0;
    for (int x = rank * kThreads + tid; x < rows * (D / 4); x += size * kThreads) {
      const int r = x / (D / 4), c = x % (D / 4) * 4;
      float mx = -INFINITY, ls = 0.f;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = 0; k < used; ++k)
        mx = fmaxf(mx, peer_f32(peer_addr(s_cta + M::kRows * D + r, k)));
#pragma unroll 4
      for (int k = 0; k < used; ++k) {
        const float a = ex2a(peer_f32(peer_addr(s_cta + M::kRows * D + r, k)) - ref_of(mx));
        const float4 v = peer_f32x4(peer_addr(s_cta + r * D + c, k));
        ls += a * peer_f32(peer_addr(s_cta + M::kRows * D + M::kRows + r, k));
        y.x += a * v.x;
        y.y += a * v.y;
        y.z += a * v.z;
        y.w += a * v.w;
      }
      const float inv = ls == 0.f ? 0.f : 1.f / ls;
      put4(p, row0 + r, D, c, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
      if (c == 0) put_lse(p, row0 + r, mx, ls);
    }
    cluster_sync();   // no CTA leaves while another reads its shared memory
  }
}

// Joins the partials of the segment that starts in CTA blockIdx.x's share and spans CTAs:
// a block takes four rows, its groups of D/4 threads every eighth (or sixteenth) partial in
// one pass with a running maximum, and then each other's sums.
template <int D, int ROWS, int WARPS>
__global__ void __launch_bounds__(256) decode_join_kernel(DecodeArgs p, int ctas_max) {
  constexpr int LN = D / 4, GRP = 256 / LN, RB = 4;
  __shared__ float4 acc[RB][256];
  __shared__ float2 ml[RB][GRP];
  asm volatile("griddepcontrol.wait;\n" ::: "memory");   // the main kernel's partials are there
  const Record rec = static_cast<const Record*>(p.work)[blockIdx.x];
  if (rec.at.b < 0) return;
  const int G = p.Hq / p.c.H, R = G * p.T, row0 = blockIdx.y * RB, tid = threadIdx.x;
  const int rows = min(min(ROWS, R - rec.at.r0) - row0, RB);
  if (rows <= 0) return;
  constexpr size_t kSlot = (size_t)ROWS * (D + 2);
  const float* slots = reinterpret_cast<const float*>(static_cast<const Record*>(p.work) + ctas_max) +
                       (size_t)ctas_max * WARPS * kSlot;
  // CTAs of the segment: blockIdx.x (slot 1), then those whose share starts inside it (slot 0)
  const int parts = rec.last - blockIdx.x + 1, c = tid % LN * 4, grp = tid / LN;
  float mx[RB], ls[RB];
  float4 y[RB];
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    mx[r] = -INFINITY;
    ls[r] = 0.f;
    y[r] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll 2
  for (int i = grp; i < parts; i += GRP) {
    const float* s = slots + ((size_t)(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * kSlot;
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      if (r >= rows) continue;
      const float m = s[ROWS * D + row0 + r], l = s[ROWS * D + ROWS + row0 + r];
      const float4 v = *reinterpret_cast<const float4*>(s + (row0 + r) * D + c);
      const float n = fmaxf(mx[r], m), e = ex2a(mx[r] - ref_of(n)), f = ex2a(m - ref_of(n));
      mx[r] = n;
      ls[r] = ls[r] * e + l * f;
      y[r].x = y[r].x * e + v.x * f;
      y[r].y = y[r].y * e + v.y * f;
      y[r].z = y[r].z * e + v.z * f;
      y[r].w = y[r].w * e + v.w * f;
    }
  }
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    acc[r][tid] = y[r];
    if (c == 0) ml[r][grp] = make_float2(mx[r], ls[r]);
  }
  __syncthreads();
  for (int x = tid; x < rows * LN; x += 256) {
    const int r = x / LN, k = x % LN;
    float top = -INFINITY, sum = 0.f;
    float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int g = 0; g < GRP; ++g) top = fmaxf(top, ml[r][g].x);
#pragma unroll
    for (int g = 0; g < GRP; ++g) {
      const float f = ex2a(ml[r][g].x - ref_of(top));
      const float4 v = acc[r][g * LN + k];
      sum += f * ml[r][g].y;
      z.x += f * v.x;
      z.y += f * v.y;
      z.z += f * v.z;
      z.w += f * v.w;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int64_t orow = ((int64_t)rec.at.b * p.Hq + rec.at.h * G) * p.T + rec.at.r0 + row0 + r;
    put4(p, orow, D, k * 4, make_float4(z.x * inv, z.y * inv, z.z * inv, z.w * inv));
    if (k == 0) put_lse(p, orow, top, sum);
  }
}

// Raises a kernel's shared-memory limit, once per device.
template <class K>
cudaError_t allow_smem(K* kern, size_t bytes, std::atomic<bool> (&ready)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && ready[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev >= 0 && dev < 64) ready[dev].store(true, std::memory_order_relaxed);
  return e;
}

// Clusters of 2, 4 or 8 CTAs that the current device runs at the same time; asked once.
template <class K>
cudaError_t clusters_at_once(K* kern, const cudaLaunchConfig_t& cfg, int size, int& n,
                             std::atomic<int> (&cache)[64][4]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int log2 = size == 2 ? 1 : size == 4 ? 2 : 3;
  if (dev >= 0 && dev < 64 && (n = cache[dev][log2].load(std::memory_order_relaxed)) > 0)
    return cudaSuccess;
  e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
  if (e == cudaSuccess && dev >= 0 && dev < 64) cache[dev][log2].store(n, std::memory_order_relaxed);
  return e;
}

// How a call of these sizes runs: clusters of `size` CTAs, or (size 0) `ctas` on the line.
struct Plan {
  int groups, size, ctas;
  size_t bytes;   // scratch
};

template <int D, class M>
cudaError_t plan(const DecodeArgs& p, cudaLaunchConfig_t& cfg, cudaLaunchAttribute& attr, Plan& pl) {
  static std::atomic<bool> ready_line[64], ready_cluster[64];
  static std::atomic<int> resident[64][4];
  const long long R = (long long)(p.Hq / p.c.H) * p.T;
  pl = Plan{(int)((R + M::kRows - 1) / M::kRows), 0, 0, 0};
  const long long segs = (long long)p.B * p.c.H * pl.groups;
  // steps of a segment whose table row (or list) is full
  const long long most =
      (((long long)(p.kv_idx ? p.cap : p.c.table_width) << p.c.page_log2) + M::kKeys - 1) / M::kKeys;
  // CTAs of the line: up to eight query rows, eight SMs in nine. 132 CTAs against 148, as
  // measured (two B200s): 4 x 16 heads x 63,960 bf16 rows 299 and 306 us against 315 and 326, as
  // e4m3 rows 159 against 174; 40 heads x 75,600 e4m3 rows 126 and 130 against 133 and 134; 64
  // ragged bf16 sequences 167 against 173, e4m3 102 and 105 against 102 and 103; 64 x 8 heads x
  // 1,500 e4m3 rows, fp32 out, 45.4 against 44.5. On a third, where the first takes 325 us, 148
  // CTAs took 321.
  // More query rows need every SM (32 rows a segment, 8 x 8 heads x 16,000: 116 against 112).
  const int line = M::kRows <= 8 ? p.sms - p.sms / 9 : p.sms;
  cfg.blockDim = dim3(M::kThreads);
  cfg.dynamicSmemBytes = M::smem(true);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;

  // A cluster per segment where all clusters run at once and that gives the SMs about as much
  // work as the line would: see kClusterSlack.
  int size = 8;
  while (size > 1 && segs * size > p.sms) size /= 2;
  const long long on_line = (segs * most + (long long)line * M::kWarps - 1) / ((long long)line * M::kWarps);
  for (; size >= 1 && segs * size <= p.sms; size /= 2) {
    const long long in_cluster = (most + size * M::kWarps - 1) / (size * M::kWarps);
    // One sequence's heads are equally long, and clusters keep up with HBM over bf16 rows of up
    // to eight queries where they hold enough SMs: 28 heads x 75,600 rows 157 us (112 CTAs)
    // against 164 on the line, 20 x 32,000 52.9 (80) against 57.7, 18 x 40,000 59.5 (144) against
    // 62.6; with 64 CTAs 16 x 32,000 45.6 against 47.5, but 32 x 75,600 191 against 183. fp32
    // outputs take more of an SM: 112 CTAs 158 us against 166, 144 69.7 against 64.9, 64 57.1
    // against 49.0. 32 heads x 32,000 rows x 16 queries 90.5 (128) against 93.2. 8-bit rows: no
    // difference in 20 shapes.
    const long long held = segs * size;
    const bool enough = M::kRows > 8 ? 6 * held >= 5ll * p.sms
                        : M::kF32    ? 8 * held >= 5ll * p.sms && held <= line
                                     : 9 * held >= 4ll * p.sms ||
                                           (12 * held >= 5ll * p.sms && in_cluster <= 2 * kClusterSteps);
    const bool even = p.B == 1 && !p.kv_idx && !M::kE4M3 && enough;
    if ((in_cluster > on_line + kClusterSlack || in_cluster > kClusterSteps) && !even) break;
    auto* kern = decode_kernel<D, M, true>;
    cudaError_t e = allow_smem(kern, M::smem(true), ready_cluster);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)(segs * size));
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = size;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    if (size > 1) {
      int at_once = 0;
      e = clusters_at_once(kern, cfg, size, at_once, resident);
      if (e != cudaSuccess) return e;
      if (segs > at_once) continue;
    }
    pl.size = size;
    return cudaSuccess;
  }
  // Never more CTAs than full tables give every warp a step.
  pl.ctas = (int)std::min<long long>(line, (segs * std::max(most, 1ll) + M::kWarps - 1) / M::kWarps);
  pl.bytes = (size_t)pl.ctas * (sizeof(Record) + (M::kWarps + 2) * (size_t)M::kRows * (D + 2) * 4);
  return allow_smem(decode_kernel<D, M, false>, M::smem(false), ready_line);
}

// Runs the call, or only says how much scratch it takes (bytes).
template <int D, class M>
cudaError_t run(const DecodeArgs& p, cudaStream_t st, size_t* bytes, bool* no_work) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  Plan pl;
  cudaError_t e = plan<D, M>(p, cfg, attr, pl);
  if (bytes) *bytes = pl.bytes;
  if (bytes || e != cudaSuccess) return e;
  if (pl.bytes && (!p.work || (reinterpret_cast<uintptr_t>(p.work) & 15u))) {
    *no_work = true;
    return cudaSuccess;
  }
  cfg.stream = st;
  if (pl.size) return cudaLaunchKernelEx(&cfg, decode_kernel<D, M, true>, p, pl.size, pl.groups);
  decode_kernel<D, M, false><<<pl.ctas, M::kThreads, M::smem(false), st>>>(p, p.kv_idx ? p.B * p.c.H : p.B,
                                                                    pl.groups);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // set up while the main kernel runs; it waits for that kernel's end before it reads
  const long long R = (long long)(p.Hq / p.c.H) * p.T;
  cfg.gridDim = dim3(pl.ctas, (unsigned)(std::min<long long>(R, M::kRows) + 3) / 4);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  return cudaLaunchKernelEx(&cfg, decode_join_kernel<D, M::kRows, M::kWarps>, p, pl.ctas);
}

// The fewest rows per segment that hold the R rows of a kv head, up to 32 (more take further
// segments, which read the keys again).
template <int D, bool E4M3, bool F32>
cudaError_t run_rows(const DecodeArgs& p, cudaStream_t st, size_t* bytes, bool* no_work) {
  const long long R = (long long)(p.Hq / p.c.H) * p.T;
  if (R <= 8) return run<D, Math<D, E4M3, F32, 1, 12, 2>>(p, st, bytes, no_work);
  if (R <= 16) return run<D, Math<D, E4M3, F32, 2, 8, 3>>(p, st, bytes, no_work);
  return run<D, Math<D, E4M3, F32, 4, 8, 2>>(p, st, bytes, no_work);
}

}  // namespace

template <int D>
cudaError_t run_decode(const DecodeArgs& p, cudaStream_t st, size_t* bytes, bool* no_work) {
  const bool f32 = p.out_dtype == SA_OUT_F32;
  if (p.c.e4m3)
    return f32 ? run_rows<D, true, true>(p, st, bytes, no_work) : run_rows<D, true, false>(p, st, bytes, no_work);
  return f32 ? run_rows<D, false, true>(p, st, bytes, no_work) : run_rows<D, false, false>(p, st, bytes, no_work);
}

}  // namespace sa
