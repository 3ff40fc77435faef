// Device helpers of the paged cache: page lookup and the 8-bit row format.
//
// A cached row of d values is stored as bf16, or as d e4m3 codes and one E8M0 byte s
// (value = code * 2^(s - 127)). The scale is a power of two so that scaling loses nothing:
// x * 2^-k and code * 2^k are exact in fp32, and the only rounding is the one to e4m3
// (at most 2^-4 of the value, or 2^-10 of the scale near zero).
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"
#include "launch.h"

namespace sa {

// 2^(s - 127); 255 is NaN, 0 is 2^-127 (a subnormal fp32).
SA_DEVI float e8m0_value(uint32_t s) {
  const uint32_t bits = (s << 23) | (((s + 1u) & 255u) < 2u ? 0x00400000u : 0u);
  return __uint_as_float(bits);
}

// Two e4m3 codes (low 16 bits of v) -> two f16, exact.
SA_DEVI uint32_t e4m3x2_to_f16x2(uint32_t v) {
  uint32_t y;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(y) : "h"(static_cast<uint16_t>(v)));
  return y;
}

// Pool page of logical page `lp` of sequence b, or -1 (and SA_FLAG_INDEX) when the table
// holds no page of the pool there.
SA_DEVI int pool_page(const PagedView& c, int b, int lp) {
  const int pg = c.table[(int64_t)b * c.table_stride + lp];
  if ((unsigned)pg < (unsigned)c.num_pages) return pg;
  if (c.err_flag) atomicOr(c.err_flag, SA_FLAG_INDEX_BIT);
  return -1;
}

// Length of sequence b clamped to what its table row can hold (nothing without a pool).
SA_DEVI int seq_len(const PagedView& c, const int32_t* lens, int b) {
  const int n = lens[b];
  const int64_t most = c.num_pages > 0 ? (int64_t)c.table_width << c.page_log2 : 0;
  if (n >= 0 && n <= most) return n;
  if (c.err_flag) atomicOr(c.err_flag, SA_FLAG_INDEX_BIT);
  return n < 0 ? 0 : (int)most;
}

}  // namespace sa
