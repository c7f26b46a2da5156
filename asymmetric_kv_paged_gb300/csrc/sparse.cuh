// What the kernels of attention over selected blocks share: the bounds records, the
// integer queries' exponents, and the checks of block sizes.
#pragma once
#include <cstdint>

#include "attn_paged.h"
#include "plan.hpp"

namespace akp {

constexpr int kOddBlock = 127;      // a record's exponent for a block with an infinity or a NaN

// Bytes of a block's record: d upper codes, d lower ones, the exponent, padding.
__host__ __device__ constexpr int bounds_row_bytes(int d) { return 2 * d + 16; }

inline bool block_size_ok(const attn_problem_t &pr, int32_t block) {
  return (block == 16 || block == 32 || block == 64 || block == 128) && pr.page_size % block == 0;
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// The least e with amax <= 127 * 2^e, at least -126; 0 for amax = 0 (amax finite).
// amax = 1.f * 2^E: 127 * 2^(E - 6) = 1.984375 * 2^E.
__device__ __forceinline__ int code_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  if (u == 0u) return 0;
  const int e = (int)(u >> 23) - 127 - ((u & 0x7FFFFFu) <= 0x7E0000u ? 6 : 5);
  return max(e, -126);
}

}  // namespace akp
