// The 4-bit cache format: rows of E2M1 codes with one E4M3 scale per 16 values.
//
// A row of d values of one KV head is a record of e2m1_row_bytes(d) bytes:
// d/2 bytes of codes (element 2i in the low nibble of byte i), d/16 scale
// bytes (block i covers elements 16i .. 16i + 15), and zeros up to a multiple
// of 16, so that rows are 16-byte aligned and loadable as TMA boxes: 112 bytes
// for d = 192 (108 used), 80 for d = 128 (72 used).  A value is
// code * scale * the tensor's own scale.
//
// E2M1 magnitudes are 0, 0.5, 1, 1.5, 2, 3, 4, 6 (code s e e m, exponent bias
// 1).  code * scale has at most 2 + 4 significant bits, is a multiple of
// 2^-10 and at most 2688, so it is exact in fp16 (11 bits, steps down to
// 2^-24, up to 65504): the widening rounds nothing.
// The E4M3 NaN scales (0x7F, 0xFF) make their whole block NaN.
#pragma once
#include <cstdint>

#include "attn_paged.h"
#include "e4m3.cuh"

namespace akp {

constexpr int kE2m1Block = 16;      // values per scale

__host__ __device__ constexpr int e2m1_row_bytes(int d) {
  return (d / 2 + d / kE2m1Block + 15) / 16 * 16;
}

// Bytes of one cached row of d values of one KV head (0: no such type).
__host__ __device__ constexpr int kv_row_bytes(int kv_dtype, int d) {
  return kv_dtype == ATTN_KV_BF16       ? 2 * d
         : kv_dtype == ATTN_KV_FP8_E4M3 ? d
         : kv_dtype == ATTN_KV_FP4_E2M1 ? e2m1_row_bytes(d)
                                        : 0;
}

// Eight codes (element i in nibble i) -> eight fp16 values, element 2j in the
// low half of word j: one conversion instruction per byte.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Two E4M3 scales (byte 0, byte 1 of `s`) as fp16, each in both halves of a word.
__device__ __forceinline__ void e4m3_scales_f16(uint32_t s, uint32_t &s0, uint32_t &s1) {
  uint32_t p;
  asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}\n" : "=r"(p) : "r"(s));
  s0 = __byte_perm(p, 0u, 0x1010);
  s1 = __byte_perm(p, 0u, 0x3232);
}

// 32 codes (one 16-byte chunk, two blocks) and their two scale bytes -> 32
// fp16 values as four 16-byte chunks, in element order.
__device__ __forceinline__ void e2m1x32_to_f16(const uint4 raw, uint32_t scales, uint4 (&out)[4]) {
  uint32_t s0, s1;
  e4m3_scales_f16(scales, s0, s1);
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t h[4];
    e2m1x8_to_f16(w[q], h);
    const uint32_t s = q < 2 ? s0 : s1;
    out[q] = make_uint4(mul_f16x2(h[0], s), mul_f16x2(h[1], s), mul_f16x2(h[2], s), mul_f16x2(h[3], s));
  }
}

}  // namespace akp
