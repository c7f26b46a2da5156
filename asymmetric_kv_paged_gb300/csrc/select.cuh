// What the two kernels of attn_select_blocks share (select.cu, select_tc.cu).
#pragma once
#include <cuda_fp16.h>

#include <cstdint>

#include "kernels.hpp"
#include "sparse.cuh"

namespace akp {

struct SelectArgs {
  const uint16_t *q;
  const uint8_t *bounds;
  const int32_t *page_table, *seq_lens, *qo_indptr;
  int32_t *block_idx, *err;
  int32_t batch, hq, hkv, group, row_tiles, page_size, pt_stride, num_pages;
  int32_t block, take, first, last, max_len, max_blocks;
  int32_t tokens;
};

// Four signed bytes -> four fp16 values: with the sign bit flipped, byte u = v + 128 is
// the low byte of fp16 1024 + u.
__device__ __forceinline__ void s8x4_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
  w ^= 0x80808080u;
  const __half2 bias = __half2half2(__ushort_as_half(0x6480));      // 1152
  uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
  const __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&a), bias);
  const __half2 y = __hsub2(*reinterpret_cast<__half2 *>(&b), bias);
  lo = *reinterpret_cast<const uint32_t *>(&x);
  hi = *reinterpret_cast<const uint32_t *>(&y);
}

// fp32 -> an unsigned integer of the same order
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// The `want` largest of n <= 32 * kHeld scores, equal ones by lowest index, as block
// numbers first + index in ascending order; a warp, its scores in registers: the smallest
// one taken is found bit by bit, until exactly `want` are not below it.
constexpr int kHeld = 16;
__device__ __forceinline__ void pick_held(const uint32_t *keys, int n, int want, int first, int32_t *out, int lane) {
  if (want <= 0) return;
  uint32_t k[kHeld];
  uint32_t least = 0xFFFFFFFFu, most = 0u;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int c = 32 * i + lane;
    k[i] = 0u;                                    // (no score is 0)
    if (c < n) {
      k[i] = keys[c];
      least = min(least, k[i]);
    }
    most = max(most, k[i]);
  }
  least = __reduce_min_sync(0xffffffffu, least);
  most = __reduce_max_sync(0xffffffffu, most);
  int bit = 31 - __clz(least ^ most);             // the first that differs (-1: none)
  uint32_t from = bit < 0 ? most : bit == 31 ? 0u : most >> (bit + 1) << (bit + 1);
  int count = n;                                  // scores >= from
  for (; bit >= 0 && count != want; --bit) {
    const uint32_t trial = from | 1u << bit;
    int c = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) c += k[i] >= trial;
    c = __reduce_add_sync(0xffffffffu, c);
    if (c >= want) {
      from = trial;
      count = c;
    }
  }
  const uint32_t below = (1u << lane) - 1u;
  if (count == want) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const bool in = k[i] >= from && 32 * i + lane < n;
      const uint32_t m = __ballot_sync(0xffffffffu, in);
      if (in) out[__popc(m & below)] = first + 32 * i + lane;
      out += __popc(m);
    }
    return;
  }
  // several equal `from`, not all of which are in
  int above = 0;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) above += k[i] > from;
  int ties = want - __reduce_add_sync(0xffffffffu, above);
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const uint32_t eq = __ballot_sync(0xffffffffu, k[i] == from);
    const bool in = k[i] > from || (k[i] == from && __popc(eq & below) < ties);
    const uint32_t m = __ballot_sync(0xffffffffu, in);
    if (in) out[__popc(m & below)] = first + 32 * i + lane;
    out += __popc(m);
    ties -= __popc(eq);
  }
}

// select_tc.cu: chunks of tokens.  CTAs of a cluster there; 0: the batch is not one for it.
int select_tc_ranks(const HostPlan &hp, const SelectArgs &a);
cudaError_t launch_select_tc(const HostPlan &hp, const SelectArgs &a, int device, cudaStream_t st);

}  // namespace akp
