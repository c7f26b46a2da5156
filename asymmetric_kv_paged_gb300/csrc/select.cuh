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

// select_tc.cu: chunks of tokens.  False: the batch is not one for it.
bool select_tc_fits(const HostPlan &hp, const SelectArgs &a);
cudaError_t launch_select_tc(const HostPlan &hp, const SelectArgs &a, int device, cudaStream_t st);

}  // namespace akp
