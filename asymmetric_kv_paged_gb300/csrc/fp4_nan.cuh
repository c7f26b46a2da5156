// NaN block scales in the V rows of a 4-bit cache.
//
// A row of weights meets a tile's V rows in one matrix product, and a weight of
// zero times NaN is NaN: the rows of a block that do not see a key (causal edge,
// start of a window) would get the NaN of its V row too.  On tiles that some row of
// the block sees only in part the kernels therefore take such scales as zeros and set
// a flag; a CTA (in the prefill kernel a segment) that ends with the flag set looks
// through the keys of those tiles once more, row by row, and makes the 16 dims of
// each such block NaN for the rows that see its key.  Where there is no NaN nothing
// but the flag is read, and on the other tiles the product itself does what it should.
#pragma once
#include "e2m1.cuh"
#include "kernels.hpp"

namespace akp {

// 0xFF for every byte of `scales` that is an E4M3 NaN code.
__device__ __forceinline__ uint32_t e4m3_nan_bytes(uint32_t scales) {
  return __vcmpeq4(scales & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
}

// The 16-dim blocks (bit c: block c) whose scale is NaN in the V row of a key of
// [j0, j1) of request b, KV head g.
__device__ __forceinline__ uint32_t v_nan_blocks(const RunArgs &a, int b, int g, int j0, int j1) {
  uint32_t lo = 0u, hi = 0u;
#pragma unroll 1
  for (int j = j0; j < j1; ++j) {
    const int32_t page = __ldg(a.page_table + (int64_t)b * a.pt_stride + j / a.page_size);
    if (page < 0 || page >= a.num_pages) continue;          // read as zeros
    const int64_t slot = (int64_t)page * a.page_size + j % a.page_size;
    const uint2 s = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(a.v_cache) +
                                                          (slot * a.hkv + g) * e2m1_row_bytes(kDv) + kDv / 2));
    lo |= e4m3_nan_bytes(s.x);
    hi |= e4m3_nan_bytes(s.y);
  }
  uint32_t m = 0u;
#pragma unroll
  for (int c = 0; c < 4; ++c) m |= ((lo >> (8 * c)) & 1u) << c | ((hi >> (8 * c)) & 1u) << (4 + c);
  return m;
}

// Keys [lo, hi) that every row of the block sees: those before the request's new
// tokens, or all but the first and last nrows of the block's range (its rows'
// tokens, hence their ranges, lie less than nrows apart).
struct SharedKeys {
  int lo, hi;
  __device__ __forceinline__ SharedKeys() : lo(0), hi(0) {}
  __device__ __forceinline__ SharedKeys(const RunArgs &a, const BlockDesc &bd) {
    lo = a.window > 0 ? bd.klo + bd.nrows : 0;
    hi = max(bd.L - bd.n, bd.khi - bd.nrows) + 1;
  }
  // whether some row does not see all of the `keys` keys from key0 on
  __device__ __forceinline__ bool cut(int key0, int keys) const { return key0 < lo || key0 + keys > hi; }
};

// The NaN blocks of a row among its keys [row_lo, row_hi) of the staged tiles
// [tile_begin, tile_end), from the bytes that the staging pass left per tile.
__device__ __forceinline__ uint32_t staged_nan_blocks(const RunArgs &a, const BlockDesc &bd, int tile_begin,
                                                      int tile_end, int row_lo, int row_hi) {
  const uint8_t *nan = a.stage_nan + bd.srow / kStageTile;
  uint32_t dims = 0u;
#pragma unroll 1
  for (int x = tile_begin; x < tile_end; ++x) {
    const uint32_t in_tile = __ldcg(nan + x);
    const int j0 = max(row_lo, x * kStageTile), j1 = min(row_hi, (x + 1) * kStageTile);
    if (!(in_tile & ~dims) || j0 >= j1) continue;
    dims |= j1 - j0 == kStageTile ? in_tile : v_nan_blocks(a, bd.b, bd.g, j0, j1);
  }
  return dims;
}

// The NaN blocks among keys [j0, j1) in those units (of `unit` keys) that
// SharedKeys::cut holds for.
__device__ __forceinline__ uint32_t cut_nan_blocks(const RunArgs &a, const BlockDesc &bd, int j0, int j1, int unit) {
  // whole units between the two borders are seen by every row
  const SharedKeys all(a, bd);
  const int lo = (all.lo + unit - 1) / unit * unit, hi = all.hi / unit * unit;
  if (lo >= hi) return v_nan_blocks(a, bd.b, bd.g, j0, j1);
  return v_nan_blocks(a, bd.b, bd.g, j0, min(j1, lo)) | v_nan_blocks(a, bd.b, bd.g, max(j0, hi), j1);
}

// NaN into the blocks `dims` of a row of kDv bf16 or (out == nullptr) fp32 values.
__device__ __forceinline__ void store_nan_blocks(uint32_t dims, uint16_t *out, float *part) {
#pragma unroll 1
  for (int c = 0; c < kDv / 16; ++c) {
    if (!((dims >> c) & 1u)) continue;
    for (int j = 16 * c; j < 16 * c + 16; ++j) {
      if (out)
        out[j] = 0x7FFFu;
      else
        part[j] = __int_as_float(0x7FFFFFFF);
    }
  }
}

// Both for all rows of the CTA's segments (tiles of `tile` keys), by all its threads
// after its last barrier, in what was written of the rows: `out`, or the partials.
__device__ __forceinline__ void patch_nan_rows(const RunArgs &a, int tile, int unit) {
  // (read again: kept in registers until here, they would cost the softmax)
  const int seg_end = a.cta_heads[blockIdx.x].seg_end;
#pragma unroll 1
  for (int sg = a.cta_heads[blockIdx.x].seg_begin; sg < seg_end; ++sg) {
    const SegDesc sd = a.segs[sg];
    const BlockDesc bd = a.blocks[sd.block];
#pragma unroll 1
    for (int r = threadIdx.x; r < bd.nrows; r += blockDim.x) {
      const int flat = bd.row0 + r;
      const int i = bd.L - bd.n + flat / a.group;        // the last key that the row sees
      const uint32_t dims = cut_nan_blocks(a, bd, max(sd.tile_begin * tile, a.window > 0 ? i - a.window + 1 : 0),
                                           min(sd.tile_end * tile, i + 1), unit);
      uint16_t *out = static_cast<uint16_t *>(a.out) +
                      ((int64_t)(bd.tok0 + flat / a.group) * a.hq + bd.g * a.group + flat % a.group) * kDv;
      float *part = a.part_o + (int64_t)(bd.part_row_base + sd.split * bd.nrows + r) * kDv;
#pragma unroll 1
      for (int d = 0; d < kDv; ++d) {
        if (!((dims >> (d / 16)) & 1u)) continue;
        if (bd.num_splits == 1)
          out[d] = 0x7FFFu;
        else
          part[d] = __int_as_float(0x7FFFFFFF);
      }
    }
  }
}

}  // namespace akp
