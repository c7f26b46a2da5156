// Bounds of the cache's blocks: attn_update_bounds and attn_read_bounds.
//
// For a block of block_size keys of one KV head, per dim hi = max k, lo = min k over the
// rows as the cache holds them; e is the least exponent with max |k| <= 127 * 2^e, and
// the record holds ceil(hi / 2^e) and floor(lo / 2^e) in 8 bits: every step is exact, so
// a record is a function of the rows alone.  Minima and maxima do not depend on the
// order either, and a block is always taken from all its rows when its last one arrives:
// nothing is accumulated from step to step, and rejected drafts leave nothing behind.
//
// A warp takes one block of one head, heads of a block side by side (their rows are
// neighbours in the cache): a lane owns 16 bytes of a row (8, 16 or 32 values) of every
// RG-th row, in 16-bit pairs (exact for every cache type: bf16, or fp16 of E4M3 and E2M1
// times its scale); the row groups meet by shuffle, so that nothing is shared and warps
// never wait for one another.  Which block a warp takes follows from the requests'
// counts of completed blocks, summed up 32 requests a step.  The kernel reads each key
// once.  For a decode step (64 requests, 8 tokens each: 6.0 us, reading back 2.5) the launch
// and a chain of dependent loads bound it.  All 17,000 records of a 4-bit cache (64 keys, 4
// heads, 124 MB of keys) take 56 us, 2.2 TB/s: the widening of the nibbles fills the issue
// slots' better half and its registers leave 34 KB in flight on an SM, four rows of 16 bytes
// a lane ahead (a CTA a block with rounded codes by comparison: 60 us for the update and 121
// in all with the reading, now 65).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "attn_paged.h"
#include "e2m1.cuh"
#include "kernels.hpp"
#include "plan.hpp"
#include "requests.cuh"
#include "sparse.cuh"

namespace akp {
namespace {

constexpr int kThreads = 256;

struct BoundsArgs {
  const void *k_cache;
  uint8_t *bounds;
  const int32_t *page_table, *seq_lens, *indptr;
  int32_t *err;
  uint16_t *out;                  // reading back
  int32_t rows;                   // flat rows (update: positions, reading: blocks)
  int32_t batch, hkv, page_size, pt_stride, num_pages, block;
};

template <int KV>
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
  uint32_t d;
  if (KV == ATTN_KV_BF16)
    asm("max.NaN.bf16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("max.NaN.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <int KV>
__device__ __forceinline__ uint32_t min_pair(uint32_t a, uint32_t b) {
  uint32_t d;
  if (KV == ATTN_KV_BF16)
    asm("min.NaN.bf16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("min.NaN.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <int KV>
__device__ __forceinline__ float2 pair_values(uint32_t w) {
  if (KV == ATTN_KV_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// How a warp takes rows of D values: VL values a lane (16 bytes of codes), NC lanes a
// row, RG rows at a time.
template <int KV, int D>
struct Rows {
  static constexpr int VL = KV == ATTN_KV_BF16 ? 8 : KV == ATTN_KV_FP8_E4M3 ? 16 : 32, NP = VL / 2;
  static constexpr int NC = D / VL, RG = 32 / NC;
  // rows in flight per lane
  static constexpr int kAhead = KV == ATTN_KV_FP4_E2M1 ? 4 : 8;
};

// A lane's piece of a row: the codes, and for 4-bit rows its two scales.
template <int KV, int D>
__device__ __forceinline__ void load_piece(const uint8_t *row, int ch, uint4 &raw, uint32_t &sc) {
  raw = __ldg(reinterpret_cast<const uint4 *>(row) + ch);
  if (KV == ATTN_KV_FP4_E2M1) sc = __ldg(reinterpret_cast<const uint16_t *>(row + D / 2) + ch);
}
template <int KV, int D>
__device__ __forceinline__ void widen_piece(const uint4 raw, uint32_t sc, uint32_t (&w)[Rows<KV, D>::NP]) {
  const uint32_t r[4] = {raw.x, raw.y, raw.z, raw.w};
  if constexpr (KV == ATTN_KV_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = r[i];
  } else if constexpr (KV == ATTN_KV_FP8_E4M3) {
    uint4 lo, hi;
    e4m3x16_to_f16(raw, lo, hi);
    w[0] = lo.x, w[1] = lo.y, w[2] = lo.z, w[3] = lo.w, w[4] = hi.x, w[5] = hi.y, w[6] = hi.z, w[7] = hi.w;
  } else {
    uint4 o[4];
    e2m1x32_to_f16(raw, sc, o);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[4 * i] = o[i].x, w[4 * i + 1] = o[i].y, w[4 * i + 2] = o[i].z, w[4 * i + 3] = o[i].w;
  }
}

// The slot of position `pos` of request b, or -1 with the error bit to set.
__device__ __forceinline__ int64_t slot_of(const BoundsArgs &a, int b, int64_t pos, int &bad) {
  bad = 4;
  if (pos < 0 || pos / a.page_size >= a.pt_stride) return -1;
  const int32_t page = __ldg(a.page_table + (int64_t)b * a.pt_stride + pos / a.page_size);
  bad = 1;
  if (page < 0 || page >= a.num_pages) return -1;
  bad = 0;
  return (int64_t)page * a.page_size + pos % a.page_size;
}

// The request whose completed blocks hold block number j of all of them, and the number
// of its block; false past the last.  All 32 lanes of a warp call it.  Blocks before
// position 0 (a length that does not hold its rows) are none.
__device__ __forceinline__ bool find_block(const BoundsArgs &a, int64_t j, int &b, int64_t &c, bool &odd) {
  const int lane = threadIdx.x & 31;
  int64_t base = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    const int r = b0 + lane;
    int64_t first = 0, cnt = 0;
    if (r < a.batch) {
      const int64_t L = __ldg(a.seq_lens + r), m = (int64_t)__ldg(a.indptr + r + 1) - __ldg(a.indptr + r);
      odd |= L < m;
      first = max((int64_t)0, L - m) / a.block;
      cnt = max((int64_t)0, max((int64_t)0, L) / a.block - first);
    }
    int64_t sum = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, base + sum > j);
    if (past) {
      const int l = __ffs(past) - 1;
      b = b0 + l;
      c = j - base - __shfl_sync(0xffffffffu, sum - cnt, l) + __shfl_sync(0xffffffffu, first, l);
      return true;
    }
    base += __shfl_sync(0xffffffffu, sum, 31);
  }
  return false;
}

// WIDE: the CTA's warps share a block's rows (few blocks: one round trip to memory for
// each instead of several).
template <int KV, int D, bool WIDE>
__global__ void __launch_bounds__(kThreads, KV == ATTN_KV_FP4_E2M1 ? 2 : 4) update_kernel(const BoundsArgs a) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  using R = Rows<KV, D>;
  constexpr int kWarps = kThreads / 32;
  __shared__ uint32_t part[WIDE ? kWarps : 1][2][D / 2];         // [warp][hi, lo][pair]
  const int lane = threadIdx.x & 31, ch = lane % R::NC, rg = lane / R::NC, warp = threadIdx.x >> 5;
  const int64_t warps = (int64_t)gridDim.x * (WIDE ? 1 : kWarps);
  const int64_t first_warp = WIDE ? blockIdx.x : (int64_t)blockIdx.x * kWarps + warp;
  // rows that kv_indptr does not hold
  if (first_warp == 0 && lane == 0 && __ldg(a.indptr + a.batch) < a.rows) atomicOr(a.err, 4);
  for (int64_t unit = first_warp;; unit += warps) {
    const int g = (int)(unit % a.hkv);
    int b;
    int64_t c;
    bool odd_len = false;
    const bool more = find_block(a, unit / a.hkv, b, c, odd_len);
    if (odd_len && first_warp == 0) atomicOr(a.err, 4);
    if (!more) break;
    int bad = 0;
    const int64_t slot = slot_of(a, b, c * a.block, bad);
    if (bad && g == 0 && lane == 0) atomicOr(a.err, bad);
    if (slot < 0) continue;
    const uint8_t *row = static_cast<const uint8_t *>(a.k_cache) + (slot * a.hkv + g) * kv_row_bytes(KV, D);
    const int64_t step = (int64_t)a.hkv * kv_row_bytes(KV, D);
    // every row group starts from row 0 .. RG - 1; the lanes past the last group repeat it
    const int mine = min(rg, R::RG - 1);
    // rows [r_lo, r_hi) are the warp's
    const int r_lo = WIDE ? a.block / kWarps * warp : 0, r_hi = WIDE ? r_lo + a.block / kWarps : a.block;
    uint32_t hi[R::NP], lo[R::NP];
    {
      uint4 raw;
      uint32_t sc = 0u;
      load_piece<KV, D>(row + min(r_lo + mine, r_hi - 1) * step, ch, raw, sc);
      widen_piece<KV, D>(raw, sc, hi);
#pragma unroll
      for (int i = 0; i < R::NP; ++i) lo[i] = hi[i];
    }
#pragma unroll 1
    for (int r0 = r_lo + mine + R::RG; r0 < r_hi; r0 += R::RG * R::kAhead) {
      uint4 raw[R::kAhead];
      uint32_t sc[R::kAhead];
#pragma unroll
      for (int k = 0; k < R::kAhead; ++k) {
        // (past the last row: that row again, which changes nothing)
        load_piece<KV, D>(row + min(r0 + k * R::RG, r_hi - 1) * step, ch, raw[k], sc[k]);
      }
#pragma unroll
      for (int k = 0; k < R::kAhead; ++k) {
        uint32_t w[R::NP];
        widen_piece<KV, D>(raw[k], sc[k], w);
#pragma unroll
        for (int i = 0; i < R::NP; ++i) {
          hi[i] = max_pair<KV>(hi[i], w[i]);
          lo[i] = min_pair<KV>(lo[i], w[i]);
        }
      }
    }
    __syncwarp();
    // the row groups meet in every lane
    if (R::RG > 1) {
#pragma unroll
      for (int i = 0; i < R::NP; ++i) {
        uint32_t h = hi[i], l = lo[i];
#pragma unroll
        for (int k = 1; k < R::RG; ++k) {
          const int from = (ch + R::NC * ((mine + k) % R::RG)) & 31;
          h = max_pair<KV>(h, __shfl_sync(0xffffffffu, hi[i], from));
          l = min_pair<KV>(l, __shfl_sync(0xffffffffu, lo[i], from));
        }
        hi[i] = h;
        lo[i] = l;
      }
    }
    if (WIDE) {
      if (rg == 0)
#pragma unroll
        for (int i = 0; i < R::NP; ++i) {
          part[warp][0][ch * R::NP + i] = hi[i];
          part[warp][1][ch * R::NP + i] = lo[i];
        }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kWarps; ++k)
#pragma unroll
        for (int i = 0; i < R::NP; ++i) {
          hi[i] = max_pair<KV>(hi[i], part[k][0][ch * R::NP + i]);
          lo[i] = min_pair<KV>(lo[i], part[k][1][ch * R::NP + i]);
        }
      __syncthreads();
      if (warp) continue;
    }
    float t = 0.f;
    bool odd = false;                              // an infinity or a NaN
#pragma unroll
    for (int i = 0; i < R::NP; ++i) {
      const float2 x = pair_values<KV>(hi[i]), y = pair_values<KV>(lo[i]);
      odd |= !(fabsf(x.x) < INFINITY) | !(fabsf(x.y) < INFINITY) | !(fabsf(y.x) < INFINITY) | !(fabsf(y.y) < INFINITY);
      t = fmaxf(fmaxf(t, fmaxf(fabsf(x.x), fabsf(x.y))), fmaxf(fabsf(y.x), fabsf(y.y)));
    }
    odd = __any_sync(0xffffffffu, odd);
    t = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(t)));      // (not negative)
    const int e = odd ? kOddBlock : code_exponent(t);
    uint8_t *rec = a.bounds + (slot / a.block * a.hkv + g) * bounds_row_bytes(D);   // pages hold whole blocks
    if (rg == 0) {
      const float unit_e = pow2(-e);
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        uint32_t words[R::VL / 4];
#pragma unroll
        for (int i = 0; i < R::VL / 4; ++i) {
          words[i] = 0u;
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const float2 v = pair_values<KV>(which ? lo[2 * i + p / 2] : hi[2 * i + p / 2]);
            const float x = p & 1 ? v.y : v.x;
            // 1.5 * 2^23 + x / 2^e rounded outwards once: the low byte is the code
            const float y = which ? __fmaf_rd(x, unit_e, 12582912.f) : __fmaf_ru(x, unit_e, 12582912.f);
            words[i] |= (__float_as_uint(y) & 0xFFu) << (8 * p);
          }
          if (odd) words[i] = 0u;
        }
        uint8_t *dst = rec + which * D + ch * R::VL;
        if constexpr (R::VL == 8) {
          *reinterpret_cast<uint2 *>(dst) = make_uint2(words[0], words[1]);
        } else {
#pragma unroll
          for (int i = 0; i < R::VL / 16; ++i)
            reinterpret_cast<uint4 *>(dst)[i] =
                make_uint4(words[4 * i], words[4 * i + 1], words[4 * i + 2], words[4 * i + 3]);
        }
      }
      if (ch == 0) *reinterpret_cast<uint4 *>(rec + 2 * D) = make_uint4((uint32_t)(e & 0xFF), 0u, 0u, 0u);
    }
  }
}

// A warp per (block, head): lane c takes codes 16c .. of the record.
template <int D>
__global__ void __launch_bounds__(kThreads) read_kernel(const BoundsArgs a) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t row = unit / a.hkv;
  const int g = (int)(unit % a.hkv);
  if (row >= a.rows) return;
  const int b = request_of(a.indptr, a.batch, row);
  int bad = 4;
  int64_t slot = -1;
  if (b < a.batch && row >= __ldg(a.indptr)) {
    const int64_t c = __ldg(a.seq_lens + b) / a.block + row - __ldg(a.indptr + b + 1);
    if (c >= 0) slot = slot_of(a, b, c * a.block, bad);
  }
  if (bad && g == 0 && lane == 0) atomicOr(a.err, bad);
  if (lane >= 2 * D / 16) return;
  uint16_t *dst = a.out + (row * a.hkv + g) * (2 * D) + lane * 16;
  uint32_t w[8] = {};
  if (slot >= 0) {
    const uint8_t *rec = a.bounds + (slot / a.block * a.hkv + g) * bounds_row_bytes(D);
    const int4 raw = *(reinterpret_cast<const int4 *>(rec) + lane);
    const int e = (int8_t)rec[2 * D];
    const int v[4] = {raw.x, raw.y, raw.z, raw.w};
    const float u = pow2(e == kOddBlock ? 0 : e), inf = lane < D / 16 ? INFINITY : -INFINITY;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int pair = v[i / 2] >> (16 * (i & 1));
      float x = (float)(int8_t)pair * u, y = (float)(int8_t)(pair >> 8) * u;
      if (e == kOddBlock) x = y = inf;
      const __nv_bfloat162 p = __floats2bfloat162_rn(x, y);
      w[i] = *reinterpret_cast<const uint32_t *>(&p);
    }
  }
  reinterpret_cast<uint4 *>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4 *>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

attn_status_t check(attn_plan_t plan, int32_t block_size, int64_t rows) {
  if (!plan || plan->device < 0 || rows < 0 || rows > INT32_MAX) return ATTN_ERR_INVALID_ARG;
  return block_size_ok(plan->host.prob, block_size) ? ATTN_OK : ATTN_ERR_UNSUPPORTED;
}

BoundsArgs make_args(attn_plan_t plan, int32_t block_size, const int32_t *page_table, const int32_t *seq_lens,
                     const int32_t *indptr, int64_t rows) {
  const attn_problem_t &pr = plan->host.prob;
  BoundsArgs a{};
  a.page_table = page_table;
  a.seq_lens = seq_lens;
  a.indptr = indptr;
  a.err = plan->dev.err;
  a.rows = (int32_t)rows;
  a.batch = pr.batch;
  a.hkv = pr.num_kv_heads;
  a.page_size = pr.page_size;
  a.pt_stride = pr.page_table_stride;
  a.num_pages = pr.num_pages;
  a.block = block_size;
  return a;
}

template <int D>
cudaError_t launch_update(const BoundsArgs &a, int kv, int64_t most, int num_sms, cudaStream_t st) {
  // a warp a block and head; where there are SMs for it, a CTA (32 requests of 128 new tokens,
  // 384 records at most: 7.7 us against 9.1; of 512, 1,152 records: 15.0 against 9.8)
  const int64_t per = kThreads / 32, room = (int64_t)num_sms * 4;
  const bool wide = most <= room;
  const dim3 grid((unsigned)std::min(wide ? most : (most + per - 1) / per, room)), block(kThreads);
  switch (kv) {
    case ATTN_KV_BF16: 
      return wide ? launch_dependent(update_kernel<ATTN_KV_BF16, D, true>, grid, block, 0, st, a)
                  : launch_dependent(update_kernel<ATTN_KV_BF16, D, false>, grid, block, 0, st, a);
    case ATTN_KV_FP8_E4M3: 
      return wide ? launch_dependent(update_kernel<ATTN_KV_FP8_E4M3, D, true>, grid, block, 0, st, a)
                  : launch_dependent(update_kernel<ATTN_KV_FP8_E4M3, D, false>, grid, block, 0, st, a);
    default: 
      return wide ? launch_dependent(update_kernel<ATTN_KV_FP4_E2M1, D, true>, grid, block, 0, st, a)
                  : launch_dependent(update_kernel<ATTN_KV_FP4_E2M1, D, false>, grid, block, 0, st, a);
  }
}

}  // namespace
}  // namespace akp

extern "C" attn_status_t attn_bounds_row_bytes(int32_t head_dim, int32_t *bytes) {
  if (!bytes) return ATTN_ERR_INVALID_ARG;
  *bytes = 0;
  if (head_dim != akp::kDqk && head_dim != akp::kDqkSym) return ATTN_ERR_UNSUPPORTED;
  *bytes = akp::bounds_row_bytes(head_dim);
  return ATTN_OK;
}

extern "C" attn_status_t attn_update_bounds(attn_plan_t plan, int32_t block_size, const void *k_cache, void *bounds,
                                            const int32_t *page_table, const int32_t *seq_lens,
                                            const int32_t *kv_indptr, int64_t rows, void *stream) {
  const attn_status_t ok = akp::check(plan, block_size, rows);
  if (ok != ATTN_OK || rows == 0) return ok;
  if (!k_cache || !bounds || !page_table || !seq_lens || !kv_indptr || !akp::aligned16(k_cache) ||
      !akp::aligned16(bounds))
    return ATTN_ERR_INVALID_ARG;
  const attn_problem_t &pr = plan->host.prob;
  akp::BoundsArgs a = akp::make_args(plan, block_size, page_table, seq_lens, kv_indptr, rows);
  a.k_cache = k_cache;
  a.bounds = static_cast<uint8_t *>(bounds);
  // blocks that the rows can complete, at most
  const int64_t most = (rows / block_size + pr.batch) * pr.num_kv_heads;
  akp::DeviceGuard dev(plan->device);
  if (!dev.ok) return ATTN_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = pr.head_dim_qk == akp::kDqk ? akp::launch_update<akp::kDqk>(a, pr.kv_dtype, most, plan->host.num_sms, st)
                                                    : akp::launch_update<akp::kDqkSym>(a, pr.kv_dtype, most, plan->host.num_sms, st);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

extern "C" attn_status_t attn_read_bounds(attn_plan_t plan, int32_t block_size, const void *bounds,
                                          const int32_t *page_table, const int32_t *seq_lens,
                                          const int32_t *block_indptr, int64_t rows, void *out, void *stream) {
  const attn_status_t ok = akp::check(plan, block_size, rows);
  if (ok != ATTN_OK || rows == 0) return ok;
  if (!bounds || !page_table || !seq_lens || !block_indptr || !out || !akp::aligned16(bounds) || !akp::aligned16(out))
    return ATTN_ERR_INVALID_ARG;
  const attn_problem_t &pr = plan->host.prob;
  akp::BoundsArgs a = akp::make_args(plan, block_size, page_table, seq_lens, block_indptr, rows);
  a.bounds = const_cast<uint8_t *>(static_cast<const uint8_t *>(bounds));
  a.out = static_cast<uint16_t *>(out);
  akp::DeviceGuard dev(plan->device);
  if (!dev.ok) return ATTN_ERR_CUDA;
  const int64_t warps = rows * pr.num_kv_heads, per = akp::kThreads / 32;
  if ((warps + per - 1) / per > INT32_MAX) return ATTN_ERR_INVALID_ARG;
  const dim3 grid((unsigned)((warps + per - 1) / per));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      pr.head_dim_qk == akp::kDqk
          ? akp::launch_dependent(akp::read_kernel<akp::kDqk>, grid, dim3(akp::kThreads), 0, st, a)
          : akp::launch_dependent(akp::read_kernel<akp::kDqkSym>, grid, dim3(akp::kThreads), 0, st, a);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
