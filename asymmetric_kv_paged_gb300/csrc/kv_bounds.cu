// Bounds of the cache's blocks: attn_update_bounds and attn_read_bounds.
//
// For a block of block_size keys of one KV head, per dim hi = max k, lo = min k over the
// rows as the cache holds them; e is the least exponent with max |k| <= 127 * 2^e, and
// the record holds ceil(hi / 2^e) and floor(lo / 2^e) in 8 bits: every step is exact, so
// a record is a function of the rows alone.  Minima and maxima do not depend on the
// order either, and a block is always taken from all its rows when its last one arrives:
// nothing is accumulated from step to step, and rejected drafts leave nothing behind.
//
// A CTA looks at a range of the new rows for one head, finds those that end a block, and
// takes these blocks one after the other: a thread owns 8 dims of every RG-th row of the
// block (16, 8 or 4 bytes a load), in 16-bit pairs (exact for every cache type: bf16, or
// fp16 of E4M3 and E2M1 times its scale); the row groups meet in shared memory.  The
// kernel reads each key once: what bounds it is memory for many blocks, and for a decode
// step the launch and four dependent loads.
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
  int32_t rows, rows_per_cta;     // flat rows (update: positions, reading: blocks)
  int32_t batch, hkv, page_size, pt_stride, num_pages, block, per_page;
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

// Chunk ch (8 values) of a cached row as four 16-bit pairs.
template <int KV, int D>
__device__ __forceinline__ void load_chunk(const uint8_t *row, int ch, uint32_t (&w)[4]) {
  if (KV == ATTN_KV_BF16) {
    const uint4 v = __ldg(reinterpret_cast<const uint4 *>(row) + ch);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if (KV == ATTN_KV_FP8_E4M3) {
    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(row) + ch);
    uint4 lo, hi;
    e4m3x16_to_f16(make_uint4(v.x, v.y, 0u, 0u), lo, hi);
    w[0] = lo.x, w[1] = lo.y, w[2] = lo.z, w[3] = lo.w;
  } else {
    const uint32_t codes = __ldg(reinterpret_cast<const uint32_t *>(row) + ch);
    uint32_t s0, s1;
    e4m3_scales_f16(__ldg(row + D / 2 + ch / 2), s0, s1);
    e2m1x8_to_f16(codes, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = mul_f16x2(w[i], s0);
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

template <int KV, int D>
__global__ void __launch_bounds__(kThreads) update_kernel(const BoundsArgs a) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  constexpr int NC = D / 8, RG = kThreads / NC, W = D / 2;      // chunks of a row, row groups, pairs
  __shared__ int found;
  __shared__ int64_t list[128];                                  // first slots of the blocks to take
  __shared__ uint32_t part[RG][2][W];                            // [row group][hi, lo][pair]
  __shared__ float top[kThreads / 32];
  __shared__ int odd;                                            // an infinity or a NaN
  const int tid = threadIdx.x, g = blockIdx.y;
  if (tid == 0) found = 0;
  __syncthreads();
  const int64_t r0 = (int64_t)blockIdx.x * a.rows_per_cta;
  if (tid < a.rows_per_cta && r0 + tid < a.rows) {
    const int64_t row = r0 + tid;
    const int b = request_of_row(a.indptr, a.batch, row);
    int bad = 0;
    if (b >= a.batch || row < __ldg(a.indptr)) {                 // a row that kv_indptr does not hold
      bad = 4;
    } else {
      const int64_t pos = row + (int64_t)__ldg(a.seq_lens + b) - __ldg(a.indptr + b + 1);
      if (pos < 0) {
        bad = 4;
      } else if ((pos + 1) % a.block == 0) {
        const int64_t slot = slot_of(a, b, pos + 1 - a.block, bad);
        if (slot >= 0) list[atomicAdd(&found, 1)] = slot;
      }
    }
    if (bad) atomicOr(a.err, bad);
  }
  __syncthreads();
  const int n = found;
  for (int k = 0; k < n; ++k) {
    const int64_t slot = list[k];
    const int ch = tid % NC, rg = tid / NC;
    uint32_t hi[4], lo[4];
    if (rg < RG) {
      const uint8_t *row = static_cast<const uint8_t *>(a.k_cache) + (slot * a.hkv + g) * kv_row_bytes(KV, D);
      const int64_t step = (int64_t)a.hkv * kv_row_bytes(KV, D);
      load_chunk<KV, D>(row + rg * step, ch, hi);
#pragma unroll
      for (int i = 0; i < 4; ++i) lo[i] = hi[i];
#pragma unroll 4
      for (int r = rg + RG; r < a.block; r += RG) {
        uint32_t w[4];
        load_chunk<KV, D>(row + r * step, ch, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          hi[i] = max_pair<KV>(hi[i], w[i]);
          lo[i] = min_pair<KV>(lo[i], w[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        part[rg][0][4 * ch + i] = hi[i];
        part[rg][1][4 * ch + i] = lo[i];
      }
    }
    if (tid == 0) odd = 0;
    __syncthreads();
    // thread tid: pair tid % W of hi (tid < W) or lo
    const bool mine = tid < 2 * W;
    float2 v = make_float2(0.f, 0.f);
    if (mine) {
      const int which = tid / W, w = tid % W;
      uint32_t x = part[0][which][w];
#pragma unroll
      for (int r = 1; r < RG; ++r)
        x = which ? min_pair<KV>(x, part[r][which][w]) : max_pair<KV>(x, part[r][which][w]);
      v = pair_values<KV>(x);
    }
    float t = fmaxf(fabsf(v.x), fabsf(v.y));
    if (!(fabsf(v.x) < INFINITY) || !(fabsf(v.y) < INFINITY)) odd = 1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
    if ((tid & 31) == 0) top[tid >> 5] = t;
    __syncthreads();
    float amax = top[0];
#pragma unroll
    for (int i = 1; i < kThreads / 32; ++i) amax = fmaxf(amax, top[i]);
    const int e = odd ? kOddBlock : code_exponent(amax);
    const int64_t entry = slot / a.block;        // pages hold whole blocks, in order
    uint8_t *rec = a.bounds + (entry * a.hkv + g) * bounds_row_bytes(D);
    if (mine) {
      const int which = tid / W, w = tid % W;
      const float unit = pow2(-e);
      uint32_t codes = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float x = i ? v.y : v.x;
        // (a product that underflows keeps its side of zero)
        int c = which ? min((int)floorf(x * unit), x < 0.f ? -1 : 127) : max((int)ceilf(x * unit), x > 0.f ? 1 : -127);
        if (e == kOddBlock) c = 0;
        codes |= (uint32_t)(c & 0xFF) << (8 * i);
      }
      reinterpret_cast<uint16_t *>(rec + which * D)[w] = (uint16_t)codes;
    }
    if (tid == 0) *reinterpret_cast<uint4 *>(rec + 2 * D) = make_uint4((uint32_t)(e & 0xFF), 0u, 0u, 0u);
    __syncthreads();
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
cudaError_t launch_update(const BoundsArgs &a, int kv, dim3 grid, cudaStream_t st) {
  switch (kv) {
    case ATTN_KV_BF16: return launch_dependent(update_kernel<ATTN_KV_BF16, D>, grid, dim3(kThreads), 0, st, a);
    case ATTN_KV_FP8_E4M3: return launch_dependent(update_kernel<ATTN_KV_FP8_E4M3, D>, grid, dim3(kThreads), 0, st, a);
    default: return launch_dependent(update_kernel<ATTN_KV_FP4_E2M1, D>, grid, dim3(kThreads), 0, st, a);
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
  // Rows a CTA looks at: at most a block's, so that the rows of one request end one
  // block at most, and few enough to give every SM four CTAs.
  const int64_t want = (int64_t)plan->host.num_sms * 4;
  a.rows_per_cta = (int32_t)std::max<int64_t>(1, std::min<int64_t>(block_size, rows * pr.num_kv_heads / want));
  const dim3 grid((unsigned)((rows + a.rows_per_cta - 1) / a.rows_per_cta), (unsigned)pr.num_kv_heads);
  akp::DeviceGuard dev(plan->device);
  if (!dev.ok) return ATTN_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = pr.head_dim_qk == akp::kDqk ? akp::launch_update<akp::kDqk>(a, pr.kv_dtype, grid, st)
                                                    : akp::launch_update<akp::kDqkSym>(a, pr.kv_dtype, grid, st);
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
