// The append of new tokens with the position rotation on the way
// (attn_append_kv_rope), the append into 4-bit caches (attn_append_kv on such
// a plan runs the same kernel without the rotation), and the reading of cached
// rows back as bfloat16 (attn_read_kv).
//
// Rotation of a row x at position p, with c_i = cos_sin[p][i] and
// s_i = cos_sin[p][rot/2 + i], over the rot dims from rot_offset on:
//   o1 = x1 c_i - x2 s_i,  o2 = x2 c_i + x1 s_i,
// (x1, x2) the pair i: dims (i, rot/2 + i), or (2i, 2i + 1) when interleaved.
// Everything is fp32, each product and sum rounded on its own (no fused
// multiply-add), so that the value written is a function of the inputs that
// any IEEE fp32 implementation reproduces bit for bit; it is rounded once,
// to what the cache (or q_out) holds.  Dims that are not rotated keep their bits
// in a bf16 cache and in q_out.
//
// 4-bit rows (e2m1.cuh): y = x / tensor scale; per 16 values the block scale
// is E4M3(max|y| / 6), nearest even, saturating at 448; the codes are
// E2M1(y / block scale), nearest even, saturating at 6 (all zeros under a zero
// scale; a block that holds a NaN gets the NaN scale).  Quotients are IEEE fp32.
//
// A unit of work is 16 values: a scale block of a K or V row, or two 8-value
// chunks of a query row (the two halves of eight rotated pairs; 16 interleaved
// values; two chunks that are only copied).  Warps are the workers: each takes a
// range of consecutive tokens and every S-th 32-unit step of them, S chosen so that
// all SMs' warps have work (decode: a step or two each; long chunks: whole
// tokens), so that the chain of dependent lookups (request, length, page) is
// walked once per range and not once per step, and the query loop keeps four
// steps' loads in flight.  Bound by HBM for large chunks (the queries are most of
// the bytes), by the launch and the lookups for decode-sized ones.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "attn_paged.h"
#include "e2m1.cuh"
#include "kernels.hpp"
#include "plan.hpp"

namespace akp {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kVGroups = kDv / kE2m1Block;
enum { kNoRope = 0, kHalves = 1, kPairs = 2 };

struct RopeAppendArgs {
  const uint16_t *q, *k_new, *v_new;
  uint16_t *q_out;
  void *k_cache, *v_cache;
  const int32_t *page_table, *seq_lens, *qo_indptr, *positions;
  const float *cos_sin;
  int32_t *err;
  int32_t tokens, chunks, slices;         // token ranges, and warps sharing each (see the top)
  int32_t batch, hq, hkv, page_size, pt_stride, num_pages;
  int32_t max_pos, rot, rot_off;
  int32_t q_units, q_turned;              // units per query row: all, and the rotated ones (first)
  float k_scale, v_scale;
};

// The request that holds flat row `t` of a prefix-sum array: the number of
// entries indptr[1 .. batch] that are <= t.  All 32 lanes of a warp call it with
// one t: whole blocks of 256 entries by bisection, then one round of loads.
__device__ __forceinline__ int request_of(const int32_t *indptr, int batch, int64_t t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = batch;               // the answer is in [lo, hi]
  while (hi - lo > 256) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(indptr + mid + 1) <= t) lo = mid + 1; else hi = mid;
  }
  int n = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = lo + i * 32 + lane;
    const bool le = e < hi && __ldg(indptr + e + 1) <= t;
    n += __popc(__ballot_sync(0xffffffffu, le));
  }
  return lo + n;
}

__device__ __forceinline__ void unpack8(const uint4 r, float (&v)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void load8f(const float *p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

__device__ __forceinline__ float rot_sub(float a, float c, float b, float s) {
  return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
}
__device__ __forceinline__ float rot_add(float a, float c, float b, float s) {
  return __fadd_rn(__fmul_rn(a, c), __fmul_rn(b, s));
}

// Interleaved pairs of one 8-value chunk, in place; cs points at the chunk's
// first cosine, the sines are `half` further.
__device__ __forceinline__ void rotate_pairs(float (&v)[8], const float *cs, int half) {
  const float4 c4 = __ldg(reinterpret_cast<const float4 *>(cs));
  const float4 s4 = __ldg(reinterpret_cast<const float4 *>(cs + half));
  const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x1 = v[2 * i], x2 = v[2 * i + 1];
    v[2 * i] = rot_sub(x1, c[i], x2, s[i]);
    v[2 * i + 1] = rot_add(x2, c[i], x1, s[i]);
  }
}

// One 8-value chunk of a K row from dim d on, rotated if it lies in the rotated
// dims (returns whether it does; `raw` is the chunk as it stands).
template <int ROPE>
__device__ __forceinline__ bool rotated_chunk(const RopeAppendArgs &a, const uint16_t *row, int d,
                                              const float *cs, uint4 raw, float (&v)[8]) {
  unpack8(raw, v);
  if (ROPE == kNoRope || d < a.rot_off || d >= a.rot_off + a.rot) return false;
  const int half = a.rot >> 1, r = d - a.rot_off;
  if (ROPE == kPairs) {
    rotate_pairs(v, cs + (r >> 1), half);
  } else {
    const bool first = r < half;
    const int i = first ? r : r - half;
    float w[8], c[8], s[8];
    unpack8(__ldg(reinterpret_cast<const uint4 *>(row + (first ? d + half : d - half))), w);
    load8f(cs + i, c);
    load8f(cs + half + i, s);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = first ? rot_sub(v[j], c[j], w[j], s[j]) : rot_add(v[j], c[j], w[j], s[j]);
  }
  return true;
}

// One E4M3 code of a non-negative value (nearest even, saturating; NaN: 0x7F).
__device__ __forceinline__ uint32_t e4m3_of(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xFFu;
}

// 16 values -> 16 E2M1 codes (8 bytes) and their E4M3 scale.
__device__ __forceinline__ uint2 quantise16(const float (&v)[16], float tensor_scale, uint32_t &scale) {
  float y[16], amax = 0.f;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    y[i] = __fdiv_rn(v[i], tensor_scale);
    amax = fmaxf(amax, fabsf(y[i]));
    nan |= y[i] != y[i];
  }
  scale = nan ? 0x7Fu : e4m3_of(__fdiv_rn(amax, 6.f));
  uint32_t h2, out[2] = {0u, 0u};
  asm("{\n .reg .b16 s;\n cvt.u16.u32 s, %1;\n cvt.rn.f16x2.e4m3x2 %0, s;\n}\n" : "=r"(h2) : "r"(scale));
  float s;
  asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %1;\n cvt.f32.f16 %0, l;\n}\n" : "=f"(s) : "r"(h2));
  if (scale != 0u && !nan) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t b;
      asm("{\n .reg .b8 t;\n cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n cvt.u32.u8 %0, t;\n}\n"
          : "=r"(b)
          : "f"(__fdiv_rn(y[2 * i + 1], s)), "f"(__fdiv_rn(y[2 * i], s)));
      out[i >> 2] |= b << (8 * (i & 3));
    }
  } else {
    // no value below half the smallest step keeps more than its sign
#pragma unroll
    for (int i = 0; i < 16; ++i) out[i >> 3] |= (__float_as_uint(y[i]) >> 31) << (4 * (i & 7) + 3);
  }
  return make_uint2(out[0], out[1]);
}

// The request of consecutive rows of a prefix-sum array, in registers: found by a
// search once, then only when a row lies past its end.
struct Request {
  int b = -1, first = 0, end = 0;      // rows [first, end)
  __device__ __forceinline__ bool seek(const int32_t *indptr, int batch, int64_t row) {
    if (b >= 0 && row < end) return false;
    b = request_of(indptr, batch, row);
    if (b < batch) {
      first = __ldg(indptr + b);
      end = __ldg(indptr + b + 1);
    }
    return true;
  }
};

// 16 values of a K or V row into the cache.
template <int KV, int ROPE, int D>
__device__ __forceinline__ void append_unit(const RopeAppendArgs &a, const uint16_t *src, uint8_t *dst, int c,
                                            const float *cs, float scale) {
  const uint4 raw[2] = {__ldg(reinterpret_cast<const uint4 *>(src) + 2 * c),
                        __ldg(reinterpret_cast<const uint4 *>(src) + 2 * c + 1)};
  float v[2][8];
  bool turned[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) turned[h] = rotated_chunk<ROPE>(a, src, 16 * c + 8 * h, cs, raw[h], v[h]);
  if (KV == ATTN_KV_BF16) {
#pragma unroll
    for (int h = 0; h < 2; ++h) reinterpret_cast<uint4 *>(dst)[2 * c + h] = turned[h] ? pack8(v[h]) : raw[h];
  } else if (KV == ATTN_KV_FP8_E4M3) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float *x = &v[e >> 1][4 * (e & 1)];
      uint16_t lo, hi;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n"
          : "=h"(lo) : "f"(__fdiv_rn(x[1], scale)), "f"(__fdiv_rn(x[0], scale)));
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n"
          : "=h"(hi) : "f"(__fdiv_rn(x[3], scale)), "f"(__fdiv_rn(x[2], scale)));
      w[e] = (uint32_t)lo | ((uint32_t)hi << 16);
    }
    reinterpret_cast<uint4 *>(dst)[c] = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    constexpr int kGroups = D / kE2m1Block, kPad = e2m1_row_bytes(D) - D / 2 - kGroups;
    static_assert(kPad == 4 || kPad == 8, "4-bit row padding");
    float x[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = v[j >> 3][j & 7];
    uint32_t s;
    reinterpret_cast<uint2 *>(dst)[c] = quantise16(x, scale, s);
    dst[D / 2 + c] = (uint8_t)s;
    if (c == kGroups - 1) {                // the row's padding
      uint32_t *pad = reinterpret_cast<uint32_t *>(dst + D / 2 + kGroups);
      pad[0] = 0u;
      if (kPad > 4) pad[1] = 0u;
    }
  }
}

template <int KV, int ROPE, int DQK>
__global__ void __launch_bounds__(kAppendThreads, 4) rope_append_kernel(const RopeAppendArgs a) {
  // A programmatic dependent of the stream's previous kernel: nothing is read
  // or written before that kernel has completed.  The kernels that follow in a
  // serving step (device planner, attention) may be scheduled now; they wait
  // for this grid.
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  constexpr int kKGroups = DQK / kE2m1Block;
  const int lane = threadIdx.x & 31;
  const int worker = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const int chunk = worker / a.slices, slice = worker % a.slices;
  if (chunk >= a.chunks) return;
  const int k_units = a.hkv * kKGroups, kv_units = k_units + a.hkv * kVGroups;
  const int q_units = a.hq * a.q_units, stride = 32 * a.slices;
  const int tok_end = (int)((int64_t)(chunk + 1) * a.tokens / a.chunks);
  Request rq;
  int64_t shift = 0;                         // position of token tok: tok + shift
  for (int tok = (int)((int64_t)chunk * a.tokens / a.chunks); tok < tok_end; ++tok) {
    if (rq.seek(a.qo_indptr, a.batch, tok)) shift = (int64_t)__ldg(a.seq_lens + rq.b) - rq.end;
    const int64_t i = tok + shift;
    const float *cs = nullptr;
    if (ROPE != kNoRope) {
      const int64_t pos = a.positions ? (int64_t)__ldg(a.positions + tok) : i;
      if (pos < 0 || pos >= a.max_pos) {            // no row of the table: the token is skipped
        if (slice == 0 && lane == 0) atomicOr(a.err, 8);
        continue;
      }
      cs = a.cos_sin + pos * a.rot;
    }
    // ---- K and V
    int64_t slot = -1;
    if (slice * 32 < kv_units) {
      int bad = 0;
      if (i < 0 || i / a.page_size >= a.pt_stride) {   // a length outside the table row
        bad = 4;
      } else {
        const int32_t page = __ldg(a.page_table + (int64_t)rq.b * a.pt_stride + i / a.page_size);
        if (page < 0 || page >= a.num_pages)
          bad = 1;
        else
          slot = (int64_t)page * a.page_size + i % a.page_size;
      }
      if (bad && slice == 0 && lane == 0) atomicOr(a.err, bad);
    }
    if (slot >= 0) {
      for (int unit = slice * 32 + lane; unit < kv_units; unit += stride) {
        if (unit < k_units) {
          const int g = unit / kKGroups, c = unit % kKGroups;
          append_unit<KV, ROPE, DQK>(a, a.k_new + ((int64_t)tok * a.hkv + g) * DQK,
                                     static_cast<uint8_t *>(a.k_cache) + (slot * a.hkv + g) * kv_row_bytes(KV, DQK),
                                     c, cs, a.k_scale);
        } else {
          const int g = (unit - k_units) / kVGroups, c = (unit - k_units) % kVGroups;
          append_unit<KV, kNoRope, kDv>(a, a.v_new + ((int64_t)tok * a.hkv + g) * kDv,
                                        static_cast<uint8_t *>(a.v_cache) + (slot * a.hkv + g) * kv_row_bytes(KV, kDv),
                                        c, cs, a.v_scale);
        }
      }
    }
    // ---- the query rows: rotated units first in each row, then the copied ones
    if constexpr (ROPE != kNoRope) {
      const int half = a.rot >> 1;
      const int64_t row0 = (int64_t)tok * a.hq * DQK;
      constexpr int kAhead = 2;
#pragma unroll 1
      for (int u0 = slice * 32 + lane; u0 < q_units; u0 += kAhead * stride) {
        uint4 x[kAhead][2];
        int at[kAhead][2], un[kAhead];             // offsets in the token's rows, unit in the row
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int unit = u0 + k * stride;
          un[k] = -1;
          if (unit < q_units) {
            const int h = unit / a.q_units, u = unit % a.q_units;
            un[k] = u;
            if (u < a.q_turned) {
              at[k][0] = a.rot_off + (ROPE == kPairs ? 16 : 8) * u;
              at[k][1] = at[k][0] + (ROPE == kPairs ? 8 : half);
            } else {
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const int d = 16 * (u - a.q_turned) + 8 * y;
                at[k][y] = d < a.rot_off ? d : d + a.rot;
              }
            }
            at[k][0] += h * DQK;
            at[k][1] += h * DQK;
#pragma unroll
            for (int y = 0; y < 2; ++y) x[k][y] = *reinterpret_cast<const uint4 *>(a.q + row0 + at[k][y]);
          }
        }
        // a unit's two chunks are read before either is written (q_out may be q)
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          if (un[k] < 0) continue;
          if (un[k] < a.q_turned) {
            float x1[8], x2[8];
            unpack8(x[k][0], x1);
            unpack8(x[k][1], x2);
            const float *c8 = cs + 8 * un[k];
            if (ROPE == kPairs) {
              rotate_pairs(x1, c8, half);
              rotate_pairs(x2, c8 + 4, half);
            } else {
              float c[8], sn[8];
              load8f(c8, c);
              load8f(c8 + half, sn);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float y1 = x1[j], y2 = x2[j];
                x1[j] = rot_sub(y1, c[j], y2, sn[j]);
                x2[j] = rot_add(y2, c[j], y1, sn[j]);
              }
            }
            x[k][0] = pack8(x1);
            x[k][1] = pack8(x2);
          }
#pragma unroll
          for (int y = 0; y < 2; ++y) *reinterpret_cast<uint4 *>(a.q_out + row0 + at[k][y]) = x[k][y];
        }
      }
    }
  }
}

struct ReadArgs {
  const void *k_cache, *v_cache;
  const int32_t *page_table, *seq_lens, *kv_indptr;
  uint16_t *k_out, *v_out;
  int32_t *err;
  int32_t rows, chunks, slices;          // as for the append's tokens
  int32_t batch, hkv, page_size, pt_stride, num_pages;
  float k_scale, v_scale;
};

// 16 cached values as bfloat16.
template <int KV, int D>
__device__ __forceinline__ void read_unit(const uint8_t *src, int c, float scale, uint4 (&o)[2]) {
  if (KV == ATTN_KV_BF16) {
    o[0] = __ldg(reinterpret_cast<const uint4 *>(src) + 2 * c);
    o[1] = __ldg(reinterpret_cast<const uint4 *>(src) + 2 * c + 1);
    return;
  }
  uint32_t h[8];                           // 16 values as fp16 pairs, exact
  if (KV == ATTN_KV_FP8_E4M3) {
    uint4 lo, hi;
    e4m3x16_to_f16(__ldg(reinterpret_cast<const uint4 *>(src) + c), lo, hi);
    h[0] = lo.x; h[1] = lo.y; h[2] = lo.z; h[3] = lo.w;
    h[4] = hi.x; h[5] = hi.y; h[6] = hi.z; h[7] = hi.w;
  } else {
    const uint2 q = __ldg(reinterpret_cast<const uint2 *>(src) + c);
    uint32_t s0, s1, p[4], u[4];
    e4m3_scales_f16(__ldg(src + D / 2 + c), s0, s1);
    e2m1x8_to_f16(q.x, p);
    e2m1x8_to_f16(q.y, u);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      h[e] = mul_f16x2(p[e], s0);
      h[4 + e] = mul_f16x2(u[e], s0);
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, u;\n}\n"
          : "=f"(v[2 * j]), "=f"(v[2 * j + 1])
          : "r"(h[4 * e + j]));
      v[2 * j] = __fmul_rn(v[2 * j], scale);
      v[2 * j + 1] = __fmul_rn(v[2 * j + 1], scale);
    }
    o[e] = pack8(v);
  }
}

// Cached rows as bfloat16, 16 values a unit; the rows of request b are its last
// kv_indptr[b + 1] - kv_indptr[b] positions.  Work is split as for the append.
template <int KV, int DQK>
__global__ void __launch_bounds__(kAppendThreads, 4) read_kernel(const ReadArgs a) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  constexpr int kKGroups = DQK / kE2m1Block;
  const int lane = threadIdx.x & 31;
  const int worker = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const int chunk = worker / a.slices, slice = worker % a.slices;
  if (chunk >= a.chunks) return;
  const int k_units = a.hkv * kKGroups, kv_units = k_units + a.hkv * kVGroups;
  const int row_end = (int)((int64_t)(chunk + 1) * a.rows / a.chunks);
  Request rq;
  int64_t shift = 0;
  for (int row = (int)((int64_t)chunk * a.rows / a.chunks); row < row_end; ++row) {
    if (rq.seek(a.kv_indptr, a.batch, row) && rq.b < a.batch)
      shift = (int64_t)__ldg(a.seq_lens + rq.b) - rq.end;
    int64_t slot = -1;
    int bad = 4;                                  // more rows than kv_indptr holds, or no such position
    if (rq.b < a.batch) {
      const int64_t i = row + shift;
      if (row >= rq.first && i >= 0 && i / a.page_size < a.pt_stride) {
        const int32_t page = __ldg(a.page_table + (int64_t)rq.b * a.pt_stride + i / a.page_size);
        bad = page >= 0 && page < a.num_pages ? 0 : 1;
        if (!bad) slot = (int64_t)page * a.page_size + i % a.page_size;
      }
    }
    if (bad && slice == 0 && lane == 0) atomicOr(a.err, bad);
#pragma unroll 2
    for (int unit = slice * 32 + lane; unit < kv_units; unit += 32 * a.slices) {
      uint4 o[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
      uint4 *dst;
      if (unit < k_units) {
        const int g = unit / kKGroups, c = unit % kKGroups;
        dst = reinterpret_cast<uint4 *>(a.k_out + ((int64_t)row * a.hkv + g) * DQK) + 2 * c;
        if (slot >= 0)
          read_unit<KV, DQK>(static_cast<const uint8_t *>(a.k_cache) + (slot * a.hkv + g) * kv_row_bytes(KV, DQK),
                             c, a.k_scale, o);
      } else {
        const int g = (unit - k_units) / kVGroups, c = (unit - k_units) % kVGroups;
        dst = reinterpret_cast<uint4 *>(a.v_out + ((int64_t)row * a.hkv + g) * kDv) + 2 * c;
        if (slot >= 0)
          read_unit<KV, kDv>(static_cast<const uint8_t *>(a.v_cache) + (slot * a.hkv + g) * kv_row_bytes(KV, kDv),
                             c, a.v_scale, o);
      }
      dst[0] = o[0];
      dst[1] = o[1];
    }
  }
}

// Restores the caller's current device on scope exit.
struct OnDevice {
  int prev = -1;
  bool ok = false;
  explicit OnDevice(int dev) {
    ok = cudaGetDevice(&prev) == cudaSuccess && (prev == dev || cudaSetDevice(dev) == cudaSuccess);
    if (prev == dev) prev = -1;
  }
  ~OnDevice() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Splits `rows` of `steps` 32-unit steps each among the warps that all SMs hold:
// ranges of rows, and the warps that share a range's steps.
struct Split {
  int32_t chunks, slices;
  unsigned ctas;
  Split(int64_t rows, int64_t steps) {
    constexpr int64_t kWarps = 152 * 4 * (kAppendThreads / 32);
    slices = (int32_t)std::max<int64_t>(1, std::min(steps, kWarps / std::max<int64_t>(rows, 1)));
    chunks = (int32_t)std::min<int64_t>(rows, std::max<int64_t>(1, kWarps / slices));
    ctas = (unsigned)(((int64_t)chunks * slices + kAppendThreads / 32 - 1) / (kAppendThreads / 32));
  }
};

template <int KV, int ROPE>
cudaError_t launch_append(const RopeAppendArgs &a, int dqk, dim3 grid, cudaStream_t st) {
  return dqk == kDqk ? launch_dependent(rope_append_kernel<KV, ROPE, kDqk>, grid, dim3(kAppendThreads), 0, st, a)
                     : launch_dependent(rope_append_kernel<KV, ROPE, kDqkSym>, grid, dim3(kAppendThreads), 0, st, a);
}

template <int ROPE>
cudaError_t launch_append_kv(const RopeAppendArgs &a, int kv, int dqk, dim3 grid, cudaStream_t st) {
  switch (kv) {
    case ATTN_KV_BF16: return launch_append<ATTN_KV_BF16, ROPE>(a, dqk, grid, st);
    case ATTN_KV_FP8_E4M3: return launch_append<ATTN_KV_FP8_E4M3, ROPE>(a, dqk, grid, st);
    default: return launch_append<ATTN_KV_FP4_E2M1, ROPE>(a, dqk, grid, st);
  }
}

bool scales_ok(int kv, float k, float v) {
  return kv == ATTN_KV_BF16 || (k > 0.f && v > 0.f && k < INFINITY && v < INFINITY);
}

}  // namespace

attn_status_t append_rows(attn_plan_t plan, const attn_rope_t *rope, const void *q, const void *k_new,
                          const void *v_new, void *q_out, void *k_cache, void *v_cache,
                          const int32_t *page_table, const int32_t *seq_lens, const int32_t *qo_indptr,
                          float k_scale, float v_scale, void *stream) {
  if (!plan || plan->device < 0) return ATTN_ERR_INVALID_ARG;
  const HostPlan &hp = plan->host;
  const attn_problem_t &pr = hp.prob;
  if (rope) {
    if (!rope->cos_sin || rope->max_pos <= 0 || rope->rot_dim <= 0 || rope->rot_offset < 0 ||
        (int64_t)rope->rot_offset + rope->rot_dim > pr.head_dim_qk)
      return ATTN_ERR_INVALID_ARG;
    // whole 8-value chunks on both sides of every border
    if (rope->rot_dim % 16 || rope->rot_offset % 8) return ATTN_ERR_UNSUPPORTED;
    if ((q == nullptr) != (q_out == nullptr) || !aligned16(rope->cos_sin) || !aligned16(q) || !aligned16(q_out))
      return ATTN_ERR_INVALID_ARG;
  }
  if (!scales_ok(pr.kv_dtype, k_scale, v_scale)) return ATTN_ERR_INVALID_ARG;
  const int64_t total_q = hp.qo_indptr.back();
  if (total_q == 0) return ATTN_OK;
  if (!k_new || !v_new || !k_cache || !v_cache || !page_table || !seq_lens || !qo_indptr)
    return ATTN_ERR_INVALID_ARG;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache))
    return ATTN_ERR_INVALID_ARG;
  RopeAppendArgs a{};
  a.k_new = static_cast<const uint16_t *>(k_new);
  a.v_new = static_cast<const uint16_t *>(v_new);
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.page_table = page_table;
  a.seq_lens = seq_lens;
  a.qo_indptr = qo_indptr;
  a.err = plan->dev.err;
  a.tokens = (int32_t)total_q;
  a.batch = pr.batch;
  a.hq = pr.num_q_heads;
  a.hkv = pr.num_kv_heads;
  a.page_size = pr.page_size;
  a.pt_stride = pr.page_table_stride;
  a.num_pages = pr.num_pages;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  const int64_t kv_units = (int64_t)pr.num_kv_heads * (pr.head_dim_qk / kE2m1Block + kVGroups);
  int64_t q_units = 0;
  if (rope) {
    a.cos_sin = rope->cos_sin;
    a.positions = rope->positions;
    a.max_pos = rope->max_pos;
    a.rot = rope->rot_dim;
    a.rot_off = rope->rot_offset;
    if (q) {
      a.q = static_cast<const uint16_t *>(q);
      a.q_out = static_cast<uint16_t *>(q_out);
      a.q_turned = rope->rot_dim / 16;
      // in place, the dims that are not rotated stay where they are
      a.q_units = q == q_out ? a.q_turned : pr.head_dim_qk / 16;
      q_units = (int64_t)pr.num_q_heads * a.q_units;
    }
  }
  const Split sp(total_q, (std::max(kv_units, q_units) + 31) / 32);
  a.chunks = sp.chunks;
  a.slices = sp.slices;
  OnDevice dev(plan->device);
  if (!dev.ok) return ATTN_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = !rope               ? launch_append_kv<kNoRope>(a, pr.kv_dtype, pr.head_dim_qk, dim3(sp.ctas), st)
                        : rope->interleaved ? launch_append_kv<kPairs>(a, pr.kv_dtype, pr.head_dim_qk, dim3(sp.ctas), st)
                                            : launch_append_kv<kHalves>(a, pr.kv_dtype, pr.head_dim_qk, dim3(sp.ctas), st);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace akp

extern "C" attn_status_t attn_append_kv_rope(attn_plan_t plan, const attn_rope_t *rope, const void *q,
                                             const void *k_new, const void *v_new, void *q_out,
                                             void *k_cache, void *v_cache, const int32_t *page_table,
                                             const int32_t *seq_lens, const int32_t *qo_indptr,
                                             float k_scale, float v_scale, void *stream) {
  if (!rope) return ATTN_ERR_INVALID_ARG;
  return akp::append_rows(plan, rope, q, k_new, v_new, q_out, k_cache, v_cache, page_table, seq_lens,
                          qo_indptr, k_scale, v_scale, stream);
}

extern "C" attn_status_t attn_read_kv(attn_plan_t plan, const void *k_cache, const void *v_cache,
                                      const int32_t *page_table, const int32_t *seq_lens,
                                      const int32_t *kv_indptr, int64_t rows, void *k_out, void *v_out,
                                      float k_scale, float v_scale, void *stream) {
  if (!plan || plan->device < 0 || rows < 0 || rows > INT32_MAX) return ATTN_ERR_INVALID_ARG;
  const attn_problem_t &pr = plan->host.prob;
  if (!akp::scales_ok(pr.kv_dtype, k_scale, v_scale)) return ATTN_ERR_INVALID_ARG;
  if (rows == 0) return ATTN_OK;
  if (!k_cache || !v_cache || !page_table || !seq_lens || !kv_indptr || !k_out || !v_out)
    return ATTN_ERR_INVALID_ARG;
  if (!akp::aligned16(k_cache) || !akp::aligned16(v_cache) || !akp::aligned16(k_out) || !akp::aligned16(v_out))
    return ATTN_ERR_INVALID_ARG;
  akp::ReadArgs a{};
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.page_table = page_table;
  a.seq_lens = seq_lens;
  a.kv_indptr = kv_indptr;
  a.k_out = static_cast<uint16_t *>(k_out);
  a.v_out = static_cast<uint16_t *>(v_out);
  a.err = plan->dev.err;
  a.rows = (int32_t)rows;
  a.batch = pr.batch;
  a.hkv = pr.num_kv_heads;
  a.page_size = pr.page_size;
  a.pt_stride = pr.page_table_stride;
  a.num_pages = pr.num_pages;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  const akp::Split sp(rows, ((int64_t)pr.num_kv_heads * (pr.head_dim_qk / akp::kE2m1Block + akp::kVGroups) + 31) / 32);
  a.chunks = sp.chunks;
  a.slices = sp.slices;
  akp::OnDevice dev(plan->device);
  if (!dev.ok) return ATTN_ERR_CUDA;
  const dim3 grid(sp.ctas), block(akp::kAppendThreads);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool wide = pr.head_dim_qk == akp::kDqk;
  cudaError_t e;
  if (pr.kv_dtype == ATTN_KV_BF16)
    e = wide ? akp::launch_dependent(akp::read_kernel<ATTN_KV_BF16, akp::kDqk>, grid, block, 0, st, a)
             : akp::launch_dependent(akp::read_kernel<ATTN_KV_BF16, akp::kDqkSym>, grid, block, 0, st, a);
  else if (pr.kv_dtype == ATTN_KV_FP8_E4M3)
    e = wide ? akp::launch_dependent(akp::read_kernel<ATTN_KV_FP8_E4M3, akp::kDqk>, grid, block, 0, st, a)
             : akp::launch_dependent(akp::read_kernel<ATTN_KV_FP8_E4M3, akp::kDqkSym>, grid, block, 0, st, a);
  else
    e = wide ? akp::launch_dependent(akp::read_kernel<ATTN_KV_FP4_E2M1, akp::kDqk>, grid, block, 0, st, a)
             : akp::launch_dependent(akp::read_kernel<ATTN_KV_FP4_E2M1, akp::kDqkSym>, grid, block, 0, st, a);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
