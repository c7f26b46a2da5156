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
// By axes (attn_append_kv_mrope) the row of pair i's cosine and sine is that of the axis
// which turns it, positions[axis(i)][token]: the axes are two bits a pair in the kernel's
// arguments, a lane picks one of its up to four positions an angle and loads cosine and
// sine one by one (one axis: four at a time).
//
// 4-bit rows (e2m1.cuh): y = x / tensor scale; per 16 values the block scale
// is E4M3(max|y| / 6), nearest even, saturating at 448; the codes are
// E2M1(y / block scale), nearest even, saturating at 6 (all zeros under a zero
// scale; a block that holds a NaN gets the NaN scale).  Quotients are IEEE fp32.
//
// A warp takes a whole row at a time (two of 128 values), a lane one 16-byte
// chunk of 8 values of it: loads and stores of a row are contiguous, the partner
// chunk of a rotated half comes from another lane by shuffle, a lane pair shares a
// scale block, and the angles of a lane's dims are the same for every head of the
// token, so that they are loaded once per token and stay in registers.  Each warp
// owns a range of consecutive tokens and every S-th row step of them, S chosen so
// that all SMs' warps have work (decode: a row each; long chunks: whole tokens),
// which walks the chain of dependent lookups (request, length, page) once per
// range and not once per row; the query loop keeps the loads of the next four rows in
// flight (two: 46.6 us on the first case below, six: 44.4 for the spilled registers).
//
// Measured (in a graph): 4096 tokens of 64 query and 4 KV heads rotated and
// quantised to E4M3, 217 MB, 40.6 us (5.3 TB/s, 0.80 of the copy rate; 7.4 us of it
// for K and V alone); 4098 tokens of 32 and 8 heads to 4 bits, 128 MB, 32.3 us, K
// and V 16 (issue: a value's two quotients, block maximum and codes); 4095 tokens of
// 4 heads to 4 bits, not rotated, 13.6 MB, 9.8 us.  A decode step's 32 tokens take
// 3.4 us, 4.5 with rotation and queries: the launch and four dependent loads.  Four
// CTAs of 64 registers an SM: three of 80 took 55 us on the first, five 12.3 us on
// the third; twice as many, shorter warps' shares 10.9 us on the third.
// Three axes in turn, 4096 tokens of 64 and 4 heads to E4M3: 50 us against 45 with one
// position (append and reading back); a decode step's 33 tokens 8.1 with the reading, in a graph.
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
#include "requests.cuh"
#include "sparse.cuh"

namespace akp {
namespace {

constexpr int kAppendThreads = 256;
// what is rotated: nothing; pairs of dims half the rotated range apart, or of neighbours;
// the same with every pair on an axis of its own
enum { kNoRope = 0, kHalves = 1, kPairs = 2, kHalvesAxes = 3, kPairsAxes = 4 };
__host__ __device__ constexpr bool halves(int rope) { return rope == kHalves || rope == kHalvesAxes; }
__host__ __device__ constexpr bool by_axes(int rope) { return rope >= kHalvesAxes; }
constexpr int kMaxAxes = 4;

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
  float k_scale, v_scale;
  // positions of several axes: positions is [axes][tokens]; two bits a pair, its axis
  int32_t axes;
  const int32_t *position_delta;          // [batch], added to the tokens' own positions
  uint32_t axis_bits[kDqk / 32];
};

// Paired fp32 arithmetic: a * b and a * b + c, two of each in one instruction.  (A
// paired addition behind a paired product is contracted into one rounding by the
// assembler in spite of its .rn, measured on a quarter of random inputs: the
// rotation's sums are scalar.)
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mul.rn.f32x2 d, a, b;\n"
      " mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
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

// What a lane's chunk does under the rotation, for the token at hand.
template <int ROPE, int NC>
struct Turn {
  static constexpr int N = halves(ROPE) ? 2 : 1;      // groups of four angles
  bool in = false;                // the chunk's dims are rotated
  int partner = 0;                // halves: the lane with the other half's chunk
  float c[4 * N], s[4 * N];
  int at = 0;                     // first cosine of the chunk
  float sign = 1.f;
  uint32_t axis = 0;              // by axes: two bits an angle

  __device__ __forceinline__ void place(const RopeAppendArgs &a, int lane) {
    if (ROPE == kNoRope) return;
    const int half = a.rot >> 1, r = 8 * (lane % NC) - a.rot_off;
    in = r >= 0 && r < a.rot;
    partner = lane;
    if (halves(ROPE)) {
      const bool first = r < half;
      at = first ? r : r - half;
      sign = first ? -1.f : 1.f;            // x1 c - x2 s, x2 c + x1 s
      if (in) partner = first ? lane + half / 8 : lane - half / 8;
    } else {
      at = r >> 1;
    }
    // (a chunk's angles start at a multiple of 8, or of 4 for neighbours: one word)
    if (by_axes(ROPE) && in) axis = a.axis_bits[at >> 4] >> (2 * (at & 15));
  }
  __device__ __forceinline__ void angles(const RopeAppendArgs &a, int64_t pos) {
    if (ROPE == kNoRope) return;
    const float *row = a.cos_sin + pos * a.rot + at;
#pragma unroll
    for (int p = 0; p < N; ++p) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
      if (in) {
        x = __ldg(reinterpret_cast<const float4 *>(row) + p);
        y = __ldg(reinterpret_cast<const float4 *>(row + (a.rot >> 1)) + p);
      }
      c[4 * p] = x.x, c[4 * p + 1] = x.y, c[4 * p + 2] = x.z, c[4 * p + 3] = x.w;
      s[4 * p] = sign * y.x, s[4 * p + 1] = sign * y.y, s[4 * p + 2] = sign * y.z, s[4 * p + 3] = sign * y.w;
    }
  }
  // The same with a position per axis.
  __device__ __forceinline__ void angles(const RopeAppendArgs &a, const int32_t (&pos)[kMaxAxes]) {
#pragma unroll
    for (int j = 0; j < 4 * N; ++j) {
      const uint32_t ax = (axis >> (2 * j)) & 3u;
      const int32_t p = ax == 0 ? pos[0] : ax == 1 ? pos[1] : ax == 2 ? pos[2] : pos[3];
      const float *cos = a.cos_sin + (int64_t)p * a.rot + at + j;
      c[j] = in ? __ldg(cos) : 0.f;
      s[j] = in ? sign * __ldg(cos + (a.rot >> 1)) : 0.f;
    }
  }
  // v = the lane's chunk, rotated; every lane of the warp calls it (shuffles).
  // Products and sums are rounded one by one (a - b s = a + b (-s) exactly).
  __device__ __forceinline__ void apply(const uint4 raw, float (&v)[8]) const {
    unpack8(raw, v);
    if (halves(ROPE)) {
      uint4 o;
      o.x = __shfl_sync(0xffffffffu, raw.x, partner);
      o.y = __shfl_sync(0xffffffffu, raw.y, partner);
      o.z = __shfl_sync(0xffffffffu, raw.z, partner);
      o.w = __shfl_sync(0xffffffffu, raw.w, partner);
      float w[8];
      unpack8(o, w);
      if (in)
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float2 x = mul2(make_float2(v[j], v[j + 1]), make_float2(c[j], c[j + 1]));
          const float2 y = mul2(make_float2(w[j], w[j + 1]), make_float2(s[j], s[j + 1]));
          v[j] = __fadd_rn(x.x, y.x);
          v[j + 1] = __fadd_rn(x.y, y.y);
        }
    } else if (ROPE != kNoRope) {
      if (in)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = make_float2(v[2 * j], v[2 * j + 1]);
          const float2 y = mul2(x, make_float2(c[j], c[j])), z = mul2(make_float2(x.y, x.x), make_float2(-s[j], s[j]));
          v[2 * j] = __fadd_rn(y.x, z.x);
          v[2 * j + 1] = __fadd_rn(y.y, z.y);
        }
    }
  }
};

// One E4M3 code of a non-negative value (nearest even, saturating; NaN: 0x7F).
__device__ __forceinline__ uint32_t e4m3_of(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xFFu;
}

// Quotients v / s as the IEEE fp32 ones, or as values that round to the same E4M3
// or E2M1 code.  With r the correctly rounded reciprocal of s, q = RN(v r) and the
// exact remainder v - q s (one fused multiply-add), RN(q + remainder r) is the
// correctly rounded quotient (Markstein's theorem) as long as nothing under- or
// overflows: |v| <= 2^60 and s within 2^+-40 leave only quotients below 2^-60
// unproven, which round to zero codes with v's sign either way.  Anything else
// (also infinities and NaN) takes the division instruction sequence.
struct Divisor {
  float s, r;                     // the divisor, RN(1 / s)
  bool plain;                     // s is in the range above
  __device__ __forceinline__ explicit Divisor(float s_) : s(s_), r(1.f / s_) {
    plain = s >= 0x1p-40f && s <= 0x1p40f;
  }
  __device__ __forceinline__ Divisor(float s_, float r_) : s(s_), r(r_), plain(true) {}
  // (zeros come out as +0)
  __device__ __forceinline__ float2 plainly(float2 v) const {
    const float2 rr = make_float2(r, r), q = mul2(v, rr);
    return fma2(fma2(q, make_float2(-s, -s), v), rr, q);
  }
};

// max(|a|, |b|, |c|), NaN if one is.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(fabsf(c)));
  return d;
}
// The largest magnitude of 8 values as fp32 bits (a NaN is above everything).
__device__ __forceinline__ uint32_t top_bits(const float (&v)[8]) {
  const float t = max3_abs(max3_abs(v[0], v[1], v[2]), max3_abs(v[3], v[4], v[5]), max3_abs(v[6], v[7], v[7]));
  return __float_as_uint(t);
}
constexpr uint32_t kPlainTop = 0x5D800000u;      // 2^60
constexpr uint32_t kInfBits = 0x7F800000u;

// v / d with v's signs, zeros included.
__device__ __forceinline__ void divide8(float (&v)[8], const Divisor &d, uint32_t top) {
  if (d.plain && top <= kPlainTop) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float2 x = make_float2(v[j], v[j + 1]), y = d.plainly(x);
      v[j] = copysignf(y.x, x.x);
      v[j + 1] = copysignf(y.y, x.y);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __fdiv_rn(v[j], d.s);
  }
}

__device__ __forceinline__ float e4m3_value(uint32_t code) {
  uint32_t h2;
  asm("{\n .reg .b16 s;\n cvt.u16.u32 s, %1;\n cvt.rn.f16x2.e4m3x2 %0, s;\n}\n" : "=r"(h2) : "r"(code));
  float s;
  asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %1;\n cvt.f32.f16 %0, l;\n}\n" : "=f"(s) : "r"(h2));
  return s;
}

// Eight quotients -> eight E2M1 codes, element i in nibble i.
__device__ __forceinline__ uint32_t e2m1_codes(const float (&y)[8]) {
  uint32_t out;
  asm("{\n .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(out)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return out;
}

// Per CTA: every finite E4M3 block scale with its correctly rounded reciprocal.
struct ScaleTable {
  float2 at[128];
  __device__ __forceinline__ void fill() {
    const int i = threadIdx.x;
    if (i < 128) {
      const float s = e4m3_value(i);
      at[i] = make_float2(s, 1.f / s);
    }
    __syncthreads();
  }
};

// A lane's 8 values of a 4-bit row (its scale block's other 8 are in lane ^ 1):
// the codes (4 bytes) and the block's scale.  Every lane of the warp calls it.
// Rounding is monotonic, so the largest quotient is the quotient of the largest.
__device__ __forceinline__ uint32_t quantise8(const float (&v)[8], const Divisor &tensor, const ScaleTable &table,
                                              uint32_t &scale) {
  uint32_t top = top_bits(v);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  float y[8];
  if (tensor.plain && top <= kPlainTop && top >= 0x21800000u) {       // 2^-60: the largest quotient is exact
    const float amax = tensor.plainly(make_float2(__uint_as_float(top), 0.f)).x;
    const float q6 = amax * (1.f / 6.f);
    scale = e4m3_of(__fmaf_rn(__fmaf_rn(-q6, 6.f, amax), 1.f / 6.f, q6));
    if (scale != 0u) {
      const float2 sr = table.at[scale];
      const Divisor block(sr.x, sr.y);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const float2 x = block.plainly(tensor.plainly(make_float2(v[j], v[j + 1])));
        y[j] = copysignf(x.x, v[j]);
        y[j + 1] = copysignf(x.y, v[j + 1]);
      }
      return e2m1_codes(y);
    }
  } else {
    // zeros, tiny or huge values, infinities, NaN (its block gets the NaN scale), odd
    // tensor scales: by the division instruction sequence
    const float amax = __fdiv_rn(__uint_as_float(top), tensor.s);
    scale = top > kInfBits ? 0x7Fu : e4m3_of(__fdiv_rn(amax, 6.f));
    if (scale != 0u && scale != 0x7Fu) {
      const float s = e4m3_value(scale);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = __fdiv_rn(__fdiv_rn(v[j], tensor.s), s);
      return e2m1_codes(y);
    }
  }
  // under a zero scale every value is below half the smallest step: its sign stays
  uint32_t out = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) out |= (__float_as_uint(v[i]) >> 31) << (4 * i + 3);
  return out;
}

// Rows of D values as a warp takes them: RPW rows a step, lane % NC the chunk.
template <int D>
struct Lanes {
  static constexpr int NC = D / 8, RPW = 32 / NC;
};

// The lane's chunk (v: rotated values, raw: as it stands) into a cached row.
// Every lane of the warp calls it; `live` lanes have a chunk.
template <int KV, int D>
__device__ __forceinline__ void store_chunk(uint8_t *row, int ch, bool live, bool turned, const uint4 raw,
                                            float (&v)[8], const Divisor &scale, const ScaleTable &table) {
  if (KV == ATTN_KV_BF16) {
    if (live) reinterpret_cast<uint4 *>(row)[ch] = turned ? pack8(v) : raw;
  } else if (KV == ATTN_KV_FP8_E4M3) {
    divide8(v, scale, top_bits(v));
    uint32_t w[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint16_t lo, hi;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(lo) : "f"(v[4 * e + 1]), "f"(v[4 * e]));
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(hi) : "f"(v[4 * e + 3]), "f"(v[4 * e + 2]));
      w[e] = (uint32_t)lo | ((uint32_t)hi << 16);
    }
    if (live) reinterpret_cast<uint2 *>(row)[ch] = make_uint2(w[0], w[1]);
  } else {
    constexpr int kGroups = D / kE2m1Block, kPad = e2m1_row_bytes(D) - D / 2 - kGroups;
    static_assert(kPad == 4 || kPad == 8, "4-bit row padding");
    uint32_t s;
    const uint32_t codes = quantise8(v, scale, table, s);
    if (live) {
      reinterpret_cast<uint32_t *>(row)[ch] = codes;
      if (!(ch & 1)) row[D / 2 + ch / 2] = (uint8_t)s;
      if (ch < kPad / 4) reinterpret_cast<uint32_t *>(row + D / 2 + kGroups)[ch] = 0u;
    }
  }
}

// The rows of one kind (K or V: D values) of a token, every `slices`-th row step
// from `slice` on.  One step's loads are ahead of the one at work, two where the row
// is rotated: its step is the longer one and starts before the lookups.
template <int KV, int ROPE, int D>
struct RowSteps {
  static constexpr int NC = Lanes<D>::NC, RPW = Lanes<D>::RPW, kAhead = ROPE == kNoRope ? 1 : 2;
  const uint4 *src;                // this lane's chunk of its next row to load
  int h, heads, step;              // that row's head; heads a step moves on
  bool lane_in;
  uint4 x[kAhead];

  __device__ __forceinline__ uint4 next() {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (lane_in && h < heads) v = __ldg(src);
    src += step * NC;
    h += step;
    return v;
  }
  __device__ __forceinline__ void start(const uint16_t *rows, int heads_, int slice, int slices) {
    const int lane = threadIdx.x & 31, sub = lane / NC;
    lane_in = sub < RPW;
    heads = heads_;
    step = slices * RPW;
    h = slice * RPW + sub;
    src = reinterpret_cast<const uint4 *>(rows + (int64_t)h * D) + lane % NC;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) x[k] = next();
  }
  __device__ __forceinline__ void store(uint8_t *rows, int slice, const Turn<ROPE, NC> &turn, const Divisor &scale,
                                        const ScaleTable &table) {
    const int lane = threadIdx.x & 31, ch = lane % NC;
    int hs = slice * RPW + lane / NC;
    uint8_t *dst = rows + (int64_t)hs * kv_row_bytes(KV, D);
    for (int first = slice * RPW; first < heads; first += step) {
      const uint4 raw = x[0];
#pragma unroll
      for (int k = 0; k + 1 < kAhead; ++k) x[k] = x[k + 1];
      x[kAhead - 1] = next();
      float v[8];
      turn.apply(raw, v);
      store_chunk<KV, D>(dst, ch, lane_in && hs < heads, turn.in, raw, v, scale, table);
      dst += step * kv_row_bytes(KV, D);
      hs += step;
    }
  }
};

template <int KV, int ROPE, int DQK>
__global__ void __launch_bounds__(kAppendThreads, 4) rope_append_kernel(const RopeAppendArgs a) {
  // A programmatic dependent of the stream's previous kernel: nothing is read
  // or written before that kernel has completed.  The kernels that follow in a
  // serving step (device planner, attention) may be scheduled now; they wait
  // for this grid.
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  constexpr int NC = Lanes<DQK>::NC, RPW = Lanes<DQK>::RPW;           // K and query rows
  const int lane = threadIdx.x & 31, sub = lane / NC, ch = lane % NC;
  const int worker = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const int chunk = worker / a.slices, slice = worker % a.slices;
  __shared__ ScaleTable table;
  if (KV == ATTN_KV_FP4_E2M1) table.fill();
  if (chunk >= a.chunks) return;
  Turn<ROPE, NC> turn;
  turn.place(a, lane);
  const Turn<kNoRope, Lanes<kDv>::NC> as_is{};
  const Divisor k_scale(a.k_scale), v_scale(a.v_scale);
  const int tok_end = (int)((int64_t)(chunk + 1) * a.tokens / a.chunks);
  Request rq;
  for (int tok = (int)((int64_t)chunk * a.tokens / a.chunks); tok < tok_end; ++tok) {
    // the first rows are on their way while the token is looked up
    RowSteps<KV, ROPE, DQK> k_rows;
    RowSteps<KV, kNoRope, kDv> v_rows;
    k_rows.start(a.k_new + (int64_t)tok * a.hkv * DQK, a.hkv, slice, a.slices);
    v_rows.start(a.v_new + (int64_t)tok * a.hkv * kDv, a.hkv, slice, a.slices);
    rq.seek(a.qo_indptr, a.seq_lens, a.batch, tok);
    if (rq.b >= a.batch || tok < rq.first) {          // a row that qo_indptr does not hold
      if (slice == 0 && lane == 0) atomicOr(a.err, 4);
      continue;
    }
    const int64_t i = tok + rq.shift;
    if (by_axes(ROPE)) {
      int32_t pos[kMaxAxes];
      bool good = true;
#pragma unroll
      for (int ax = 0; ax < kMaxAxes; ++ax) {
        int64_t p = 0;
        if (ax < a.axes) {
          p = a.positions ? (int64_t)__ldg(a.positions + (int64_t)ax * a.tokens + tok)
                          : i + (a.position_delta ? __ldg(a.position_delta + rq.b) : 0);
          good &= p >= 0 && p < a.max_pos;
        }
        pos[ax] = good ? (int32_t)p : 0;
      }
      if (!good) {                                  // as below
        if (slice == 0 && lane == 0) atomicOr(a.err, 8);
        continue;
      }
      turn.angles(a, pos);
    } else if (ROPE != kNoRope) {
      const int64_t pos = a.positions ? (int64_t)__ldg(a.positions + tok) : i;
      if (pos < 0 || pos >= a.max_pos) {            // no row of the table: the token is skipped
        if (slice == 0 && lane == 0) atomicOr(a.err, 8);
        continue;
      }
      turn.angles(a, pos);
    }
    // ---- K and V
    if (slice < a.hkv) {
      int64_t slot = -1;
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
      if (slot >= 0) {
        k_rows.store(static_cast<uint8_t *>(a.k_cache) + slot * a.hkv * kv_row_bytes(KV, DQK), slice, turn, k_scale,
                     table);
        v_rows.store(static_cast<uint8_t *>(a.v_cache) + slot * a.hkv * kv_row_bytes(KV, kDv), slice, as_is, v_scale,
                     table);
      }
    }
    // ---- the query rows; a row is read by its warp before it is written (q_out
    // may be q: then only the rotated chunks move)
    if constexpr (ROPE != kNoRope) {
      if (a.q) {
        const bool moves = sub < RPW && (turn.in || a.q != a.q_out);
        const int steps = (a.hq + RPW - 1) / RPW;
        constexpr int kAhead = 4;
        const int h0 = slice * RPW + sub;
        const int64_t at = ((int64_t)tok * a.hq + h0) * DQK + ch * 8;
        const uint16_t *src = a.q + at;
        uint16_t *dst = a.q_out + at;
        const int stride = a.slices * RPW * DQK;
        int h = h0, h_next = h0;
        auto next = [&]() {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (moves && h_next < a.hq) v = *reinterpret_cast<const uint4 *>(src);
          h_next += a.slices * RPW;
          src += stride;
          return v;
        };
        uint4 x[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) x[k] = next();
#pragma unroll 1
        for (int st0 = slice; st0 < steps; st0 += kAhead * a.slices) {
#pragma unroll
          for (int k = 0; k < kAhead; ++k) {
            if (st0 + k * a.slices >= steps) break;
            float v[8];
            turn.apply(x[k], v);
            if (moves && h < a.hq) *reinterpret_cast<uint4 *>(dst) = turn.in ? pack8(v) : x[k];
            x[k] = next();
            h += a.slices * RPW;
            dst += stride;
          }
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

// The heads of one cached slot (cache == nullptr: zeros) as bfloat16 rows.
template <int KV, int D>
__device__ __forceinline__ void read_rows_of(const uint8_t *cache, uint16_t *out, int heads, int slice, int slices,
                                             float scale) {
  constexpr int NC = Lanes<D>::NC, RPW = Lanes<D>::RPW, kAhead = 4;
  const int lane = threadIdx.x & 31, sub = lane / NC, ch = lane % NC;
  const int steps = (heads + RPW - 1) / RPW;
#pragma unroll 1
  for (int st0 = slice; st0 < steps; st0 += kAhead * slices) {
    uint4 x[kAhead];                       // raw: 16, 8 or 4 bytes, and a scale byte in .w
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int h = (st0 + k * slices) * RPW + sub;
      x[k] = make_uint4(0u, 0u, 0u, 0u);
      if (cache && sub < RPW && h < heads) {
        const uint8_t *row = cache + (int64_t)h * kv_row_bytes(KV, D);
        if (KV == ATTN_KV_BF16) {
          x[k] = __ldg(reinterpret_cast<const uint4 *>(row) + ch);
        } else if (KV == ATTN_KV_FP8_E4M3) {
          const uint2 r = __ldg(reinterpret_cast<const uint2 *>(row) + ch);
          x[k].x = r.x;
          x[k].y = r.y;
        } else {
          x[k].x = __ldg(reinterpret_cast<const uint32_t *>(row) + ch);
          x[k].w = __ldg(row + D / 2 + ch / 2);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int h = (st0 + k * slices) * RPW + sub;
      if (sub >= RPW || h >= heads) continue;
      uint4 o = x[k];
      if (KV != ATTN_KV_BF16) {
        uint32_t p[4];                     // 8 values as fp16 pairs, exact
        if (KV == ATTN_KV_FP8_E4M3) {
          uint4 lo, hi;
          e4m3x16_to_f16(make_uint4(x[k].x, x[k].y, 0u, 0u), lo, hi);
          p[0] = lo.x, p[1] = lo.y, p[2] = lo.z, p[3] = lo.w;
        } else {
          uint32_t s0, s1;
          e4m3_scales_f16(x[k].w, s0, s1);
          e2m1x8_to_f16(x[k].x, p);
#pragma unroll
          for (int e = 0; e < 4; ++e) p[e] = mul_f16x2(p[e], s0);
        }
        float v[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, u;\n}\n"
              : "=f"(v[2 * e]), "=f"(v[2 * e + 1])
              : "r"(p[e]));
          v[2 * e] = __fmul_rn(v[2 * e], scale);
          v[2 * e + 1] = __fmul_rn(v[2 * e + 1], scale);
        }
        o = pack8(v);
      }
      reinterpret_cast<uint4 *>(out + (int64_t)h * D)[ch] = o;
    }
  }
}

// Cached rows as bfloat16; the rows of request b are its last kv_indptr[b + 1] -
// kv_indptr[b] positions.  Work is split as for the append.
template <int KV, int DQK>
__global__ void __launch_bounds__(kAppendThreads, 4) read_kernel(const ReadArgs a) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int worker = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const int chunk = worker / a.slices, slice = worker % a.slices;
  if (chunk >= a.chunks) return;
  const int row_end = (int)((int64_t)(chunk + 1) * a.rows / a.chunks);
  Request rq;
  for (int row = (int)((int64_t)chunk * a.rows / a.chunks); row < row_end; ++row) {
    rq.seek(a.kv_indptr, a.seq_lens, a.batch, row);
    int64_t slot = -1;
    int bad = 4;                                  // more rows than kv_indptr holds, or no such position
    if (rq.b < a.batch) {
      const int64_t i = row + rq.shift;
      if (row >= rq.first && i >= 0 && i / a.page_size < a.pt_stride) {
        const int32_t page = __ldg(a.page_table + (int64_t)rq.b * a.pt_stride + i / a.page_size);
        bad = page >= 0 && page < a.num_pages ? 0 : 1;
        if (!bad) slot = (int64_t)page * a.page_size + i % a.page_size;
      }
    }
    if (bad && slice == 0 && lane == 0) atomicOr(a.err, bad);
    const int64_t row_heads = slot * a.hkv;
    read_rows_of<KV, DQK>(slot < 0 ? nullptr : static_cast<const uint8_t *>(a.k_cache) + row_heads * kv_row_bytes(KV, DQK),
                          a.k_out + (int64_t)row * a.hkv * DQK, a.hkv, slice, a.slices, a.k_scale);
    read_rows_of<KV, kDv>(slot < 0 ? nullptr : static_cast<const uint8_t *>(a.v_cache) + row_heads * kv_row_bytes(KV, kDv),
                          a.v_out + (int64_t)row * a.hkv * kDv, a.hkv, slice, a.slices, a.v_scale);
  }
}

// Splits `rows` of `heads` rows of one kind each among the warps that all SMs hold
// (four CTAs an SM): ranges of rows, and the warps that share a range's heads.  (A
// step of 128-value rows takes two heads, so that with few rows some of the warps
// have nothing to take.)
struct Split {
  int32_t chunks, slices;
  unsigned ctas;
  Split(int64_t rows, int64_t heads, int num_sms) {
    const int64_t warps = (int64_t)num_sms * 4 * (kAppendThreads / 32);
    slices = (int32_t)std::max<int64_t>(1, std::min(heads, warps / std::max<int64_t>(rows, 1)));
    chunks = (int32_t)std::min<int64_t>(rows, std::max<int64_t>(1, warps / slices));
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

attn_status_t append_rows(attn_plan_t plan, const attn_rope_t *rope, const attn_mrope_t *axes, const void *q,
                          const void *k_new, const void *v_new, void *q_out, void *k_cache, void *v_cache,
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
  if (axes) {
    if (axes->num_axes < 1 || axes->num_axes > kMaxAxes || !axes->pair_axis_host ||
        (rope->positions && axes->position_delta))
      return ATTN_ERR_INVALID_ARG;
    for (int i = 0; i < rope->rot_dim / 2; ++i)
      if (axes->pair_axis_host[i] >= axes->num_axes) return ATTN_ERR_INVALID_ARG;
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
  int64_t heads = pr.num_kv_heads;
  if (rope) {
    a.cos_sin = rope->cos_sin;
    a.positions = rope->positions;
    a.max_pos = rope->max_pos;
    a.rot = rope->rot_dim;
    a.rot_off = rope->rot_offset;
    if (axes) {
      a.axes = axes->num_axes;
      a.position_delta = axes->position_delta;
      for (int i = 0; i < rope->rot_dim / 2; ++i)
        a.axis_bits[i / 16] |= (uint32_t)axes->pair_axis_host[i] << (2 * (i % 16));
    }
    if (q) {
      a.q = static_cast<const uint16_t *>(q);
      a.q_out = static_cast<uint16_t *>(q_out);
      heads = std::max<int64_t>(heads, pr.num_q_heads);
    }
  }
  const Split sp(total_q, heads, hp.num_sms);
  a.chunks = sp.chunks;
  a.slices = sp.slices;
  DeviceGuard dev(plan->device);
  if (!dev.ok) return ATTN_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 grid(sp.ctas);
  // (without a rotation only 4-bit caches come here: kv_append.cu)
  const int kv = pr.kv_dtype, dqk = pr.head_dim_qk;
  const cudaError_t e = !rope               ? launch_append<ATTN_KV_FP4_E2M1, kNoRope>(a, dqk, grid, st)
                        : rope->interleaved ? axes ? launch_append_kv<kPairsAxes>(a, kv, dqk, grid, st)
                                                   : launch_append_kv<kPairs>(a, kv, dqk, grid, st)
                        : axes              ? launch_append_kv<kHalvesAxes>(a, kv, dqk, grid, st)
                                            : launch_append_kv<kHalves>(a, kv, dqk, grid, st);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace akp

extern "C" attn_status_t attn_append_kv_rope(attn_plan_t plan, const attn_rope_t *rope, const void *q,
                                             const void *k_new, const void *v_new, void *q_out,
                                             void *k_cache, void *v_cache, const int32_t *page_table,
                                             const int32_t *seq_lens, const int32_t *qo_indptr,
                                             float k_scale, float v_scale, void *stream) {
  if (!rope) return ATTN_ERR_INVALID_ARG;
  return akp::append_rows(plan, rope, nullptr, q, k_new, v_new, q_out, k_cache, v_cache, page_table, seq_lens,
                          qo_indptr, k_scale, v_scale, stream);
}

extern "C" attn_status_t attn_append_kv_mrope(attn_plan_t plan, const attn_mrope_t *mrope, const void *q,
                                              const void *k_new, const void *v_new, void *q_out,
                                              void *k_cache, void *v_cache, const int32_t *page_table,
                                              const int32_t *seq_lens, const int32_t *qo_indptr,
                                              float k_scale, float v_scale, void *stream) {
  if (!mrope) return ATTN_ERR_INVALID_ARG;
  return akp::append_rows(plan, &mrope->rope, mrope, q, k_new, v_new, q_out, k_cache, v_cache, page_table,
                          seq_lens, qo_indptr, k_scale, v_scale, stream);
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
  const akp::Split sp(rows, pr.num_kv_heads, plan->host.num_sms);
  a.chunks = sp.chunks;
  a.slices = sp.slices;
  akp::DeviceGuard dev(plan->device);
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
