// attn_run_sparse: attention of every new token over its own list of blocks.
//
// For a token at position i and KV head g, over the keys j <= i of the listed blocks:
//   s_j = scale <q, k_j>,  out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m),
// one pass with a running maximum and sum per row, as in the other kernels.
//
// Tokens choose their blocks apart from each other, so a block of keys meets the query
// rows of one token: the 16 rows of a group (or as many as there are, padded), which is
// the M of one register-operand MMA (m16n8k16).  The tcgen05 instructions want 64 or 128
// rows; with 16 they would spend their time on padding.  A "unit" is a token's tile of at
// most 16 heads of one KV head, and a warp holds a unit's queries, maxima, sums and output
// in registers.
//
// A CTA has eight such warps and one that loads.  Keys come in tiles of 64 (a block of
// 64, half a block of 128, or several smaller blocks), as TMA boxes in a ring that all
// eight warps pass through in order, each waiting for every tile (so that no barrier
// phase can be taken for another):
//   SHARED  (groups of more than 128 heads) eight neighbouring units, a warp each.  The
//           loader merges their lists in ascending order, so that a block that several of
//           them chose is fetched once; a warp skips the tiles that its unit has not chosen.
//   REDO    the same for the jobs that attn_sparse_tc.cu has marked; writes their marked
//           rows.
//   SPLIT   (decode, verify) one unit for all eight warps, each taking half of every
//           fourth tile; a cluster of up to eight CTAs shares out the list.  The warps'
//           partial results meet in shared memory, the CTAs' through distributed shared
//           memory.
// 32 requests (16/2 heads, 16 blocks of 64, bf16) take 12.3 us, 4 x 8 verified tokens of an
// E4M3 cache 13.0: 42 MB at 3.4 TB/s on the first, behind a chain of dependent loads
// (layout, list, pages, keys) and in front of a combine over the cluster.
//
// K fragments come from shared memory by ldmatrix (bf16), or as 16- or 8-byte pieces
// that are widened in registers (E4M3, E2M1: the order of a contraction's index is free,
// and Q's fragments use the same order); V fragments by ldmatrix.trans, or as the
// pieces of four keys whose bytes or nibbles are paired up before the conversion.
// 8- and 4-bit caches run in fp16 with queries scaled by a power of two per row, and P
// times 2^7, as attn_fp4.cu does.
//
// Keys that a unit does not see (behind its token, blocks of other units, pieces of a
// tile that were not filled) have their scores set to -inf and their V operands to zero
// in registers, so that what the slots hold does not matter.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <limits>

#include "attn_paged.h"
#include "e2m1.cuh"
#include "kernels.hpp"
#include "requests.cuh"
#include "sparse_attn.cuh"
#include "tc_common.cuh"

namespace akp {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 8;                      // consumer warps
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kRows = 16;                      // query rows of a unit
constexpr int kTile = 64;                      // keys of a tile
constexpr int kHalf = 32;                      // keys a warp takes at a time
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGrow = 8.0f;                  // base-2 growth of a maximum before O is rescaled
constexpr int kStride = 132;                   // floats per row of the partial results

template <int KV, int DQK>
struct Tile {
  static constexpr bool kRaw = KV != ATTN_KV_BF16;
  static constexpr int kKrow = kv_row_bytes(KV, DQK), kVrow = kv_row_bytes(KV, kDv);
  static constexpr int kKBytes = kTile * kKrow, kVBytes = kTile * kVrow, kBytes = kKBytes + kVBytes;
  static constexpr int kKBoxes = kRaw ? 1 : DQK / 64, kVBoxes = kRaw ? 1 : kDv / 64, kBoxes = kKBoxes + kVBoxes;
  static constexpr int kStages = KV == ATTN_KV_FP4_E2M1 ? 12 : KV == ATTN_KV_FP8_E4M3 ? 8 : DQK == kDqk ? 5 : 6;
  static constexpr int kRing = kStages * kBytes;
  static_assert(kKBytes % 1024 == 0 || KV == ATTN_KV_FP4_E2M1, "swizzled boxes start on 1024 bytes");
  static_assert(kRing >= (kWarps + 1) * kRows * kStride * 4, "the partial results use the ring");
};

struct Desc {                 // a tile's pieces: first key and the units that chose it
  int32_t key0[4];
  uint32_t units[4];
  int32_t end, pad[3];
};

constexpr int kMaxStages = 12;

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  Desc desc[kMaxStages];
  int32_t count[kWarps], pos[kWarps], req[kWarps];      // a unit's blocks, position (-1: no unit), request
  float m[kWarps][kRows], l[kWarps][kRows];
  float pm[kRows], pl[kRows];
  int abort;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

template <bool BF>
__device__ __forceinline__ uint32_t pair16(float lo, float hi) {
  if (BF) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// c (16 x 8, fp32) += a (16 x 16) . b (16 x 8), bf16 or fp16
template <bool BF>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
  asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, u;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t lo16) {
  uint32_t p;
  asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}\n" : "=r"(p) : "r"(lo16));
  return p;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2,
                                            uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(tc::smem_u32(bar))
      : "memory");
}

// What a warp holds of its unit's rows g and g + 8 (lane = 4 g + t).  Output column of
// o[nt][x], o[nt][2 + x] (x = 0, 1; rows g, g + 8): bf16 caches 8 nt + 2 t + x, others
// 32 t + 16 x + nt.
template <int KV, int DQK>
struct Unit {
  static constexpr bool kBf = KV == ATTN_KV_BF16;
  static constexpr float kLift = kBf ? 0.f : 7.f;
  using T = Tile<KV, DQK>;
  uint32_t qf[DQK / 16][4];
  float o[16][4];
  float m[2], l[2], sc[2];

  // rows of the unit, `rows` of them from `row0` on (row stride DQK)
  __device__ __forceinline__ void load(const uint16_t *row0, int rows, float scale_log2, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const uint16_t *r0 = row0 + (int64_t)g * DQK, *r1 = r0 + 8 * DQK;
    if (kBf) {
#pragma unroll
      for (int k = 0; k < DQK / 16; ++k)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int at = 16 * k + 8 * x + 2 * t;
          qf[k][2 * x] = g < rows ? __ldg(reinterpret_cast<const uint32_t *>(r0 + at)) : 0u;
          qf[k][2 * x + 1] = g + 8 < rows ? __ldg(reinterpret_cast<const uint32_t *>(r1 + at)) : 0u;
        }
      sc[0] = sc[1] = scale_log2;
    } else {
      // k-step 4 j + s: dims 64 j + 16 t + 4 s + {0, 1} and {2, 3}
      uint32_t e[2] = {0u, 0u};
#pragma unroll
      for (int k = 0; k < DQK / 16; ++k) {
        const int at = 64 * (k >> 2) + 16 * t + 4 * (k & 3);
        const uint2 v0 = g < rows ? __ldg(reinterpret_cast<const uint2 *>(r0 + at)) : make_uint2(0u, 0u);
        const uint2 v1 = g + 8 < rows ? __ldg(reinterpret_cast<const uint2 *>(r1 + at)) : make_uint2(0u, 0u);
        qf[k][0] = v0.x, qf[k][2] = v0.y, qf[k][1] = v1.x, qf[k][3] = v1.y;
#pragma unroll
        for (int x = 0; x < 4; ++x)
          e[x & 1] = max(e[x & 1], max((qf[k][x] >> 7) & 0xFFu, (qf[k][x] >> 23) & 0xFFu));
      }
      float up[2];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        e[y] = max(e[y], __shfl_xor_sync(0xffffffffu, e[y], 1));
        e[y] = max(e[y], __shfl_xor_sync(0xffffffffu, e[y], 2));
        const int sh = min(141 - (int)e[y], 126);
        up[y] = __int_as_float((sh + 127) << 23);
        sc[y] = tc::row_score_scale(scale_log2, sh);
      }
#pragma unroll
      for (int k = 0; k < DQK / 16; ++k)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t w = qf[k][x];
          qf[k][x] = pair16<false>(__uint_as_float(w << 16) * up[x & 1], __uint_as_float(w & 0xFFFF0000u) * up[x & 1]);
        }
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      m[y] = -INFINITY;
      l[y] = 0.f;
    }
#pragma unroll
    for (int nt = 0; nt < 16; ++nt)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[nt][x] = 0.f;
  }

  // Keys [r0, r0 + 32) of the tile at `kt`; vis[q]: how many of the 16 keys r0 + 16 q ..
  // are seen (EDGE; otherwise all are).
  template <bool EDGE>
  __device__ __forceinline__ void step(const uint8_t *kt, int r0, const int (&vis)[2], int lane) {
    const int g = lane >> 2, t = lane & 3;
    float s[4][4];
#pragma unroll
    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
      for (int x = 0; x < 4; ++x) s[nt][x] = 0.f;
    // ---- S = Q . K^T
    if (kBf) {
      const uint32_t base = tc::smem_u32(kt);
      const int row = r0 + (lane & 7) + (lane >> 4) * 8, hi = (lane >> 3) & 1;
#pragma unroll
      for (int k = 0; k < DQK / 16; ++k) {
        const uint32_t at = base + (k >> 2) * (kTile * 128) + row * 128 + ((((2 * k) & 7) + hi) ^ (row & 7)) * 16;
        uint32_t f[4];
        ldmatrix4(f, at);
        mma<true>(s[0], qf[k], f[0], f[1]);
        mma<true>(s[1], qf[k], f[2], f[3]);
        ldmatrix4(f, at + 16 * 128);
        mma<true>(s[2], qf[k], f[0], f[1]);
        mma<true>(s[3], qf[k], f[2], f[3]);
      }
    } else if (KV == ATTN_KV_FP8_E4M3) {
#pragma unroll
      for (int j = 0; j < DQK / 64; ++j)
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          const uint4 w = *reinterpret_cast<const uint4 *>(kt + (r0 + 8 * nt + g) * T::kKrow + 16 * (t + 4 * j));
          const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t b0, b1;
            e4m3x4_to_f16(x[k], b0, b1);
            mma<false>(s[nt], qf[4 * j + k], b0, b1);
          }
        }
    } else {
#pragma unroll
      for (int j = 0; j < DQK / 64; ++j)
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          const uint8_t *row = kt + (r0 + 8 * nt + g) * T::kKrow;
          const uint2 w = *reinterpret_cast<const uint2 *>(row + 8 * (t + 4 * j));
          uint32_t s0, s1, h[8];
          e4m3_scales_f16(row[DQK / 2 + t + 4 * j], s0, s1);
          uint32_t x[4];
          e2m1x8_to_f16(w.x, x);
          h[0] = x[0], h[1] = x[1], h[2] = x[2], h[3] = x[3];
          e2m1x8_to_f16(w.y, x);
          h[4] = x[0], h[5] = x[1], h[6] = x[2], h[7] = x[3];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma<false>(s[nt], qf[4 * j + k], mul_f16x2(h[2 * k], s0), mul_f16x2(h[2 * k + 1], s0));
        }
    }
    // ---- softmax: base-2 scores against the running maximum
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        float v = s[nt][x] * sc[x >> 1];
        if (EDGE && (nt & 1) * 8 + 2 * t + (x & 1) >= vis[nt >> 1]) v = -INFINITY;
        s[nt][x] = v;
        top[x >> 1] = fmaxf(top[x >> 1], v);
      }
    if (__any_sync(0xffffffffu, top[0] > m[0] + kGrow || top[1] > m[1] + kGrow)) {
      float alpha[2];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float mx = top[y];
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const bool up = mx > m[y] + kGrow;            // also from -inf
        alpha[y] = up ? ex2(m[y] - mx) : 1.f;
        if (up) m[y] = mx;
        l[y] *= alpha[y];
      }
#pragma unroll
      for (int nt = 0; nt < 16; ++nt)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[nt][x] *= alpha[x >> 1];
    }
    uint32_t p[2][4];
#pragma unroll
    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const float n = m[y] == -INFINITY ? 0.f : kLift - m[y];
        const float p0 = ex2(s[nt][2 * y] + n), p1 = ex2(s[nt][2 * y + 1] + n);
        l[y] += p0 + p1;
        p[nt >> 1][2 * (nt & 1) + y] = pair16<kBf>(p0, p1);
      }
    // ---- O += P . V
    const uint8_t *vt = kt + T::kKBytes;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (EDGE && vis[q] <= 0) continue;
      // keys 2t, 2t + 1, 2t + 8, 2t + 9 of the 16, those that are not seen as zeros
      bool see[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) see[y] = !EDGE || 2 * t + (y & 1) + 8 * (y >> 1) < vis[q];
      if (kBf) {
        const uint32_t base = tc::smem_u32(vt);
        const int row = r0 + 16 * q + (lane & 7) + ((lane >> 3) & 1) * 8, hi = lane >> 4;
        const uint32_t m0 = (see[0] ? 0xFFFFu : 0u) | (see[1] ? 0xFFFF0000u : 0u);
        const uint32_t m1 = (see[2] ? 0xFFFFu : 0u) | (see[3] ? 0xFFFF0000u : 0u);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t f[4];
          ldmatrix4_trans(f, base + (c >> 2) * (kTile * 128) + row * 128 + ((((2 * c) & 7) + hi) ^ (row & 7)) * 16);
          if (EDGE) f[0] &= m0, f[1] &= m1, f[2] &= m0, f[3] &= m1;
          mma<true>(o[2 * c], p[q], f[0], f[1]);
          mma<true>(o[2 * c + 1], p[q], f[2], f[3]);
        }
      } else if (KV == ATTN_KV_FP8_E4M3) {
        uint4 w[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int row = r0 + 16 * q + 2 * t + (y & 1) + 8 * (y >> 1);
          w[y] = *reinterpret_cast<const uint4 *>(vt + row * 128 + ((g ^ (row & 7)) * 16));     // swizzled box
          if (EDGE && !see[y]) w[y] = make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t k0 = i == 0 ? w[0].x : i == 1 ? w[0].y : i == 2 ? w[0].z : w[0].w;
          const uint32_t k1 = i == 0 ? w[1].x : i == 1 ? w[1].y : i == 2 ? w[1].z : w[1].w;
          const uint32_t k2 = i == 0 ? w[2].x : i == 1 ? w[2].y : i == 2 ? w[2].z : w[2].w;
          const uint32_t k3 = i == 0 ? w[3].x : i == 1 ? w[3].y : i == 2 ? w[3].z : w[3].w;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t a0, a1, b0, b1;
            e4m3x4_to_f16(__byte_perm(k0, k1, h ? 0x7362 : 0x5140), a0, a1);
            e4m3x4_to_f16(__byte_perm(k2, k3, h ? 0x7362 : 0x5140), b0, b1);
            mma<false>(o[4 * i + 2 * h], p[q], a0, b0);
            mma<false>(o[4 * i + 2 * h + 1], p[q], a1, b1);
          }
        }
      } else {
        uint2 w[4];
        uint32_t sb[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const uint8_t *row = vt + (r0 + 16 * q + 2 * t + (y & 1) + 8 * (y >> 1)) * T::kVrow;
          w[y] = *reinterpret_cast<const uint2 *>(row + 8 * g);
          sb[y] = see[y] ? row[kDv / 2 + g] : 0u;
        }
        const uint32_t sA = e4m3x2_to_f16(sb[0] | sb[1] << 8), sB = e4m3x2_to_f16(sb[2] | sb[3] << 8);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t k0 = h ? w[0].y : w[0].x, k1 = h ? w[1].y : w[1].x;
          const uint32_t k2 = h ? w[2].y : w[2].x, k3 = h ? w[3].y : w[3].x;
          constexpr uint32_t L4 = 0x0F0F0F0Fu;
          uint32_t eA[4], oA[4], eB[4], oB[4];
          e2m1x8_to_f16((k0 & L4) | ((k1 << 4) & ~L4), eA);          // even codes, (key, key + 1)
          e2m1x8_to_f16(((k0 >> 4) & L4) | (k1 & ~L4), oA);          // odd codes
          e2m1x8_to_f16((k2 & L4) | ((k3 << 4) & ~L4), eB);
          e2m1x8_to_f16(((k2 >> 4) & L4) | (k3 & ~L4), oB);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            mma<false>(o[8 * h + 2 * i], p[q], mul_f16x2(eA[i], sA), mul_f16x2(eB[i], sB));
            mma<false>(o[8 * h + 2 * i + 1], p[q], mul_f16x2(oA[i], sA), mul_f16x2(oB[i], sB));
          }
        }
      }
    }
  }

  // The rows' sums, and a maximum of 0 for a row of nothing but NaN scores.
  __device__ __forceinline__ void close() {
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      l[y] += __shfl_xor_sync(0xffffffffu, l[y], 1);
      l[y] += __shfl_xor_sync(0xffffffffu, l[y], 2);
      if (l[y] != l[y] && m[y] == -INFINITY) m[y] = 0.f;
    }
  }
};

// A unit's list as ascending blocks and the slots they start at (whole pool: a page id
// outside it).  All 32 lanes of a warp call it; returns the number of blocks.
__device__ __forceinline__ int prepare_list(const SparseArgs &a, const int32_t *idx, int b, int own, int32_t *list,
                                            int32_t *slots, int lane) {
  const uint32_t below = (1u << lane) - 1u;
  int cnt = 0, prev = -1;
  bool sorted = true;
  for (int at = 0; at < a.take; at += 32) {
    int c = at + lane < a.take ? __ldg(idx + at + lane) : -1;
    if (c > own) {
      atomicOr(a.err, 16);
      c = -1;
    }
    c = max(c, -1);
    int up = c;                                  // the largest up to this lane
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up = max(up, y);
    }
    int before = __shfl_up_sync(0xffffffffu, up, 1);
    before = max(lane ? before : -1, prev);
    sorted &= __all_sync(0xffffffffu, c < 0 || c > before);
    const uint32_t in = __ballot_sync(0xffffffffu, c >= 0);
    if (c >= 0) list[cnt + __popc(in & below)] = c;
    cnt += __popc(in);
    prev = max(prev, __shfl_sync(0xffffffffu, up, 31));
  }
  __syncwarp();
  if (!sorted) {                                 // any order, repetitions: by rank
    constexpr int N = ATTN_SPARSE_MAX_TAKE / 32;
    int mine[N], rank[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      mine[k] = lane + 32 * k < cnt ? list[lane + 32 * k] : INT_MAX;
      rank[k] = 0;
    }
    for (int j = 0; j < cnt; ++j) {              // a repetition: an equal entry further ahead
      const int v = list[j];
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (v == mine[k] && j < lane + 32 * k) rank[k] = -1;
    }
    __syncwarp();
    int gone = 0;
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (rank[k] < 0) {
        list[lane + 32 * k] = INT_MAX;
        ++gone;
      }
    __syncwarp();
    for (int j = 0; j < cnt; ++j) {
      const int v = list[j];
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (rank[k] >= 0 && v < mine[k]) ++rank[k];
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (lane + 32 * k < cnt && rank[k] >= 0) list[rank[k]] = mine[k];
    cnt -= __reduce_add_sync(0xffffffffu, gone);
    __syncwarp();
  }
  const int per_page = a.page_size / a.block;
  for (int e = lane; e < cnt; e += 32) {
    const int c = list[e];
    const int32_t page = __ldg(a.page_table + (int64_t)b * a.pt_stride + c / per_page);
    const bool bad = page < 0 || page >= a.num_pages;
    if (bad) atomicOr(a.err, 1);
    slots[e] = bad ? a.num_pages * a.page_size : page * a.page_size + c % per_page * a.block;
  }
  return cnt;
}

enum { kShared = 0, kSplit = 1, kRedo = 2 };     // kRedo: the marked jobs of attn_sparse_tc.cu, as kShared

template <int KV, int DQK, int MODE>
__global__ void __launch_bounds__(kThreads, 1) sparse_kernel(const SparseArgs a, const __grid_constant__ TmaMaps maps) {
  constexpr bool SPLIT = MODE == kSplit;
  using T = Tile<KV, DQK>;
  using U = Unit<KV, DQK>;
  constexpr int kUnits = SPLIT ? 1 : kWarps, kStages = T::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *ring = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
  int32_t *lists = reinterpret_cast<int32_t *>(ring + T::kRing);       // [units][take] blocks, then slots
  __shared__ Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, t = lane & 3;
  const int ranks = SPLIT ? (int)cg::this_cluster().num_blocks() : 1;
  const int rank = SPLIT ? (int)cg::this_cluster().block_rank() : 0;
  int g = blockIdx.y;
  int unit0 = SPLIT ? (int)blockIdx.x / ranks : (int)blockIdx.x * kWarps;
  int total_units = a.tokens * a.row_tiles;
  if (tid == 0) sh.abort = 0;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  int job = (int)blockIdx.x - (int)gridDim.x, job_left = 0;
  for (bool again = false;; again = true) {
  if (MODE != kRedo && again) break;
  if (MODE == kRedo) {                       // the next eight units of a marked job
    unit0 += kWarps;
    while (--job_left < 0) {
      for (job += gridDim.x; job < a.jobs && !__ldcg(a.redo + job);) job += gridDim.x;
      if (job >= a.jobs) return;
      SparseJob x;
      if (!find_job(a, job, x, false)) continue;
      g = x.g;
      unit0 = x.tok0 * a.row_tiles;
      total_units = (x.tok0 + x.ntok) * a.row_tiles;
      job_left = (total_units - unit0 + kWarps - 1) / kWarps;
    }
    if (again) {
      __syncthreads();
      if (sh.abort) return;
      if (tid == 0)
        for (int s = 0; s < kStages; ++s) {
          asm volatile("mbarrier.inval.shared::cta.b64 [%0];\n" ::"r"(tc::smem_u32(&sh.full[s])) : "memory");
          asm volatile("mbarrier.inval.shared::cta.b64 [%0];\n" ::"r"(tc::smem_u32(&sh.empty[s])) : "memory");
        }
    }
  }
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(&sh.full[s], 1);
      tc::mbar_init(&sh.empty[s], kWarps);
    }
    tc::fence_mbar_init();
  }
  // ---- the units: their lists, their query rows
  U u;
  const int unit = SPLIT ? unit0 : unit0 + warp;
  const int tok = unit / a.row_tiles, row0 = unit % a.row_tiles * kRows;       // the unit's first head
  const int rows = warp < kWarps && unit < total_units ? min(kRows, a.group - row0) : 0;
  if (warp < kWarps) {
    if (!SPLIT || warp == 0) {
      int cnt = 0, pos = -1, b = a.batch;
      if (rows > 0) {
        b = request_of(a.qo_indptr, a.batch, tok);
        int q0 = 0, n = 0;
        if (b < a.batch) {
          q0 = __ldg(a.qo_indptr + b);
          n = __ldg(a.qo_indptr + b + 1) - q0;
        }
        // a row that qo_indptr does not hold, or a request longer than the plan's: left as it was
        if (b >= a.batch || tok < q0 || n > a.max_len) {
          b = a.batch;
          if (lane == 0) atomicOr(a.err, 4);
        } else {
          const int L0 = __ldg(a.seq_lens + b), L = max(min(L0, a.max_len), n);
          if (L != L0 && lane == 0) atomicOr(a.err, 4);
          pos = L - n + tok - q0;
          cnt = prepare_list(a, a.block_idx + ((int64_t)tok * a.hkv + g) * a.take, b, pos / a.block,
                             lists + warp * a.take, lists + (kUnits + warp) * a.take, lane);
        }
      }
      if (lane == 0) {
        sh.count[warp] = cnt;
        sh.pos[warp] = pos;
        sh.req[warp] = b;
      }
    }
  }
  __syncthreads();
  // after the lists: the loader's start waits for those, and their loads do not queue behind these
  // (32 requests, 16/2 heads, 16 blocks of 64: 12.8 -> 12.3 us)
  if (rows > 0) u.load(a.q + ((int64_t)tok * a.hq + g * a.group + row0) * DQK, rows, a.scale_log2, lane);

  if (warp == kWarps) {
    // ------------------------------------------------------------ loader
    const int per_tile = a.block < kTile ? kTile / a.block : 1;        // pieces of a tile
    const int piece = min(a.block, kTile);                             // keys of a piece
    const bool halves = a.block > kTile;                               // two tiles a block
    // lane u < units: where unit u's list stands
    int at = 0, end = 0, pos = -1;
    uint32_t request = 0;
    if (lane < kUnits) {
      end = sh.count[lane];
      pos = sh.pos[lane];
      request = lane > 0 && sh.req[lane] != sh.req[lane - 1];
    }
    if (SPLIT) {                                                       // this CTA's share, whole tiles
      const int tiles = halves ? 2 * end : (end + per_tile - 1) / per_tile;
      const int lo = (int)((int64_t)tiles * rank / ranks), hi = (int)((int64_t)tiles * (rank + 1) / ranks);
      at = halves ? lo : lo * per_tile;                                // (in halves)
      end = halves ? hi : min(end, hi * per_tile);
    } else {
#pragma unroll
      for (int o = 1; o < kWarps; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, request, o);
        if (lane >= o) request += y;
      }
      if (halves) end *= 2;
    }
    const int32_t *list = lists + lane * a.take, *slot_list = lists + (kUnits + lane) * a.take;
    // lists are merged on (request, piece) as one number: requests ascend with the units
    auto key_at = [&](int i) -> uint32_t {
      if (lane >= kUnits || i >= end) return 0xFFFFFFFFu;
      return request << 29 | (uint32_t)(halves ? 2 * list[i >> 1] + (i & 1) : list[i]);
    };
    uint32_t key = key_at(at);
    int issued = 0;
    bool more = true;
    while (more) {
      int pieces = 0, my_key0 = 0, my_slot = 0;
      uint32_t my_units = 0u;
      for (int s = 0; s < per_tile; ++s) {
        int slot = 0, key0 = 0;
        uint32_t units = 0u;
        for (;;) {
          const uint32_t least = __reduce_min_sync(0xffffffffu, key);
          if (least == 0xFFFFFFFFu) {
            more = false;
            break;
          }
          key0 = (int)(least & 0x1FFFFFFFu) * piece;
          const bool has = key == least;
          units = __ballot_sync(0xffffffffu, has);
          if (has) slot = halves ? slot_list[at >> 1] + ((at & 1) * kTile) : slot_list[at];
          // (a page id outside the pool: past the pool for both halves)
          slot = __shfl_sync(0xffffffffu, slot, __ffs(units) - 1);
          const bool any = __any_sync(0xffffffffu, has && pos >= key0);
          if (has) key = key_at(++at);
          if (any) break;                                              // the far half of an own block may be empty
        }
        if (!more) break;
        if (lane == s) {
          my_key0 = key0;
          my_slot = slot;
          my_units = units;
        }
        ++pieces;
      }
      const int st = issued % kStages;
      if (issued >= kStages && !tc::mbar_wait_warp(&sh.empty[st], (issued / kStages - 1) & 1, &sh.abort)) break;
      if (lane < 4) {
        sh.desc[st].key0[lane] = my_key0;
        sh.desc[st].units[lane] = my_units;
      }
      if (lane == 4) sh.desc[st].end = !more;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_expect_tx(&sh.full[st], pieces * piece * (T::kKrow + T::kVrow));
      __syncwarp();
      ++issued;
      uint8_t *tile = ring + st * T::kBytes;
      const int s = lane / T::kBoxes, box = lane % T::kBoxes;
      const int slot = __shfl_sync(0xffffffffu, my_slot, s & 3);
      if (s < pieces) {
        const bool is_k = box < T::kKBoxes;
        const int col = is_k ? box : box - T::kKBoxes;
        uint8_t *dst = tile + (is_k ? 0 : T::kKBytes);
        dst += T::kRaw ? s * piece * (is_k ? T::kKrow : T::kVrow) : col * (kTile * 128) + s * piece * 128;
        tma_load_3d(tc::smem_u32(dst), is_k ? &maps.k : &maps.v, 64 * col, g, slot, &sh.full[st]);
      }
      __syncwarp();
    }
    if (sh.abort) {                    // the copies in flight land before the CTA ends
      int no_abort = 0;
      for (int i = max(0, issued - kStages); i < issued; ++i)
        tc::mbar_wait(&sh.full[i % kStages], (i / kStages) & 1, &no_abort, 100000000ull);
    }
  } else {
    // ------------------------------------------------------------ attention
    const int pos = sh.pos[SPLIT ? 0 : warp];
    const uint32_t me = SPLIT ? 1u : 1u << warp;
    for (int n = 0;; ++n) {
      const int st = n % kStages;
      if (!tc::mbar_wait_warp(&sh.full[st], (n / kStages) & 1, &sh.abort)) break;
      const uint8_t *kt = ring + st * T::kBytes;
      const bool last = sh.desc[st].end != 0;
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        if (SPLIT && ((n & 3) != (warp >> 1) || h != (warp & 1))) continue;
        int vis[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int r = kHalf * h + 16 * q, s = a.block < kTile ? r / a.block : 0;
          const int k0 = sh.desc[st].key0[s] + (a.block < kTile ? r % a.block : r);
          vis[q] = sh.desc[st].units[s] & me ? min(16, pos + 1 - k0) : 0;
        }
        if (vis[0] == 16 && vis[1] == 16)
          u.template step<false>(kt, kHalf * h, vis, lane);
        else if (vis[0] > 0 || vis[1] > 0)
          u.template step<true>(kt, kHalf * h, vis, lane);
      }
      tc::mbar_arrive_warp(&sh.empty[st]);
      if (last) break;
    }
    if (rows > 0) u.close();
  }
  auto sink_of = [&](int head) { return a.sinks ? __ldg(a.sinks + head) * kLog2e : -INFINITY; };
  if constexpr (!SPLIT) {
    if (rows > 0 && sh.req[warp] < a.batch) {
      bool write[2];                                  // REDO: the marked rows
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int r = gq + 8 * y;
        write[y] = r < rows;
        if (MODE == kRedo && write[y]) {
          const uint16_t *at = a.out + ((int64_t)tok * a.hq + g * a.group + row0 + r) * kDv;
          write[y] = __ldcg(at) == kMark || __ldcg(at + 64) == kMark;
        }
      }
      __syncwarp();
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int r = gq + 8 * y;
        if (!write[y]) continue;
        const int head = g * a.group + row0 + r;
        float lse;
        const float f = finish(u.m[y], u.l[y], U::kLift, sink_of(head), a.v_scale, lse);
        uint16_t *dst = a.out + ((int64_t)tok * a.hq + head) * kDv;
        if (U::kBf) {
#pragma unroll
          for (int nt = 0; nt < 16; ++nt)
            *reinterpret_cast<uint32_t *>(dst + 8 * nt + 2 * t) = pair16<true>(u.o[nt][2 * y] * f, u.o[nt][2 * y + 1] * f);
        } else {
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[i] = pair16<true>(u.o[8 * k + 2 * i][2 * y + x] * f, u.o[8 * k + 2 * i + 1][2 * y + x] * f);
              *reinterpret_cast<uint4 *>(dst + 32 * t + 16 * x + 8 * k) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        if (a.lse && t == 0) a.lse[(int64_t)tok * a.hq + head] = lse;
      }
    }
  } else {
    // ---- the warps' results, then the CTAs'
    __syncthreads();                                  // the ring is no longer read or written
    float *part = reinterpret_cast<float *>(ring);    // [warp][row][kStride], then the CTA's own
    if (warp < kWarps) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int r = gq + 8 * y;
        float *dst = part + (warp * kRows + r) * kStride;
        if (t == 0) {
          sh.m[warp][r] = u.m[y];
          sh.l[warp][r] = u.l[y];
        }
#pragma unroll
        for (int nt = 0; nt < 16; ++nt)
#pragma unroll
          for (int x = 0; x < 2; ++x) dst[U::kBf ? 8 * nt + 2 * t + x : 32 * t + 16 * x + nt] = u.o[nt][2 * y + x];
      }
    }
    __syncthreads();
    float *own = part + kWarps * kRows * kStride;
    if (warp < kWarps) {
      for (int r = warp; r < rows; r += kWarps) {
        float M = -INFINITY, l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sh.m[w][r]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          if (sh.m[w][r] == -INFINITY) continue;      // (nothing seen)
          const float f = exp2f(sh.m[w][r] - M);      // (0 for a warp far below the others, whose NaN stays one)
          const float4 v = *reinterpret_cast<const float4 *>(part + (w * kRows + r) * kStride + 4 * lane);
          l += f * sh.l[w][r];
          acc.x += f * v.x;
          acc.y += f * v.y;
          acc.z += f * v.z;
          acc.w += f * v.w;
        }
        *reinterpret_cast<float4 *>(own + r * kStride + 4 * lane) = acc;
        if (lane == 0) {
          sh.pm[r] = M;
          sh.pl[r] = l;
        }
      }
    }
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    if (warp < kWarps && sh.req[0] < a.batch) {
      for (int r = rank + ranks * warp; r < rows; r += ranks * kWarps) {
        float M = -INFINITY, l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < ranks; ++k) M = fmaxf(M, *cluster.map_shared_rank(&sh.pm[r], k));
        for (int k = 0; k < ranks; ++k) {
          const float mk = *cluster.map_shared_rank(&sh.pm[r], k);
          if (mk == -INFINITY) continue;
          const float f = exp2f(mk - M);
          const float4 v = *reinterpret_cast<const float4 *>(cluster.map_shared_rank(own + r * kStride + 4 * lane, k));
          l += f * *cluster.map_shared_rank(&sh.pl[r], k);
          acc.x += f * v.x;
          acc.y += f * v.y;
          acc.z += f * v.z;
          acc.w += f * v.w;
        }
        const int head = g * a.group + row0 + r;
        float lse;
        const float f = finish(M, l, U::kLift, sink_of(head), a.v_scale, lse);
        uint16_t *dst = a.out + ((int64_t)tok * a.hq + head) * kDv + 4 * lane;
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pair16<true>(acc.x * f, acc.y * f), pair16<true>(acc.z * f, acc.w * f));
        if (a.lse && lane == 0) a.lse[(int64_t)tok * a.hq + head] = lse;
      }
    }
    cluster.sync();                                   // (no CTA leaves while another reads from it)
  }
  if (tid == 0 && sh.abort) atomicOr(a.err, 2);
  }
}

template <int KV, int DQK, int MODE>
cudaError_t launch_one(const SparseArgs &a, const TmaMaps &maps, int ranks, int num_sms, int device, cudaStream_t st) {
  constexpr bool SPLIT = MODE == kSplit;
  using T = Tile<KV, DQK>;
  const size_t smem = 1024 + T::kRing + (size_t)(SPLIT ? 1 : kWarps) * a.take * 8;
  auto kernel = sparse_kernel<KV, DQK, MODE>;
  static SmemLimit limit;
  const cudaError_t e = limit.raise(reinterpret_cast<const void *>(kernel), device,
                                    1024 + T::kRing + (SPLIT ? 1 : kWarps) * ATTN_SPARSE_MAX_TAKE * 8);
  if (e != cudaSuccess) return e;
  const int units = a.tokens * a.row_tiles;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = MODE == kRedo ? dim3((unsigned)std::min(a.jobs, num_sms))
                              : dim3((unsigned)(SPLIT ? units * ranks : (units + kWarps - 1) / kWarps), (unsigned)a.hkv);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ranks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = SPLIT ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, maps);
}

template <int KV, int DQK>
cudaError_t launch_kv(const HostPlan &hp, const SparseArgs &a, const TmaMaps &maps, int device, cudaStream_t st) {
  // With up to a unit for each SM: a unit a CTA, its list over as many CTAs as there are SMs
  // for (up to eight, with two tiles for each).  With more, tiles of neighbouring tokens
  // (attn_sparse_tc.cu) where they hold 1.5 units a job or more, however empty their 128
  // rows: a job takes about as long as a unit, whose blocks it shares.  Measured at 4,000 to
  // 8,000 tokens, 16 blocks of 64, 64/4 heads, us, a unit a CTA against tiles:
  //                                      bf16        E4M3        4-bit
  //   1,024 units of 1 token a request   163 / 161   133 / 172   143 / 170
  //   1,024 units of 2                   138 / 107   129 / 115   139 / 114
  //   1,024 units of 4                   126 / 67    128 / 71    138 / 71
  //   1,024 units of 8                   122 / 44    126 / 47    137 / 47
  //   192 units of 2                     35 / 27     35 / 32     38 / 32
  //   192 units of 8                     35 / 31     35 / 39     38 / 39
  // (24 jobs of eight tokens leave most SMs idle: there the rule costs E4M3 4 us.)  The more
  // neighbours' lists differ, the longer a job's union: 4,096 tokens in a row take 485 (E4M3
  // 624, 4-bit 632) us with lists alike for 16 tokens, 43 blocks a job of eight tokens, and
  // 886 (1,166, 1,187) with independent ones, 97 blocks; a unit a CTA 1,870 (1,941, 2,101)
  // whatever the lists.
  // A group of more than 128 heads fits no tile: its row tiles have one list, and eight
  // units of a CTA share the blocks (256 heads, 64 tokens: 45 us, a unit a CTA 120; from about
  // two units an SM on).
  const int num_sms = hp.num_sms;
  const int64_t units = (int64_t)a.tokens * a.row_tiles * a.hkv;
  if (units > num_sms && a.jobs > 0 && 2 * units >= 3 * (int64_t)a.jobs) {
    const cudaError_t e = launch_sparse_tc(hp, a, maps, device, st);
    return e != cudaSuccess ? e : launch_one<KV, DQK, kRedo>(a, maps, 1, num_sms, device, st);
  }
  if (a.group > kSparseTileRows && units > 2 * num_sms) return launch_one<KV, DQK, kShared>(a, maps, 1, num_sms, device, st);
  const int tiles = (int)((int64_t)a.take * a.block / kTile);
  int ranks = 1;
  while (ranks < 8 && units * ranks * 2 <= num_sms && ranks * 4 <= tiles) ranks *= 2;
  return launch_one<KV, DQK, kSplit>(a, maps, ranks, num_sms, device, st);
}

template <int DQK>
cudaError_t launch(const HostPlan &hp, const SparseArgs &a, const TmaMaps &maps, int device, cudaStream_t st) {
  switch (hp.prob.kv_dtype) {
    case ATTN_KV_BF16: return launch_kv<ATTN_KV_BF16, DQK>(hp, a, maps, device, st);
    case ATTN_KV_FP8_E4M3: return launch_kv<ATTN_KV_FP8_E4M3, DQK>(hp, a, maps, device, st);
    default: return launch_kv<ATTN_KV_FP4_E2M1, DQK>(hp, a, maps, device, st);
  }
}

}  // namespace
}  // namespace akp

extern "C" attn_status_t attn_run_sparse(attn_plan_t plan, const attn_sparse_t *sparse, const void *q,
                                         const void *k_cache, const void *v_cache, const int32_t *page_table,
                                         const int32_t *seq_lens, const int32_t *qo_indptr,
                                         const int32_t *block_idx, const float *sinks, float softmax_scale,
                                         float k_scale, float v_scale, void *out, float *lse_out, void *stream) {
  if (!plan || plan->device < 0) return ATTN_ERR_INVALID_ARG;
  const akp::HostPlan &hp = plan->host;
  const attn_problem_t &pr = hp.prob;
  const attn_status_t ok = akp::check_sparse(hp, sparse);
  if (ok != ATTN_OK) return ok;
  const bool raw = pr.kv_dtype != ATTN_KV_BF16;
  if ((sinks != nullptr) != (pr.has_sinks != 0)) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(softmax_scale) || !std::isfinite(k_scale) || !std::isfinite(v_scale) || !(softmax_scale > 0.f) ||
      (raw && !(k_scale > 0.f)))
    return ATTN_ERR_INVALID_ARG;
  const int64_t slots = (int64_t)pr.num_pages * pr.page_size, tokens = hp.qo_indptr.back();
  if (slots > INT32_MAX - akp::kTile) return ATTN_ERR_UNSUPPORTED;
  if (tokens == 0) return ATTN_OK;
  if (!q || !k_cache || !v_cache || !page_table || !seq_lens || !qo_indptr || !block_idx || !out ||
      !akp::aligned16(q) || !akp::aligned16(k_cache) || !akp::aligned16(v_cache) || !akp::aligned16(out))
    return ATTN_ERR_INVALID_ARG;
  akp::SparseArgs a{};
  a.q = static_cast<const uint16_t *>(q);
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.page_table = page_table;
  a.seq_lens = seq_lens;
  a.qo_indptr = qo_indptr;
  a.block_idx = block_idx;
  a.sinks = sinks;
  a.out = static_cast<uint16_t *>(out);
  a.lse = lse_out;
  a.err = plan->dev.err;
  a.scale_log2 = std::max(softmax_scale * (raw ? k_scale : 1.f) * 1.4426950408889634f,
                          std::numeric_limits<float>::denorm_min());
  a.v_scale = raw ? v_scale : 1.f;
  a.batch = pr.batch;
  a.hq = pr.num_q_heads;
  a.hkv = pr.num_kv_heads;
  a.group = hp.group;
  a.row_tiles = (hp.group + akp::kRows - 1) / akp::kRows;
  a.page_size = pr.page_size;
  a.pt_stride = pr.page_table_stride;
  a.num_pages = pr.num_pages;
  a.tokens = (int32_t)tokens;
  a.block = sparse->block_size;
  a.take = sparse->num_blocks;
  a.max_len = akp::longest_request(hp);
  a.job_tokens = akp::sparse_job_tokens(hp.group);
  a.jobs = plan->dev.sparse_redo ? (int32_t)akp::sparse_jobs(hp) : 0;
  a.redo = plan->dev.sparse_redo;
  const int box = std::min(sparse->block_size, akp::kTile);
  akp::TmaMaps maps{};
  if (!akp::make_cache_map(&maps.k, k_cache, raw ? akp::kv_row_bytes(pr.kv_dtype, pr.head_dim_qk) : 0, pr.head_dim_qk,
                           pr.num_kv_heads, slots, box) ||
      !akp::make_cache_map(&maps.v, v_cache, raw ? akp::kv_row_bytes(pr.kv_dtype, akp::kDv) : 0, akp::kDv,
                           pr.num_kv_heads, slots, box, pr.kv_dtype == ATTN_KV_FP8_E4M3))
    return ATTN_ERR_CUDA;
  akp::DeviceGuard dev(plan->device);
  if (!dev.ok) return ATTN_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = pr.head_dim_qk == akp::kDqk
                            ? akp::launch<akp::kDqk>(hp, a, maps, plan->device, st)
                            : akp::launch<akp::kDqkSym>(hp, a, maps, plan->device, st);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
