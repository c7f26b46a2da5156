// attn_select_blocks for chunks of tokens: the scores as tcgen05 products.
//
// The same whole numbers as in select.cu, d(h, c) = q^+ . hi + q^- . lo over 2 Dqk dims,
// here with blocks as the rows of the product (M = 128 blocks a tile, operand A) and
// query rows as its columns (N = 128: a token tile of 128 / Gp tokens with Gp rows each,
// Gp the group's heads rounded up to a power of two, 4 at least): a thread of the
// epilogue then holds one block's scores for a token's heads side by side and takes
// their maximum without a shuffle.  A row that is missing or takes no part repeats one
// that does, which leaves the maximum as it is.  Rows carry their factor 2^(e_h - max e)
// in the fp16 integers (exact down to 2^-16; what is left of smaller ones is multiplied
// to the scores, as two powers of two where one would round twice or vanish).
//
// The bounds stay and the tokens stream by: a cluster of CTAs shares out the blocks of
// one (request, KV head), two tiles of 128 for each CTA, widened once into tensor memory,
// and goes through a range of token tiles.  For each, every CTA stages the query rows,
// multiplies, and hands each token's scores to the CTA of the cluster that makes its
// list (token t to CTA t mod size, through distributed shared memory).  Warps:
//   0-3    epilogue: maxima, exponents, ordered integers into the owners' shared memory
//   4-11   the bounds at the start of a range (a block a lane); then operand B of each
//          token tile in two halves of 64 rows (query rows in integers, 48 KB of 128-byte
//          swizzled rows each): one half is written while the other is multiplied
//   12-15  the lists: a token a warp, a radix select over its scores and the list in order
//   16     TMEM allocation; one thread issues the MMAs, 64 columns at a time, into two
//          accumulators in turn, so that the epilogue overlaps the next products
//   17     the query rows of the next token tile, as bulk copies
// TMEM: A 2 x Dqk columns, D 128.  Every wait is bounded in time.
//
// Up to 512 scored blocks a list is found in one warp's registers; beyond that by radix passes
// of one warp over the scores, and with larger clusters, which have room for fewer tokens a CTA,
// fewer of its four warps have a list to make.  4096 tokens (64/4 heads) over 500 blocks 150 us,
// 514 422, 768 659, 1,024 763, 1,500 1,939, 2,047 3,194.
//
// 4096 tokens (64/4 heads) over 470 blocks take 150 us; with the tokens at rest and the
// bounds widened for every token tile 316, a token a CTA (select.cu) 800.  Its 47 GFLOP
// (94 with q^+ and q^- apart) are 49 us of the tensor cores, which are busy 28% of the time:
// staging, epilogue, MMA issue and lists each need 7 to 9 thousand of a token tile's 11
// thousand cycles, side by side on 54% of the issue slots.  Every CTA of a cluster
// stages all query rows; to share that out is what is left.  Not kept: eight epilogue
// warps (80 registers: 173 us), the rounding by packed bf16 FMAs (fewer instructions, the same
// 150), the staging loops unrolled (153 to 157), scores by asynchronous remote stores (158).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "attn_paged.h"
#include "kernels.hpp"
#include "requests.cuh"
#include "select.cuh"
#include "tc_common.cuh"

namespace akp {
namespace {

constexpr int kThreads = 18 * 32;
constexpr int kStageWarps = 8, kPickWarps = 4, kMmaWarp = 16;
constexpr int kM = 128, kN = 128;              // blocks and query rows of a tile
constexpr int kTiles = 2;                      // block tiles of a CTA
constexpr int kSpan = kM * kTiles;             // its blocks
constexpr int kMaxRanks = 8;
constexpr int kMaxSmem = 216 * 1024;           // dynamic
constexpr int kOdd = INT_MIN;

template <int D>
struct Op {
  static constexpr int kColBlk = 64 * 128;                 // one 64-element column block of half of B
  static constexpr int kHalf = 2 * D / 64 * kColBlk;       // 48 KB at 192
  static constexpr int kRow = 2 * D;                       // bytes of a query row
  static constexpr int kRaw = kN * kRow;                   // a tile's rows as they are
  static constexpr int kACols = D;                         // 2 D fp16 values: D columns
  static constexpr uint32_t kTmemD = kTiles * kACols;
};

struct TcArgs {
  SelectArgs s;
  int32_t gp, gp_log2, tile_tokens;            // rows a token, tokens a tile
  int32_t range, ranges;                       // token tiles a range, ranges of all requests
  int32_t nr, ns;                              // row and score buffers
};

struct Bars {
  uint64_t b_full[2], b_empty[2], d_full[2], d_empty[2], s_full[2], s_empty[2], r_full[2], r_empty[2];
  uint64_t raw_full[2], raw_empty[2], a_full, a_empty, side, done;
};

// How a query row becomes integers: row `from` (-1: zeros) times 2^-e, rounded, times `sh`.
struct RowScale {
  float unit;
  uint32_t sh;
  int from, pad;
};

// One range of token tiles: tokens [tok0, tok0 + ntok) of request b at positions pos0 ..;
// blocks [c_lo, c_hi) are scored, this CTA's from c_lo + rank * kSpan on.
struct Item {
  int g, b, tok0, ntok, pos0, c_lo, c_hi;
};

// All 32 lanes of a warp call it; false: past the device's layout.
__device__ __forceinline__ bool find_item(const TcArgs &t, int item, Item &it, bool report) {
  const SelectArgs &a = t.s;
  const int lane = threadIdx.x & 31;
  it.g = item % a.hkv;
  const int want = item / a.hkv;
  const int per = t.range * t.tile_tokens;
  int base = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    const int r = b0 + lane;
    int q0 = 0, n = 0, L = 0;
    if (r < a.batch) {
      q0 = __ldg(a.qo_indptr + r);
      n = max(0, __ldg(a.qo_indptr + r + 1) - q0);
      L = __ldg(a.seq_lens + r);
    }
    const int cnt = (n + per - 1) / per;
    int sum = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, base + sum > want);
    if (past) {
      const int l = __ffs(past) - 1;
      const int k = want - base - __shfl_sync(0xffffffffu, sum - cnt, l);      // the request's range
      const int Lc = max(min(L, a.max_len), n);
      if (report && lane == l && Lc != L) atomicOr(a.err, 4);
      it.b = b0 + l;
      n = __shfl_sync(0xffffffffu, n, l);
      it.tok0 = __shfl_sync(0xffffffffu, q0, l) + k * per;
      it.ntok = min(per, n - k * per);
      it.pos0 = __shfl_sync(0xffffffffu, Lc, l) - n + k * per;
      // (a layout of more tokens than the plan's, or longer: nothing past the arrays)
      if (it.tok0 < 0 || it.tok0 + it.ntok > a.tokens || it.pos0 + it.ntok > a.max_len) return false;
      const int own = (it.pos0 + it.ntok - 1) / a.block;
      it.c_lo = a.first;
      it.c_hi = own < a.take ? it.c_lo : max(it.c_lo, own - a.last + 1);       // (every token takes all)
      return true;
    }
    base += __shfl_sync(0xffffffffu, sum, 31);
  }
  return false;
}

// Where the record of block c is (c past the scored ones: of the last of them).
struct Record {
  const uint8_t *rec;
  bool bad;                        // a page outside the pool
  __device__ __forceinline__ void find(const SelectArgs &a, const Item &it, int c, int row_bytes) {
    const int per_page = a.page_size / a.block;
    c = min(c, it.c_hi - 1);
    const int32_t page = __ldg(a.page_table + (int64_t)it.b * a.pt_stride + c / per_page);
    bad = page < 0 || page >= a.num_pages;
    rec = a.bounds + (((int64_t)(bad ? 0 : page) * per_page + c % per_page) * a.hkv + it.g) * row_bytes;
  }
};

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t max_h2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t min_h2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Shared memory of the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void store_remote(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(addr), "r"(v) : "memory");
}
// One arrival of the warp on a barrier of every CTA of the cluster, its lanes' earlier
// stores to any of them before it.
__device__ __forceinline__ void arrive_all(uint64_t *bar, int ranks) {
  asm volatile("fence.acq_rel.cluster;\n" ::: "memory");
  __syncwarp();
  const int lane = threadIdx.x & 31;
  if (lane < ranks)
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(
                     map_rank(tc::smem_u32(bar), lane))
                 : "memory");
}
// tc::mbar_wait_warp for barriers that other CTAs of the cluster arrive on.
__device__ __forceinline__ bool wait_cluster(uint64_t *bar, uint32_t parity, volatile int *abort) {
  const bool ok = tc::mbar_wait_warp(bar, parity, abort);
  asm volatile("fence.acq_rel.cluster;\n" ::: "memory");
  return ok;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) select_tc_kernel(const TcArgs ta) {
  const SelectArgs &a = ta.s;
  constexpr int kRec = bounds_row_bytes(D);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
  __shared__ Bars bars;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  // the rows' exponents and scales; of the token tiles in turn, factors that do not fit the
  // integers, and whether there are any
  __shared__ int exps[kN];
  __shared__ __align__(16) RowScale scale_of[kN];
  __shared__ float resid_of[2][2][kN];
  __shared__ int spread[2];
  __shared__ uint32_t home[kN / 4];              // where a token's scores go (buffer 0)
  __shared__ __align__(16) int hist[kPickWarps][256];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int rank, ranks;
  asm("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctarank;\n" : "=r"(ranks));
  // scores of this CTA's tokens: [ns][tokens / ranks][ranks * kSpan]
  const int stride = ranks * kSpan, own_tokens = (ta.tile_tokens + ranks - 1) / ranks;
  uint32_t *scores = reinterpret_cast<uint32_t *>(smem + 2 * Op<D>::kHalf + ta.nr * Op<D>::kRaw);
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&bars.b_full[i], kStageWarps);
      tc::mbar_init(&bars.b_empty[i], 1);
      tc::mbar_init(&bars.d_full[i], 1);
      tc::mbar_init(&bars.d_empty[i], 4);
      tc::mbar_init(&bars.s_full[i], 4 * ranks);
      tc::mbar_init(&bars.s_empty[i], kPickWarps * ranks);
      tc::mbar_init(&bars.r_full[i], kStageWarps);
      tc::mbar_init(&bars.r_empty[i], 4);
      tc::mbar_init(&bars.raw_full[i], 1);
      tc::mbar_init(&bars.raw_empty[i], kStageWarps);
    }
    tc::mbar_init(&bars.a_full, kStageWarps);
    tc::mbar_init(&bars.a_empty, 1);
    tc::mbar_init(&bars.side, kStageWarps);
    tc::mbar_init(&bars.done, 1);
    tc::fence_mbar_init();
  }
  if (tid < ta.tile_tokens) home[tid] = map_rank(tc::smem_u32(scores + tid / ranks * stride), tid % ranks);
  if (warp == kMmaWarp) tc::tmem_alloc(&tmem_slot, 512);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  asm volatile("barrier.cluster.arrive.aligned;\n barrier.cluster.wait.aligned;\n" ::: "memory");
  const uint32_t tmem = tmem_slot;
  const int items = ta.ranges * a.hkv, step = gridDim.x / ranks;
  auto wait = [&](uint64_t *bar, uint32_t parity) { return tc::mbar_wait_warp(bar, parity, &abort_flag); };
  auto my_blocks = [&](const Item &x) { return x.c_lo + rank * kSpan; };
  auto my_tiles = [&](const Item &x) { return min(kTiles, max(0, (x.c_hi - my_blocks(x) + kM - 1) / kM)); };
  auto token_tiles = [&](const Item &x) { return (x.ntok + ta.tile_tokens - 1) / ta.tile_tokens; };
  Item it;
  bool ok = true;

  if (warp < 4) {
    // ------------------------------------------------------------ epilogue
    const uint32_t d_addr = tmem + ((uint32_t)(warp * 32) << 16) + Op<D>::kTmemD;
    int seq = 0, staged = 0, tile = 0;            // token tiles so far, those with products here, block tiles
    for (int item = blockIdx.x / ranks; item < items && ok; item += step) {
      if (!find_item(ta, item, it, false)) continue;
      if (it.c_hi == it.c_lo) continue;
      const int na = my_tiles(it), nt = token_tiles(it);
      int e[kTiles] = {0, 0};
#pragma unroll
      for (int j = 0; j < kTiles; ++j) {
        if (j >= na) break;
        Record rec;
        rec.find(a, it, my_blocks(it) + j * kM + warp * 32 + lane, kRec);
        e[j] = rec.bad ? 0 : (int)(int8_t)__ldg(rec.rec + 2 * D);
        if (rec.bad) atomicOr(a.err, 1);
      }
      for (int k = 0; k < nt && ok; ++k, ++seq) {
        const int sb = seq % ta.ns, rb = staged & 1, tokens = min(ta.tile_tokens, it.ntok - k * ta.tile_tokens);
        if (seq >= ta.ns && !(ok = wait_cluster(&bars.s_empty[sb], (seq / ta.ns - 1) & 1, &abort_flag))) break;
        if (na > 0 && !(ok = wait(&bars.r_full[rb], (staged >> 1) & 1))) break;
        const uint32_t out = sb * own_tokens * stride * 4;
        const bool odd_factors = na > 0 && spread[rb];
        float over[kTiles] = {-INFINITY, -INFINITY};      // Gp = 128: the first half's maxima
        for (int h = 0; h < 2 && ok; ++h)
#pragma unroll
          for (int j = 0; j < kTiles; ++j) {
            if (j >= na) break;
            const int at = rank * kSpan + j * kM + warp * 32 + lane;     // the block among the scored ones
            const bool live = it.c_lo + at < it.c_hi;
            const float unit = pow2(e[j] == kOddBlock ? 0 : max(e[j], -126));
            auto put = [&](int tt, float s) {
              if (live && tt < tokens) store_remote(home[tt] + out + at * 4, ordered(e[j] == kOddBlock ? INFINITY : s * unit));
            };
            const int d = tile & 1;
            if (!(ok = wait(&bars.d_full[d], (tile >> 1) & 1))) break;
            ++tile;
            tc::tc_fence_after();
            uint32_t x[2][32];
            tc::tmem_ld32(d_addr + 64 * d, x[0]);
            tc::tmem_ld32(d_addr + 64 * d + 32, x[1]);
            tc::tmem_wait_ld_regs64(x[0], x[1]);
            tc::tc_fence_before();
            tc::mbar_arrive_warp(&bars.d_empty[d]);
            float v[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(x[i / 32][i % 32]);
            if (odd_factors) {
#pragma unroll
              for (int i = 0; i < 64; ++i) v[i] = v[i] * resid_of[rb][0][64 * h + i] * resid_of[rb][1][64 * h + i];
            }
            // maxima of 4, 8, .. columns side by side
#pragma unroll
            for (int w = 64, g = 1; w >= 1; w >>= 1, g <<= 1) {
              if (g >= 4 && ta.gp == g) {
#pragma unroll
                for (int i = 0; i < w; ++i) put(h * w + i, v[i]);
                break;
              }
              if (w > 1)
#pragma unroll
                for (int i = 0; i < w / 2; ++i) v[i] = fmaxf(v[2 * i], v[2 * i + 1]);
            }
            if (ta.gp == 128) {
              if (h) put(0, fmaxf(over[j], v[0]));
              over[j] = v[0];
            }
          }
        if (!ok) break;
        if (na > 0) {
          tc::mbar_arrive_warp(&bars.r_empty[rb]);
          ++staged;
        }
        arrive_all(&bars.s_full[sb], ranks);
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ bounds, query rows
    const int w = warp - 4;
    int staged = 0;                               // token tiles staged so far
    // Query rows of token tile k of a range: row r is head r % Gp of its token r / Gp.
    int synced = 0;
    auto side_sync = [&]() {
      tc::mbar_arrive_warp(&bars.side);
      return wait(&bars.side, synced++ & 1);
    };
    auto stage = [&](const Item &x, int k_tile) -> bool {
      const int tokens = min(ta.tile_tokens, x.ntok - k_tile * ta.tile_tokens);
      const int qb = staged % ta.nr, rb = staged & 1;
      if (staged >= 2 && !wait(&bars.r_empty[rb], ((staged >> 1) - 1) & 1)) return false;
      if (!wait(&bars.raw_full[qb], (staged / ta.nr) & 1)) return false;
      const uint8_t *raw = smem + 2 * Op<D>::kHalf + qb * Op<D>::kRaw;
      const bool in = lane < D / 8;
      // the largest magnitude of each of the warp's 16 rows; lane i (and i + 16) keeps row i's
      const int r = w * 16 + (lane & 15);
      uint32_t mine = 0u;
#pragma unroll 4
      for (int i = 0; i < 16; ++i) {
        const uint4 v = in ? *reinterpret_cast<const uint4 *>(raw + (w * 16 + i) * Op<D>::kRow + lane * 16)
                           : make_uint4(0u, 0u, 0u, 0u);
        constexpr uint32_t kAbs = 0x7FFF7FFFu;
        const uint32_t m2 = max_u16x2(max_u16x2(v.x & kAbs, v.y & kAbs), max_u16x2(v.z & kAbs, v.w & kAbs));
        const uint32_t m = __reduce_max_sync(0xffffffffu, max(m2 & 0xFFFFu, m2 >> 16));
        if ((lane & 15) == i) mine = m;
      }
      const bool odd = mine >= 0x7F80u || (r >> ta.gp_log2) >= tokens || (r & (ta.gp - 1)) >= a.group;
      const int e = odd ? kOdd : min(code_exponent(__uint_as_float(mine << 16)), 121);
      // the token's largest exponent and its first row that takes part: within the warp, or
      // (more than 16 rows a token) through shared memory
      int top = e, first = odd ? INT_MAX : r;
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) {
        if (o >= ta.gp) break;
        top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
      }
      if (w == 0 && lane == 0) spread[rb] = 0;
      if (lane < 16) exps[r] = e;
      if (!side_sync()) return false;
      if (ta.gp > 16) {
        top = kOdd;
        first = INT_MAX;
        const int t_row = w * 16 & ~(ta.gp - 1);
        for (int h = lane; h < ta.gp; h += 32) {
          top = max(top, exps[t_row + h]);
          if (exps[t_row + h] != kOdd) first = min(first, t_row + h);
        }
        top = __reduce_max_sync(0xffffffffu, top);
        first = __reduce_min_sync(0xffffffffu, first);
      }
      // a row that takes no part repeats `first`; the factor 2^(e - top) goes into the
      // integers as far as that goes
      const int from = odd ? first : r;
      const int ef = from == INT_MAX ? 0 : odd ? exps[from] : e, k = from == INT_MAX ? 0 : top - ef;
      if (lane < 16) {
        // (a whole number times 2^-122 is a normal fp32, still exact: one rounding, with the rest)
        resid_of[rb][0][r] = pow2(min(16 - min(k, 122), 0));
        resid_of[rb][1][r] = pow2(min(122 - k, 0));
        if (k > 16) spread[rb] = 1;
        const __half2 sh2 = __float2half2_rn(pow2(-min(k, 16)));
        scale_of[r] = RowScale{pow2(-ef), *reinterpret_cast<const uint32_t *>(&sh2), from == INT_MAX ? -1 : from, 0};
      }
      if (!side_sync()) return false;
      tc::mbar_arrive_warp(&bars.r_full[rb]);
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        if (staged > 0 && !wait(&bars.b_empty[h], (staged - 1) & 1)) return false;
        uint8_t *dst0 = smem + h * Op<D>::kHalf + (lane >> 3) * Op<D>::kColBlk;
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
          const int row = w * 8 + i;
          const int4 sc = *reinterpret_cast<const int4 *>(&scale_of[h * 64 + row]);
          const float unit = __int_as_float(sc.x);
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (in && sc.z >= 0) v = *reinterpret_cast<const uint4 *>(raw + sc.z * Op<D>::kRow + lane * 16);
          const uint32_t x4[4] = {v.x, v.y, v.z, v.w};
          uint32_t up[4], dn[4];
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            constexpr float kMagic = 12582912.f;    // 1.5 * 2^23: rounds to whole numbers, nearest even
            const float lo = __fadd_rn(__fmaf_rn(__uint_as_float(x4[p] << 16), unit, kMagic), -kMagic);
            const float hi = __fadd_rn(__fmaf_rn(__uint_as_float(x4[p] & 0xFFFF0000u), unit, kMagic), -kMagic);
            const __half2 h2 = __floats2half2_rn(lo, hi);
            const uint32_t q = mul_h2(*reinterpret_cast<const uint32_t *>(&h2), (uint32_t)sc.y);
            up[p] = max_h2(q, 0u);
            dn[p] = min_h2(q, 0u);
          }
          if (in) {
            // dims 8 lane .. of q+ in the first D / 64 column blocks, of q- in the others
            uint8_t *dst = dst0 + tc::sw128_offset(row, lane & 7);
            *reinterpret_cast<uint4 *>(dst) = make_uint4(up[0], up[1], up[2], up[3]);
            *reinterpret_cast<uint4 *>(dst + D / 64 * Op<D>::kColBlk) = make_uint4(dn[0], dn[1], dn[2], dn[3]);
          }
        }
        tc::fence_proxy_async_smem();
        tc::mbar_arrive_warp(&bars.b_full[h]);
      }
      tc::mbar_arrive_warp(&bars.raw_empty[qb]);
      ++staged;
      return true;
    };
    // The CTA's bounds as operand A: warp w takes block quadrant w % 4 (its TMEM lanes) of
    // the upper (w < 4) or lower codes.
    auto widen = [&](const Item &x, int na) {
      const int low = w >= 4;
      const uint32_t lane_base = (uint32_t)((w & 3) * 32) << 16;
#pragma unroll 1
      for (int j = 0; j < na; ++j) {
        Record rec;
        rec.find(a, x, my_blocks(x) + j * kM + (w & 3) * 32 + lane, kRec);
        uint4 raw[D / 16];
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          raw[i] = rec.bad ? make_uint4(0u, 0u, 0u, 0u) : __ldg(reinterpret_cast<const uint4 *>(rec.rec + low * D) + i);
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          uint32_t v[16];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint4 r = raw[2 * q + i];
            s8x4_to_f16(r.x, v[8 * i], v[8 * i + 1]);
            s8x4_to_f16(r.y, v[8 * i + 2], v[8 * i + 3]);
            s8x4_to_f16(r.z, v[8 * i + 4], v[8 * i + 5]);
            s8x4_to_f16(r.w, v[8 * i + 6], v[8 * i + 7]);
          }
          tc::tmem_st16(tmem + lane_base + j * Op<D>::kACols + low * (D / 2) + 16 * q, v);
        }
      }
      tc::tmem_wait_st();
      tc::tc_fence_before();
      tc::mbar_arrive_warp(&bars.a_full);
    };
    int with_products = 0;                        // ranges with products here
    for (int item = blockIdx.x / ranks; item < items && ok; item += step) {
      if (!find_item(ta, item, it, item % a.hkv == 0 && w == 0 && rank == 0)) {
        if (w == 0 && lane == 0) atomicOr(a.err, 4);         // a layout of fewer tokens
        continue;
      }
      const int na = my_tiles(it), nt = token_tiles(it);
      if (na == 0) continue;
      // (every product with the last range's bounds is done)
      if (with_products > 0 && !(ok = wait(&bars.a_empty, (with_products - 1) & 1))) break;
      ++with_products;
      tc::tc_fence_after();
      widen(it, na);
      for (int k = 0; k < nt && ok; ++k) ok = stage(it, k);
    }
  } else if (warp < kMmaWarp) {
    // ------------------------------------------------------------ lists
    // The list of the range's token tt from its scores, keys[c - c_lo].
    auto pick = [&](const Item &x, int tt, const uint32_t *keys) {
      const int own = (x.pos0 + tt) / a.block, total = own + 1;
      int32_t *out = a.block_idx + ((int64_t)(x.tok0 + tt) * a.hkv + x.g) * a.take;
      if (own < a.take) {
        for (int k = lane; k < a.take; k += 32) out[k] = k <= own ? k : -1;
        return;
      }
      const int c_hi = own - a.last + 1;          // [c_lo, c_hi) are scored, the others always in
      const int n = c_hi - x.c_lo;
      if (n <= 32 * kHeld) {
        pick_held(keys, n, a.take - (own + 1 - n), x.c_lo, out + x.c_lo, lane);
        for (int c = lane; c < x.c_lo; c += 32) out[c] = c;
        for (int c = c_hi + lane; c <= own; c += 32) out[a.take - (own + 1 - c)] = c;
        return;
      }
      int *bins = hist[warp - 12];
      uint32_t prefix = 0;
      int want = a.take - (x.c_lo + own + 1 - max(c_hi, x.c_lo));
      bool whole = want <= 0;                     // every key from `prefix` on is in
      if (whole) prefix = 0xFFFFFFFFu;
      // the bits that all scores share need no pass
      uint32_t least = 0xFFFFFFFFu, most = 0u;
#pragma unroll 4
      for (int c = x.c_lo + lane; c < c_hi; c += 32) {
        least = min(least, keys[c - x.c_lo]);
        most = max(most, keys[c - x.c_lo]);
      }
      least = __reduce_min_sync(0xffffffffu, least);
      most = __reduce_max_sync(0xffffffffu, most);
      int bits = 32 - __clz(least ^ most);        // that differ, 0 to 32
      if (!whole) prefix = bits < 32 ? most >> bits << bits : 0u;
      while (bits > 0 && !whole) {
        const int shift = max(bits - 8, 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) bins[i * 32 + lane] = 0;
        __syncwarp();
#pragma unroll 4
        for (int c = x.c_lo + lane; c < c_hi; c += 32) {
          const uint32_t k = keys[c - x.c_lo];
          if (bits == 32 || (k ^ prefix) >> bits == 0u) atomicAdd(&bins[(k >> shift) & ((1u << (bits - shift)) - 1u)], 1);
        }
        __syncwarp();
        // lane owns bins 255 - 8 lane .. downwards
        int cnt[8], sum = 0;
        const int4 lo4 = *reinterpret_cast<const int4 *>(&bins[248 - 8 * lane]);
        const int4 hi4 = *reinterpret_cast<const int4 *>(&bins[252 - 8 * lane]);
        cnt[0] = hi4.w, cnt[1] = hi4.z, cnt[2] = hi4.y, cnt[3] = hi4.x;
        cnt[4] = lo4.w, cnt[5] = lo4.z, cnt[6] = lo4.y, cnt[7] = lo4.x;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += cnt[i];
        int before = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, before, o);
          if (lane >= o) before += y;
        }
        before -= sum;
        int bin = 0, rest = 0, full = 0;
        bool here = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (before < want && before + cnt[i] >= want) {
            here = true;
            bin = 255 - (8 * lane + i);
            rest = want - before;
            full = rest == cnt[i];
          }
          before += cnt[i];
        }
        const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
        prefix |= (uint32_t)__shfl_sync(0xffffffffu, bin, src) << shift;
        want = __shfl_sync(0xffffffffu, rest, src);
        whole = __shfl_sync(0xffffffffu, full, src) != 0;
        bits = shift;
        __syncwarp();
      }
      // in order; of keys equal to `prefix` the first `want`
      int at = 0;
#pragma unroll 4
      for (int c0 = 0; c0 < total; c0 += 32) {
        const int c = c0 + lane;
        const uint32_t below = (1u << lane) - 1u;
        const bool forced = c < total && (c < x.c_lo || c >= c_hi);
        const uint32_t k = c >= x.c_lo && c < c_hi ? keys[c - x.c_lo] : 0u;
        const bool scored = c >= x.c_lo && c < c_hi;
        const bool is_eq = scored && !whole && k == prefix;
        const uint32_t eq = __ballot_sync(0xffffffffu, is_eq);
        const bool in = forced || (scored && (whole ? k >= prefix && prefix != 0xFFFFFFFFu : k > prefix)) ||
                        (is_eq && __popc(eq & below) < want);
        const uint32_t m = __ballot_sync(0xffffffffu, in);
        const int pos = at + __popc(m & below);
        if (in && pos < a.take) out[pos] = c;
        at += __popc(m);
        want -= __popc(eq);
      }
    };
    int seq = 0;
    for (int item = blockIdx.x / ranks; item < items && ok; item += step) {
      if (!find_item(ta, item, it, false)) continue;
      const bool scored = it.c_hi > it.c_lo;
      const int nt = token_tiles(it);
      for (int k = 0; k < nt; ++k) {
        const int sb = seq % ta.ns;
        if (scored && !(ok = wait_cluster(&bars.s_full[sb], (seq / ta.ns) & 1, &abort_flag))) break;
        const int t0 = k * ta.tile_tokens, tokens = min(ta.tile_tokens, it.ntok - t0);
        for (int i = warp - 12; i * ranks + rank < tokens; i += kPickWarps)
          pick(it, t0 + i * ranks + rank, scores + (sb * own_tokens + i) * stride);
        if (scored) {
          arrive_all(&bars.s_empty[sb], ranks);
          ++seq;
        }
      }
    }
  } else if (warp > kMmaWarp) {
    // ------------------------------------------------------------ query rows as they are
    int staged = 0;
    for (int item = blockIdx.x / ranks; item < items && ok; item += step) {
      if (!find_item(ta, item, it, false)) continue;
      if (my_tiles(it) == 0) continue;
      const int nt = token_tiles(it);
      for (int k = 0; k < nt; ++k, ++staged) {
        const int qb = staged % ta.nr, tokens = min(ta.tile_tokens, it.ntok - k * ta.tile_tokens);
        if (staged >= ta.nr && !(ok = wait(&bars.raw_empty[qb], (staged / ta.nr - 1) & 1))) break;
        const uint32_t bytes = a.group * Op<D>::kRow;
        if (lane == 0) tc::mbar_arrive_expect_tx(&bars.raw_full[qb], tokens * bytes);
        __syncwarp();
        if (lane < tokens) {
          const uint16_t *src = a.q + ((int64_t)(it.tok0 + k * ta.tile_tokens + lane) * a.hq + it.g * a.group) * D;
          const uint32_t dst = tc::smem_u32(smem + 2 * Op<D>::kHalf + qb * Op<D>::kRaw + lane * ta.gp * Op<D>::kRow);
          asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst),
                       "l"(src), "r"(bytes), "r"(tc::smem_u32(&bars.raw_full[qb]))
                       : "memory");
        }
        __syncwarp();
      }
    }
    if (!ok || abort_flag) {            // the copies in flight land before the CTA ends
      int no_abort = 0;
      for (int i = max(0, staged - ta.nr); i < staged; ++i)
        tc::mbar_wait(&bars.raw_full[i % ta.nr], (i / ta.nr) & 1, &no_abort, 100000000ull);
    }
  } else {
    // ------------------------------------------------------------ MMAs
    const uint32_t idesc = tc::idesc_f16(0, 0, 0, kM, 64);
    const uint32_t sbase = tc::smem_u32(smem);
    int staged = 0, with_products = 0, tile = 0;
    for (int item = blockIdx.x / ranks; item < items && ok; item += step) {
      if (!find_item(ta, item, it, false)) continue;
      const int na = my_tiles(it), nt = token_tiles(it);
      if (na == 0) continue;
      if (!(ok = wait(&bars.a_full, with_products & 1))) break;
      ++with_products;
      for (int k = 0; k < nt && ok; ++k, ++staged) {
        for (int h = 0; h < 2 && ok; ++h) {
          if (!(ok = wait(&bars.b_full[h], staged & 1))) break;
          for (int j = 0; j < na; ++j, ++tile) {
            const int d = tile & 1;
            if (tile >= 2 && !(ok = wait(&bars.d_empty[d], ((tile >> 1) - 1) & 1))) break;
            tc::tc_fence_after();
            if (lane == 0) {
              const uint64_t b_desc = tc::smem_desc_sw128(sbase + h * Op<D>::kHalf, 16, 1024);
              const uint32_t d_tmem = tmem + Op<D>::kTmemD + 64 * d, a_tmem = tmem + j * Op<D>::kACols;
#pragma unroll
              for (int q = 0; q < 2 * D / 16; ++q)      // (the descriptor's address counts 16 bytes)
                tc::mma_f16_ts(d_tmem, a_tmem + 8 * q, b_desc + ((q >> 2) * Op<D>::kColBlk + (q & 3) * 32) / 16, idesc,
                               q > 0);
              tc::mma_commit(&bars.d_full[d]);
              if (j + 1 == na) {
                tc::mma_commit(&bars.b_empty[h]);
                if (h == 1 && k + 1 == nt) tc::mma_commit(&bars.a_empty);
              }
            }
            __syncwarp();
          }
        }
      }
    }
    if (lane == 0) {                              // every MMA is complete before TMEM goes back
      tc::mma_commit(&bars.done);
      int no_abort = 0;
      tc::mbar_wait(&bars.done, 0, &no_abort, 100000000ull);
    }
    __syncwarp();
  }
  tc::tc_fence_before();
  __syncthreads();
  if (tid == 0 && abort_flag) atomicOr(a.err, 2);
  if (warp == kMmaWarp) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
  // no CTA leaves while another may still write to it
  asm volatile("barrier.cluster.arrive.aligned;\n barrier.cluster.wait.aligned;\n" ::: "memory");
}

// Rows of a token: a power of two, at least 4 (more tokens a tile would need more room
// for scores than there is).
int rows_of(int group) {
  int gp = 4;
  while (gp < group) gp *= 2;
  return gp;
}

// Shared memory for operand B, nr row buffers and ns score buffers.
size_t smem_for(int d, int nr, int ns, int tokens, int ranks) {
  return 1024 + (size_t)2 * d / 64 * kN * 128 + (size_t)nr * kN * 2 * d + (size_t)ns * ((tokens + ranks - 1) / ranks) * ranks * kSpan * 4;
}

// False: not a batch for this kernel.
bool shape(const HostPlan &hp, const SelectArgs &a, TcArgs *t, int *ranks) {
  t->gp = rows_of(a.group);
  if (t->gp > kN) return false;
  t->gp_log2 = 0;
  while ((1 << t->gp_log2) < t->gp) ++t->gp_log2;
  t->tile_tokens = kN / t->gp;
  // Eight CTAs a cluster at most, 2,048 scored blocks of the plan's longest request.  At that
  // limit both kernels take the same time (4,096 tokens, 64/4 heads: 2,047 blocks 3,194 us here,
  // 2,050 3,311 token by token, then in proportion: 4,096 6,068, 8,192 11,494).  A replayable
  // plan's bounds decide: 470 blocks under a bound of 2,047 take 1,061 us, of 8,192 1,171.
  *ranks = std::max(1, (a.max_blocks - a.first + kSpan - 1) / kSpan);
  if (*ranks > kMaxRanks) return false;
  constexpr int kChoices[4][2] = {{2, 2}, {1, 2}, {2, 1}, {1, 1}};
  t->nr = 0;
  for (const auto &n : kChoices)
    if (!t->nr && smem_for(hp.prob.head_dim_qk, n[0], n[1], t->tile_tokens, *ranks) <= (size_t)kMaxSmem) {
      t->nr = n[0];
      t->ns = n[1];
    }
  if (!t->nr) return false;
  // Two tokens a request or more, which share its widened bounds however empty their tile
  // (4,000 to 8,000 tokens, blocks of 64, 1,024 tokens x KV heads, us, select.cu against this:
  // 16 heads a group 44 / 69, 44 / 40, 44 / 24 with 1, 2, 4 tokens a request; 64 heads 72 / 103,
  // 70 / 48, 68 / 35), and more than two tokens x KV heads for each SM (one request, 256 tokens
  // x KV heads 12.8 / 17.2, 384 18.0 / 17.2, 512 23.2 / 16.2).
  int64_t tiles = 0, requests = 0;
  const auto &qo = hp.qo_indptr;
  for (size_t b = 0; b + 1 < qo.size(); ++b) {
    tiles += (qo[b + 1] - qo[b] + t->tile_tokens - 1) / t->tile_tokens;
    requests += qo[b + 1] > qo[b];
  }
  const int64_t clusters = std::max(1, hp.num_sms / *ranks);
  if (a.tokens < 2 * requests || (int64_t)a.tokens * a.hkv <= 2 * hp.num_sms) return false;
  // ranges of as many token tiles as give every cluster one
  t->range = (int32_t)std::max<int64_t>(1, (tiles * a.hkv + clusters - 1) / clusters);
  int64_t ranges = 0;
  const int64_t per = (int64_t)t->range * t->tile_tokens;
  for (size_t b = 0; b + 1 < qo.size(); ++b) ranges += (qo[b + 1] - qo[b] + per - 1) / per;
  if (ranges * a.hkv > INT32_MAX) return false;
  t->ranges = (int32_t)ranges;
  return true;
}

template <int D>
cudaError_t launch(const TcArgs &t, int ranks, int num_sms, int device, cudaStream_t st) {
  static SmemLimit limit;
  const cudaError_t e = limit.raise(reinterpret_cast<const void *>(select_tc_kernel<D>), device, kMaxSmem);
  if (e != cudaSuccess) return e;
  const int64_t items = (int64_t)t.ranges * t.s.hkv;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(std::min<int64_t>(items, std::max(1, num_sms / ranks)) * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_for(D, t.nr, t.ns, t.tile_tokens, ranks);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ranks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, select_tc_kernel<D>, t);
}

}  // namespace

int select_tc_ranks(const HostPlan &hp, const SelectArgs &a) {
  TcArgs t{};
  int ranks;
  return shape(hp, a, &t, &ranks) ? ranks : 0;
}

cudaError_t launch_select_tc(const HostPlan &hp, const SelectArgs &a, int device, cudaStream_t st) {
  TcArgs t{};
  int ranks;
  if (!shape(hp, a, &t, &ranks)) return cudaErrorInvalidValue;
  t.s = a;
  return hp.prob.head_dim_qk == kDqk ? launch<kDqk>(t, ranks, hp.num_sms, device, st)
                                     : launch<kDqkSym>(t, ranks, hp.num_sms, device, st);
}

}  // namespace akp
