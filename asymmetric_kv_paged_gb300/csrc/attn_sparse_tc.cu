// attn_run_sparse for chunks of tokens, on tcgen05: neighbouring tokens together over the
// union of their blocks.
//
// Neighbouring queries choose much the same blocks.  A CTA takes up to 2 x (128 / G)
// consecutive tokens of one request and KV head as two Q tiles of 128 rows (token-major,
// G heads a token), walks through the union of their lists in ascending order, 128 keys
// a tile (two blocks of 64, one of 128, or four or eight smaller ones), and leaves out of
// each row's softmax the blocks that its token did not list: their weights are zeros.  A
// Q tile none of whose tokens listed a tile's blocks skips the tile.  What is multiplied
// in vain is bounded by what has to be loaded anyway: a tile's 80 KB take about as long
// from L2 as one Q tile's products with it.
//
// Roles, TMEM and the tile pipeline are those of attn_prefill.cu (512 threads):
//   warps 0-3, 4-7  softmax and epilogue of Q tile 0 / 1 (row p in TMEM lane p)
//   warps 8-11      Q rows; K and V tiles: TMA boxes of the paged cache (bf16), or rows
//                   read by a thread per key, widened to fp16 and stored (8 and 4 bits)
//   warps 12, 13    one thread each issues the MMAs of Q tile 0 / 1
//   warp  14        merges the lists (a token a lane, four in turn) and looks the pages
//                   up, some tiles ahead; a tile's blocks and who listed them go through
//                   a ring of descriptors
//   warp  15        completes the warpgroup
//
// Keys behind the request's end are zeroed in V tiles.  What else a row must not see (a NaN
// or an infinity in a block that only its neighbours listed, or behind its token) could
// still reach it as 0 * NaN: a job with any NaN or infinity in its sums, and one whose lists
// are not ascending, is marked and done again by the kernel of attn_sparse.cu, unit by unit.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>

#include "e2m1.cuh"
#include "kernels.hpp"
#include "sparse_attn.cuh"
#include "tc_common.cuh"

namespace akp {
namespace {

constexpr int kPN = 128;                      // keys of a tile
constexpr int kPM = kSparseTileRows;          // rows of a Q tile (MMA M)
constexpr int kMmaWarp = 12, kMergeWarp = 14;
constexpr int kPThreads = 16 * 32;
constexpr int kTileBlk = 128 * 128;           // one 64-column block of a 128-row tile: 16 KB
constexpr int kVStage = 2 * kTileBlk;
constexpr uint32_t kTmemCols = 512, kTmemO = 256;
constexpr int kDescs = 6;                     // descriptors in the ring
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGrow = 8.0f;                 // base-2 growth of a maximum before O is rescaled

template <int DQK>
struct Lay {
  static constexpr int kQTile = DQK / 64 * kTileBlk, kKStage = DQK / 64 * kTileBlk;
  static constexpr int kOffK = 2 * kQTile, kOffV = kOffK + 2 * kKStage;
  static constexpr int kSmem = kOffV + kVStage + 1024;     // + room to align the base to 1024 B
  static_assert(kSmem + 2048 <= 227 * 1024, "shared memory layout too large");
};

// A tile: its pieces (blocks) in order.
struct TileDesc {
  int32_t key0[8], slot[8];        // first key, first slot (the pool's size: read as zeros)
  uint32_t tokens[8][4];           // the job's tokens that listed it
  int32_t tiles;                   // bit t: some token of Q tile t did
  int32_t end;                     // no tile: the list has ended
  int32_t edge;                    // keys that not every token of the job is past
  int32_t pad;
};

struct Bars {
  uint64_t desc_full[kDescs], desc_empty[kDescs];
  uint64_t k_full[2], k_empty[2], v_full, v_empty, v_edge, q_full;
  uint64_t s_full[2], p_hi[2], p_full[2], pv_done[2], done[2];
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

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2,
                                            uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(tc::smem_u32(bar))
      : "memory");
}

// The power of two that a query row is multiplied by on its way to fp16 (attn_prefill.cu).
template <int DQK>
__device__ __forceinline__ int q_row_shift(const uint4 *row) {
  uint32_t e = 0;
#pragma unroll 1
  for (int c0 = 0; c0 < DQK / 8; c0 += 8) {
    uint4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = __ldg(row + c0 + u);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) e = max(e, max((w[q] >> 7) & 0xFFu, (w[q] >> 23) & 0xFFu));
    }
  }
  return min(141 - (int)e, 126);
}

template <int KV, int DQK>
__global__ void __launch_bounds__(kPThreads, 1)
    sparse_tc_kernel(const SparseArgs a, const __grid_constant__ TmaMaps maps) {
  constexpr bool F16 = KV != ATTN_KV_BF16, E2M1 = KV == ATTN_KV_FP4_E2M1;
  constexpr float kLift = F16 ? 7.f : 0.f;
  using Y = Lay<DQK>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
  __shared__ Bars bars;
  __shared__ TileDesc descs[kDescs];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag, odd_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const int job = blockIdx.x;
  SparseJob x;
  if (!find_job(a, job, x, warp == 0)) {
    if (tid == 0) {
      atomicOr(a.err, 4);                          // a layout of fewer tokens
      a.redo[job] = 0;
    }
    return;
  }
  // the lists are ascending, their empty entries last, none past the token's own block
  bool bad_list = false;
  for (int i = tid; i < x.ntok * a.take; i += kPThreads) {
    const int tt = i / a.take, k = i % a.take;
    const int32_t *list = a.block_idx + ((int64_t)(x.tok0 + tt) * a.hkv + x.g) * a.take;
    const int c = __ldg(list + k), next = k + 1 < a.take ? __ldg(list + k + 1) : -1;
    bad_list |= (next >= 0 && (c < 0 || next <= c)) || c > (x.pos0 + tt) / a.block;
  }
  if (tid == 0) {
    abort_flag = odd_flag = 0;
    for (int i = 0; i < kDescs; ++i) {
      tc::mbar_init(&bars.desc_full[i], 1);
      tc::mbar_init(&bars.desc_empty[i], 14);     // softmax, load and issuing warps
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&bars.k_full[i], F16 ? 4 : 1);
      tc::mbar_init(&bars.k_empty[i], 2);
      tc::mbar_init(&bars.s_full[i], 1);
      tc::mbar_init(&bars.p_hi[i], 4);
      tc::mbar_init(&bars.p_full[i], 4);
      tc::mbar_init(&bars.pv_done[i], 1);
      tc::mbar_init(&bars.done[i], 1);
    }
    tc::mbar_init(&bars.v_full, 4);
    tc::mbar_init(&bars.v_empty, 2);
    tc::mbar_init(&bars.v_edge, 1);
    tc::mbar_init(&bars.q_full, 4);
    tc::fence_mbar_init();
  }
  if (__syncthreads_or(bad_list)) {                // left to the other kernel
    if (tid == 0) a.redo[job] = 1;
    return;
  }
  if (warp == kMmaWarp) tc::tmem_alloc(&tmem_slot, kTmemCols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = tmem_slot, sbase = tc::smem_u32(smem);
  const int tile_tokens = a.job_tokens / 2;
  const int num_slots = a.num_pages * a.page_size;
  auto wait = [&](uint64_t *bar, uint32_t parity) { return tc::mbar_wait_warp(bar, parity, &abort_flag); };
  auto desc_wait = [&](int k) { return wait(&bars.desc_full[k % kDescs], (k / kDescs) & 1); };
  auto desc_done = [&](int k) { tc::mbar_arrive_warp(&bars.desc_empty[k % kDescs]); };

  // Registers per warpgroup as in attn_prefill.cu: 168 + 168 + 120 + 56 = 4 x 128.
  if (warp >= 8 && warp < kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 120;\n" ::: "memory");
    // ------------------------------------------------------------ load warps
    const int lt = tid - 256;
    // Q rows: row p of Q tile t is head p % G of token t * tile_tokens + p / G; others zero
#pragma unroll 1
    for (int rr = 0; rr < 2; ++rr) {
      const int tt = rr * tile_tokens + lt / a.group;
      const bool live = lt / a.group < tile_tokens && tt < x.ntok;
      const uint4 *src = reinterpret_cast<const uint4 *>(
          a.q + ((int64_t)(x.tok0 + (live ? tt : 0)) * a.hq + x.g * a.group + lt % a.group) * DQK);
      const float f = F16 ? __int_as_float(((live ? q_row_shift<DQK>(src) : 0) + 127) << 23) : 1.f;
#pragma unroll 1
      for (int c0 = 0; c0 < DQK / 8; c0 += 8) {
        uint4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = live ? __ldg(src + c0 + u) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          uint32_t h[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
          if (F16)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              h[q] = pair16<false>(__uint_as_float(h[q] << 16) * f, __uint_as_float(h[q] & 0xFFFF0000u) * f);
          *reinterpret_cast<uint4 *>(smem + rr * Y::kQTile + (c0 >> 3) * kTileBlk + tc::sw128_offset(lt, u)) =
              make_uint4(h[0], h[1], h[2], h[3]);
        }
      }
    }
    tc::fence_proxy_async_smem();
    tc::mbar_arrive_warp(&bars.q_full);

    if constexpr (F16) {
      // Thread `lt` owns that key of every tile; the K stream runs one tile ahead of the V
      // stream (attn_prefill.cu).
      constexpr int KCH = E2M1 ? e2m1_row_bytes(DQK) / 16 : DQK / 16;
      constexpr int VCH = E2M1 ? e2m1_row_bytes(kDv) / 16 : kDv / 16;
      const uint8_t *kc = static_cast<const uint8_t *>(a.k_cache), *vc = static_cast<const uint8_t *>(a.v_cache);
      auto put_row = [&](uint32_t base, const uint4 *src, int n) {
        auto put = [&](int ch, uint4 v) {
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(
                           base + (ch >> 3) * kTileBlk + tc::sw128_offset(lt, ch & 7)),
                       "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                       : "memory");
        };
        if constexpr (E2M1) {
          const uint32_t sc[4] = {src[n - 1].x, src[n - 1].y, src[n - 1].z, src[n - 1].w};
#pragma unroll
          for (int i = 0; i + 1 < n; ++i) {
            uint4 w[4];
            e2m1x32_to_f16(src[i], i & 1 ? sc[i >> 1] >> 16 : sc[i >> 1], w);
#pragma unroll
            for (int u = 0; u < 4; ++u) put(4 * i + u, w[u]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < n; ++i) {
            uint4 lo, hi;
            e4m3x16_to_f16(src[i], lo, hi);
            put(2 * i, lo);
            put(2 * i + 1, hi);
          }
        }
      };
      // the thread's slot in tile k: -1 read as zeros; false: the list has ended
      auto next = [&](int k, int64_t &slot, bool &more) -> bool {
        if (!desc_wait(k)) return false;
        const TileDesc &d = descs[k % kDescs];
        more = !d.end;
        const int p = lt / a.block, in = lt % a.block;
        const int s = d.slot[p];
        slot = s < num_slots && d.key0[p] + in < x.len ? s + in : -1;
        desc_done(k);
        return true;
      };
      uint4 kr[KCH], vr[VCH];
      auto load = [&](uint4 *dst, int n, const uint8_t *cache, int64_t slot) {
        const uint4 *row = reinterpret_cast<const uint4 *>(cache) + ((slot >= 0 ? slot : 0) * a.hkv + x.g) * n;
#pragma unroll
        for (int i = 0; i < n; ++i) dst[i] = slot >= 0 ? __ldg(row + i) : make_uint4(0u, 0u, 0u, 0u);
      };
      int64_t slot = -1;
      bool more = false, ok = next(0, slot, more);
      if (ok && more) load(kr, KCH, kc, slot);
      for (int k = 0; ok; ++k) {
        int64_t v_slot = -1;
        const bool here = more;
        if (here) {
          const int s = k & 1;
          if (k >= 2 && !(ok = wait(&bars.k_empty[s], ((k >> 1) - 1) & 1))) break;
          put_row(sbase + Y::kOffK + s * Y::kKStage, kr, KCH);
          tc::fence_proxy_async_smem();
          tc::mbar_arrive_warp(&bars.k_full[s]);
          v_slot = slot;
          if (!(ok = next(k + 1, slot, more))) break;
          if (more) load(kr, KCH, kc, slot);
        }
        if (k >= 1) {
          if (k >= 2 && !(ok = wait(&bars.v_empty, (k - 2) & 1))) break;
          put_row(sbase + Y::kOffV, vr, VCH);
          tc::fence_proxy_async_smem();
          tc::mbar_arrive_warp(&bars.v_full);
        }
        if (!here) break;
        load(vr, VCH, vc, v_slot);
      }
    } else {
      // Boxes of `rows` keys x 64 columns; lane i of warp 8 issues box i % nb of column block
      // i / nb.
      const int rows = min(a.block, 64), nb = kPN / rows;
      const int col = lane / nb, box = lane % nb;
      int v_slot = 0, dead = 0, v_dead = 0, v_tail = 0;
      bool ok = true;
      int issued_v = 0, issued_k = 0, edges = 0;
      for (int k = 0; ok; ++k) {
        if (!(ok = desc_wait(k))) break;
        const TileDesc &d = descs[k % kDescs];
        const bool more = !d.end;
        const int at = box * rows, p = at / a.block;
        const int slot = d.slot[p] + at % a.block;
        // the thread's key lies behind the request's end; does any key of the tile?
        dead = d.key0[lt / a.block] + lt % a.block >= x.len;
        int tail = 0;
        if (d.edge)
          for (int i = 0; i < kPN / a.block; ++i) tail |= d.key0[i] + a.block > x.len;
        desc_done(k);
        if (more && warp == 8) {
          const int s = k & 1;
          if (k >= 2 && !(ok = wait(&bars.k_empty[s], ((k >> 1) - 1) & 1))) break;
          if (lane == 0) tc::mbar_arrive_expect_tx(&bars.k_full[s], Y::kKStage);
          __syncwarp();
          if (col < DQK / 64)
            tma_load_3d(sbase + Y::kOffK + s * Y::kKStage + col * kTileBlk + box * rows * 128, &maps.k, 64 * col, x.g,
                        slot, &bars.k_full[s]);
          __syncwarp();
          ++issued_k;
        }
        if (k >= 1) {
          if (k >= 2 && !(ok = wait(&bars.v_empty, (k - 2) & 1))) break;
          uint64_t *bar = v_tail ? &bars.v_edge : &bars.v_full;
          if (warp == 8) {
            if (lane == 0) tc::mbar_arrive_expect_tx(bar, kVStage);
            __syncwarp();
            if (col < kDv / 64)
              tma_load_3d(sbase + Y::kOffV + col * kTileBlk + box * rows * 128, &maps.v, 64 * col, x.g, v_slot, bar);
            __syncwarp();
            ++issued_v;
          }
          if (v_tail) {                            // zeros behind the request's end
            if (!(ok = wait(&bars.v_edge, edges & 1))) break;
            if (v_dead)
#pragma unroll
              for (int ch = 0; ch < kDv / 8; ++ch)
                *reinterpret_cast<uint4 *>(smem + Y::kOffV + (ch >> 3) * kTileBlk + tc::sw128_offset(lt, ch & 7)) =
                    make_uint4(0u, 0u, 0u, 0u);
            tc::fence_proxy_async_smem();
            tc::mbar_arrive_warp(&bars.v_full);
          } else if (warp != 8) {
            tc::mbar_arrive_warp(&bars.v_full);
          }
          edges += v_tail;
        }
        if (!more) break;
        v_slot = slot;
        v_dead = dead;
        v_tail = tail;
      }
      if (abort_flag && warp == 8) {               // the copies in flight land before the CTA ends
        int no_abort = 0;
        for (int i = max(0, issued_k - 2); i < issued_k; ++i)
          tc::mbar_wait(&bars.k_full[i & 1], (i >> 1) & 1, &no_abort, 100000000ull);
        if (issued_v > 0) {
          if (v_tail)
            tc::mbar_wait(&bars.v_edge, (edges > 0 ? edges - 1 : 0) & 1, &no_abort, 100000000ull);
          else
            tc::mbar_wait(&bars.v_full, (issued_v - 1) & 1, &no_abort, 100000000ull);
        }
      }
    }
  } else if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;\n" ::: "memory");
    if (warp == kMergeWarp) {
      // ------------------------------------------------------------ the union of the lists
      const int pieces = kPN / a.block, per_page = a.page_size / a.block;
      // lane: tokens lane, lane + 32, ..; the entry at hand and the one behind it
      const int32_t *next_at[4];
      int left[4];
      uint32_t cur[4], ahead[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tt = lane + 32 * i;
        next_at[i] = a.block_idx + ((int64_t)(x.tok0 + tt) * a.hkv + x.g) * a.take;
        left[i] = tt < x.ntok ? a.take : 0;
        auto take = [&]() -> uint32_t {
          if (left[i] <= 0) return 0xFFFFFFFFu;
          --left[i];
          return (uint32_t)__ldg(next_at[i]++);    // (an empty entry is the largest)
        };
        cur[i] = take();
        ahead[i] = take();
      }
      bool ok = true, more = true;
      for (int k = 0; more && ok; ++k) {
        uint32_t block = 0xFFFFFFFFu, who[4] = {0u, 0u, 0u, 0u};
        int found = 0;
        for (int s = 0; s < pieces; ++s) {
          const uint32_t least =
              __reduce_min_sync(0xffffffffu, min(min(cur[0], cur[1]), min(cur[2], cur[3])));
          if ((int32_t)least < 0) break;
          uint32_t m[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool has = cur[i] == least;
            m[i] = __ballot_sync(0xffffffffu, has);
            if (has) {
              cur[i] = ahead[i];
              ahead[i] = 0xFFFFFFFFu;
              if (left[i] > 0) {
                --left[i];
                ahead[i] = (uint32_t)__ldg(next_at[i]++);
              }
            }
          }
          if (lane == s) {
            block = least;
#pragma unroll
            for (int i = 0; i < 4; ++i) who[i] = m[i];
          }
          ++found;
        }
        more = found > 0;
        int slot = num_slots;
        const int key0 = lane < found ? (int)block * a.block : 0;
        if (lane < found) {
          const int32_t page = __ldg(a.page_table + (int64_t)x.b * a.pt_stride + (int)block / per_page);
          if (page >= 0 && page < a.num_pages)
            slot = page * a.page_size + (int)block % per_page * a.block;
          else
            atomicOr(a.err, 1);
        }
        // Q tile 0: tokens below tile_tokens
        uint32_t tiles = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int cut = min(32, max(0, tile_tokens - 32 * i));
          const uint32_t low = cut == 32 ? 0xFFFFFFFFu : (1u << cut) - 1u;
          tiles |= (who[i] & low ? 1u : 0u) | (who[i] & ~low ? 2u : 0u);
        }
        tiles = __reduce_or_sync(0xffffffffu, tiles);
        const bool edge = __any_sync(0xffffffffu, lane < found && key0 + a.block - 1 > x.pos0);
        if (k >= kDescs && !(ok = wait(&bars.desc_empty[k % kDescs], (k / kDescs - 1) & 1))) break;
        TileDesc &d = descs[k % kDescs];
        if (lane < 8) {
          d.key0[lane] = key0;
          d.slot[lane] = slot;
#pragma unroll
          for (int i = 0; i < 4; ++i) d.tokens[lane][i] = who[i];
        }
        if (lane == 0) {
          d.tiles = (int)tiles;
          d.end = !more;
          d.edge = edge;
        }
        tc::mbar_arrive_warp(&bars.desc_full[k % kDescs]);
      }
    } else if (warp < kMergeWarp) {
      // ------------------------------------------------------------ MMA issuers
      const int t = warp - kMmaWarp;
      const uint32_t id_s = tc::idesc_f16(F16 ? 0 : 1, 0, 0, kPM, kPN), id_pv = tc::idesc_f16(F16 ? 0 : 1, 0, 1, kPM, kDv);
      const uint32_t q_smem = sbase + t * Y::kQTile, s_tmem = tmem + kPN * t, o_tmem = tmem + kTmemO + kDv * t;
      int c = 0;                                   // tiles of this Q tile so far
      bool ok = wait(&bars.q_full, 0);
      for (int k = 0; ok; ++k) {
        if (!(ok = desc_wait(k))) break;
        const bool end = descs[k % kDescs].end != 0, mine = descs[k % kDescs].tiles >> t & 1;
        desc_done(k);
        if (end) break;
        const int s = k & 1;
        if (!(ok = wait(&bars.k_full[s], (k >> 1) & 1))) break;
        if (lane == 0) {
          if (mine) {
            tc::tc_fence_after();
#pragma unroll
            for (int kq = 0; kq < DQK / 16; ++kq) {
              const uint32_t off = (kq & 3) * 32 + (kq >> 2) * kTileBlk;
              const uint64_t ad = tc::smem_desc_sw128(q_smem + off, 16, 1024);
              const uint64_t bd = tc::smem_desc_sw128(sbase + Y::kOffK + s * Y::kKStage + off, 16, 1024);
              tc::mma_f16_ss(s_tmem, ad, bd, id_s, kq > 0 ? 1u : 0u);
            }
            tc::mma_commit(&bars.s_full[t]);
          }
          tc::mma_commit(&bars.k_empty[s]);
        }
        __syncwarp();
        if (!(ok = wait(&bars.v_full, k & 1))) break;
        if (mine) {
          auto pv = [&](int kk, bool acc) {
            const uint64_t bd = tc::smem_desc_sw128(sbase + Y::kOffV + kk * 16 * 128, kTileBlk, 1024);
            tc::mma_f16_ts(o_tmem, s_tmem + kPN / 2 + kk * 8, bd, id_pv, acc ? 1u : 0u);
          };
          if (!(ok = wait(&bars.p_hi[t], c & 1))) break;
          if (lane == 0) {
            tc::tc_fence_after();
#pragma unroll
            for (int kk = kPN / 32; kk < kPN / 16; ++kk) pv(kk, c > 0 || kk > kPN / 32);
          }
          __syncwarp();
          if (!(ok = wait(&bars.p_full[t], c & 1))) break;
          if (lane == 0) {
            tc::tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < kPN / 32; ++kk) pv(kk, true);
            tc::mma_commit(&bars.pv_done[t]);
          }
          __syncwarp();
          ++c;
        }
        if (lane == 0) tc::mma_commit(&bars.v_empty);
        __syncwarp();
      }
      if (lane == 0) {                             // every MMA is complete before TMEM goes back
        tc::mma_commit(&bars.done[t]);
        int no_abort = 0;
        tc::mbar_wait(&bars.done[t], 0, &no_abort, 100000000ull);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 168;\n" ::: "memory");
    // ------------------------------------------------------------ softmax + epilogue
    const int t = warp >> 2, wq = warp & 3;
    const int p = wq * 32 + lane;                  // row of the Q tile, TMEM lane
    const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
    const uint32_t s_addr = tmem + lane_base + kPN * t, o_addr = tmem + lane_base + kTmemO + kDv * t;
    const int tt = t * tile_tokens + p / a.group;
    const bool valid = p / a.group < tile_tokens && tt < x.ntok;
    const int head = x.g * a.group + p % a.group;
    const int pos = valid ? x.pos0 + tt : -1;
    const uint32_t bit = valid ? 1u << (tt & 31) : 0u;
    float sc = a.scale_log2;
    if (F16 && valid)
      sc = tc::row_score_scale(a.scale_log2,
                               q_row_shift<DQK>(reinterpret_cast<const uint4 *>(
                                   a.q + ((int64_t)(x.tok0 + tt) * a.hq + head) * DQK)));
    const int block_log2 = 31 - __clz(a.block);
    float m_run = -INFINITY, l_run = 0.f;
    int c = 0;
    bool ok = true;
    for (int k = 0;; ++k) {
      if (!(ok = desc_wait(k))) break;
      const TileDesc &d = descs[k % kDescs];
      const bool end = d.end != 0, mine = d.tiles >> t & 1, edge = d.edge != 0;
      // the eight groups of 16 keys: a bit each if listed, and (edge) how many keys are seen
      uint32_t sel = 0u, lim[2] = {0u, 0u};
      if (mine && !end) {
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const int pc = (g * 16) >> block_log2;
          if (d.tokens[pc][(tt >> 5) & 3] & bit) {
            sel |= 1u << g;
            if (edge) lim[g >> 2] |= (uint32_t)min(16, max(0, pos + 1 - d.key0[pc] - ((g * 16) & (a.block - 1)))) << (8 * (g & 3));
          }
        }
      }
      desc_done(k);
      if (end) break;
      if (!mine) continue;
      if (!(ok = wait(&bars.s_full[t], c & 1))) break;
      tc::tc_fence_after();
      uint32_t s[4][32];
      tc::tmem_ld32(s_addr, s[0]);
      tc::tmem_ld32(s_addr + 32, s[1]);
      tc::tmem_ld32(s_addr + 64, s[2]);
      tc::tmem_ld32(s_addr + 96, s[3]);
      tc::tmem_wait_ld_regs64(s[0], s[1]);
      tc::tmem_wait_ld_regs64(s[2], s[3]);
      if (edge) {
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const int n = (int)(lim[g >> 2] >> (8 * (g & 3)) & 31u);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            uint32_t &v = s[g >> 1][16 * (g & 1) + j];
            v = j < n ? v : 0xFF800000u;
          }
        }
      }
      // the listed groups' maximum
      float mx = -INFINITY;
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const uint32_t *v = &s[g >> 1][16 * (g & 1) + j];
          m0 = tc::max3(m0, __uint_as_float(v[0]), __uint_as_float(v[1]));
          m1 = tc::max3(m1, __uint_as_float(v[2]), __uint_as_float(v[3]));
        }
        if (sel >> g & 1u) mx = tc::max3(mx, m0, m1);
      }
      const float m_tile = mx * sc;
      const bool need = m_tile > m_run + kGrow;    // also from -inf
      if (__any_sync(0xffffffffu, need)) {
        const bool rescale = need && m_run != -INFINITY;
        if (__any_sync(0xffffffffu, rescale)) {
          if (!(ok = wait(&bars.pv_done[t], (c - 1) & 1))) break;
          tc::tc_fence_after();
          const float alpha = rescale ? ex2(m_run - m_tile) : 1.f;
#pragma unroll 1
          for (int q = 0; q < kDv / 16; ++q) {
            uint32_t o[16];
            tc::tmem_ld16(o_addr + q * 16, o);
            tc::tmem_wait_ld_regs(o);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
            tc::tmem_st16(o_addr + q * 16, o);
          }
          tc::tmem_wait_st();
          l_run *= alpha;
        }
        if (need) m_run = m_tile;
      }
      // P: key j's 16-bit value in the low or high half of column 64 + j / 2 of S; keys 64-127
      // first.  A group that the row's token did not list gets zeros.
      const float off = m_run == -INFINITY ? 0.f : kLift - m_run;
      float rs[2] = {0.f, 0.f};
#pragma unroll
      for (int half = 1; half >= 0; --half) {
        const bool any = __any_sync(0xffffffffu, (sel >> (4 * half) & 15u) != 0u);
#pragma unroll
        for (int g = 4 * half; g < 4 * half + 4; ++g) {
          uint32_t pk[8];
          if (any) {
            const float og = sel >> g & 1u ? off : -INFINITY;
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const uint32_t *v = &s[g >> 1][16 * (g & 1) + j];
              float y0, y1;
              tc::ffma2(y0, y1, __uint_as_float(v[0]), __uint_as_float(v[1]), sc, og);
              const float p0 = ex2(y0), p1 = ex2(y1);
              tc::fadd2(rs[0], rs[1], p0, p1);
              pk[j >> 1] = pair16<!F16>(p0, p1);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) pk[j] = 0u;
          }
          tc::tmem_st8(s_addr + kPN / 2 + 8 * g, pk);
        }
        tc::tmem_wait_st();
        tc::tc_fence_before();
        tc::mbar_arrive_warp(half ? &bars.p_hi[t] : &bars.p_full[t]);
      }
      l_run += rs[0] + rs[1];
      ++c;
    }
    // ---------------- normalise and write the rows
    if (ok && c > 0) ok = wait(&bars.pv_done[t], (c - 1) & 1);
    if (ok) {
      tc::tc_fence_after();
      float lse;
      const float sink2 = a.sinks && valid ? __ldg(a.sinks + head) * kLog2e : -INFINITY;
      const float f = finish(m_run, l_run, kLift, sink2, a.v_scale, lse);
      bool odd = l_run != l_run;
      uint16_t *row = a.out + ((int64_t)(x.tok0 + (valid ? tt : 0)) * a.hq + head) * kDv;
#pragma unroll 1
      for (int q = 0; q < kDv / 32; ++q) {
        uint32_t o[32];
        if (c > 0) {
          tc::tmem_ld32(o_addr + q * 32, o);
          tc::tmem_wait_ld_regs32(o);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = 0u;
        }
        if (!valid) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float v0 = __uint_as_float(o[8 * e + 2 * j]), v1 = __uint_as_float(o[8 * e + 2 * j + 1]);
            odd |= !(fabsf(v0) < INFINITY) | !(fabsf(v1) < INFINITY);
            w[j] = pair16<true>(v0 * f, v1 * f);
          }
          reinterpret_cast<uint4 *>(row + q * 32)[e] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      if (valid && a.lse) a.lse[(int64_t)(x.tok0 + tt) * a.hq + head] = lse;
      if (valid && odd) odd_flag = 1;
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (tid == 0) {
    if (abort_flag) atomicOr(a.err, 2);
    a.redo[job] = odd_flag;
  }
  if (warp == kMmaWarp) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

template <int KV, int DQK>
cudaError_t launch_one(const SparseArgs &a, const TmaMaps &maps, int device, cudaStream_t st) {
  static SmemLimit limit;
  const cudaError_t e = limit.raise(reinterpret_cast<const void *>(sparse_tc_kernel<KV, DQK>), device, Lay<DQK>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_dependent(sparse_tc_kernel<KV, DQK>, dim3((unsigned)a.jobs), dim3(kPThreads), Lay<DQK>::kSmem, st, a,
                          maps);
}

template <int DQK>
cudaError_t launch_kv(int kv, const SparseArgs &a, const TmaMaps &maps, int device, cudaStream_t st) {
  switch (kv) {
    case ATTN_KV_BF16: return launch_one<ATTN_KV_BF16, DQK>(a, maps, device, st);
    case ATTN_KV_FP8_E4M3: return launch_one<ATTN_KV_FP8_E4M3, DQK>(a, maps, device, st);
    default: return launch_one<ATTN_KV_FP4_E2M1, DQK>(a, maps, device, st);
  }
}

}  // namespace

cudaError_t launch_sparse_tc(const HostPlan &hp, const SparseArgs &a, const TmaMaps &maps, int device,
                             cudaStream_t st) {
  return hp.prob.head_dim_qk == kDqk ? launch_kv<kDqk>(hp.prob.kv_dtype, a, maps, device, st)
                                     : launch_kv<kDqkSym>(hp.prob.kv_dtype, a, maps, device, st);
}

}  // namespace akp
