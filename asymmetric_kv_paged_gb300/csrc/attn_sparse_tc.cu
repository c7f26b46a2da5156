// attn_run_sparse for chunks of tokens, on tcgen05: neighbouring tokens together over the
// union of their blocks.
//
// Neighbouring queries choose much the same blocks.  A CTA takes up to 128 / G consecutive
// tokens of one request and KV head as a Q tile of 128 rows (token-major, G heads a
// token), walks through the union of their lists in ascending order, 128 keys a tile (two
// blocks of 64, one of 128, or four or eight smaller ones), and leaves out of each row's
// softmax the blocks that its token did not list: their weights are zeros.  Multiplied in
// vain is what the union has beyond a token's own list (2.8 times its length on the case
// below), while a block is loaded once for all that listed it.
//
// One chain S = Q.K^T, softmax, O += P.V spends most of its time waiting for its own parts.
// Two chains share the Q tile: tile k belongs to chain k % 2, which has K and V buffers, S,
// O and running maxima and sums of its own (the TMEM is full: 2 x 128 columns of S, 2 x 128
// of O); at the end the two are merged, each chain's warps writing half the columns.  (Two
// Q tiles of 128 rows on one chain each, over the union of all 256 rows' blocks as in
// attn_prefill.cu, took 531 us on the case below: 96 KB of Q leave no room for the tiles
// that only one of the two needs.)
//
// 4096 tokens behind 26,000 (64/4 heads, 16 blocks of 64, bf16) take 485 us, with every unit
// by itself (attn_sparse.cu) 1,870, with eight neighbouring units of register operands a CTA
// 822; dense attention of the same chunk takes about 3 ms.  That is with lists that stay alike
// for 16 tokens, from a job's first token on (43 blocks a job); shifted by 4 tokens (52 blocks)
// it takes 546, with lists independent from token to token (97) 886.  The 172 GFLOP of the
// listed keys would be 89 us at the tensor cores' rate.  A chain needs 4.4 thousand cycles a tile, half a tile's time as there are two: 12 + 8 MMAs of 66 cycles, 1.9
// thousand cycles of softmax and the hand-offs between them; 10 of a CTA's 65 thousand cycles
// pass before its first tile and 5 behind its last.  Two threads a row for the softmax gave
// 479 us (of 481 then), a persistent form 504, spinning waits 495: the hand-offs remain, and no room in
// shared memory or TMEM for a third chain.  4-bit caches (3 x 777 tokens, 12 blocks of 128):
// 435 us, unit by unit 2,810; there the widening of a tile by four warps is the chain's longest part.
//
// Roles (512 threads; the tile pipeline is that of attn_prefill.cu):
//   warps 0-3, 4-7  Q rows, then softmax and epilogue of chain 0 / 1 (row p in TMEM lane p)
//   warps 8-11      widen the tiles of 8- and 4-bit caches to fp16, in place (the raw rows
//                   arrive in the operand's own buffer, which they fill a half or a quarter);
//                   zeros behind the request's end; whether the lists are ascending
//   warps 12, 13    one thread each issues the MMAs of chain 0 / 1
//   warp  14        merges the lists (a token a lane, two in turn) and looks the pages up,
//                   some tiles ahead; a tile's blocks and who listed them go through a ring
//                   of descriptors
//   warp  15        issues the tiles' TMA boxes (of the paged cache itself)
//
// Keys behind the request's end are zeroed in V tiles.  What else a row must not see (a NaN
// or an infinity in a block that only its neighbours listed, or behind its token) could
// still reach it as 0 * NaN: rows with a NaN or an infinity in their sums are marked (so is
// the job) and done again by the kernel of attn_sparse.cu, unit by unit.  Lists in any other order are searched
// for their next entry instead of read on: the same tiles, the same bits.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "e2m1.cuh"
#include "kernels.hpp"
#include "sparse_attn.cuh"
#include "tc_common.cuh"

namespace akp {
namespace {

constexpr int kPN = 128;                      // keys of a tile
constexpr int kPM = kSparseTileRows;          // rows of a Q tile (MMA M)
constexpr int kMmaWarp = 12, kMergeWarp = 14;
constexpr int kPThreads = 16 * 32, kLoadThreads = 128;
constexpr int kTileBlk = 128 * 128;           // one 64-column block of a 128-row tile: 16 KB
constexpr int kVStage = 2 * kTileBlk;
constexpr uint32_t kTmemCols = 512, kTmemO = 256;
constexpr int kDescs = 8;                     // descriptors in the ring
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGrow = 8.0f;                 // base-2 growth of a maximum before O is rescaled

template <int DQK>
struct Lay {
  static constexpr int kQTile = DQK / 64 * kTileBlk, kKStage = DQK / 64 * kTileBlk;
  static constexpr int kOffK = kQTile, kOffV = kOffK + 2 * kKStage;
  static constexpr int kSmem = kOffV + 2 * kVStage + 1024;     // + room to align the base to 1024 B
  static_assert(kSmem + 2048 <= 227 * 1024, "shared memory layout too large");
};

// A tile: its pieces (blocks) in order.
struct TileDesc {
  int32_t key0[8], slot[8];        // first key, first slot (the pool's size: read as zeros)
  uint8_t listed[64];              // of every token of the job, a bit per 16 keys: listed
  int32_t end;                     // no tile: the list has ended
  int32_t edge;                    // bit 0: keys that not every token of the job is past; bit 1: behind the end
};

struct Bars {
  uint64_t desc_full[kDescs], desc_empty[kDescs];
  uint64_t k_raw[2], k_full[2], k_empty[2], v_raw[2], v_full[2], v_empty[2], load, checked, q_full, merge;
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
  __shared__ int abort_flag, odd_flag, mixed_flag;
  __shared__ float row_sc[kPM], row_m[2][kPM], row_l[2][kPM];     // the rows' score scales, the chains' results
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
  if (warp < 8) {
    // The query rows into the operand tile, 16 a warp, 16 bytes a lane: row r is head r % G of
    // token r / G; others zeros.  (Rolled, as asynchronous copies: a CTA runs this once, and
    // unrolled its time was the fetching of its code.)
    uint8_t *mine = smem + (lane >> 3) * kTileBlk;
    int tt = warp * 16 / a.group, h = warp * 16 % a.group;
#pragma unroll 1
    for (int r = warp * 16; r < warp * 16 + 16; ++r) {
      const bool live = tt < x.ntok;
      const uint16_t *src =
          a.q + ((int64_t)(x.tok0 + (live ? tt : 0)) * a.hq + x.g * a.group + (live ? h : 0)) * DQK + lane * 8;
      if (lane < DQK / 8)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(
                         tc::smem_u32(mine + tc::sw128_offset(r, lane & 7))),
                     "l"(src), "r"(live ? 16 : 0)
                     : "memory");
      if (++h == a.group) {
        h = 0;
        ++tt;
      }
    }
  }
  if (tid == 0) {
    abort_flag = odd_flag = mixed_flag = 0;
    for (int i = 0; i < kDescs; ++i) {
      tc::mbar_init(&bars.desc_full[i], 1);
      tc::mbar_init(&bars.desc_empty[i], 10);     // warps that read it: the loading ones, the chain's
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&bars.k_raw[i], 1);
      tc::mbar_init(&bars.v_raw[i], 1);
      tc::mbar_init(&bars.k_full[i], F16 ? 4 : 1);
      tc::mbar_init(&bars.k_empty[i], 1);
      tc::mbar_init(&bars.v_full[i], 4);
      tc::mbar_init(&bars.v_empty[i], 1);
      tc::mbar_init(&bars.s_full[i], 1);
      tc::mbar_init(&bars.p_hi[i], 4);
      tc::mbar_init(&bars.p_full[i], 4);
      tc::mbar_init(&bars.pv_done[i], 1);
      tc::mbar_init(&bars.done[i], 1);
    }
    tc::mbar_init(&bars.merge, 8);
    tc::mbar_init(&bars.load, 4);
    tc::mbar_init(&bars.checked, 4);
    tc::mbar_init(&bars.q_full, 8);
    tc::fence_mbar_init();
  }
  if (warp == kMmaWarp) tc::tmem_alloc(&tmem_slot, kTmemCols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = tmem_slot, sbase = tc::smem_u32(smem);
  const int num_slots = a.num_pages * a.page_size;
  auto wait = [&](uint64_t *bar, uint32_t parity) { return tc::mbar_wait_warp(bar, parity, &abort_flag); };
  auto desc_wait = [&](int k) { return wait(&bars.desc_full[k % kDescs], (k / kDescs) & 1); };
  auto desc_done = [&](int k) { tc::mbar_arrive_warp(&bars.desc_empty[k % kDescs]); };

  if (warp >= 8 && warp < kMmaWarp) {
    // ------------------------------------------------------------ load warps
    const int lt = tid - 256;
    // Are the lists ascending, their empty entries last, none past the token's own block?
    {
      // (a token a warp, the entries of up to eight tokens on their way together)
      bool mixed = false, past = false;
      const int lw = lt >> 5, blk = 31 - __clz(a.block);
      for (int e0 = 0; e0 < a.take; e0 += 32) {
        const int e = e0 + lane;
        const int32_t *list = a.block_idx + ((int64_t)(x.tok0 + lw) * a.hkv + x.g) * a.take + e;
#pragma unroll 1
        for (int t0 = lw; t0 < x.ntok; t0 += 32) {
          int c[8], next[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const bool in = t0 + 4 * i < x.ntok;
            c[i] = in && e < a.take ? __ldg(list) : -1;
            next[i] = in && e + 1 < a.take ? __ldg(list + 1) : -1;
            list += (int64_t)4 * a.hkv * a.take;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            past |= c[i] > (x.pos0 + t0 + 4 * i) >> blk;
            mixed |= next[i] >= 0 && (c[i] < 0 || next[i] <= c[i]);
          }
        }
      }
      if (past) atomicOr(a.err, 16);
      mixed |= past;
      if (mixed) mixed_flag = 1;
      tc::mbar_arrive_warp(&bars.checked);
    }
    int synced = 0;
    auto load_sync = [&]() {
      tc::mbar_arrive_warp(&bars.load);
      return wait(&bars.load, synced++ & 1);
    };
    // A raw tile of ROWB-byte rows in its stage, widened in place: every thread holds its
    // part in registers before any is written.  4-bit rows go by a row a thread (scales at
    // the row's end; 112 and 80 bytes are an odd number of 16-byte banks), E4M3 by 16-byte
    // pieces in order.  `dead(row)`: a key behind the request's end, zeros.
    auto widen = [&](auto row_bytes, bool swizzled, uint8_t *tile, auto dead) -> bool {
      constexpr int ROWB = decltype(row_bytes)::value, NCH = ROWB / 16;
      uint4 r[NCH];
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        const int idx = E2M1 ? lt * NCH + i : lt + i * kLoadThreads;
        const int row = idx / NCH, ch = idx % NCH;
        r[i] = *reinterpret_cast<const uint4 *>(tile + row * ROWB + (swizzled ? ch ^ (row & 7) : ch) * 16);
        if (dead(row)) r[i] = make_uint4(0u, 0u, 0u, 0u);
      }
      if (!load_sync()) return false;
      auto put = [&](int row, int ch, uint4 v) {
        *reinterpret_cast<uint4 *>(tile + (ch >> 3) * kTileBlk + tc::sw128_offset(row, ch & 7)) = v;
      };
      if constexpr (E2M1) {
        const uint32_t sc[4] = {r[NCH - 1].x, r[NCH - 1].y, r[NCH - 1].z, r[NCH - 1].w};
#pragma unroll
        for (int i = 0; i + 1 < NCH; ++i) {
          uint4 w[4];
          e2m1x32_to_f16(r[i], i & 1 ? sc[i >> 1] >> 16 : sc[i >> 1], w);
#pragma unroll
          for (int u = 0; u < 4; ++u) put(lt, 4 * i + u, w[u]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
          const int idx = lt + i * kLoadThreads;
          uint4 lo, hi;
          e4m3x16_to_f16(r[i], lo, hi);
          put(idx / NCH, 2 * (idx % NCH), lo);
          put(idx / NCH, 2 * (idx % NCH) + 1, hi);
        }
      }
      tc::fence_proxy_async_smem();
      return true;
    };
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!(ok = desc_wait(k))) break;
      const TileDesc &d = descs[k % kDescs];
      const bool end = d.end != 0;
      const bool tail = d.edge & 2;
      bool dead = false;                           // the thread's key lies behind the request's end
      if (tail) dead = d.key0[lt / a.block] + lt % a.block >= x.len;
      uint32_t dead_rows[4] = {0u, 0u, 0u, 0u};
      if (F16 && !E2M1 && tail) {                  // (pieces of other keys too)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 32 * i + lane;
          const uint32_t m = __ballot_sync(0xffffffffu, d.key0[row / a.block] + row % a.block >= x.len);
          dead_rows[i] = m;
        }
      }
      desc_done(k);
      if (end) break;
      const int s = k & 1, phase = (k >> 1) & 1;
      uint8_t *kt = smem + Y::kOffK + s * Y::kKStage, *vt = smem + Y::kOffV + s * kVStage;
      if constexpr (F16) {
        if (!(ok = wait(&bars.k_raw[s], phase))) break;
        if (!(ok = widen(std::integral_constant<int, kv_row_bytes(KV, DQK)>{}, false, kt, [](int) { return false; }))) break;
        tc::mbar_arrive_warp(&bars.k_full[s]);
      }
      if (!(ok = wait(&bars.v_raw[s], phase))) break;
      if constexpr (F16) {
        // E4M3: a thread's pieces are of the rows lt / NCH + multiples of kLoadThreads / NCH
        auto is_dead = [&](int row) {
          if (E2M1) return dead;
          const uint32_t w = row < 32 ? dead_rows[0] : row < 64 ? dead_rows[1] : row < 96 ? dead_rows[2] : dead_rows[3];
          return (w >> (row & 31) & 1u) != 0u;
        };
        if (!(ok = widen(std::integral_constant<int, kv_row_bytes(KV, kDv)>{}, !E2M1, vt, is_dead))) break;
      } else if (tail) {                           // zeros behind the request's end
        if (dead)
#pragma unroll
          for (int ch = 0; ch < kDv / 8; ++ch)
            *reinterpret_cast<uint4 *>(vt + (ch >> 3) * kTileBlk + tc::sw128_offset(lt, ch & 7)) = make_uint4(0u, 0u, 0u, 0u);
        tc::fence_proxy_async_smem();
      }
      tc::mbar_arrive_warp(&bars.v_full[s]);
    }
  } else if (warp >= kMmaWarp) {
    if (warp == kMergeWarp) {
      // ------------------------------------------------------------ the union of the lists
      const int pieces = kPN / a.block, per_page = a.page_size / a.block;
      const uint32_t own = (uint32_t)((x.pos0 + x.ntok - 1) / a.block);
      // Lists in ascending order are read on, others searched for their next entry.  False: the
      // lists are not in order, and nothing has been passed on.
      auto merge = [&](auto in_order) -> bool {
        constexpr bool kInOrder = decltype(in_order)::value;
        // lane: tokens lane, lane + 32, ..; the entry at hand and the one behind it
        const int32_t *list[2] = {a.block_idx, a.block_idx};
        uint32_t cur[2], ahead[2];
        int left[2] = {0, 0};                      // entries unread; searched: the least block still to come
        auto entry = [&](int i) -> uint32_t {      // (none: the largest number)
          if (kInOrder) {
            if (left[i] <= 0) return 0xFFFFFFFFu;
            --left[i];
            const uint32_t c = (uint32_t)__ldg(list[i]++);
            return c <= own ? c : 0xFFFFFFFFu;     // (not past the job's last block)
          }
          const int tt = lane + 32 * i;
          const uint32_t last = (uint32_t)((x.pos0 + tt) / a.block);
          uint32_t best = 0xFFFFFFFFu;
#pragma unroll 4
          for (int e = 0; e < (tt < x.ntok ? a.take : 0); ++e) {
            const uint32_t c = (uint32_t)__ldg(list[i] + e);
            if (c >= (uint32_t)left[i] && c <= last) best = min(best, c);
          }
          left[i] = best == 0xFFFFFFFFu ? INT_MAX : (int)best + 1;
          return best;
        };
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int tt = lane + 32 * i;
          list[i] = a.block_idx + ((int64_t)(x.tok0 + tt) * a.hkv + x.g) * a.take;
          if (kInOrder) left[i] = tt < x.ntok ? a.take : 0;
          cur[i] = entry(i);
          ahead[i] = entry(i);
        }
        bool ok = true;
        int ends = 0;                              // one for each chain
        for (int k = 0; ok && ends < 2; ++k) {
          uint32_t block = 0u, listed[2] = {0u, 0u};
          int found = 0;
          const uint32_t groups = (1u << (a.block >> 4)) - 1u;
          for (int s = 0; s < pieces; ++s) {
            const uint32_t least = __reduce_min_sync(0xffffffffu, min(cur[0], cur[1]));
            if (least == 0xFFFFFFFFu) break;
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (cur[i] == least) {
                listed[i] |= groups << (s * (a.block >> 4));
                cur[i] = ahead[i];
                ahead[i] = entry(i);
              }
            if (lane == s) block = least;
            ++found;
          }
          ends += found == 0;
          const bool in = lane < found;
          int slot = num_slots, key0 = 0;
          if (in) {
            key0 = (int)block * a.block;
            const int32_t page = __ldg(a.page_table + (int64_t)x.b * a.pt_stride + (int)block / per_page);
            if (page >= 0 && page < a.num_pages)
              slot = page * a.page_size + (int)block % per_page * a.block;
            else
              atomicOr(a.err, 1);
          }
          const int edge = (__any_sync(0xffffffffu, in && key0 + a.block - 1 > x.pos0) ? 1 : 0) |
                           (__any_sync(0xffffffffu, in && key0 + a.block > x.len) ? 2 : 0);
          if (kInOrder && k == 0) {                // (asked first thing, it took 1% more)
            if (!(ok = wait(&bars.checked, 0))) break;
            if (mixed_flag) return false;
          }
          if (k >= kDescs && !(ok = wait(&bars.desc_empty[k % kDescs], (k / kDescs - 1) & 1))) break;
          TileDesc &d = descs[k % kDescs];
          if (lane < 8) {
            d.key0[lane] = key0;
            d.slot[lane] = slot;
          }
          d.listed[lane] = (uint8_t)listed[0];
          d.listed[lane + 32] = (uint8_t)listed[1];
          if (lane == 0) {
            d.end = found == 0;
            d.edge = edge;
          }
          tc::mbar_arrive_warp(&bars.desc_full[k % kDescs]);
        }
        return true;
      };
      if (!merge(std::true_type{})) merge(std::false_type{});
    } else if (warp < kMergeWarp) {
      // ------------------------------------------------------------ MMA issuers
      const int t = warp - kMmaWarp;
      const uint32_t id_s = tc::idesc_f16(F16 ? 0 : 1, 0, 0, kPM, kPN), id_pv = tc::idesc_f16(F16 ? 0 : 1, 0, 1, kPM, kDv);
      const uint32_t s_tmem = tmem + kPN * t, o_tmem = tmem + kTmemO + kDv * t;
      if (lane == 0) {
        auto wait1 = [&](uint64_t *bar, uint32_t parity) { return tc::mbar_wait(bar, parity, &abort_flag); };
        // (descriptors' addresses count 16 bytes: a step is one addition.  Each built anew, an MMA's
        // issue took 97 cycles in place of the 47 to 66 that it runs.)
        const uint64_t q_desc = tc::smem_desc_sw128(sbase, 16, 1024);
        const uint64_t k_desc = tc::smem_desc_sw128(sbase + Y::kOffK + t * Y::kKStage, 16, 1024);
        const uint64_t v_desc = tc::smem_desc_sw128(sbase + Y::kOffV + t * kVStage, kTileBlk, 1024);
        bool ok = wait1(&bars.q_full, 0);
        for (int c = 0; ok; ++c) {                 // tile 2 c + t
          const int ds = (2 * c + t) % kDescs;
          if (!(ok = wait1(&bars.desc_full[ds], (2 * c + t) / kDescs & 1))) break;
          const bool end = descs[ds].end != 0;
          tc::mbar_arrive(&bars.desc_empty[ds]);
          if (end) break;
          if (!(ok = wait1(&bars.k_full[t], c & 1))) break;
          tc::tc_fence_after();
#pragma unroll
          for (int kq = 0; kq < DQK / 16; ++kq) {
            const uint32_t off = ((kq & 3) * 32 + (kq >> 2) * kTileBlk) / 16;
            tc::mma_f16_ss(s_tmem, q_desc + off, k_desc + off, id_s, kq > 0 ? 1u : 0u);
          }
          tc::mma_commit(&bars.s_full[t]);
          tc::mma_commit(&bars.k_empty[t]);
          if (!(ok = wait1(&bars.v_full[t], c & 1))) break;
          auto pv = [&](int kk, bool acc) {
            tc::mma_f16_ts(o_tmem, s_tmem + 32 * (kk >> 1) + 8 * (kk & 1), v_desc + kk * (16 * 128 / 16), id_pv,
                           acc ? 1u : 0u);
          };
          if (!(ok = wait1(&bars.p_hi[t], c & 1))) break;
          tc::tc_fence_after();
#pragma unroll
          for (int kk = kPN / 32; kk < kPN / 16; ++kk) pv(kk, c > 0 || kk > kPN / 32);
          if (!(ok = wait1(&bars.p_full[t], c & 1))) break;
          tc::tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < kPN / 32; ++kk) pv(kk, true);
          tc::mma_commit(&bars.pv_done[t]);
          tc::mma_commit(&bars.v_empty[t]);
        }
        // every MMA is complete before TMEM goes back
        tc::mma_commit(&bars.done[t]);
        int no_abort = 0;
        tc::mbar_wait(&bars.done[t], 0, &no_abort, 100000000ull);
      }
    } else {
      // ------------------------------------------------------------ K and V tiles
      // Boxes of `rows` keys of a 64-column block (bf16), or of whole rows: box i of a column
      // block by lane col * boxes + i.
      const int rows = min(a.block, 64), boxes = kPN / rows;
      const int col = lane / boxes, box = lane % boxes;
      constexpr int kKCols = F16 ? 1 : DQK / 64, kVCols = F16 ? 1 : kDv / 64;
      constexpr uint32_t kKRow = F16 ? kv_row_bytes(KV, DQK) : 128, kVRow = F16 ? kv_row_bytes(KV, kDv) : 128;
      uint64_t *k_bar = F16 ? bars.k_raw : bars.k_full;
      int issued = 0;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        if (!(ok = desc_wait(k))) break;
        const TileDesc &d = descs[k % kDescs];
        const bool end = d.end != 0;
        const int at = box * rows, slot = d.slot[at / a.block] + at % a.block;
        desc_done(k);
        if (end) break;
        const int s = k & 1;
        if (k >= 2 && !(ok = wait(&bars.k_empty[s], ((k >> 1) - 1) & 1))) break;
        if (lane == 0) tc::mbar_arrive_expect_tx(&k_bar[s], kPN * kKRow * kKCols);
        __syncwarp();
        if (col < kKCols)
          tma_load_3d(sbase + Y::kOffK + s * Y::kKStage + col * kTileBlk + at * kKRow, &maps.k, 64 * col, x.g, slot,
                      &k_bar[s]);
        __syncwarp();
        ++issued;
        if (k >= 2 && !(ok = wait(&bars.v_empty[s], ((k >> 1) - 1) & 1))) break;
        if (lane == 0) tc::mbar_arrive_expect_tx(&bars.v_raw[s], kPN * kVRow * kVCols);
        __syncwarp();
        if (col < kVCols)
          tma_load_3d(sbase + Y::kOffV + s * kVStage + col * kTileBlk + at * kVRow, &maps.v, 64 * col, x.g, slot,
                      &bars.v_raw[s]);
        __syncwarp();
        ++issued;
      }
      if (!ok) {                                   // the copies in flight land before the CTA ends
        int no_abort = 0;
        for (int i = max(0, issued - 4); i < issued; ++i)
          tc::mbar_wait(i & 1 ? &bars.v_raw[(i >> 1) & 1] : &k_bar[(i >> 1) & 1], (i >> 2) & 1, &no_abort, 100000000ull);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax + epilogue
    const int t = warp >> 2, wq = warp & 3;
    const int p = wq * 32 + lane;                  // row of the Q tile, TMEM lane
    const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
    const uint32_t s_addr = tmem + lane_base + kPN * t;
    auto o_addr = [&](int chain) { return tmem + lane_base + kTmemO + kDv * chain; };
    const int tt = p / a.group;
    const bool valid = tt < x.ntok;
    const int head = x.g * a.group + p % a.group;
    const int pos = valid ? x.pos0 + tt : -1;
    // The warp's 16 rows have been on their way since the start; 8- and 4-bit caches: times the
    // power of two that puts the row's largest |q| in [2^14, 2^15), in fp16 (attn_prefill.cu).
    {
      uint8_t *mine = smem + (lane >> 3) * kTileBlk;
      asm volatile("cp.async.wait_all;\n" ::: "memory");
      if (F16) {
#pragma unroll 1
        for (int r = warp * 16; r < warp * 16 + 16; ++r) {
          uint4 *at = reinterpret_cast<uint4 *>(mine + tc::sw128_offset(r, lane & 7));
          const uint4 v = lane < DQK / 8 ? *at : make_uint4(0u, 0u, 0u, 0u);
          uint32_t h[4] = {v.x, v.y, v.z, v.w}, e = 0u;
#pragma unroll
          for (int q = 0; q < 4; ++q) e = max(e, max((h[q] >> 7) & 0xFFu, (h[q] >> 23) & 0xFFu));
          const int sh = min(141 - (int)__reduce_max_sync(0xffffffffu, e), 126);
          const float f = __int_as_float((sh + 127) << 23);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            h[q] = pair16<false>(__uint_as_float(h[q] << 16) * f, __uint_as_float(h[q] & 0xFFFF0000u) * f);
          if (lane < DQK / 8) *at = make_uint4(h[0], h[1], h[2], h[3]);
          if (lane == 0) row_sc[r] = tc::row_score_scale(a.scale_log2, sh);
        }
      }
    }
    tc::fence_proxy_async_smem();
    tc::mbar_arrive_warp(&bars.q_full);
    bool ok = wait(&bars.q_full, 0);               // the other warps' row_sc
    const float sc = F16 && ok ? row_sc[p] : a.scale_log2;
    const int block_log2 = 31 - __clz(a.block);
    float m_run = -INFINITY, l_run = 0.f;
    int c = 0;                                     // the chain's tiles so far
    while (ok) {
      const int k = 2 * c + t;
      if (!(ok = desc_wait(k))) break;
      const TileDesc &d = descs[k % kDescs];
      const bool end = d.end != 0, edge = d.edge & 1;
      // the eight groups of 16 keys: a bit each if listed, and (edge) how many keys are seen
      const uint32_t sel = valid ? d.listed[tt & 63] : 0u;
      uint64_t lim = 0u;
      if (edge)
#pragma unroll 1
        for (int g = 0; g < 8; ++g) {
          const int n = pos + 1 - d.key0[(g * 16) >> block_log2] - ((g * 16) & (a.block - 1));
          lim |= (uint64_t)(sel >> g & 1u ? min(16, max(0, n)) : 0) << (8 * g);
        }
      desc_done(k);
      if (end) break;
      if (!(ok = wait(&bars.s_full[t], c & 1))) break;
      tc::tc_fence_after();
      // Rolled over the tile's four 32-column chunks: the four roles share each scheduler's
      // instruction cache, and this loop is what they wait for (unrolled, with the next chunk
      // on its way, 5.3 thousand cycles a tile against 1.9).  Tiles with an edge: keys that the
      // token does not see go to -inf first.  Groups of 16 that it did not list are left out of
      // the maximum and get a weight of 2^-inf.
      if (edge) {
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          uint32_t v[32];
          tc::tmem_ld32(s_addr + 32 * q, v);
          const uint32_t n0 = (uint32_t)(lim >> (16 * q)) & 31u, n1 = (uint32_t)(lim >> (16 * q + 8)) & 31u;
          const uint32_t seen = ((1u << n0) - 1u) | ((1u << n1) - 1u) << 16;
          tc::tmem_wait_ld_regs32(v);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = seen >> j & 1u ? v[j] : 0xFF800000u;
          tc::tmem_st32(s_addr + 32 * q, v);
        }
        tc::tmem_wait_st();
      }
      float mx = -INFINITY;
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        const uint32_t here = sel >> (2 * q) & 3u;
        if (!__any_sync(0xffffffffu, here != 0u)) continue;
        uint32_t v[32];
        tc::tmem_ld32(s_addr + 32 * q, v);
        tc::tmem_wait_ld_regs32(v);
        float g[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 32; j += 2)
          g[j >> 4] = tc::max3(g[j >> 4], __uint_as_float(v[j]), __uint_as_float(v[j + 1]));
        if (here & 1u) mx = fmaxf(mx, g[0]);
        if (here & 2u) mx = fmaxf(mx, g[1]);
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
            tc::tmem_ld16(o_addr(t) + q * 16, o);
            tc::tmem_wait_ld_regs(o);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
            tc::tmem_st16(o_addr(t) + q * 16, o);
          }
          tc::tmem_wait_st();
          l_run *= alpha;
        }
        if (need) m_run = m_tile;
      }
      // P of a chunk's 32 keys (16-bit values, key j in a half of column j / 2) over the first
      // half of its own columns; keys 64-127 first
      const float off = m_run == -INFINITY ? 0.f : kLift - m_run;
      float rs[2] = {0.f, 0.f};
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        const int q = i ^ 2;
        const uint32_t here = sel >> (2 * q) & 3u;
        uint32_t pk[16];
        if (__any_sync(0xffffffffu, here != 0u)) {
          uint32_t v[32];
          tc::tmem_ld32(s_addr + 32 * q, v);
          const float og[2] = {here & 1u ? off : -INFINITY, here & 2u ? off : -INFINITY};
          tc::tmem_wait_ld_regs32(v);
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            float y0, y1;
            tc::ffma2(y0, y1, __uint_as_float(v[j]), __uint_as_float(v[j + 1]), sc, og[j >> 4]);
            const float p0 = ex2(y0), p1 = ex2(y1);
            tc::fadd2(rs[0], rs[1], p0, p1);
            pk[j >> 1] = pair16<!F16>(p0, p1);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) pk[j] = 0u;
        }
        tc::tmem_st16(s_addr + 32 * q, pk);
        if (i & 1) {
          tc::tmem_wait_st();
          tc::tc_fence_before();
          tc::mbar_arrive_warp(i == 1 ? &bars.p_hi[t] : &bars.p_full[t]);
        }
      }
      l_run += rs[0] + rs[1];
      ++c;
    }
    // ---------------- the chains' results together; a warp writes half the columns
    if (ok && c > 0) ok = wait(&bars.pv_done[t], (c - 1) & 1);
    bool odd = l_run != l_run;
    // (a chain without a tile has nothing in its O, one that saw none of the row's blocks zeros)
    row_m[t][p] = c > 0 ? m_run : -INFINITY;
    row_l[t][p] = l_run;
    tc::tc_fence_before();
    tc::mbar_arrive_warp(&bars.merge);
    if (ok) ok = wait(&bars.merge, 0);
    if (ok) {
      tc::tc_fence_after();
      const float m0 = row_m[0][p], m1 = row_m[1][p], M = fmaxf(m0, m1);
      // (a chain far below the other has a weight of 0 and counts all the same: its NaN is the row's)
      const bool saw0 = m0 != -INFINITY, saw1 = m1 != -INFINITY;
      const float w0 = saw0 ? exp2f(m0 - M) : 0.f, w1 = saw1 ? exp2f(m1 - M) : 0.f;
      const float l = (saw0 ? w0 * row_l[0][p] : 0.f) + (saw1 ? w1 * row_l[1][p] : 0.f);
      float lse;
      const float sink2 = a.sinks && valid ? __ldg(a.sinks + head) * kLog2e : -INFINITY;
      const float f = finish(M, l, kLift, sink2, a.v_scale, lse);
      const float f0 = f * w0, f1 = f * w1;
      uint16_t *row = a.out + ((int64_t)(x.tok0 + (valid ? tt : 0)) * a.hq + head) * kDv;
#pragma unroll 1
      for (int q = 4 * t; q < 4 * t + 4; ++q) {
        uint32_t o0[16], o1[16];
        tc::tmem_ld16(o_addr(0) + q * 16, o0);
        tc::tmem_ld16(o_addr(1) + q * 16, o1);
        tc::tmem_wait_ld_regs(o0);
        tc::tmem_wait_ld_regs(o1);
        uint32_t w[8];
        float sum = 0.f;                           // NaN if any of what counts is NaN or infinite
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          float u[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float u0 = saw0 ? __uint_as_float(o0[j + y]) : 0.f, u1 = saw1 ? __uint_as_float(o1[j + y]) : 0.f;
            sum += 0.f * u0 + 0.f * u1;
            u[y] = u0 * f0 + u1 * f1;
          }
          w[j >> 1] = pair16<true>(u[0], u[1]);
        }
        odd |= sum != sum;
        if (!valid) continue;
        reinterpret_cast<uint4 *>(row + q * 16)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4 *>(row + q * 16)[1] = make_uint4(w[4], w[5], w[6], w[7]);
      }
      if (valid && a.lse && t == 0) a.lse[(int64_t)(x.tok0 + tt) * a.hq + head] = lse;
      if (valid && odd) {                          // a mark on the row: no other row's output is NaN
        row[64 * t] = kMark;
        odd_flag = 1;
      }
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
