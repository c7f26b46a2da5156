// Split-KV attention over a 4-bit cache for row blocks of at most 32 query rows
// (decode, and a few draft tokens on small groups; of 17 to 32 rows where the batch
// has three key tiles an SM or more, see planner.cpp).
//
// At these sizes a key's 192 bytes feed few rows, and what bounds the tcgen05 kernel
// (attn_tc.cu) is not the tensor pipe but getting there: its operands have to be
// 16-bit tiles in shared memory, so every 4-bit tile is read, written four times as
// wide, and read again, and a 64-key tile passes through four warp roles.  Here the
// codes go from the TMA ring straight into registers, are widened there, and feed
// register-operand MMAs (m16n8k16, fp16, fp32 accumulation).  Both products are
// computed transposed, so that the padded side is the 8-row granule (1, 2 or 4 of
// them: NB) and not 64 rows of MMA:
//   S^T (keys x rows) = K (16 keys x 16 dims) . Q^T (16 dims x 8 rows),
//   O^T (dv x rows)   = V^T (16 dv x 16 keys) . P^T (16 keys x 8 rows).
// The order of a contraction's index is free, so lanes take what is
// contiguous in the cache: lane (g, t) (g = lane / 4, t = lane % 4) of a K
// operand owns the whole 16-code blocks t, t + 4, t + 8 of keys g and g + 8
// (Q's fragments use the same order), and of a V operand the block g of keys 2t,
// 2t + 1, 2t + 8, 2t + 9; a lane needs one scale per 8-byte load.  V^T wants two
// keys in one register: the nibbles of two keys are interleaved into bytes
// first (one shift and one bit-select per four pairs), and the byte's one
// conversion then yields the pair.  P^T comes out of S^T's accumulators with an
// 8x8 transpose (movmatrix).
//
// Codes times scales are exact in fp16 (e2m1.cuh).  Q rows are scaled by the power
// of two that puts the row's largest |q| in [2^14, 2^15) (exact down to 2^-31 of
// it) and the scores divided by it in fp32.  P is held in fp16 relative to the
// running maximum times 2^7, so that weights down to 2^-21 of the maximum keep
// 11 bits and none above 2^-32 is lost; the maximum may grow by 2^8 before O is
// rescaled (P <= 2^15).  Row sums are fp32, of the weights before rounding.
//
// A unit of work is half a 64-key tile (32 keys); unit u of the CTA belongs to
// warp u % kWarps, which keeps running maxima, sums and O of its own for the
// whole segment, so nothing is shared between tiles; at the end of a segment
// the warps' partials are combined through shared memory.  Each warp also
// fetches its own units, into a ring of its own, a unit or two ahead: it alone
// fills, waits for and frees the ring's stages, in order, so that no barrier
// phase can be mistaken for another and no warp ever waits for another one's
// data.  With page sizes TMA can tile a unit is one K and one V box per page
// piece, issued by a lane each after up to 32 page lookups in one round trip;
// otherwise its rows are gathered with 16-byte asynchronous copies.
// Every wait is bounded in time, as in attn_tc.cu.
//
// Measured (16 query heads on 2 KV heads unless said, merge included): a ragged
// decode batch of 32 requests, 195 MB of rows, 50 us (3.9 TB/s, 0.58 of the copy rate;
// fetching alone, without any arithmetic, takes 42.7 us, so what is left is the
// fetch and the warps' issue slots, 58% busy); four requests of 46K keys 23 us with
// 8 rows and 43 with 32 (there it is the latency of one warp's chain: 2 warps a
// scheduler, 0.36 instructions a cycle); pages of one token, 16 rows, 109 MB, 54 us
// (16-byte copies).  12 warps for 8 rows, 8 beyond: what the registers allow; 16 of
// 128 registers took 54 us on the batch, a ring of three units 53.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>

#include "e2m1.cuh"
#include "fp4_nan.cuh"
#include "kernels.hpp"
#include "tc_common.cuh"

namespace akp {
namespace {

constexpr int kN = kKeyTile;
constexpr int kUnitKeys = kFp4UnitKeys;
constexpr int kUnits = kN / kUnitKeys;        // units per tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGrow = 8.0f;                 // base-2 growth of a maximum before O is rescaled
constexpr float kLift = 7.0f;                 // P is held times 2^kLift
constexpr int kCombStride = 130;              // floats per row of the combine buffer (see its use)

template <int DQK>
struct Unit {
  static constexpr int kKrow = e2m1_row_bytes(DQK), kVrow = e2m1_row_bytes(kDv);
  static constexpr int kKBytes = kUnitKeys * kKrow;
  static constexpr int kBytes = kKBytes + kUnitKeys * kVrow;      // 6 KB at 192
};

template <int DQK, int NB>
struct Cfg {
  static constexpr int kWarps = NB == 1 ? 12 : 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kDepth = NB == 2 ? 3 : 2;     // units in a warp's ring
  // Q's fragments in shared memory but for 8-row blocks (16 rows: 5% faster than
  // in registers; 32 rows: O alone takes 128 registers)
  static constexpr bool kQsmem = NB >= 2;
  static constexpr int kQBytes = kQsmem ? NB * (DQK / 16) * 32 * 8 : 0;
  static constexpr int kCombRows = NB > 2 ? 16 : NB * 8;     // rows combined at a time
  // 8-row blocks: a warp's partial goes into its own ring's free stage
  static constexpr bool kCombInRing = NB == 1;
  static constexpr int kOffQ = kWarps * kDepth * Unit<DQK>::kBytes;
  static constexpr int kOffComb = kOffQ + kQBytes;
  static constexpr int kSmem = kOffComb + (kCombInRing ? 0 : kWarps * kCombRows * kCombStride * 4) + 1024;
  static_assert(!kCombInRing || kCombRows * kCombStride * 4 <= Unit<DQK>::kBytes, "partial larger than a stage");
  static_assert(kSmem + 3 * 1024 <= 227 * 1024, "shared memory layout too large");
};

struct FBars {
  uint64_t full[12][3];       // [warp][stage of its ring]
  uint64_t sync;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t f16_pair(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&h);
}

// c (16 x 8, fp32) += a (16 x 16, fp16) . b (16 x 8, fp16)
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8x8 transpose of 16-bit elements held as one row per four lanes.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t lo16) {
  uint32_t p;
  asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}\n" : "=r"(p) : "r"(lo16));
  return p;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int c1, int c2, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(c1), "r"(c2), "r"(tc::smem_u32(bar))
      : "memory");
}

// The page pieces ("boxes") of a warp's units, up to 32 looked up at a time:
// lane i holds box i % nbox of the batch's unit i / nbox.  A page id is loaded when
// its batch is looked up, one batch ahead, and first used when that becomes the
// current one.
struct Boxes {
  int32_t page, off, g;      // page id, first slot in the page (-1: no visible key in the box), KV head
};

template <int DQK, int NB, bool TMA>
__global__ void __launch_bounds__(Cfg<DQK, NB>::kThreads, 1)
    attn_fp4_kernel(const RunArgs args, const __grid_constant__ TmaMaps maps) {
  const RunArgs a = args;
  using C = Cfg<DQK, NB>;
  using T = Unit<DQK>;
  constexpr int kWarps = C::kWarps, kDepth = C::kDepth;
  constexpr int NJ = DQK / 64;                 // K blocks per lane
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
  __shared__ FBars bars;
  __shared__ int abort_flag;
  __shared__ int v_nan;           // a NaN V block of a unit cut by some row's range (fp4_nan.cuh)
  __shared__ float sm_m[kWarps][NB * 8], sm_l[kWarps][NB * 8];
  __shared__ __align__(8) float sm_sc[C::kQsmem ? NB * 8 : 2];     // the rows' score scales

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // programmatic dependent: see attn_tc.cu
  // (a plan that is not replayable never changes: its head record is read while the
  // previous kernel ends)
  CtaHead head;
  if (!a.replayed) head = a.cta_heads[blockIdx.x];
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  if (a.replayed) head = a.cta_heads[blockIdx.x];
  if (head.seg_begin >= head.seg_end) return;
  const int total_units = head.total * kUnits;
  if (tid == 0) {
    abort_flag = 0;
    v_nan = 0;
    for (int w = 0; w < kWarps; ++w)
      for (int d = 0; d < kDepth; ++d) tc::mbar_init(&bars.full[w][d], 1);
    tc::mbar_init(&bars.sync, kWarps);
    tc::fence_mbar_init();
  }
  __syncthreads();

  // ------------------------------------------------------------ fetching
  // This warp's units are warp, warp + kWarps, ... of the CTA; its n-th unit goes
  // to stage n % kDepth of its ring.
  const int my_units = total_units > warp ? (total_units - warp + kWarps - 1) / kWarps : 0;
  uint8_t *ring = smem + warp * (kDepth * T::kBytes);
  const uint32_t ring_addr = tc::smem_u32(ring);
  const int box = TMA ? min(a.page_size, kUnitKeys) : 1;
  const int nbox = TMA ? kUnitKeys / box : 32;            // boxes per unit (TMA: 1, 2 or 4)
  const int batch = TMA ? 32 / nbox : 1;                  // units per lookup
  const int mine = lane / nbox, bx = lane % nbox;
  int lk_seg = head.seg_begin, lk_at = warp, lk_next = 0; // where the next lookup starts
  SegDesc lk_sd = head.seg;
  BlockDesc lk_bd = head.blk;
  auto lookup = [&]() -> Boxes {
    Boxes r{0, -1, 0};
    const int cnt = min(batch, my_units - lk_next);
    lk_next += batch;
    if (cnt <= 0) return r;
    // the lane's unit: past whole segments first (the batch's last unit is where
    // the next batch goes on from; its segment and block stay in registers)
    int sg = lk_seg, at = lk_at + min(mine, cnt - 1) * kWarps;
    SegDesc sd = lk_sd;
    while (at >= (sd.tile_end - sd.tile_begin) * kUnits && sg + 1 < head.seg_end) {
      at -= (sd.tile_end - sd.tile_begin) * kUnits;
      sd = a.segs[++sg];
    }
    int b = lk_bd.b, klo = lk_bd.klo, khi = lk_bd.khi;
    r.g = lk_bd.g;
    if (sd.block != lk_sd.block) {
      const BlockDesc bd = a.blocks[sd.block];
      b = bd.b;
      klo = bd.klo;
      khi = bd.khi;
      r.g = bd.g;
    }
    const int j = sd.tile_begin * kN + at * kUnitKeys + bx * box;
    if (mine < cnt && j + box > klo && j < khi) {
      r.page = __ldg(a.page_table + (int64_t)b * a.pt_stride + j / a.page_size);
      r.off = j % a.page_size;
    }
    const int last = __shfl_sync(0xffffffffu, sg, 31);
    lk_at = __shfl_sync(0xffffffffu, at, 31) + kWarps;
    if (last != lk_seg) {
      lk_seg = last;
      lk_sd = a.segs[last];
      lk_bd = a.blocks[lk_sd.block];
    }
    return r;
  };
  // the batch's first slots, -1 where nothing is to be read (ids outside the pool
  // are reported, and read as zeros)
  auto resolve = [&](const Boxes &b) -> int64_t {
    if (b.off < 0) return -1;
    if (b.page < 0 || b.page >= a.num_pages) {
      atomicOr(a.err, 1);
      return -1;
    }
    return (int64_t)b.page * a.page_size + b.off;
  };
  Boxes nxt = lookup();
  int64_t slot = resolve(nxt);
  int cur_g = nxt.g;
  nxt = lookup();
  int issued = 0;
  auto issue = [&]() {
    const int d = issued % kDepth, u = issued & (batch - 1);
    const uint32_t dst = ring_addr + d * T::kBytes;
    if constexpr (TMA) {
      uint64_t *bar = &bars.full[warp][d];
      if (lane == 0) tc::mbar_arrive_expect_tx(bar, T::kBytes);
      __syncwarp();
      if (mine == u) {
        // a box without a visible key reads past the pool: zero fill
        const int first = slot >= 0 ? (int)slot : a.num_pages * a.page_size;
        tma_load_3d(dst + bx * box * T::kKrow, &maps.k, cur_g, first, bar);
        tma_load_3d(dst + T::kKBytes + bx * box * T::kVrow, &maps.v, cur_g, first, bar);
      }
    } else {
      // lane i holds key i's slot; the lanes copy the unit's 16-byte chunks in
      // order (a row's neighbouring chunks by neighbouring lanes); keys without
      // a slot are filled with zeros
      const int64_t row = slot >= 0 ? slot * a.hkv + cur_g : -1;
      auto rows = [&](const void *cache, int row_bytes, uint32_t to) {
        const int nch = row_bytes / 16;
#pragma unroll
        for (int i = 0; i < nch; ++i) {
          const int c = i * 32 + lane, key = c / nch, ch = c % nch;
          const int64_t s = __shfl_sync(0xffffffffu, row, key);
          const uint8_t *src = static_cast<const uint8_t *>(cache) + (s >= 0 ? s : 0) * row_bytes + ch * 16;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(to + c * 16), "l"(src),
                       "r"(s >= 0 ? 16 : 0)
                       : "memory");
        }
      };
      rows(a.k_cache, T::kKrow, dst);
      rows(a.v_cache, T::kVrow, dst + T::kKBytes);
    }
    ++issued;
    if ((issued & (batch - 1)) == 0) {
      slot = resolve(nxt);
      cur_g = nxt.g;
      nxt = lookup();
    }
  };
  // every stage but one is filled ahead; without TMA each fill is one group of
  // asynchronous copies, empty past the last unit, so that their count is fixed
  auto fill = [&]() {
    if (issued < my_units) issue();
    if (!TMA) asm volatile("cp.async.commit_group;\n" ::: "memory");
  };
  for (int i = 0; i < kDepth - 1; ++i) fill();
  int done = 0;                                // units this warp has finished

  {
    // ------------------------------------------------------------ attention
    const int g = lane >> 2, t = lane & 3;
    uint32_t qf[C::kQsmem ? 1 : NB][NJ * 4][2];
    float o[8][NB][4];
    float m[NB][2], l[NB][2], sc[C::kQsmem ? 1 : NB][2];
    uint2 *qsm = reinterpret_cast<uint2 *>(smem + C::kOffQ);      // [NB][NJ * 4][32 lanes]
    uint32_t sync_phase = 0;
    auto group_sync = [&]() -> bool {
      tc::mbar_arrive_warp(&bars.sync);
      const bool ok = __all_sync(0xffffffffu, tc::mbar_wait_spin(&bars.sync, sync_phase, &abort_flag));
      sync_phase ^= 1;
      return ok;
    };
    SegDesc sd = head.seg;
    BlockDesc bd = head.blk;
    int u0 = 0;                                // the segment's first unit among the CTA's
    bool alive = true;
    for (int seg = head.seg_begin; seg < head.seg_end && alive; ++seg) {
      if (seg > head.seg_begin) {
        sd = a.segs[seg];
        bd = a.blocks[sd.block];
      }
      const int u_end = u0 + (sd.tile_end - sd.tile_begin) * kUnits;
      // this warp's first unit of the segment
      int u = u0 + (warp - u0 % kWarps + kWarps) % kWarps;
      const bool has = u < u_end;
      // ---- rows: Q fragments (scaled to fp16), score scales, visible keys
      const int i_first = bd.L - bd.n + bd.row0 / a.group;
      const int i_last = bd.L - bd.n + (bd.row0 + bd.nrows - 1) / a.group;
      // keys every row sees
      const int all_lo = a.window > 0 ? max(0, i_last - a.window + 1) : 0, all_hi = i_first + 1;
      // Row group nb as B fragments of fp16, scaled; returns this lane's row's shift.
      auto load_q = [&](int nb, uint32_t (&f)[NJ * 4][2]) -> int {
        const int r = nb * 8 + g;
        uint32_t e = 0;
        const bool live = r < bd.nrows;
        const int flat = bd.row0 + (live ? r : 0);
        const uint2 *src = reinterpret_cast<const uint2 *>(
            static_cast<const uint16_t *>(a.q) +
            ((int64_t)(bd.tok0 + flat / a.group) * a.hq + bd.g * a.group + flat % a.group) * DQK);
#pragma unroll
        for (int i = 0; i < NJ * 4; ++i) {
          const uint2 v = live ? __ldg(src + (t + 4 * (i >> 2)) * 4 + (i & 3)) : make_uint2(0u, 0u);
          f[i][0] = v.x;
          f[i][1] = v.y;
          e = max(e, max(max((v.x >> 7) & 0xFFu, (v.x >> 23) & 0xFFu),
                         max((v.y >> 7) & 0xFFu, (v.y >> 23) & 0xFFu)));
        }
        e = max(e, __shfl_xor_sync(0xffffffffu, e, 1));
        e = max(e, __shfl_xor_sync(0xffffffffu, e, 2));
        const int sh = min(141 - (int)e, 126);
        const float up = __int_as_float((sh + 127) << 23);
#pragma unroll
        for (int i = 0; i < NJ * 4; ++i)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t w = f[i][x];
            f[i][x] = f16_pair(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xFFFF0000u) * up);
          }
        return sh;
      };
      if constexpr (C::kQsmem) {
        // warp nb stages row group nb for all warps (the previous segment's
        // combine has ended: nobody reads the old fragments any more)
        if (warp < NB) {
          uint32_t f[NJ * 4][2];
          const int sh = load_q(warp, f);
#pragma unroll
          for (int i = 0; i < NJ * 4; ++i) qsm[(warp * NJ * 4 + i) * 32 + lane] = make_uint2(f[i][0], f[i][1]);
          if (t == 0) sm_sc[warp * 8 + g] = a.scale_log2 * __int_as_float((127 - sh) << 23);
        }
        if (!group_sync()) break;
      }
      if (has) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          if constexpr (!C::kQsmem) {
            const int sh = load_q(nb, qf[nb]);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int shr = __shfl_sync(0xffffffffu, sh, (2 * t + x) * 4);
              sc[nb][x] = a.scale_log2 * __int_as_float((127 - shr) << 23);
            }
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            m[nb][x] = -INFINITY;
            l[nb][x] = 0.f;
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[i][nb][x] = 0.f;
      }
#pragma unroll 1
      for (; u < u_end; u += kWarps) {
        const int d = done % kDepth;
        const int key0 = sd.tile_begin * kN + (u - u0) * kUnitKeys;
        fill();                                   // the stage freed by the previous unit
        if constexpr (TMA) {
          if (!tc::mbar_wait_warp(&bars.full[warp][d], (done / kDepth) & 1, &abort_flag)) {
            alive = false;
            break;
          }
        } else {
          asm volatile("cp.async.wait_group %0;\n" ::"n"(kDepth - 1) : "memory");
          __syncwarp();
        }
        const uint8_t *kt = ring + d * T::kBytes, *vt = kt + T::kKBytes;
        // ---- S^T = K . Q^T for 2 x 16 keys
        float sacc[2][NB][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int x = 0; x < 4; ++x) sacc[mt][nb][x] = 0.f;
        const uint8_t *krow = kt + g * T::kKrow;       // keys g, g + 8, g + 16, g + 24
        uint32_t ws[4][NJ];                            // their scales
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const uint4 w = *reinterpret_cast<const uint4 *>(krow + 8 * y * T::kKrow + DQK / 2);
          ws[y][0] = w.x;
          ws[y][1] = w.y;
          if (NJ > 2) ws[y][NJ - 1] = w.z;
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          uint32_t h[4][8], s[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const uint2 c = *reinterpret_cast<const uint2 *>(krow + 8 * y * T::kKrow + 8 * (t + 4 * j));
            uint32_t x[4];
            e2m1x8_to_f16(c.x, x);
            h[y][0] = x[0], h[y][1] = x[1], h[y][2] = x[2], h[y][3] = x[3];
            e2m1x8_to_f16(c.y, x);
            h[y][4] = x[0], h[y][5] = x[1], h[y][6] = x[2], h[y][7] = x[3];
          }
#pragma unroll
          for (int y = 0; y < 4; y += 2) {
            // byte t of two rows' scale words -> both scales, doubled up
            const uint32_t p2 = e4m3x2_to_f16(__byte_perm(ws[y][j], ws[y + 1][j], t | (t + 4) << 4));
            s[y] = __byte_perm(p2, 0u, 0x1010);
            s[y + 1] = __byte_perm(p2, 0u, 0x3232);
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint2 qs[NB];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
              qs[nb] = C::kQsmem ? qsm[(nb * NJ * 4 + 4 * j + q) * 32 + lane]
                                 : make_uint2(qf[C::kQsmem ? 0 : nb][4 * j + q][0], qf[C::kQsmem ? 0 : nb][4 * j + q][1]);
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
              const uint32_t a0 = mul_f16x2(h[2 * mt][2 * q], s[2 * mt]);
              const uint32_t a2 = mul_f16x2(h[2 * mt][2 * q + 1], s[2 * mt]);
              const uint32_t a1 = mul_f16x2(h[2 * mt + 1][2 * q], s[2 * mt + 1]);
              const uint32_t a3 = mul_f16x2(h[2 * mt + 1][2 * q + 1], s[2 * mt + 1]);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) mma16816(sacc[mt][nb], a0, a1, a2, a3, qs[nb].x, qs[nb].y);
            }
          }
        }
        // ---- softmax: base-2 scores, the running maximum, P in fp16
        const bool full = key0 >= all_lo && key0 + kUnitKeys <= all_hi;
        float lm[NB][2];
        bool grow = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float mx = -INFINITY;
            const float scx = C::kQsmem ? sm_sc[nb * 8 + 2 * t + x] : sc[C::kQsmem ? 0 : nb][x];
            int row_lo = 0, row_hi = 0;
            if (!full) {
              // (rows past the block have zero queries and are never written: any
              // range does for them)
              const int rr = min(nb * 8 + 2 * t + x, bd.nrows - 1);
              const int i = bd.L - bd.n + (bd.row0 + rr) / a.group;
              row_hi = i + 1;
              row_lo = a.window > 0 ? max(0, i - a.window + 1) : 0;
            }
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float v = sacc[mt][nb][2 * h + x] * scx;
                if (!full) {
                  const int j = key0 + mt * 16 + h * 8 + g;
                  if (j < row_lo || j >= row_hi) v = -INFINITY;
                }
                sacc[mt][nb][2 * h + x] = v;
                mx = fmaxf(mx, v);
              }
            lm[nb][x] = mx;
            grow |= mx > m[nb][x] + kGrow;
          }
        if (__any_sync(0xffffffffu, grow)) {
          float alpha[NB][2];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float mx = lm[nb][x];
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
              const bool up = mx > m[nb][x] + kGrow;       // also from -inf
              alpha[nb][x] = up ? ex2(m[nb][x] - mx) : 1.f;
              if (up) m[nb][x] = mx;
              l[nb][x] *= alpha[nb][x];
            }
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int x = 0; x < 4; ++x) o[i][nb][x] *= alpha[nb][x & 1];
        }
        uint32_t pf[2][NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const float n0 = m[nb][0] == -INFINITY ? 0.f : kLift - m[nb][0];
          const float n1 = m[nb][1] == -INFINITY ? 0.f : kLift - m[nb][1];
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float p0 = ex2(sacc[mt][nb][2 * h] + n0), p1 = ex2(sacc[mt][nb][2 * h + 1] + n1);
              l[nb][0] += p0;
              l[nb][1] += p1;
              pf[mt][nb][h] = transpose8(f16_pair(p0, p1));
            }
        }
        // ---- O^T += V^T . P^T
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const uint8_t *vr = vt + (mt * 16 + 2 * t) * T::kVrow + 8 * g;
          const uint8_t *vs = vt + (mt * 16 + 2 * t) * T::kVrow + kDv / 2 + g;
          uint2 c[4];                                      // keys 2t, 2t + 1, 2t + 8, 2t + 9
          uint32_t sb[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int kk = (y & 1) + 8 * (y >> 1);
            c[y] = *reinterpret_cast<const uint2 *>(vr + kk * T::kVrow);
            sb[y] = vs[kk * T::kVrow];
          }
          if (!full) {
            // keys outside the block's range may hold anything: NaN scales to zero, and
            // those that only some rows see must not reach the others (fp4_nan.cuh)
            const int j0 = key0 + mt * 16 + 2 * t;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int j = j0 + (y & 1) + 8 * (y >> 1);
              if (j < bd.klo || j >= bd.khi) sb[y] = 0u;
            }
            const uint32_t nan = e4m3_nan_bytes(sb[0] | sb[1] << 8 | sb[2] << 16 | sb[3] << 24);
            if (nan) {
              v_nan = 1;
#pragma unroll
              for (int y = 0; y < 4; ++y) sb[y] &= ~(nan >> (8 * y));
            }
          }
          const uint32_t sA = e4m3x2_to_f16(sb[0] | sb[1] << 8), sB = e4m3x2_to_f16(sb[2] | sb[3] << 8);
#pragma unroll
          for (int w = 0; w < 2; ++w) {                    // eight codes of each key
            const uint32_t k0w = w ? c[0].y : c[0].x, k1w = w ? c[1].y : c[1].x;
            const uint32_t k2w = w ? c[2].y : c[2].x, k3w = w ? c[3].y : c[3].x;
            constexpr uint32_t L4 = 0x0F0F0F0Fu;
            uint32_t eA[4], oA[4], eB[4], oB[4];
            e2m1x8_to_f16((k0w & L4) | ((k1w << 4) & ~L4), eA);      // even codes, (key, key + 1)
            e2m1x8_to_f16(((k0w >> 4) & L4) | (k1w & ~L4), oA);      // odd codes
            e2m1x8_to_f16((k2w & L4) | ((k3w << 4) & ~L4), eB);
            e2m1x8_to_f16(((k2w >> 4) & L4) | (k3w & ~L4), oB);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t a0 = mul_f16x2(eA[i], sA), a1 = mul_f16x2(oA[i], sA);
              const uint32_t a2 = mul_f16x2(eB[i], sB), a3 = mul_f16x2(oB[i], sB);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
                mma16816(o[4 * w + i][nb], a0, a1, a2, a3, pf[mt][nb][0], pf[mt][nb][1]);
            }
          }
        }
        ++done;
        if (TMA) tc::fence_proxy_async_smem();   // the refill must not overtake these reads
        __syncwarp();
      }
      if (!alive) break;

      // ---- end of the segment: this warp's partial, then the common result.
      // Row r of the buffer starts at r * 130 and the pair of dv (16g + 2i, + 1)
      // sits at 16g + ((2i + 2(g / 2)) & 15): the 16 lanes of a half-warp write 32
      // different banks.
      // (the partials in the rings' stages: the one a warp freed last, which nothing is
      // fetched into before the next segment)
      auto part_of = [&](int w) -> float * {
        if constexpr (C::kCombInRing) {
          const int n = u_end > w ? (u_end - w + kWarps - 1) / kWarps : 1;      // units warp w has finished
          return reinterpret_cast<float *>(smem + (w * kDepth + (n - 1) % kDepth) * T::kBytes);
        } else {
          return reinterpret_cast<float *>(smem + C::kOffComb) + w * (C::kCombRows * kCombStride);
        }
      };
      // Row r of an uncut block: its normalised sum `acc` (of this lane's dv) and
      // base-2 log-sum-exp; the sink joins here.
      auto finish = [&](int r, float lse2, float4 acc) {
        const int flat = bd.row0 + r;
        const int tok = bd.tok0 + flat / a.group, h = bd.g * a.group + flat % a.group;
        const float sink2 = a.sinks ? __ldg(a.sinks + h) * kLog2e : -INFINITY;
        const float M = fmaxf(lse2, sink2);
        float f = a.v_scale, lse = lse2 * kLn2;
        if (sink2 != -INFINITY) {
          const float w = exp2f(lse2 - M), Z = w + exp2f(sink2 - M);
          f *= w / Z;
          lse = (M + log2f(Z)) * kLn2;
        }
        __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * f, acc.y * f);
        __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * f, acc.w * f);
        uint2 w2;
        w2.x = *reinterpret_cast<uint32_t *>(&lo);
        w2.y = *reinterpret_cast<uint32_t *>(&hi);
        *(reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + ((int64_t)tok * a.hq + h) * kDv) + lane) = w2;
        if (a.lse_out && lane == 0) a.lse_out[(int64_t)tok * a.hq + h] = lse;
      };
      bool synced = true;
#pragma unroll
      for (int nb0 = 0; nb0 < NB; nb0 += C::kCombRows / 8) {
      if (nb0 > 0 && nb0 * 8 >= bd.nrows) break;
      if (nb0 > 0 && !(synced = group_sync())) break;     // the previous rows have been read
      if (has) {
        float *dst = part_of(warp);
#pragma unroll
        for (int nc = 0; nc < C::kCombRows / 8; ++nc)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int nb = nb0 + nc;
            float sum = l[nb][x];
            sum += __shfl_xor_sync(0xffffffffu, sum, 4);
            sum += __shfl_xor_sync(0xffffffffu, sum, 8);
            sum += __shfl_xor_sync(0xffffffffu, sum, 16);
            const int r = 2 * t + x;
            if (g == 0) {
              // (nothing but NaN scores: no maximum, but the NaN sum counts)
              sm_m[warp][nb * 8 + r] = sum != sum && m[nb][x] == -INFINITY ? 0.f : m[nb][x];
              sm_l[warp][nb * 8 + r] = sum;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float2 *>(dst + (nc * 8 + r) * kCombStride + 16 * g +
                                          ((2 * i + 2 * (g >> 1)) & 15)) =
                  make_float2(o[i][nb][x], o[i][nb][2 + x]);
          }
      } else if (lane < C::kCombRows) {
        sm_m[warp][nb0 * 8 + lane] = -INFINITY;
      }
      if (!(synced = group_sync())) break;
      // a warp combines whole rows: lane owns dv 4 lane .. 4 lane + 3.  (Rolled loops:
      // this runs once per segment, and its time is the fetch of its code.)
#pragma unroll 1
      for (int r = nb0 * 8 + warp; r < min(bd.nrows, nb0 * 8 + C::kCombRows); r += kWarps) {
        float M = -INFINITY;
#pragma unroll 4
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w][r]);
        float Lsum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        const int gg = lane >> 2;
        const int p0 = 16 * gg + ((4 * (lane & 3) + 2 * (gg >> 1)) & 15);
        const int p1 = 16 * gg + ((4 * (lane & 3) + 2 + 2 * (gg >> 1)) & 15);
        if (M != -INFINITY) {
#pragma unroll 4
          for (int w = 0; w < kWarps; ++w) {
            const float mw = sm_m[w][r];
            if (mw == -INFINITY) continue;             // nothing written by this warp
            const float f = exp2f(mw - M);
            const float *src = part_of(w) + (r - nb0 * 8) * kCombStride;
            const float2 x = *reinterpret_cast<const float2 *>(src + p0);
            const float2 y = *reinterpret_cast<const float2 *>(src + p1);
            Lsum += f * sm_l[w][r];
            acc.x += f * x.x;
            acc.y += f * x.y;
            acc.z += f * y.x;
            acc.w += f * y.y;
          }
        }
        // O and the sums are both 2^kLift times what they stand for; a NaN stays one
        const float scale = Lsum == 0.f ? 0.f : 1.f / Lsum;
        const float lse = Lsum == 0.f ? -INFINITY : M + log2f(Lsum * 0.0078125f);
        acc.x *= scale, acc.y *= scale, acc.z *= scale, acc.w *= scale;
        if (bd.num_splits == 1) {
          finish(r, lse, acc);
        } else {
          const int prow = bd.part_row_base + sd.split * bd.nrows + r;
          acc.x *= a.v_scale, acc.y *= a.v_scale, acc.z *= a.v_scale, acc.w *= a.v_scale;
          reinterpret_cast<float4 *>(a.part_o + (int64_t)prow * kDv)[lane] = acc;
          if (lane == 0) a.part_lse[prow] = lse;
        }
      }
      }
      if (!synced) break;
      u0 = u_end;
      // the partials are free for the next segment once every warp has read them
      if (C::kCombInRing && TMA) tc::fence_proxy_async_smem();
      if (seg + 1 < head.seg_end && !group_sync()) break;
    }
  }
  if constexpr (TMA) {
    // after a give-up, the copies still in flight land before the CTA ends (a
    // bounded wait of its own that ignores the abort)
    int no_abort = 0;
    for (; done < issued; ++done)
      tc::mbar_wait(&bars.full[warp][done % kDepth], (done / kDepth) & 1, &no_abort, 100000000ull);
  } else {
    asm volatile("cp.async.wait_all;\n" ::: "memory");
  }
  __syncthreads();
  if (tid == 0 && abort_flag) atomicOr(a.err, 2);
  if (v_nan) patch_nan_rows(a, kN, kUnitKeys);
}

template <int DQK, int NB, bool TMA>
cudaError_t launch_one(const HostPlan &hp, const RunArgs &a, const TmaMaps &m, cudaStream_t st) {
  return launch_dependent(attn_fp4_kernel<DQK, NB, TMA>, dim3(hp.num_ctas), dim3(Cfg<DQK, NB>::kThreads), Cfg<DQK, NB>::kSmem, st, a, m);
}

template <int DQK, int NB, bool TMA>
cudaError_t prepare_one() {
  return cudaFuncSetAttribute(attn_fp4_kernel<DQK, NB, TMA>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Cfg<DQK, NB>::kSmem);
}

template <int DQK, int NB>
cudaError_t launch_nb(const HostPlan &hp, const RunArgs &a, const TmaMaps &m, cudaStream_t st) {
  return hp.use_tma ? launch_one<DQK, NB, true>(hp, a, m, st) : launch_one<DQK, NB, false>(hp, a, m, st);
}

template <int DQK, int NB>
cudaError_t prepare_nb(const HostPlan &hp) {
  return hp.use_tma ? prepare_one<DQK, NB, true>() : prepare_one<DQK, NB, false>();
}

template <int DQK>
cudaError_t launch_dqk(const HostPlan &hp, const RunArgs &a, const TmaMaps &m, cudaStream_t st) {
  switch (hp.fp4_rows) {
    case 8: return launch_nb<DQK, 1>(hp, a, m, st);
    case 16: return launch_nb<DQK, 2>(hp, a, m, st);
    default: return launch_nb<DQK, 4>(hp, a, m, st);
  }
}

template <int DQK>
cudaError_t prepare_dqk(const HostPlan &hp) {
  switch (hp.fp4_rows) {
    case 8: return prepare_nb<DQK, 1>(hp);
    case 16: return prepare_nb<DQK, 2>(hp);
    default: return prepare_nb<DQK, 4>(hp);
  }
}

}  // namespace

cudaError_t launch_attn_fp4(const HostPlan &hp, const RunArgs &a, const TmaMaps &m, cudaStream_t st) {
  if (hp.num_ctas == 0) return cudaSuccess;
  return hp.prob.head_dim_qk == kDqkSym ? launch_dqk<kDqkSym>(hp, a, m, st) : launch_dqk<kDqk>(hp, a, m, st);
}

cudaError_t prepare_attn_fp4(const HostPlan &hp) {
  return hp.prob.head_dim_qk == kDqkSym ? prepare_dqk<kDqkSym>(hp) : prepare_dqk<kDqk>(hp);
}

}  // namespace akp
