// attn_select_blocks: which blocks of the cache a new token attends to.
//
// For a token and KV head, with q^ the group's query rows in integers (|q^| <= 128, a
// power of two apart from the bf16 row) and hi, lo a block's 8-bit bounds:
//   d(h, c) = sum_d max(q^ hi, q^ lo) = q^+ . hi + q^- . lo,   q^+ = max(q^, 0), q^- = min(q^, 0),
// a contraction of 2 Dqk whole numbers that every step of fp16 x fp16 -> fp32 MMAs holds
// exactly (partial sums stay below 2^22), so that the order of summation plays no part
// and equal scores are equal bits.  The score is the largest over the group's heads.
//
// A cluster of CTAs takes one token of one KV head.  A warp scores 8 blocks at a time:
// lane (g, t) (g = lane / 4, t = lane % 4) reads 16-byte pieces t, t + 4, .. of the bounds
// of block g straight into registers (the order of a contraction's index is free, so
// that a piece feeds four MMAs) and widens them to fp16 there; the query rows wait in
// shared memory as operand fragments.  A row's factor 2^(e_h - max e) is applied as two powers
// of two, the first of which keeps every whole number exact, so that the product is rounded
// once however far the heads lie apart.  Scores meet as ordered integers in the shared
// memory of the cluster's first CTA, which finds the smallest one taken (by a warp bit by
// bit up to 512 scores, else by a radix select of 8 bits a pass) and writes the list in order.
//
// 32 requests of 1,024 to 32,767 tokens (16/2 heads, blocks of 64): 8.9 us, one of 16,384
// blocks (64/4 heads) 26 us, which the 26 MB of bounds would take 3.9 us to read: a chain
// of dependent loads (layout, page, bounds), the cluster's barriers and the passes over the
// scores by one CTA bound it, not the bandwidth.  Eight warps, no step ahead and clusters of
// eight at most: 13.9 and 87 us.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "attn_paged.h"
#include "kernels.hpp"
#include "plan.hpp"
#include "requests.cuh"
#include "select.cuh"

namespace akp {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxSmem = 224 * 1024;

// c (16 x 8, fp32) += a (16 x 16, fp16) . b (16 x 8, fp16)
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// The smallest factor that is one multiplication: from 2^-122 on a whole number times it is a
// normal fp32; what is left of it (2^-125 at least) is multiplied behind it.
constexpr int kLeastLog2 = -122;

template <int D>
struct QTile {                         // 16 query rows as A fragments, and their factors
  uint4 frag[D / 16][32];
  float factor[16];                    // 2^(e_h - E), at least 2^kLeastLog2; -1: no such row, or one that takes no part
};

// Row r of a token's query heads (r < group) as integers, D / 32 a lane in element order
// of the fragments; returns its exponent, or INT_MIN for a row that takes no part.
// Fragment order: k-step (j, s) holds for lane column t the dims 64 j + 16 t + 4 s + {0..3}.
template <int D>
__device__ __forceinline__ void stage_row(QTile<D> &tile, int r, const uint16_t *row, int lane, int *exps) {
  // lane owns dims 4 (lane + 32 k) ..: piece p = dims / 4
  constexpr int NP = D / 4, PL = (NP + 31) / 32;
  uint2 w[PL];
  float amax = 0.f;
  bool odd = false;
#pragma unroll
  for (int k = 0; k < PL; ++k) {
    const int p = lane + 32 * k;
    w[k] = make_uint2(0u, 0u);
    if (row && p < NP) w[k] = __ldg(reinterpret_cast<const uint2 *>(row) + p);
    const uint32_t x[2] = {w[k].x, w[k].y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float a = fabsf(__uint_as_float(x[i] << 16)), b = fabsf(__uint_as_float(x[i] & 0xFFFF0000u));
      odd |= !(a < INFINITY) || !(b < INFINITY);
      amax = fmaxf(amax, fmaxf(a, b));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  odd = __any_sync(0xffffffffu, odd) || !row;
  const int e = odd ? 0 : min(code_exponent(amax), 121);
  if (lane == 0) exps[r] = odd ? INT_MIN : e;
  const float unit = odd ? 0.f : pow2(-e);
#pragma unroll
  for (int k = 0; k < PL; ++k) {
    const int p = lane + 32 * k;
    if (p >= NP) break;
    float v[4] = {__uint_as_float(w[k].x << 16), __uint_as_float(w[k].x & 0xFFFF0000u),
                  __uint_as_float(w[k].y << 16), __uint_as_float(w[k].y & 0xFFFF0000u)};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = odd ? 0.f : rintf(v[i] * unit);
    const __half2 lo = __floats2half2_rn(v[0], v[1]), hi = __floats2half2_rn(v[2], v[3]);
    // dims 4p = 64 j + 16 t + 4 s: a lane (r % 8, t)'s words 0 (first pair), 2 (second), + 1 for rows 8..15
    const int j = p / 16, t = p / 4 % 4, s = p % 4;
    uint32_t *f = reinterpret_cast<uint32_t *>(&tile.frag[4 * j + s][(r & 7) * 4 + t]) + (r >> 3);
    f[0] = *reinterpret_cast<const uint32_t *>(&lo);
    f[2] = *reinterpret_cast<const uint32_t *>(&hi);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) select_kernel(const SelectArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  QTile<D> *tiles = reinterpret_cast<QTile<D> *>(smem);                        // [row_tiles]
  int *exps = reinterpret_cast<int *>(smem + a.row_tiles * sizeof(QTile<D>));  // [row_tiles * 16]
  uint32_t *keys = reinterpret_cast<uint32_t *>(exps + a.row_tiles * 16);      // [max_blocks]
  __shared__ int hist[256], sums[2][kWarps], pick[3];
  __shared__ int top_exp, far_apart;      // E, and whether a factor is below 2^kLeastLog2
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tok = blockIdx.x / ranks, g = blockIdx.y;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  Request rq;
  rq.seek(a.qo_indptr, a.seq_lens, a.batch, tok);
  const int b = rq.b;
  int32_t *out = a.block_idx + ((int64_t)tok * a.hkv + g) * a.take;
  const int q0 = rq.first, n = rq.end - q0;
  // a row that qo_indptr does not hold, or a request longer than the plan's (the whole
  // cluster): left as it was
  if (b >= a.batch || tok < q0 || n > a.max_len) {
    if (rank == 0 && tid == 0) atomicOr(a.err, 4);
    return;
  }
  const int L0 = (int)(rq.shift + rq.end), L = max(min(L0, a.max_len), n);
  if (L != L0 && tid == 0 && rank == 0) atomicOr(a.err, 4);
  const int own = (L - n + tok - q0) / a.block;             // the token's own block
  if (own < a.take) {                                       // all of them
    if (rank == 0)
      for (int k = tid; k < a.take; k += kThreads) out[k] = k <= own ? k : -1;
    return;
  }
  const int c_lo = a.first, c_hi = own - a.last + 1;        // the scored ones (take < own + 1: there are some)
  // the first CTA's keys may be written once all have started
  asm volatile("barrier.cluster.arrive.aligned;\n" ::: "memory");
  uint32_t *dst = cluster.map_shared_rank(keys, 0);
  // ---- a warp's bounds: 8 blocks at a time, on their way while the 8 before are at work,
  // their pages one step ahead of them
  const int gq = lane >> 2, t = lane & 3;
  const int per_page = a.page_size / a.block, step = ranks * kWarps * 8;
  struct Bounds {
    uint4 raw[2][D / 64];
    int e;
  } ahead;
  int c_at = c_lo + (rank * kWarps + warp) * 8;
  int32_t page = 0;
  auto look = [&](int c) { page = __ldg(a.page_table + (int64_t)b * a.pt_stride + min(c + gq, c_hi - 1) / per_page); };
  auto fetch = [&](int c) {
    c = min(c + gq, c_hi - 1);
    const bool bad = page < 0 || page >= a.num_pages;
    if (bad && t == 0) atomicOr(a.err, 1);
    const uint8_t *rec = a.bounds + (((int64_t)(bad ? 0 : page) * per_page + c % per_page) * a.hkv + g) *
                                        bounds_row_bytes(D);
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int j = 0; j < D / 64; ++j)
        ahead.raw[w][j] = bad ? make_uint4(0u, 0u, 0u, 0u) : __ldg(reinterpret_cast<const uint4 *>(rec + w * D) + 4 * j + t);
    ahead.e = bad ? 0 : (int)(int8_t)__ldg(rec + 2 * D);
  };
  if (c_at < c_hi) {
    look(c_at);
    fetch(c_at);
    look(c_at + step);
  }
  // ---- the query rows
  if (tid == 0) far_apart = 0;
  for (int r = warp; r < a.row_tiles * 16; r += kWarps) {
    const uint16_t *row = r < a.group ? a.q + ((int64_t)tok * a.hq + g * a.group + r) * D : nullptr;
    stage_row<D>(tiles[r >> 4], r & 15, row, lane, exps + (r & ~15));
  }
  __syncthreads();
  for (int r = tid; r < a.row_tiles * 16; r += kThreads) {
    int top = INT_MIN;
    for (int i = 0; i < a.group; ++i) top = max(top, exps[i]);
    const bool in = exps[r] != INT_MIN;
    tiles[r >> 4].factor[r & 15] = in ? pow2(max(exps[r] - top, kLeastLog2)) : -1.f;
    if (r == 0) top_exp = top;
    if (in && exps[r] - top < kLeastLog2) far_apart = 1;
  }
  __syncthreads();
  asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");
  // ---- scores
  for (; c_at < c_hi; c_at += step) {
    const Bounds now = ahead;
    if (c_at + step < c_hi) {
      fetch(c_at + step);
      look(c_at + 2 * step);
    }
    float best[2] = {-INFINITY, -INFINITY};
    for (int rt = 0; rt < a.row_tiles; ++rt) {
      float acc[2][4] = {};
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        const uint32_t up[4] = {now.raw[0][j].x, now.raw[0][j].y, now.raw[0][j].z, now.raw[0][j].w};
        const uint32_t dn[4] = {now.raw[1][j].x, now.raw[1][j].y, now.raw[1][j].z, now.raw[1][j].w};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const uint4 f = tiles[rt].frag[4 * j + s][lane];
          uint32_t b0, b1;
          const uint32_t pos[4] = {max_h2(f.x, 0u), max_h2(f.y, 0u), max_h2(f.z, 0u), max_h2(f.w, 0u)};
          s8x4_to_f16(up[s], b0, b1);
          mma16816(acc[0], pos, b0, b1);
          const uint32_t neg[4] = {min_h2(f.x, 0u), min_h2(f.y, 0u), min_h2(f.z, 0u), min_h2(f.w, 0u)};
          s8x4_to_f16(dn[s], b0, b1);
          mma16816(acc[1], neg, b0, b1);
        }
      }
      const float f0 = tiles[rt].factor[gq], f1 = tiles[rt].factor[gq + 8];
      float s[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) s[x] = (acc[0][x] + acc[1][x]) * (x < 2 ? f0 : f1);
      if (far_apart) {
        const int *e = exps + rt * 16 + gq;
        const float r0 = f0 < 0.f ? 1.f : pow2(min(e[0] - top_exp - kLeastLog2, 0));
        const float r1 = f1 < 0.f ? 1.f : pow2(min(e[8] - top_exp - kLeastLog2, 0));
#pragma unroll
        for (int x = 0; x < 4; ++x) s[x] *= x < 2 ? r0 : r1;
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (f0 >= 0.f) best[x] = fmaxf(best[x], s[x]);
        if (f1 >= 0.f) best[x] = fmaxf(best[x], s[2 + x]);
      }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) best[x] = fmaxf(best[x], __shfl_xor_sync(0xffffffffu, best[x], o));
      // column 2 t + x is block c_at + 2 t + x, whose exponent lane (2 t + x) * 4 holds
      const int ec = __shfl_sync(0xffffffffu, now.e, (2 * t + x) * 4);
      const int cc = c_at + 2 * t + x;
      if (gq == 0 && cc < c_hi) dst[cc] = ordered(ec == kOddBlock ? INFINITY : best[x] * pow2(max(ec, -126)));
    }
  }
  cluster.sync();
  if (rank != 0) return;
  // ---- the list: a warp by itself where its registers hold the scores
  const int total = own + 1, n_scored = c_hi - c_lo;
  if (n_scored <= 32 * kHeld) {
    if (warp == 0) pick_held(keys + c_lo, n_scored, a.take - (total - n_scored), c_lo, out + c_lo, lane);
    for (int c = tid; c < c_lo; c += kThreads) out[c] = c;
    for (int c = c_hi + tid; c <= own; c += kThreads) out[a.take - (total - c)] = c;
    return;
  }
  // forced blocks are above every score
  uint32_t least = 0xFFFFFFFFu, most = 0u;
#pragma unroll 4
  for (int c = c_lo + tid; c < c_hi; c += kThreads) {
    least = min(least, keys[c]);
    most = max(most, keys[c]);
  }
  least = __reduce_min_sync(0xffffffffu, least);
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) {
    sums[0][warp] = (int)least;
    sums[1][warp] = (int)most;
  }
  for (int c = tid; c < c_lo; c += kThreads) keys[c] = 0xFFFFFFFFu;
  for (int c = c_hi + tid; c <= own; c += kThreads) keys[c] = 0xFFFFFFFFu;
  __syncthreads();
  for (int w = 0; w < kWarps; ++w) {
    least = min(least, (uint32_t)sums[0][w]);
    most = max(most, (uint32_t)sums[1][w]);
  }
  // The bits that all scores share need no pass; the others by 8 a pass, until all that share
  // the prefix are in.
  int bits = 32 - __clz(least ^ most);
  uint32_t prefix = bits < 32 ? most >> bits << bits : 0u;
  int want = a.take - (total - n_scored);      // rank within the scores that share the prefix
  bool whole = want <= 0;
  if (whole) prefix = 0xFFFFFFFFu;
  while (bits > 0 && !whole) {
    const int shift = max(bits - 8, 0);
    __syncthreads();
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
#pragma unroll 4
    for (int c = c_lo + tid; c < c_hi; c += kThreads) {
      const uint32_t k = keys[c];
      if (bits == 32 || (k ^ prefix) >> bits == 0u) atomicAdd(&hist[(k >> shift) & ((1u << (bits - shift)) - 1u)], 1);
    }
    __syncthreads();
    if (warp == 0) {                           // from the highest bin down: lane owns 8 bins
      int cnt[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        cnt[i] = hist[255 - (lane * 8 + i)];
        sum += cnt[i];
      }
      int before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
      }
      before -= sum;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (before < want && before + cnt[i] >= want) {
          pick[0] = 255 - (lane * 8 + i);
          pick[1] = want - before;
          pick[2] = want - before == cnt[i];
        }
        before += cnt[i];
      }
    }
    __syncthreads();
    prefix |= (uint32_t)pick[0] << shift;
    want = pick[1];
    whole = pick[2] != 0;
    bits = shift;
  }
  if (whole) {                                 // all from `prefix` on: above its predecessor
    --prefix;
    want = 0;
  }
  // keys above `prefix` are in, and the first `want` equal to it; a warp takes a range
  __syncthreads();
  const int span = ((total + kWarps - 1) / kWarps + 31) & ~31;
  const int w_lo = warp * span, w_hi = min(total, w_lo + span);
  int above = 0, equal = 0;
  for (int c = w_lo + lane; c < w_hi; c += 32) {
    above += keys[c] > prefix;
    equal += keys[c] == prefix;
  }
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) {
    sums[0][warp] = above;
    sums[1][warp] = equal;
  }
  __syncthreads();
  int eq_before = 0, at = 0;
  for (int w = 0; w < warp; ++w) {
    at += sums[0][w];
    eq_before += sums[1][w];
  }
  at += min(eq_before, want);
  for (int c = w_lo; c < w_hi; c += 32) {
    const uint32_t k = c + lane < w_hi ? keys[c + lane] : 0u;
    const bool is_eq = c + lane < w_hi && k == prefix;
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t eq = __ballot_sync(0xffffffffu, is_eq);
    const bool in = c + lane < w_hi && (k > prefix || (is_eq && eq_before + __popc(eq & below) < want));
    const uint32_t m = __ballot_sync(0xffffffffu, in);
    if (in) out[at + __popc(m & below)] = c + lane;
    at += __popc(m);
    eq_before += __popc(eq);
  }
}

template <int D>
size_t smem_of(int row_tiles, int max_blocks) {
  return row_tiles * (sizeof(QTile<D>) + 16 * sizeof(int)) + (size_t)max_blocks * 4;
}

template <int D>
cudaError_t launch(const SelectArgs &a, int64_t tokens, int num_sms, int device, cudaStream_t st) {
  const size_t smem = smem_of<D>(a.row_tiles, a.max_blocks);
  static SmemLimit limit;
  const void *kernel = reinterpret_cast<const void *>(select_kernel<D>);
  cudaError_t e = limit.raise(kernel, device, kMaxSmem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  // CTAs of a cluster: while there are SMs for them, and 64 blocks for each (16: more than
  // every device has to offer; this one does)
  int ranks = 1;
  while (ranks < 16 && tokens * a.hkv * ranks * 2 <= num_sms && a.max_blocks >= ranks * 2 * 64) ranks *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(tokens * ranks), (unsigned)a.hkv);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, select_kernel<D>, a);
}

}  // namespace

attn_status_t check_sparse(const HostPlan &hp, const attn_sparse_t *s) {
  if (!s) return ATTN_ERR_INVALID_ARG;
  if (!block_size_ok(hp.prob, s->block_size)) return ATTN_ERR_UNSUPPORTED;
  if (s->num_blocks < 1 || s->num_blocks > ATTN_SPARSE_MAX_TAKE || s->first_blocks < 0 || s->last_blocks < 1 ||
      (int64_t)s->first_blocks + s->last_blocks > s->num_blocks || hp.prob.window > 0)
    return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

int32_t longest_request(const HostPlan &hp) {
  const int64_t slots = (int64_t)hp.prob.page_table_stride * hp.prob.page_size;
  int32_t top = 0;
  for (const int32_t L : hp.seq_lens) top = std::max(top, L);
  return (int32_t)std::min<int64_t>(top, slots);
}

// What a selection has of its plan, and whether its longest request may have so many blocks.
static attn_status_t plan_args(const HostPlan &hp, const attn_sparse_t *sparse, SelectArgs *a) {
  const attn_status_t ok = check_sparse(hp, sparse);
  if (ok != ATTN_OK) return ok;
  const attn_problem_t &pr = hp.prob;
  a->max_len = longest_request(hp);
  a->max_blocks = (a->max_len + sparse->block_size - 1) / sparse->block_size;
  if (a->max_blocks > ATTN_SPARSE_MAX_BLOCKS) return ATTN_ERR_UNSUPPORTED;
  a->batch = pr.batch;
  a->hq = pr.num_q_heads;
  a->hkv = pr.num_kv_heads;
  a->group = hp.group;
  a->row_tiles = (hp.group + 15) / 16;
  a->page_size = pr.page_size;
  a->pt_stride = pr.page_table_stride;
  a->num_pages = pr.num_pages;
  a->block = sparse->block_size;
  a->take = sparse->num_blocks;
  a->first = sparse->first_blocks;
  a->last = sparse->last_blocks;
  a->tokens = hp.qo_indptr.back();
  return ATTN_OK;
}

static bool fits_smem(const HostPlan &hp, const SelectArgs &a) {
  return (hp.prob.head_dim_qk == kDqk ? smem_of<kDqk>(a.row_tiles, a.max_blocks)
                                      : smem_of<kDqkSym>(a.row_tiles, a.max_blocks)) <= kMaxSmem;
}

}  // namespace akp

extern "C" attn_status_t attn_plan_select_ctas(attn_plan_t plan, const attn_sparse_t *sparse, int32_t *ctas) {
  if (!plan || !ctas) return ATTN_ERR_INVALID_ARG;
  *ctas = 0;
  akp::SelectArgs a{};
  const attn_status_t ok = akp::plan_args(plan->host, sparse, &a);
  if (ok != ATTN_OK || a.tokens == 0) return ok;
  if (!akp::fits_smem(plan->host, a)) return ATTN_ERR_UNSUPPORTED;
  *ctas = akp::select_tc_ranks(plan->host, a);
  return ATTN_OK;
}

extern "C" attn_status_t attn_select_blocks(attn_plan_t plan, const attn_sparse_t *sparse, const void *q,
                                            const void *bounds, const int32_t *page_table, const int32_t *seq_lens,
                                            const int32_t *qo_indptr, int32_t *block_idx, void *stream) {
  if (!plan || plan->device < 0) return ATTN_ERR_INVALID_ARG;
  const akp::HostPlan &hp = plan->host;
  const attn_problem_t &pr = hp.prob;
  akp::SelectArgs a{};
  const attn_status_t ok = akp::plan_args(hp, sparse, &a);
  if (ok != ATTN_OK || a.tokens == 0) return ok;
  if (!q || !bounds || !page_table || !seq_lens || !qo_indptr || !block_idx || !akp::aligned16(q) ||
      !akp::aligned16(bounds))
    return ATTN_ERR_INVALID_ARG;
  a.q = static_cast<const uint16_t *>(q);
  a.bounds = static_cast<const uint8_t *>(bounds);
  a.page_table = page_table;
  a.seq_lens = seq_lens;
  a.qo_indptr = qo_indptr;
  a.block_idx = block_idx;
  a.err = plan->dev.err;
  if (!akp::fits_smem(hp, a)) return ATTN_ERR_UNSUPPORTED;
  akp::DeviceGuard dev(plan->device);
  if (!dev.ok) return ATTN_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (akp::select_tc_ranks(hp, a))
    return akp::launch_select_tc(hp, a, plan->device, st) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
  const cudaError_t e = pr.head_dim_qk == akp::kDqk ? akp::launch<akp::kDqk>(a, a.tokens, hp.num_sms, plan->device, st)
                                                    : akp::launch<akp::kDqkSym>(a, a.tokens, hp.num_sms, plan->device, st);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
