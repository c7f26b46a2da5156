// What the kernels of attn_run_sparse share (attn_sparse.cu, attn_sparse_tc.cu).
#pragma once
#include <cstdint>

#include "kernels.hpp"
#include "sparse.cuh"

namespace akp {

struct SparseArgs {
  const uint16_t *q;
  const void *k_cache, *v_cache;
  const int32_t *page_table, *seq_lens, *qo_indptr, *block_idx;
  const float *sinks;
  uint16_t *out;
  float *lse;
  int32_t *err;
  float scale_log2, v_scale;
  int32_t batch, hq, hkv, group, row_tiles, page_size, pt_stride, num_pages;
  int32_t tokens, block, take, max_len;
  // chunks of tokens (attn_sparse_tc.cu): jobs of job_tokens tokens of one request and KV
  // head, and whether a job is left to the kernel that takes every unit by itself
  int32_t jobs, job_tokens;
  int32_t *redo;
};

// Job number `job` as its KV head, request and tokens [tok0, tok0 + ntok), whose first one
// stands at pos0 of `len` keys.  All 32 lanes of a warp call it; false: past the device's
// layout.
struct SparseJob {
  int g, b, tok0, ntok, pos0, len;
};
__device__ __forceinline__ bool find_job(const SparseArgs &a, int job, SparseJob &x, bool report) {
  const int lane = threadIdx.x & 31;
  x.g = job % a.hkv;
  const int want = job / a.hkv;
  int base = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    const int r = b0 + lane;
    int q0 = 0, n = 0, L = 0;
    if (r < a.batch) {
      q0 = __ldg(a.qo_indptr + r);
      n = max(0, __ldg(a.qo_indptr + r + 1) - q0);
      L = __ldg(a.seq_lens + r);
    }
    const int cnt = (n + a.job_tokens - 1) / a.job_tokens;
    int sum = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, base + sum > want);
    if (past) {
      const int l = __ffs(past) - 1;
      const int k = want - base - __shfl_sync(0xffffffffu, sum - cnt, l);      // the request's job
      const int Lc = max(min(L, a.max_len), n);
      if (report && lane == l && Lc != L) atomicOr(a.err, 4);
      x.b = b0 + l;
      n = __shfl_sync(0xffffffffu, n, l);
      x.len = __shfl_sync(0xffffffffu, Lc, l);
      x.tok0 = __shfl_sync(0xffffffffu, q0, l) + k * a.job_tokens;
      x.ntok = min(a.job_tokens, n - k * a.job_tokens);
      x.pos0 = x.len - n + k * a.job_tokens;
      // (a layout of more tokens than the plan's, or longer: nothing past the arrays)
      return x.tok0 >= 0 && x.tok0 + x.ntok <= a.tokens && x.pos0 + x.ntok <= a.max_len;
    }
    base += __shfl_sync(0xffffffffu, sum, 31);
  }
  return false;
}

// The mark of a row that attn_sparse_tc.cu leaves to the other kernel: a NaN as the first
// value of either half of its output.
constexpr uint16_t kMark = 0x7FFF;

// What a row's maximum and sum make of its output: the factor of O and the natural
// log-sum-exp; sink2 in base 2.
__device__ __forceinline__ float finish(float m, float l, float lift, float sink2, float v_scale, float &lse) {
  const float lse2 = l == 0.f ? -INFINITY : m + log2f(l) - lift;
  float f = l == 0.f ? 0.f : v_scale / l;
  const float M = fmaxf(lse2, sink2);
  lse = lse2 * 0.6931471805599453f;
  if (sink2 != -INFINITY) {
    const float w = exp2f(lse2 - M), Z = w + exp2f(sink2 - M);
    f *= w / Z;
    lse = (M + log2f(Z)) * 0.6931471805599453f;
  }
  return f;
}

// Tokens of a job for a group of `group` heads (0: the group is too large).
constexpr int kSparseTileRows = 128;
inline int sparse_job_tokens(int group) {
  return group > kSparseTileRows ? 0 : kSparseTileRows / group < 64 ? kSparseTileRows / group : 64;
}
inline int64_t sparse_jobs(const HostPlan &hp) {
  const int per = sparse_job_tokens(hp.group);
  if (per == 0) return 0;
  int64_t jobs = 0;
  for (size_t b = 0; b + 1 < hp.qo_indptr.size(); ++b) jobs += (hp.qo_indptr[b + 1] - hp.qo_indptr[b] + per - 1) / per;
  return jobs * hp.prob.num_kv_heads;
}

cudaError_t launch_sparse_tc(const HostPlan &hp, const SparseArgs &a, const TmaMaps &maps, int device,
                             cudaStream_t st);

}  // namespace akp
