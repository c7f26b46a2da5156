// Which request a flat row of a prefix-sum array (qo_indptr, kv_indptr) belongs to.
#pragma once
#include <cstdint>

namespace akp {

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

// The request of consecutive rows of a prefix-sum array, in registers: looked up
// once, then only when a row lies past its end.  `shift`: the position of row t in
// its request is t + shift (the last row is the request's last key).
struct Request {
  int b = -1, first = 0, end = 0;      // rows [first, end)
  int64_t shift = 0;
  __device__ __forceinline__ void seek(const int32_t *indptr, const int32_t *seq_lens, int batch, int64_t row) {
    if (b >= 0 && row < end) return;
    if (batch <= 32) {                 // everything in one round of loads, a request a lane
      const int lane = threadIdx.x & 31;
      int lo = 0, hi = 0, len = 0;
      if (lane < batch) {
        lo = __ldg(indptr + lane);
        hi = __ldg(indptr + lane + 1);
        len = __ldg(seq_lens + lane);
      }
      b = __popc(__ballot_sync(0xffffffffu, lane < batch && hi <= row));
      first = __shfl_sync(0xffffffffu, lo, b & 31);
      end = __shfl_sync(0xffffffffu, hi, b & 31);
      shift = (int64_t)__shfl_sync(0xffffffffu, len, b & 31) - end;
      return;
    }
    b = request_of(indptr, batch, row);
    if (b < batch) {
      first = __ldg(indptr + b);
      end = __ldg(indptr + b + 1);
      shift = (int64_t)__ldg(seq_lens + b) - end;
    }
  }
};

}  // namespace akp
