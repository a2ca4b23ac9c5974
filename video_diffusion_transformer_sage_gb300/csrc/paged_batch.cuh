// paged_batch.cuh -- device side: finding a token's sequence and its bounds; a row's log-sum-exp.
#pragma once
#include <cmath>

#include "paged_internal.h"
#include "sm103_ptx.cuh"
#include "status.cuh"

namespace sage {

// The rows of sequence b, [start, end), whatever cu_q holds: inside [0, n_tokens), never reversed.
__device__ __forceinline__ void seq_rows(const PagedBatchDev& b, int s, int& start, int& end) {
  start = min(max(__ldg(b.cu_q + s), 0), b.n_tokens);
  end = min(max(__ldg(b.cu_q + s + 1), start), b.n_tokens);
}

// The sequence whose rows hold row t, or -1.  Every lane of the warp calls it with the same t: each
// step compares 32 evenly spaced entries of cu_q, so 1024 sequences take two loads in a row.
__device__ __forceinline__ int find_seq(const PagedBatchDev& b, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = b.n_seqs;
  while (true) {
    const int step = (n + 31) / 32;
    const int off = lane * step;
    const bool le = off < n && __ldg(b.cu_q + lo + off) <= t;
    const uint32_t m = __ballot_sync(0xffffffffu, le);
    if (m == 0) return -1;
    const int k = (31 - __clz(m)) * step;
    lo += k;
    n = min(step, n - k);
    if (step == 1) break;
  }
  return t < __ldg(b.cu_q + lo + 1) ? lo : -1;
}

// log2 of how far P is lifted where it is held as fp16 (E4M3 cache): with the running maximum taken 2^7 lower than it is, P
// lies in [0, 2^15], still inside fp16, and the subnormals, where it loses precision, begin at 2^-21 of the row's
// largest instead of 2^-14 (weights of 2^-22 beside one with V = 0 came out up to 15 % off).
constexpr float kLiftE4M3 = 7.0f;

// A row's natural log-sum-exp of its maximum (log2 units) and sum: -infinity for a row that saw no key (l = 0), NaN where
// its scores are no numbers.
__device__ __forceinline__ float lse_of(float m, float l) {
  return l > 0.0f ? (m + log2f(l)) * 0.6931471805599453f : l == 0.0f ? -INFINITY : l;
}

}  // namespace sage
