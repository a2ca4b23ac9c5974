// paged_kept.h -- which items of a long list sage_paged_compact has to read before it writes an item.  Plain integer arithmetic,
// the same on host and device.
//
// Entry i of a list moves to place first + i, and keep[i] >= first + i ascends.  So the tokens that stand in the new places of
// an item's entries [i0, i0 + count) and move themselves in an earlier item are the entries before i0 whose keep lies in
// [first + i0, first + i0 + count): as many as the item has, at most, from the first that is not below first + i0 (in a list with
// gaps fewer: an item may then wait for one more than it has to).
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define SAGE_HD __host__ __device__ __forceinline__
#else
#define SAGE_HD inline
#endif

namespace sage {

// The last entry of part `lane` of 32 parts of `step` entries (the last ones shorter, or empty), of n from `lo` on.
SAGE_HD int kept_part_end(int lo, int step, int n, int lane) {
  const int end = (lane + 1) * step;
  return lo + (end < n ? end : n) - 1;
}

// The first of n ascending entries that is not below a place (n: none).  below(lo, step, n): how many of the 32 parts' last
// entries (kept_part_end) are below it.
template <typename F>
SAGE_HD int kept_search(int n, F&& below) {
  int lo = 0;
  while (n > 0) {
    const int step = (n + 31) / 32, whole = below(lo, step, n) * step;   // entries of parts that lie below as a whole
    const int skip = whole < n ? whole : n;
    lo += skip;
    if (step == 1 || skip == n) break;
    n = (step < n - skip ? step : n - skip) - 1;   // (a part's last entry is known)
  }
  return lo;
}

// The items `near` .. `far` before this one (far 0: none) hold those; `from`: the first entry before i0 not below
// first + i0; `tokens`: entries of an item.
struct KeptWait {
  uint32_t near, far;
};
SAGE_HD KeptWait kept_wait(int i0, int count, int tokens, int from) {
  const int end = i0 < from + count ? i0 : from + count;
  if (from >= end) return {0, 0};
  return {static_cast<uint32_t>(i0 / tokens - (end - 1) / tokens), static_cast<uint32_t>(i0 / tokens - from / tokens)};
}

}  // namespace sage
