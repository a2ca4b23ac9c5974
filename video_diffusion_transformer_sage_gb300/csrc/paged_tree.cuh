// paged_tree.cuh -- device side: which keys a drafted token sees when a sequence's new tokens are a tree.
//
// Of n new tokens behind P = len - n cached ones, row j sees the keys below P (with a window those from
// P + depth_j + 1 - window on) and the new tokens whose bit is set in its row of the mask.
#pragma once
#include "paged_internal.h"

namespace sage {

// Keys that every row of a sequence sees, [alo, ahi), and those that some row may see, [ulo, uhi): depths lie in [0, n).
__device__ __forceinline__ void tree_keys(const PagedAttnArgs& a, int len, int n_new, int& alo, int& ahi, int& ulo, int& uhi) {
  const int prefix = len - n_new;
  ulo = a.window > 0 ? max(0, prefix + 1 - a.window) : 0;
  alo = a.window > 0 ? max(0, prefix + n_new - a.window) : 0;
  ahi = max(0, prefix);
  uhi = len;
}

// The cached keys [lo, hi) that row j of the sequence sees (`start`: its row 0); lo >= hi: none.
__device__ __forceinline__ void tree_row_keys(const PagedAttnArgs& a, int start, int len, int n_new, int j, int& lo, int& hi) {
  const int prefix = len - n_new;
  hi = max(0, prefix);
  lo = 0;
  if (a.window > 0) lo = max(0, prefix + 1 - a.window + min(max(__ldg(a.depth + start + j), 0), n_new - 1));
}

// Bits [at, at + kBits) of row t's mask, at any offset: 0 outside its words.
template <int kBits>
__device__ __forceinline__ uint64_t tree_bits(const PagedAttnArgs& a, int t, int at) {
  const uint32_t* row = a.mask + t * a.mask_stride;
  const int w0 = at >> 5, shift = at & 31;   // (rounds down for a negative offset)
  auto word = [&](int w) -> uint32_t { return w >= 0 && w < a.mask_words ? __ldg(row + w) : 0u; };
  const uint32_t x0 = word(w0), x1 = word(w0 + 1), x2 = kBits > 32 ? word(w0 + 2) : 0u;
  return static_cast<uint64_t>(__funnelshift_r(x1, x2, shift)) << 32 | __funnelshift_r(x0, x1, shift);
}

// Bits [lo, hi) of 64, any lo and hi.
__device__ __forceinline__ uint64_t key_range(int lo, int hi) {
  lo = max(lo, 0);
  hi = min(hi, 64);
  return lo >= hi ? 0ull : (~0ull >> (64 - (hi - lo))) << lo;
}

// Whether key k0 + lane is cached text or a new token that some of the tokens j0 .. j1 (of the sequence with row 0 `start`)
// sees.  Called by a whole warp with the same arguments.
__device__ __forceinline__ bool tree_key_seen(const PagedAttnArgs& a, int start, int j0, int j1, int k0, int prefix) {
  if (k0 + 32 <= prefix) return true;
  const int lane = threadIdx.x & 31;
  uint32_t some = 0;
  for (int j = j0 + lane; j <= j1; j += 32) some |= static_cast<uint32_t>(tree_bits<32>(a, start + j, k0 - prefix));
  some = __reduce_or_sync(0xffffffffu, some);
  return k0 + lane < prefix || ((some >> lane) & 1u);
}

}  // namespace sage
