// paged_pool_walk.h -- how the accounting walks through the counts of all pages: which part is whose, in which steps.  Plain
// integer arithmetic, the same on host and device.
//
// Page numbers are below 2^31 and steps of kPoolStep pages may end up to a step behind the last one, so they are counted
// without sign: in 32 bits with one the last step's end is negative, and the walk begins again in front of the counts.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define SAGE_HD __host__ __device__ __forceinline__
#else
#define SAGE_HD inline
#endif

namespace sage {

constexpr int kPoolTile = 128;                          // pages that a warp looks at together, four to a lane
constexpr int kPoolKept = 16;                           // tiles of a step
constexpr uint32_t kPoolStep = kPoolTile * kPoolKept;

struct PoolPart {
  uint32_t from, to;
};
// Warp `warp` of `warps` takes the pages [from, to).
SAGE_HD PoolPart pool_part(uint32_t n_pages, int warp, int warps) {
  const uint64_t tiles = (static_cast<uint64_t>(n_pages) + kPoolTile - 1) / kPoolTile;
  const uint64_t from = tiles * warp / warps * kPoolTile, to = tiles * (warp + 1) / warps * kPoolTile;
  return {static_cast<uint32_t>(from < n_pages ? from : n_pages), static_cast<uint32_t>(to < n_pages ? to : n_pages)};
}
// The first of a lane's four pages in tile k of the step at p0.
SAGE_HD uint32_t pool_four(uint32_t p0, int k, int lane) { return p0 + k * kPoolTile + lane * 4; }
// Whether the four pages from p on lie before `to`.
SAGE_HD bool pool_four_whole(uint32_t p, uint32_t to) { return p < to && to - p >= 4; }

}  // namespace sage
