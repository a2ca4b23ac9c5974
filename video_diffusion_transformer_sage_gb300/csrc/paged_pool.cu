// paged_pool.cu -- the accounting of the cache's pages (include/sage_paged_pool.h): which are free, who holds which.
//
// What bounds it: launches and chains of dependent loads; the counts of all pages are read once or twice (4 bytes a page).
//
// Release is a plain kernel, an entry to a thread.  Reserve and fork hand out the free pages in ascending order, which needs
// the number of free pages before each one: one cluster of eight CTAs does the whole call, with barriers of the cluster
// between its steps (a launch each would cost more than the steps do):
//   1  each warp counts what its rows need and the free pages of its part of the counts;
//   2  every CTA adds up both (sums of a few hundred numbers, cheaper than a barrier more), each warp writes the numbers of
//      its free pages to their places in the list, as far as they are needed;
//   3  each warp gives its rows the pages from their place in the list on.
// A fork's full pages are shared in step 2 already: whether anybody holds them is asked of counts that no page given out has
// changed yet, and those that change there, of pages held, stay above 0.
#include "paged_batch.cuh"
#include "paged_check.h"
#include "paged_pool_walk.h"
#include "sage_paged_pool.h"

namespace sage {
namespace {

constexpr int kPoolCtas = 8, kPoolThreads = 1024, kPoolWarps = kPoolThreads / 32;
constexpr int kReleaseThreads = 256, kReleasePer = 4;

struct PoolArgs {
  int32_t* refs;
  int n_pages;
  int32_t* table;
  int64_t table_stride;
  int n_rows, max_pages, page_shift;
  const int32_t *lo, *hi;          // release, reserve
  const int32_t *src, *dst, *len;  // fork
  int n_forks;
  int32_t *copy_src, *copy_dst, *copy_tokens;
  int32_t* ok;
  int32_t* status;
  int32_t* need;   // [n_rows] (or [n_forks]): pages asked for
  int32_t* sums;   // [kPoolCtas * kPoolWarps]: free pages of each warp's part
  int32_t* list;   // [n_pages]: the free pages in ascending order
};

// What one CTA of the cluster wrote before it, the others read behind it (past L1: __ldcg).
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ int warp_sum(int x) { return __reduce_add_sync(0xffffffffu, x); }
__device__ __forceinline__ int warp_scan(int x) {   // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += up;
  }
  return x;
}

// ------------------------------------------------------------------------------------------- release
__global__ void __launch_bounds__(kReleaseThreads) paged_release_kernel(const __grid_constant__ PoolArgs a) {
  for (int row = blockIdx.y; row < a.n_rows; row += gridDim.y) {
    const int lo = a.lo ? __ldg(a.lo + row) : 0, hi = __ldg(a.hi + row);
    int32_t* entries = a.table + row * a.table_stride;
    int page[kReleasePer];
#pragma unroll
    for (int k = 0; k < kReleasePer; ++k) {
      const int i = (blockIdx.x * kReleasePer + k) * kReleaseThreads + threadIdx.x;
      // Positions [i, i + 1) << page_shift, at most 2^30.
      const bool out = i < a.max_pages && (((i + 1) << a.page_shift) <= lo || (i << a.page_shift) >= hi || hi <= lo);
      page[k] = out ? entries[i] : -1;
    }
#pragma unroll
    for (int k = 0; k < kReleasePer; ++k) {
      if (page[k] < 0) continue;
      entries[(blockIdx.x * kReleasePer + k) * kReleaseThreads + threadIdx.x] = -1;
      if (page[k] >= a.n_pages) {
        record_bad_index(a.status, kWherePage);
      } else if (atomicSub(a.refs + page[k], 1) <= 0) {
        atomicAdd(a.refs + page[k], 1);
        record_bad_index(a.status, kWhereCount);
      }
    }
  }
}

// ------------------------------------------------------------------------------------------- reserve, fork
// This warp's part of the counts.
__device__ __forceinline__ PoolPart part_of_counts(const PoolArgs& a) {
  return pool_part(a.n_pages, blockIdx.x * kPoolWarps + (threadIdx.x >> 5), kPoolCtas * kPoolWarps);
}
// Bit j: page p + j is free, of the four from p on.
__device__ __forceinline__ uint32_t free_of_four(const PoolArgs& a, uint32_t p, uint32_t to) {
  int c[4] = {1, 1, 1, 1};
  if (pool_four_whole(p, to)) {
    const int4 v = __ldcg(reinterpret_cast<const int4*>(a.refs + p));
    c[0] = v.x; c[1] = v.y; c[2] = v.z; c[3] = v.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (p + j < to) c[j] = __ldcg(a.refs + p + j);
  }
  return (c[0] == 0) | (c[1] == 0) << 1 | (c[2] == 0) << 2 | (c[3] == 0) << 3;
}
// A warp's part of up to kPoolStep pages (all of 2^19) is kept as bits between counting and listing.
__device__ __forceinline__ uint64_t count_free(const PoolArgs& a) {
  const int lane = threadIdx.x & 31;
  const PoolPart part = part_of_counts(a);
  int n = 0;
  uint64_t kept = 0;
  for (uint32_t p0 = part.from; p0 < part.to; p0 += kPoolStep) {
    uint32_t f[kPoolKept];
#pragma unroll
    for (int k = 0; k < kPoolKept; ++k) {
      const uint32_t p = pool_four(p0, k, lane);
      f[k] = p < part.to ? free_of_four(a, p, part.to) : 0;
    }
    kept = 0;
#pragma unroll
    for (int k = 0; k < kPoolKept; ++k) kept |= static_cast<uint64_t>(f[k]) << (4 * k);
    n += __popcll(kept);
  }
  n = warp_sum(n);
  if (lane == 0) a.sums[blockIdx.x * kPoolWarps + (threadIdx.x >> 5)] = n;
  return kept;
}
// Writes this warp's free pages to the list, which begins with `before` of other warps', up to `most` in all.
__device__ __forceinline__ void list_free(const PoolArgs& a, uint64_t kept, int before, int64_t most) {
  const int lane = threadIdx.x & 31;
  const PoolPart part = part_of_counts(a);
  for (uint32_t p0 = part.from; p0 < part.to && before < most; p0 += kPoolStep) {
    if (part.to - part.from > kPoolStep) {   // more than was kept: read again
      kept = 0;
      for (int k = 0; k < kPoolKept; ++k) {
        const uint32_t p = pool_four(p0, k, lane);
        if (p < part.to) kept |= static_cast<uint64_t>(free_of_four(a, p, part.to)) << (4 * k);
      }
    }
    // The free pages of four groups of 128 added up at a time, a byte each (at most 128).
#pragma unroll
    for (int k4 = 0; k4 < kPoolKept; k4 += 4) {
      const uint32_t bits = static_cast<uint32_t>(kept >> (4 * k4)) & 0xFFFFu;
      uint32_t mine = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) mine |= __popc((bits >> (4 * k)) & 15u) << (8 * k);
      const uint32_t incl = static_cast<uint32_t>(warp_scan(static_cast<int>(mine)));
      const uint32_t all = __shfl_sync(0xffffffffu, incl, 31);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        int at = before + static_cast<int>(((incl >> (8 * k)) & 255u) - ((mine >> (8 * k)) & 255u));
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if ((bits >> (4 * k + j)) & 1u) {
            if (at < most) a.list[at] = static_cast<int>(pool_four(p0, k4 + k, lane) + j);
            ++at;
          }
        before += static_cast<int>((all >> (8 * k)) & 255u);
      }
    }
  }
}

// Of the needs [0, n) whose own part is [from, to): the sums before `from` and of all, by every thread of the CTA; the free
// pages of warps before this one, and of all.
struct PoolSums {
  int64_t before, all;
  int free_before, free_all;
};
template <typename F>
__device__ __forceinline__ PoolSums add_up(const PoolArgs& a, int n, int from, F need, int64_t (*sh)[kPoolWarps]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t s0 = 0, s1 = 0;
  for (int i = threadIdx.x; i < n; i += kPoolThreads) {
    const int x = need(i);
    s1 += x;
    s0 += i < from ? x : 0;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s0 += __shfl_xor_sync(0xffffffffu, s0, o);
    s1 += __shfl_xor_sync(0xffffffffu, s1, o);
  }
  if (lane == 0) {
    sh[0][warp] = s0;
    sh[1][warp] = s1;
  }
  PoolSums r;
  r.free_before = r.free_all = 0;
  const int me = blockIdx.x * kPoolWarps + warp;
#pragma unroll
  for (int k = 0; k < kPoolCtas * kPoolWarps / 32; ++k) {
    const int x = __ldcg(a.sums + k * 32 + lane);
    r.free_all += x;
    r.free_before += k * 32 + lane < me ? x : 0;
  }
  r.free_all = warp_sum(r.free_all);
  r.free_before = warp_sum(r.free_before);
  __syncthreads();
  s0 = sh[0][lane];
  s1 = sh[1][lane];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s0 += __shfl_xor_sync(0xffffffffu, s0, o);
    s1 += __shfl_xor_sync(0xffffffffu, s1, o);
  }
  r.before = s0;
  r.all = s1;
  return r;
}
// For each of the CTA's items in turn, a warp to an item: place(item, its first place in the list), with the needs of the items
// before it.
template <typename F, typename G>
__device__ __forceinline__ void for_each_in_order(int from, int to, int64_t before, F need, G place) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i0 = from; i0 < to; i0 += kPoolWarps) {
    // (Warp w's item is i0 + w; every warp adds up the 32 needs.)
    const int x = i0 + lane < to ? need(i0 + lane) : 0;
    int64_t incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    const int64_t at = before + __shfl_sync(0xffffffffu, incl - x, warp);
    if (i0 + warp < to) place(i0 + warp, __shfl_sync(0xffffffffu, x, warp), at);
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
}

__device__ __forceinline__ void part_of_items(int n, int& from, int& to) {
  from = static_cast<int>(static_cast<int64_t>(n) * blockIdx.x / kPoolCtas);
  to = static_cast<int>(static_cast<int64_t>(n) * (blockIdx.x + 1) / kPoolCtas);
}

__global__ void __cluster_dims__(kPoolCtas, 1, 1) __launch_bounds__(kPoolThreads, 1)
    paged_reserve_kernel(const __grid_constant__ PoolArgs a) {
  __shared__ int64_t sh[2][kPoolWarps];
  __shared__ int32_t mine[kMaxSeqs / kPoolCtas];   // the needs of the CTA's rows
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cap = a.max_pages << a.page_shift;   // at most 2^30
  int from, to;
  part_of_items(a.n_rows, from, to);
  // The entries [first, last) of row r's positions.
  auto range = [&](int r, int& first, int& last) {
    const int lo = a.lo ? __ldg(a.lo + r) : 0, hi = __ldg(a.hi + r);
    first = min(max(lo, 0), cap) >> a.page_shift;
    last = (min(max(hi, 0), cap) + (1 << a.page_shift) - 1) >> a.page_shift;
    if (hi <= lo) last = first;
    return hi;
  };
  for (int r = from + warp; r < to; r += kPoolWarps) {
    int first, last, n = 0;
    if (range(r, first, last) > cap && lane == 0) record_bad_index(a.status, kWhereLength);
    const int32_t* entries = a.table + r * a.table_stride;
    for (int i = first + lane; i < last; i += 32) n += entries[i] < 0;
    n = warp_sum(n);
    if (lane == 0) a.need[r] = mine[r - from] = n;
  }
  const uint64_t kept = count_free(a);
  cluster_barrier();
  const PoolSums s = add_up(a, a.n_rows, from, [&](int r) { return __ldcg(a.need + r); }, sh);
  list_free(a, kept, s.free_before, s.all);
  cluster_barrier();
  for_each_in_order(from, to, s.before, [&](int r) { return mine[r - from]; }, [&](int r, int n, int64_t at) {
    const bool good = n == 0 || at + n <= s.free_all;
    if (a.ok && lane == 0) a.ok[r] = good;
    if (n == 0 || !good) return;
    int first, last;
    range(r, first, last);
    int32_t* entries = a.table + r * a.table_stride;
    for (int i0 = first; i0 < last; i0 += 32) {
      const bool missing = i0 + lane < last && entries[i0 + lane] < 0;
      const uint32_t all = __ballot_sync(0xffffffffu, missing);
      if (missing) {
        const int page = __ldcg(a.list + at + __popc(all & ((1u << lane) - 1u)));
        entries[i0 + lane] = page;
        a.refs[page] = 1;
      }
      at += __popc(all);
    }
  });
}

// A child's row is marked by the number of its fork in entry 0: the smallest stays, whoever comes when.
__device__ __forceinline__ int fork_mark(int k) { return INT32_MIN + k; }

__global__ void __cluster_dims__(kPoolCtas, 1, 1) __launch_bounds__(kPoolThreads, 1)
    paged_fork_kernel(const __grid_constant__ PoolArgs a) {
  __shared__ int64_t sh[2][kPoolWarps];
  __shared__ uint8_t mine[kMaxSeqs / kPoolCtas];   // of the CTA's forks: 1 has its row, 2 is possible, 4 needs a page
  __shared__ uint8_t in_order[kMaxSeqs / kPoolCtas];   // of their sources: 1 the first page, 2 the begun one is somebody's
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cap = a.max_pages << a.page_shift;
  int from, to;
  part_of_items(a.n_forks, from, to);
  auto row_of = [&](int r) { return a.table + r * a.table_stride; };
  auto exists = [&](int r) { return r >= 0 && r < a.n_rows; };
  for (int k = from + warp; k < to; k += kPoolWarps) {
    const int src = __ldg(a.src + k), dst = __ldg(a.dst + k), len = __ldg(a.len + k);
    bool good = exists(src) && exists(dst) && src != dst;
    if (good) {
      bool held = false;
      const int32_t* entries = row_of(dst);
      for (int i = lane; i < a.max_pages; i += 32) held |= __ldcg(entries + i) >= 0;
      good = !__any_sync(0xffffffffu, held);
    }
    if (lane == 0) {
      if (good) atomicMin(row_of(dst), fork_mark(k));
      if (len < 0 || len > cap) record_bad_index(a.status, kWhereLength);
    }
  }
  const uint64_t kept = count_free(a);
  cluster_barrier();
  auto length = [&](int k) { return min(max(__ldg(a.len + k), 0), cap); };
  // Whether fork k has its row (its mark stands there), its source is no child itself, and a begun page is to be had.  Every CTA
  // asks for all forks, before any row is written (behind the second barrier).
  const PoolSums s = add_up(a, a.n_forks, from, [&](int k) {
    const int src = __ldg(a.src + k), dst = __ldg(a.dst + k);
    int state = exists(src) && exists(dst) && src != dst && __ldcg(row_of(dst)) == fork_mark(k) ? 1 : 0;
    if (state && __ldcg(row_of(src)) >= fork_mark(a.n_forks)) state |= 2;
    if (state == 3 && (length(k) & ((1 << a.page_shift) - 1)) != 0) state |= 4;
    if (k >= from && k < to) mine[k - from] = static_cast<uint8_t>(state);
    return state >> 2;
  }, sh);
  list_free(a, kept, s.free_before, s.all);
  auto need = [&](int k) { return mine[k - from] >> 2; };
  // Whether fork k of `state` is made, its page at `at` of the list.
  auto made = [&](int state, int n, int64_t at) { return (state & 2) && (n == 0 || at < s.free_all); };
  for_each_in_order(from, to, s.before, need, [&](int k, int n, int64_t at) {
    if (!made(mine[k - from], n, at)) return;
    const int32_t* parent = row_of(__ldg(a.src + k));
    int32_t* child = row_of(__ldg(a.dst + k));
    const int full = length(k) >> a.page_shift, entries = full + n;   // the begun page's too
    constexpr int kAhead = 4;   // entries of a lane whose loads are in flight together
    int flags = 0;
    for (int i0 = 0; i0 < entries; i0 += 32 * kAhead) {
      int page[kAhead], count[kAhead];
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {
        const int i = i0 + x * 32 + lane;
        page[x] = i < entries ? __ldcg(parent + i) : -1;
      }
#pragma unroll
      for (int x = 0; x < kAhead; ++x) count[x] = page[x] >= 0 && page[x] < a.n_pages ? __ldcg(a.refs + page[x]) : 0;
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {
        const int i = i0 + x * 32 + lane;
        if (i >= entries) continue;
        if (count[x] <= 0) record_bad_index(a.status, page[x] >= 0 && page[x] < a.n_pages ? kWhereCount : kWherePage);
        if (i == full) {
          flags |= count[x] > 0 ? 2 : 0;
          continue;
        }
        if (count[x] > 0) atomicAdd(a.refs + page[x], 1);
        if (i > 0) child[i] = count[x] > 0 ? page[x] : -1;   // (entry 0 holds the mark until step 3)
        else flags |= count[x] > 0 ? 1 : 0;
      }
    }
    flags = __reduce_or_sync(0xffffffffu, flags);
    if (lane == 0) in_order[k - from] = static_cast<uint8_t>(flags);
  });
  cluster_barrier();
  for_each_in_order(from, to, s.before, need, [&](int k, int n, int64_t at) {
    const int state = mine[k - from];
    const bool good = made(state, n, at);
    const int len = length(k), full = len >> a.page_shift, part = len & ((1 << a.page_shift) - 1);
    int c_src = -1, c_dst = -1, c_tokens = 0;
    if (lane == 0 && !(state & 2)) record_bad_index(a.status, kWhereRow);
    if (lane == 0 && (state & 1)) {   // the row is this fork's, with a mark in entry 0
      int32_t* child = row_of(__ldg(a.dst + k));
      const int32_t* parent = row_of(__ldg(a.src + k));
      const int flags = good ? in_order[k - from] : 0;
      if (good && n) {
        if (flags & 2) c_src = __ldcg(parent + full);
        c_dst = __ldcg(a.list + at);
        c_tokens = part;
        child[full] = c_dst;
        a.refs[c_dst] = 1;
      }
      if (!good || full > 0 || n == 0) child[0] = flags & 1 ? __ldcg(parent) : -1;
    }
    if (lane == 0) {
      a.copy_src[k] = c_src;
      a.copy_dst[k] = c_dst;
      a.copy_tokens[k] = c_tokens;
      a.ok[k] = good;
    }
  });
}

// ------------------------------------------------------------------------------------------- host side
sage_status check_pool(const sage_paged_pool* p) {
  if (!p || !p->refs || !p->page_table || p->n_pages <= 0 || p->n_rows <= 0 || p->max_pages <= 0) return SAGE_ERR_INVALID_ARG;
  if (p->page_size < 8 || p->page_size > 1024 || (p->page_size & (p->page_size - 1)) != 0) return SAGE_ERR_UNSUPPORTED;
  if (p->n_pages > INT32_MAX || p->n_rows > kMaxSeqs || p->max_pages > (int64_t(1) << 30) / p->page_size)
    return SAGE_ERR_UNSUPPORTED;
  if (p->n_rows > 1 && p->table_stride < p->max_pages) return SAGE_ERR_INVALID_ARG;
  if (!aligned(p->refs, 16) || !aligned(p->page_table, 4)) return SAGE_ERR_ALIGNMENT;
  return SAGE_OK;
}

constexpr size_t kPoolSumsOff = kPagedStatusBytes;
constexpr size_t kPoolNeedOff = kPoolSumsOff + sizeof(int32_t) * kPoolCtas * kPoolWarps;

size_t pool_bytes(int64_t n_rows, int64_t n_pages) {
  return kPoolNeedOff + sizeof(int32_t) * static_cast<size_t>(n_rows + n_pages);
}

sage_status check_pool_ws(const sage_paged_pool* p, void* ws, size_t ws_bytes) {
  if (!ws) return SAGE_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return SAGE_ERR_ALIGNMENT;
  return ws_bytes < pool_bytes(p->n_rows, p->n_pages) ? SAGE_ERR_WORKSPACE : SAGE_OK;
}

PoolArgs pool_args(const sage_paged_pool* p, void* ws) {
  PoolArgs a{};
  a.refs = p->refs;
  a.n_pages = static_cast<int>(p->n_pages);
  a.table = p->page_table;
  a.table_stride = p->table_stride;
  a.n_rows = static_cast<int>(p->n_rows);
  a.max_pages = static_cast<int>(p->max_pages);
  while ((int64_t(1) << a.page_shift) < p->page_size) ++a.page_shift;
  a.status = static_cast<int32_t*>(ws);
  char* w = static_cast<char*>(ws);
  a.sums = reinterpret_cast<int32_t*>(w + kPoolSumsOff);
  a.need = reinterpret_cast<int32_t*>(w + kPoolNeedOff);
  a.list = a.need + p->n_rows;
  return a;
}

}  // namespace
}  // namespace sage

using namespace sage;

extern "C" {

size_t sage_paged_pool_workspace_bytes(int64_t n_rows, int64_t n_pages) {
  if (n_rows <= 0 || n_rows > kMaxSeqs || n_pages <= 0 || n_pages > INT32_MAX) return 0;
  return pool_bytes(n_rows, n_pages);
}

sage_status sage_paged_release(const sage_paged_pool* pool, const int32_t* lo, const int32_t* hi, void* status_block,
                               void* stream) {
  const sage_status st = check_pool(pool);
  if (st != SAGE_OK) return st;
  if (!hi || !status_block) return SAGE_ERR_INVALID_ARG;
  if (!aligned(lo, 4) || !aligned(hi, 4) || !aligned(status_block, 4)) return SAGE_ERR_ALIGNMENT;
  PoolArgs a = pool_args(pool, status_block);
  a.lo = lo;
  a.hi = hi;
  constexpr int kPer = kReleaseThreads * kReleasePer;
  const unsigned parts = static_cast<unsigned>((pool->max_pages + kPer - 1) / kPer);
  const unsigned rows = static_cast<unsigned>(a.n_rows < 65535 ? a.n_rows : 65535);
  paged_release_kernel<<<dim3(parts, rows), kReleaseThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return cuda_status(cudaGetLastError());
}

sage_status sage_paged_reserve(const sage_paged_pool* pool, const int32_t* lo, const int32_t* hi, int32_t* ok, void* ws,
                               size_t ws_bytes, void* stream) {
  sage_status st;
  if ((st = check_pool(pool)) != SAGE_OK) return st;
  if (!hi) return SAGE_ERR_INVALID_ARG;
  if (!aligned(lo, 4) || !aligned(hi, 4) || !aligned(ok, 4)) return SAGE_ERR_ALIGNMENT;
  if ((st = check_pool_ws(pool, ws, ws_bytes)) != SAGE_OK) return st;
  PoolArgs a = pool_args(pool, ws);
  a.lo = lo;
  a.hi = hi;
  a.ok = ok;
  paged_reserve_kernel<<<kPoolCtas, kPoolThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return cuda_status(cudaGetLastError());
}

sage_status sage_paged_fork(const sage_paged_pool* pool, const int32_t* src_rows, const int32_t* dst_rows,
                            const int32_t* n_tokens, int64_t n_forks, int32_t* copy_src, int32_t* copy_dst,
                            int32_t* copy_tokens, int32_t* ok, void* ws, size_t ws_bytes, void* stream) {
  sage_status st;
  if ((st = check_pool(pool)) != SAGE_OK) return st;
  if (n_forks < 0) return SAGE_ERR_INVALID_ARG;
  if (n_forks > 0 && (!src_rows || !dst_rows || !n_tokens || !copy_src || !copy_dst || !copy_tokens || !ok))
    return SAGE_ERR_INVALID_ARG;
  if (n_forks > pool->n_rows) return SAGE_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(src_rows), static_cast<const void*>(dst_rows),
                        static_cast<const void*>(n_tokens), static_cast<const void*>(copy_src),
                        static_cast<const void*>(copy_dst), static_cast<const void*>(copy_tokens),
                        static_cast<const void*>(ok)})
    if (!aligned(p, 4)) return SAGE_ERR_ALIGNMENT;
  if ((st = check_pool_ws(pool, ws, ws_bytes)) != SAGE_OK) return st;
  if (n_forks == 0) return SAGE_OK;
  PoolArgs a = pool_args(pool, ws);
  a.src = src_rows;
  a.dst = dst_rows;
  a.len = n_tokens;
  a.n_forks = static_cast<int>(n_forks);
  a.copy_src = copy_src;
  a.copy_dst = copy_dst;
  a.copy_tokens = copy_tokens;
  a.ok = ok;
  paged_fork_kernel<<<kPoolCtas, kPoolThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return cuda_status(cudaGetLastError());
}

}  // extern "C"
