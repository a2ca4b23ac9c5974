// paged_move.cu -- copies inside the paged cache (include/sage_paged_pool.h): pages to pages, and the kept tokens of a sequence
// moved together in place.
//
// What bounds it: every moved byte is read and written once, so HBM; for a few tokens the chain launch -> numbers -> page table ->
// row -> row.
//
// Copy: a CTA takes 32 KB of a page's K or V, eight 16-byte loads in flight per thread, then the stores.
//
// Compact moves every token to an earlier place of its own sequence, so a place may be written only when the tokens before
// it in the list, which may stand there, have been read.  A token's own place lies before all that later tokens are read
// from (keep[i] >= first + i), so that is all.  An item is a run of tokens of one sequence, of K or V, and some of the heads,
// held in shared memory between reading and writing:
//   lists that fit one item (64 KB)   a CTA for each item, nothing to wait for;
//   longer ones                       one CTA per SM with eight items in work, four of them with 48 KB of shared memory, each step
//                                     of an item by warps of their own: drawn (in the order of the lists' tokens), its
//                                     places found, its rows read, announced, and written after a look at whether
//                                     the items that read from its new places have done so.  In an ascending list these are
//                                     as many entries as the item has tokens, found by search; most often they were
//                                     read long ago.  Rows go by bulk copies where a token's heads lie together, by 16 bytes a
//                                     thread where they do not (a bulk copy takes ~20 ns whatever its size).
// Which items have been read stands in a ring of 8 numbers per CTA: in place `item mod its length` the round of the last item read,
// each put there after the one a round before it.  Items ascend within a CTA, reading waits for nothing but that and a buffer, and
// the lowest item not yet read finds its place ready: so every wait ends.
// The long kernel's steps on compact_frames (23184 tokens of 56 heads, 1.33 GB; floor 196 us): an item read, waited for and written
// in turn, two CTAs per SM 554 us; reading and writing by warps of their own 420-520, 200 of it waiting for all items drawn
// before; the search and bulk copies 337; eight items found ahead, the lists side by side, a place in the ring for every
// item in work 220 (207 without looking at the ring); a fence an item, which that one lacked, 230 (5.8 TB/s).  Rows of 256 bytes,
// by 16 bytes a thread, before the fence: 24000 tokens 354, where heads lie together 270.
#include <algorithm>

#include "paged_batch.cuh"
#include "paged_check.h"
#include "paged_kept.h"
#include "sage_paged_pool.h"

namespace sage {
namespace {

constexpr int kMoveThreads = 256;
constexpr int kCopyPer = 8;                                    // 16-byte pieces of a thread
constexpr int kCopyPieces = kMoveThreads * kCopyPer;           // 32 KB
constexpr int kItemPieces = 64 * 64, kLongPieces = 48 * 64;    // 16 bytes each, of an item: 64 KB, of a long list 48 KB
constexpr int kLongItems = 8, kLongBuffers = 4;                // in work in a CTA
constexpr int kMovePlaces = 8;                                 // of the ring, for each CTA: no item waits for one that is not drawn
static_assert(kMovePlaces >= kLongItems, "items wait for their places");
constexpr int kItemTokens = 256;                               // at most, of an item
constexpr uint64_t kMoveWaitNs = 2000000000ull;

struct PageSide {   // K or V: bytes
  uint8_t* pages;
  int64_t page, token, head;
};

// ------------------------------------------------------------------------------------------- copy
struct CopyArgs {
  PageSide side[2];
  const int32_t *src, *dst, *tokens;
  int n_pages, page_size;
  int row_shift;        // log2 of the 16-byte pieces of a head's row
  int heads;
  bool by_head;         // rows of a head's slots lie closer together than those of a slot's heads
  int32_t* status;
};

__global__ void __launch_bounds__(kMoveThreads) paged_copy_kernel(const __grid_constant__ CopyArgs a) {
  const int i = blockIdx.y;
  const int src = __ldg(a.src + i), dst = __ldg(a.dst + i);
  const bool first = blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0;
  if (src == -1 || dst == -1) return;
  if (src < 0 || src >= a.n_pages || dst < 0 || dst >= a.n_pages) {
    if (first) record_bad_index(a.status, kWherePage);
    return;
  }
  int n = a.page_size;
  if (a.tokens) {
    n = __ldg(a.tokens + i);
    if (first && (n < 0 || n > a.page_size)) record_bad_index(a.status, kWhereLength);
    n = min(max(n, 0), a.page_size);
  }
  if (src == dst) return;
  const PageSide& s = a.side[blockIdx.z];
  const uint8_t* from = s.pages + src * s.page;
  uint8_t* to = s.pages + dst * s.page;
  const uint32_t pieces = static_cast<uint32_t>(n * a.heads) << a.row_shift;   // below 2^26
  const uint32_t inner = a.by_head ? n : a.heads;
  const uint32_t p0 = blockIdx.x * kCopyPieces + threadIdx.x;
  uint4 v[kCopyPer];
  int64_t at[kCopyPer];
#pragma unroll
  for (int k = 0; k < kCopyPer; ++k) {
    const uint32_t p = p0 + k * kMoveThreads;
    at[k] = -1;
    if (p < pieces) {
      const uint32_t row = p >> a.row_shift, outer = row / inner, in = row - outer * inner;
      at[k] = (a.by_head ? outer * s.head + in * s.token : outer * s.token + in * s.head) +
              ((p & ((1u << a.row_shift) - 1u)) << 4);
      v[k] = __ldcs(reinterpret_cast<const uint4*>(from + at[k]));
    }
  }
#pragma unroll
  for (int k = 0; k < kCopyPer; ++k)
    if (at[k] >= 0) __stcs(reinterpret_cast<uint4*>(to + at[k]), v[k]);
}

// ------------------------------------------------------------------------------------------- compact
struct CompactArgs {
  PageSide side[2];
  PagedBatchDev b;
  const int32_t *first, *keep, *n_keep;
  int64_t keep_stride;
  int max_keep;
  int row_shift, heads;
  int slab, slabs;             // heads of an item, items side by side
  int tokens, runs;            // tokens of an item, items of a list of max_keep
  int sides;                   // 2, or 1 where K and V are the same pages
  uint32_t units, items;       // n_seqs * sides * slabs; times runs
  int32_t* status;
  int32_t* counters;           // next item, CTAs done, ring of 16-bit numbers: 1 + the round last read in each place
};

__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 load_shared16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

// The ring's numbers, put and looked at without an order of their own; fence_gpu between what they stand for and them.
__device__ __forceinline__ void ring_put(uint16_t* place, uint32_t n) {
  asm volatile("st.relaxed.gpu.global.u16 [%0], %1;" ::"l"(place), "h"(static_cast<uint16_t>(n)) : "memory");
}
__device__ __forceinline__ uint32_t ring_get(const uint16_t* place) {
  uint16_t n;
  asm volatile("ld.relaxed.gpu.global.u16 %0, [%1];" : "=h"(n) : "l"(place) : "memory");
  return n;
}
__device__ __forceinline__ void fence_gpu() { asm volatile("fence.acq_rel.gpu;" ::: "memory"); }
// What this thread has seen done comes before its bulk stores to global memory.
__device__ __forceinline__ void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

struct MoveShared {
  int64_t from[kItemTokens], to[kItemTokens];   // bytes from the pages' beginning; from < 0: not moved
};
// An item: what it takes to read and to write it.
struct Item {
  uint32_t pieces, per;   // 16-byte pieces, and those of a token
  const PageSide* side;
  int64_t head0;          // bytes to its first head
  int b, i0, count;       // sequence, first token of its list, tokens
};
__device__ __forceinline__ Item find_item(const CompactArgs& a, uint32_t item) {
  // The lists side by side, so that an item's predecessors were drawn long before it.
  const uint32_t run = item / a.units, unit = item - run * a.units, half = unit / a.slabs;
  const int slab = unit - half * a.slabs;
  Item it;
  it.b = a.sides == 2 ? half >> 1 : half;
  it.side = &a.side[a.sides == 2 ? half & 1 : 0];
  it.head0 = static_cast<int64_t>(slab) * a.slab * it.side->head;
  it.per = static_cast<uint32_t>(min(a.slab, a.heads - slab * a.slab)) << a.row_shift;
  it.i0 = run * a.tokens;
  it.count = max(0, min(a.tokens, min(max(__ldg(a.n_keep + it.b), 0), a.max_keep) - it.i0));
  it.pieces = it.count * it.per;
  return it;
}
// Where its tokens lie and go to, by `n` threads.
__device__ __forceinline__ void find_places(const CompactArgs& a, const Item& it, MoveShared& sh, int me, int n) {
  const bool first_head = it.head0 == 0 && it.side == &a.side[0];   // one item of each run records what is wrong
  if (me == 0 && first_head && it.i0 == 0) {
    const int k = __ldg(a.n_keep + it.b);
    if (k < 0 || k > a.max_keep) record_bad_index(a.status, kWhereLength);
  }
  for (int t = me; t < it.count; t += n) {
    const int i = it.i0 + t;
    const int64_t old = __ldg(a.keep + it.b * a.keep_stride + i), now = static_cast<int64_t>(__ldg(a.first + it.b)) + i;
    int64_t from = -1, to = -1;
    const int64_t last = i > 0 ? __ldg(a.keep + it.b * a.keep_stride + i - 1) : -1;
    if (now < 0 || old < now || old <= last || old >= min(__ldg(a.b.kv_len + it.b), a.b.cap)) {
      if (first_head) record_bad_index(a.status, kWhereKept);
    } else if (old != now) {
      const int32_t* row = a.b.table + it.b * a.b.table_stride;
      const int p0 = __ldg(row + (old >> a.b.page_shift)), p1 = __ldg(row + (now >> a.b.page_shift));
      if (p0 < 0 || p0 >= a.b.n_pages || p1 < 0 || p1 >= a.b.n_pages) {
        if (first_head) record_bad_index(a.status, kWherePage);
      } else {
        const int mask = (1 << a.b.page_shift) - 1;
        from = p0 * it.side->page + (old & mask) * it.side->token + it.head0;
        to = p1 * it.side->page + (now & mask) * it.side->token + it.head0;
      }
    }
    sh.from[t] = from;
    sh.to[t] = to;
  }
}
// Reads its tokens into shared memory by `n` threads; the calling thread's copies have landed when it returns.
__device__ __forceinline__ void read_item(const CompactArgs& a, const Item& it, const MoveShared& sh, uint32_t smem, int me, int n) {
  for (uint32_t p = me; p < it.pieces; p += n) {
    const uint32_t tok = p / it.per, in = p - tok * it.per;
    const int64_t from = sh.from[tok];
    if (from >= 0)
      copy_async16(smem + p * 16, it.side->pages + from + (in >> a.row_shift) * it.side->head +
                                      ((in & ((1u << a.row_shift) - 1u)) << 4));
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}
__device__ __forceinline__ void write_item(const CompactArgs& a, const Item& it, const MoveShared& sh, uint32_t smem, int me,
                                           int n) {
  for (uint32_t p = me; p < it.pieces; p += n) {
    const uint32_t tok = p / it.per, in = p - tok * it.per;
    if (sh.from[tok] < 0) continue;
    const uint4 v = load_shared16(smem + p * 16);
    *reinterpret_cast<uint4*>(it.side->pages + sh.to[tok] + (in >> a.row_shift) * it.side->head +
                              ((in & ((1u << a.row_shift) - 1u)) << 4)) = v;
  }
}
__device__ __forceinline__ bool timed_out(const int32_t* status) {
  return *reinterpret_cast<const volatile int32_t*>(status) == kStatusTimeout;
}

__global__ void __launch_bounds__(kMoveThreads) paged_compact_kernel(const __grid_constant__ CompactArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ MoveShared sh;
  if (__syncthreads_or(threadIdx.x == 0 && timed_out(a.status))) return;   // no work until the status has been read
  const Item it = find_item(a, blockIdx.x);
  find_places(a, it, sh, threadIdx.x, kMoveThreads);
  __syncthreads();
  read_item(a, it, sh, smem_u32(smem_raw), threadIdx.x, kMoveThreads);
  __syncthreads();   // the whole list has been read
  write_item(a, it, sh, smem_u32(smem_raw), threadIdx.x, kMoveThreads);
}

// Warp 0 draws, 1-4 find, 5-8 announce and look at the ring (a buffer each: both are chains of waits for L2); then those that
// read and those that write: one warp each for bulk copies, eight each (reading in two groups of four, items in turn) without.
constexpr int kFinders = 4;
static_assert(kLongBuffers == kFinders, "an end for each warp that finds, and for each buffer");
template <bool kBulk>
struct LongCfg {
  static constexpr int kReaders = kBulk ? 32 : 128, kReadGroups = kBulk ? 1 : 2, kWriters = kBulk ? 32 : 256;
  static constexpr int kReader0 = (1 + kFinders + kLongBuffers) * 32, kWriter0 = kReader0 + kReaders * kReadGroups;
  static constexpr int kThreads = kWriter0 + kWriters;
};
template <int kThreads>
__device__ __forceinline__ void role_sync(int barrier) {
  if (kThreads == 32) __syncwarp();
  else asm volatile("bar.sync %0, %1;" ::"r"(barrier), "n"(kThreads) : "memory");
}

// What the steps of an item need of it.
struct LongItem {
  uint32_t item;
  uint32_t moved;       // tokens that move
  uint32_t near, far;   // items `near` .. `far` before this one read from its new places (far 0: none)
  Item it;
};

// The first entry of b's list, among the n before entry i0, that is not below `place` (n: none), by a warp.  The list ascends.
__device__ __forceinline__ int first_not_below(const CompactArgs& a, int b, int n, int64_t place) {
  const int lane = threadIdx.x & 31;
  const int32_t* keep = a.keep + b * a.keep_stride;
  return kept_search(n, [&](int lo, int step, int m) {
    return __popc(__ballot_sync(0xffffffffu, __ldg(keep + kept_part_end(lo, step, m, lane)) < place));
  });
}

template <bool kBulk>
__global__ void __launch_bounds__(LongCfg<kBulk>::kThreads, 1) paged_compact_long_kernel(const __grid_constant__ CompactArgs a) {
  using C = LongCfg<kBulk>;
  constexpr uint32_t M = kLongItems, B = kLongBuffers;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ MoveShared sh[M];
  __shared__ LongItem li[M];   // item a.items: no more
  __shared__ uint64_t drawn[M], found[M], done[M], full[B], go[B], empty[B];
  __shared__ volatile int s_abort;
  __shared__ int s_last;
  int32_t* next = a.counters;
  uint16_t* ring = reinterpret_cast<uint16_t*>(next + 2);
  const uint32_t places = kMovePlaces * gridDim.x;   // at most kPagedMoveRing
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    s_abort = timed_out(a.status);
    for (uint32_t i = 0; i < M; ++i) {
      mbar_init(drawn + i, 1);
      mbar_init(found + i, 1);
      mbar_init(done + i, 1);
    }
    for (uint32_t i = 0; i < B; ++i) {
      mbar_init(full + i, 1);
      mbar_init(go + i, 1);
      mbar_init(empty + i, 1);
    }
    fence_mbar_init();
  }
  __syncthreads();
  if (s_abort) return;   // an earlier wait ran out: no work until the status has been read
  // After a wait that ran out nothing more is drawn or written, but the turns still go round.
  auto fail = [&] {
    if (lane == 0) {
      record_timeout(a.status, kWherePagedMove);
      s_abort = 1;
    }
    __syncwarp();
  };
  auto wait = [&](uint64_t* bar, uint32_t k, uint32_t n) {   // by a whole warp: turn k of n barriers
    const bool ok = __all_sync(0xffffffffu, mbar_wait(bar + k % n, (k / n) & 1, 4 * kMoveWaitNs));
    if (!ok) fail();
    return ok;
  };
  auto pass = [&](uint64_t* bar, uint32_t k, uint32_t n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar + k % n);
  };
  // Turn k's item, or a.items.
  auto item_of = [&](bool ok, uint32_t k) { return ok ? li[k % M].item : a.items; };
  if (warp == 0) {
    for (uint32_t k = 0, ends = 0; ends < kFinders; ++k) {   // an end for each warp that finds
      const bool ok = k < M || wait(done, k - M, M);
      uint32_t item = a.items;
      if (lane == 0 && ok && !s_abort && ends == 0) item = min(static_cast<uint32_t>(atomicAdd(next, 1)), a.items);
      item = __shfl_sync(0xffffffffu, item, 0);
      if (lane == 0) li[k % M].item = item;
      pass(drawn, k, M);
      ends += item >= a.items;
    }
  } else if (warp <= kFinders) {
    for (uint32_t k = warp - 1;; k += kFinders) {
      const bool ok = wait(drawn, k, M);
      const uint32_t item = item_of(ok, k);
      if (item < a.items) {
        const Item it = find_item(a, item);
        MoveShared& m = sh[k % M];
        find_places(a, it, m, lane, 32);
        __syncwarp();
        uint32_t moved = 0;
        for (int t = lane; t < it.count; t += 32) moved += m.from[t] >= 0;
        moved = __reduce_add_sync(0xffffffffu, moved);
        const int from = it.count > 0 && it.i0 > 0
                             ? first_not_below(a, it.b, it.i0, static_cast<int64_t>(__ldg(a.first + it.b)) + it.i0)
                             : it.i0;
        const KeptWait w = kept_wait(it.i0, it.count, a.tokens, from);
        if (lane == 0) {
          LongItem& l = li[k % M];
          l.it = it;
          l.moved = moved;
          l.near = w.near;
          l.far = w.far;
        }
      }
      pass(found, k, M);
      if (item >= a.items) break;
    }
  } else if (warp <= kFinders + static_cast<int>(B)) {
    // ------------------------------------------------------------ announce, and look at the ring
    // An item's rows have arrived in shared memory (`full`), its place in the ring holds the round before, and most often the
    // items that it waits for are there: one fence of all lanes stands behind all three and before the item's own number and its
    // writing.  So whoever sees that number, or a later one of its place, writes after the rows were read.  (Without a fence,
    // in no order that PTX's memory model gives: 195 us instead of 205 of compact_frames, 303 instead of 325 where heads lie
    // apart; with an acquire at each look and a release at each number 204 and 330.)
    for (uint32_t k = warp - kFinders - 1;; k += B) {
      const bool ok = wait(found, k, M);
      const uint32_t item = item_of(ok, k), round = item / places, far = li[k % M].far, near = li[k % M].near;
      uint16_t* at = ring + item % places;
      const uint64_t t0 = global_timer_ns();
      auto late = [&] {
        __nanosleep(40);
        if (__any_sync(0xffffffffu, global_timer_ns() - t0 > kMoveWaitNs)) fail();
      };
      // Whether the items that have to be read before this one is written are.
      auto clear = [&] {
        bool all = true;
        for (uint32_t d = near + lane; d <= far; d += 32) {
          const uint32_t other = item - d * a.units;
          all &= ring_get(ring + other % places) >= other / places + 1;
        }
        return __all_sync(0xffffffffu, all);
      };
      bool all = true;
      if (item < a.items) {
        while (!__all_sync(0xffffffffu, s_abort || ring_get(at) >= round)) late();   // the item a round before
        all = far == 0 || clear();
      }
      if (wait(full, k, B) && item < a.items) {
        fence_gpu();
        if (lane == 0) ring_put(at, round + 1);
        if (!all) {
          while (!clear() && !__any_sync(0xffffffffu, s_abort)) late();
          fence_gpu();
        }
      }
      pass(go, k, B);
      if (item >= a.items) break;
    }
  } else if (static_cast<int>(threadIdx.x) < C::kWriter0) {
    // ------------------------------------------------------------ read
    const int group = (threadIdx.x - C::kReader0) / C::kReaders, me = threadIdx.x - C::kReader0 - group * C::kReaders;
    for (uint32_t k = group, ends = 0; ends < B / C::kReadGroups; k += C::kReadGroups) {   // an end for each buffer
      const uint32_t buf = k % B;
      bool ok = wait(found, k, M);
      ok = (k < B || wait(empty, k - B, B)) && ok;
      const uint32_t item = item_of(ok, k), moved = item < a.items ? li[k % M].moved : 0;
      if (kBulk) {
        const Item it = li[k % M].it;
        if (me == 0) {
          if (moved > 0) mbar_arrive_expect_tx(full + buf, moved * it.per * 16);
          else mbar_arrive(full + buf);
        }
        __syncwarp();
        if (moved > 0)
          for (int t = me; t < it.count; t += 32)
            if (sh[k % M].from[t] >= 0)
              bulk_load(smem_raw + buf * kLongPieces * 16 + t * it.per * 16, it.side->pages + sh[k % M].from[t], it.per * 16, full + buf);
      } else {
        if (moved > 0) read_item(a, li[k % M].it, sh[k % M], smem_u32(smem_raw) + buf * kLongPieces * 16, me, C::kReaders);
        role_sync<C::kReaders>(1 + group);   // every thread's copies have landed
        if (me == 0) mbar_arrive(full + buf);
      }
      ends += item >= a.items;
    }
  } else {
    // ------------------------------------------------------------ write
    const int me = threadIdx.x - C::kWriter0;
    for (uint32_t k = 0;; ++k) {
      const uint32_t buf = k % B;
      const bool ok = wait(go, k, B);
      const uint32_t item = item_of(ok, k);
      if (item < a.items && li[k % M].moved > 0 && !s_abort) {
        const Item it = li[k % M].it;
        if (kBulk) {
          fence_proxy_async_global();
          for (int t = me; t < it.count; t += 32)
            if (sh[k % M].from[t] >= 0)
              bulk_store(it.side->pages + sh[k % M].to[t], smem_raw + buf * kLongPieces * 16 + t * it.per * 16, it.per * 16);
          bulk_commit();
          bulk_wait_read<0>();
        } else {
          write_item(a, it, sh[k % M], smem_u32(smem_raw) + buf * kLongPieces * 16, me, C::kWriters);
        }
      }
      role_sync<C::kWriters>(3);
      if (me == 0) {
        mbar_arrive(empty + buf);
        mbar_arrive(done + k % M);
      }
      if (item >= a.items) break;
    }
    if (kBulk) bulk_wait_all();
  }
  // The last CTA to draw no more leaves the counters at zero for the next call.
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicAdd(next + 1, 1) == static_cast<int>(gridDim.x) - 1;
  }
  __syncthreads();
  if (s_last && !s_abort)
    for (uint32_t w = threadIdx.x; w < 2 + (places + 1) / 2; w += C::kThreads) a.counters[w] = 0;
}

void page_sides(const sage_paged_kv* c, PageSide side[2]) {
  const int64_t e = c->format == 1 ? 1 : 2;
  // (Strides of a dimension with one element are ignored.)
  const int64_t p = c->n_pages > 1, t = c->page_size > 1, h = c->n_heads > 1;
  side[0] = {static_cast<uint8_t*>(c->k_pages), c->k_stride_page * e * p, c->k_stride_token * e * t, c->k_stride_head * e * h};
  side[1] = {static_cast<uint8_t*>(c->v_pages), c->v_stride_page * e * p, c->v_stride_token * e * t, c->v_stride_head * e * h};
}
// Values that are the keys themselves move once.
int page_side_count(const sage_paged_kv* c, const PageSide side[2]) {
  return c->k_pages == c->v_pages && side[0].page == side[1].page && side[0].token == side[1].token && side[0].head == side[1].head ? 1 : 2;
}
int pieces_shift(const sage_paged_kv* c) {   // 16-byte pieces of a row: 4, 8 or 16
  const int64_t row = c->head_dim * (c->format == 1 ? 1 : 2);
  return row == 64 ? 2 : row == 128 ? 3 : 4;
}

}  // namespace
}  // namespace sage

using namespace sage;

extern "C" {

sage_status sage_paged_copy(const sage_paged_kv* cache, const int32_t* src, const int32_t* dst, const int32_t* n_tokens,
                            int64_t n_copies, void* status_block, void* stream) {
  sage_status st;
  if ((st = check_cache(cache)) != SAGE_OK) return st;
  if (n_copies < 0 || (n_copies > 0 && (!src || !dst)) || !status_block) return SAGE_ERR_INVALID_ARG;
  if (n_copies > kMaxRows) return SAGE_ERR_UNSUPPORTED;
  if (!aligned(src, 4) || !aligned(dst, 4) || !aligned(n_tokens, 4) || !aligned(status_block, 4)) return SAGE_ERR_ALIGNMENT;
  if (n_copies == 0) return SAGE_OK;
  CopyArgs a{};
  page_sides(cache, a.side);
  a.src = src;
  a.dst = dst;
  a.tokens = n_tokens;
  a.n_pages = static_cast<int>(cache->n_pages);
  a.page_size = static_cast<int>(cache->page_size);
  a.row_shift = pieces_shift(cache);
  a.heads = static_cast<int>(cache->n_heads);
  a.by_head = a.heads > 1 && a.side[0].head > a.side[0].token;
  a.status = static_cast<int32_t*>(status_block);
  const int64_t pieces = cache->page_size * cache->n_heads << a.row_shift;   // at most 2^26
  for (int64_t at = 0; at < n_copies; at += 65535) {
    const int64_t n = std::min<int64_t>(n_copies - at, 65535);
    a.src = src + at;
    a.dst = dst + at;
    a.tokens = n_tokens ? n_tokens + at : nullptr;
    const dim3 grid(static_cast<unsigned>((pieces + kCopyPieces - 1) / kCopyPieces), static_cast<unsigned>(n),
                    static_cast<unsigned>(page_side_count(cache, a.side)));
    paged_copy_kernel<<<grid, kMoveThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
    if ((st = cuda_status(cudaGetLastError())) != SAGE_OK) return st;
  }
  return SAGE_OK;
}

sage_status sage_paged_compact(const sage_paged_kv* cache, const sage_paged_batch* batch, const int32_t* first,
                               const int32_t* keep, int64_t max_keep, int64_t keep_stride, const int32_t* n_keep, void* ws,
                               size_t ws_bytes, void* stream) {
  sage_status st;
  if ((st = check_cache(cache)) != SAGE_OK || (st = check_batch(batch, cache->page_size)) != SAGE_OK) return st;
  if (max_keep < 0) return SAGE_ERR_INVALID_ARG;
  const bool any = batch->n_seqs > 0 && max_keep > 0;
  if (any && (!first || !keep || !n_keep || (batch->n_seqs > 1 && keep_stride < max_keep))) return SAGE_ERR_INVALID_ARG;
  if (max_keep > (int64_t(1) << 30)) return SAGE_ERR_UNSUPPORTED;
  if (!aligned(first, 4) || !aligned(keep, 4) || !aligned(n_keep, 4)) return SAGE_ERR_ALIGNMENT;
  if (!ws) return SAGE_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return SAGE_ERR_ALIGNMENT;
  if (ws_bytes < SAGE_PAGED_WS_HEADER) return SAGE_ERR_WORKSPACE;
  if (!any) return SAGE_OK;
  CompactArgs a{};
  page_sides(cache, a.side);
  a.b = batch_dev(batch, cache, 0);
  a.first = first;
  a.keep = keep;
  a.n_keep = n_keep;
  a.keep_stride = keep_stride;
  a.max_keep = static_cast<int>(max_keep);
  a.row_shift = pieces_shift(cache);
  a.heads = static_cast<int>(cache->n_heads);
  a.status = static_cast<int32_t*>(ws);
  a.counters = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + kCountersOff);
  // As many heads to an item as leave room for the whole list, where one head does; else rows of about 4 KB.
  const int64_t row = int64_t(1) << a.row_shift;
  int64_t slab = std::min<int64_t>(a.heads, kItemPieces / row / max_keep), pieces = kItemPieces;
  const bool whole = max_keep <= kItemTokens && slab >= 1;
  if (!whole) {
    slab = std::min<int64_t>(a.heads, 256 / row);
    pieces = kLongPieces;
  }
  a.slabs = static_cast<int>((a.heads + slab - 1) / slab);
  a.slab = static_cast<int>(slab);
  a.tokens = static_cast<int>(std::min<int64_t>({kItemTokens, pieces / (slab * row), max_keep}));
  a.runs = static_cast<int>((max_keep + a.tokens - 1) / a.tokens);
  a.sides = page_side_count(cache, a.side);
  const int64_t items = batch->n_seqs * a.sides * a.slabs * a.runs;
  if (items > (whole ? INT32_MAX : int64_t(1) << 25)) return SAGE_ERR_UNSUPPORTED;   // (rounds of the ring in 16 bits)
  a.units = static_cast<uint32_t>(items / a.runs);
  a.items = static_cast<uint32_t>(items);
  // Bulk copies where a token's rows of K and of V lie together.
  const bool bulk = slab == 1 || (a.side[0].head == row * 16 && a.side[1].head == row * 16);
  auto* kernel = whole ? paged_compact_kernel : bulk ? paged_compact_long_kernel<true> : paged_compact_long_kernel<false>;
  int dev = 0, sms = 0;
  cudaError_t e = cudaSuccess;
  if (!whole && (e = cudaGetDevice(&dev)) == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t ctas = whole ? items : std::min<int64_t>({items, sms, kPagedMoveRing / kMovePlaces});
  const int threads = whole ? kMoveThreads : bulk ? LongCfg<true>::kThreads : LongCfg<false>::kThreads;
  const int smem = whole ? static_cast<int>(a.tokens * slab * row * 16) : kLongBuffers * kLongPieces * 16;
  if (e == cudaSuccess && smem > 40 * 1024)   // (less needs no leave, which takes a microsecond)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, whole ? kItemPieces * 16 : smem);
  if (e != cudaSuccess) return cuda_status(e);
  kernel<<<static_cast<unsigned>(ctas), threads, smem, static_cast<cudaStream_t>(stream)>>>(a);
  return cuda_status(cudaGetLastError());
}

}  // extern "C"
