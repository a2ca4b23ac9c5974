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
// from (keep[i] >= first + i), so that is all.  An item is a run of tokens of one sequence, of K or V, and some of the heads, up
// to 64 KB, held in shared memory between reading and writing:
//   lists that fit one item     a CTA for each item, nothing to wait for;
//   longer ones                 CTAs draw items in the order of a list's tokens; an item is written when all items drawn
//                               before it have been read.  Reading waits for nothing, so every wait ends.  While an item is
//                               not read, every later one is held by a CTA of its own, which waits for it: with G CTAs
//                               only the G - 1 items before an item can be outstanding, and a ring of G numbers, the last
//                               item read in each place, tells which are.
#include <algorithm>

#include "paged_batch.cuh"
#include "paged_check.h"
#include "sage_paged_pool.h"

namespace sage {
namespace {

constexpr int kMoveThreads = 256;
constexpr int kCopyPer = 8;                                    // 16-byte pieces of a thread
constexpr int kCopyPieces = kMoveThreads * kCopyPer;           // 32 KB
constexpr int kItemPieces = 4096;                              // 64 KB
constexpr int kItemTokens = 256;                               // at most, of an item
constexpr int kMoveCtasPerSm = 2;
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
  uint32_t items;              // n_seqs * 2 * slabs * runs
  int32_t* status;
  int32_t* counters;           // next item, CTAs done, ring [kPagedMoveRing]: 1 + the last item read in each place
};

__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 load_shared16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

struct MoveShared {
  int64_t from[kItemTokens], to[kItemTokens];   // bytes from the pages' beginning; from < 0: not moved
  uint32_t item;
  int go;
};

// Reads an item's tokens; what write() needs of it.
struct Item {
  uint32_t pieces, per;   // 16-byte pieces, and those of a token
  const PageSide* side;
  int64_t head0;          // bytes to its first head
};
__device__ __forceinline__ Item read_item(const CompactArgs& a, uint32_t item, MoveShared& sh, uint32_t smem) {
  const uint32_t unit = item / a.runs, run = item - unit * a.runs, half = unit / a.slabs;
  const int slab = unit - half * a.slabs, b = half >> 1;
  Item it;
  it.side = &a.side[half & 1];
  it.head0 = static_cast<int64_t>(slab) * a.slab * it.side->head;
  it.per = static_cast<uint32_t>(min(a.slab, a.heads - slab * a.slab)) << a.row_shift;
  const int n_all = __ldg(a.n_keep + b), n = min(max(n_all, 0), a.max_keep);
  const int i0 = run * a.tokens, count = min(a.tokens, n - i0);
  const bool first = slab == 0 && !(half & 1) && threadIdx.x == 0;
  if (first && run == 0 && n_all != n) record_bad_index(a.status, kWhereLength);
  it.pieces = count > 0 ? count * it.per : 0;
  __syncthreads();   // the last item's places are no longer needed
  if (static_cast<int>(threadIdx.x) < count) {
    const int i = i0 + threadIdx.x;
    const int64_t old = __ldg(a.keep + b * a.keep_stride + i), now = static_cast<int64_t>(__ldg(a.first + b)) + i;
    int64_t from = -1, to = -1;
    const int where_slab = slab == 0 && !(half & 1);
    if (now < 0 || old < now || old >= min(__ldg(a.b.kv_len + b), a.b.cap)) {
      if (where_slab) record_bad_index(a.status, kWhereKept);
    } else if (old != now) {
      const int32_t* row = a.b.table + b * a.b.table_stride;
      const int p0 = __ldg(row + (old >> a.b.page_shift)), p1 = __ldg(row + (now >> a.b.page_shift));
      if (p0 < 0 || p0 >= a.b.n_pages || p1 < 0 || p1 >= a.b.n_pages) {
        if (where_slab) record_bad_index(a.status, kWherePage);
      } else {
        const int mask = (1 << a.b.page_shift) - 1;
        from = p0 * it.side->page + (old & mask) * it.side->token + it.head0;
        to = p1 * it.side->page + (now & mask) * it.side->token + it.head0;
      }
    }
    sh.from[threadIdx.x] = from;
    sh.to[threadIdx.x] = to;
  }
  __syncthreads();
  for (uint32_t p = threadIdx.x; p < it.pieces; p += kMoveThreads) {
    const uint32_t tok = p / it.per, in = p - tok * it.per;
    const int64_t from = sh.from[tok];
    if (from >= 0)
      copy_async16(smem + p * 16, it.side->pages + from + (in >> a.row_shift) * it.side->head +
                                      ((in & ((1u << a.row_shift) - 1u)) << 4));
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  return it;
}
// Each thread writes the pieces that it has read.
__device__ __forceinline__ void write_item(const CompactArgs& a, const Item& it, const MoveShared& sh, uint32_t smem) {
  for (uint32_t p = threadIdx.x; p < it.pieces; p += kMoveThreads) {
    const uint32_t tok = p / it.per, in = p - tok * it.per;
    if (sh.from[tok] < 0) continue;
    const uint4 v = load_shared16(smem + p * 16);
    *reinterpret_cast<uint4*>(it.side->pages + sh.to[tok] + (in >> a.row_shift) * it.side->head +
                              ((in & ((1u << a.row_shift) - 1u)) << 4)) = v;
  }
}

__global__ void __launch_bounds__(kMoveThreads) paged_compact_kernel(const __grid_constant__ CompactArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ MoveShared sh;
  const uint32_t smem = smem_u32(smem_raw);
  if (threadIdx.x == 0) sh.go = *reinterpret_cast<volatile int32_t*>(a.status) != kStatusTimeout;
  __syncthreads();
  if (!sh.go) return;   // an earlier wait ran out: no work until the status has been read
  if (a.runs == 1) {
    // The list is one item: it has been read whole before any of it is written.
    const Item it = read_item(a, blockIdx.x, sh, smem);
    __syncthreads();
    write_item(a, it, sh, smem);
    return;
  }
  int32_t *next = a.counters, *ring = next + 2;
  const uint32_t ctas = gridDim.x;   // at most kPagedMoveRing
  while (true) {
    __syncthreads();
    if (threadIdx.x == 0) sh.item = static_cast<uint32_t>(atomicAdd(next, 1));
    __syncthreads();
    const uint32_t item = sh.item;
    if (item >= a.items) break;
    const Item it = read_item(a, item, sh, smem);
    __syncthreads();   // every thread's copies have landed
    if (threadIdx.x == 0) {
      __threadfence();
      *reinterpret_cast<volatile int32_t*>(ring + item % ctas) = static_cast<int32_t>(item + 1);
    }
    // Each thread looks after the items `back` before this one (those that have nothing to write wait too: see above).
    bool ok = true;
    for (uint32_t back = threadIdx.x + 1; back < ctas && back <= item; back += kMoveThreads) {
      const volatile int32_t* at = ring + (item - back) % ctas;
      const uint64_t t0 = global_timer_ns();
      while (ok && static_cast<uint32_t>(*at) < item - back + 1) ok = global_timer_ns() - t0 < kMoveWaitNs;
    }
    if (!ok) record_timeout(a.status, kWherePagedMove);
    __threadfence();
    if (!__syncthreads_and(ok)) return;
    write_item(a, it, sh, smem);
  }
  // The last CTA to draw no more leaves the counters at zero for the next call.
  __shared__ int s_last;
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicAdd(next + 1, 1) == static_cast<int>(ctas) - 1;
  }
  __syncthreads();
  if (s_last)
    for (uint32_t w = threadIdx.x; w < ctas + 2; w += kMoveThreads) a.counters[w] = 0;
}

void page_sides(const sage_paged_kv* c, PageSide side[2]) {
  const int64_t e = c->format == 1 ? 1 : 2;
  // (Strides of a dimension with one element are ignored.)
  const int64_t p = c->n_pages > 1, t = c->page_size > 1, h = c->n_heads > 1;
  side[0] = {static_cast<uint8_t*>(c->k_pages), c->k_stride_page * e * p, c->k_stride_token * e * t, c->k_stride_head * e * h};
  side[1] = {static_cast<uint8_t*>(c->v_pages), c->v_stride_page * e * p, c->v_stride_token * e * t, c->v_stride_head * e * h};
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
    const dim3 grid(static_cast<unsigned>((pieces + kCopyPieces - 1) / kCopyPieces), static_cast<unsigned>(n), 2);
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
  a.counters = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + kCountersOff) + kPagedMoveCounters;
  // As many heads to an item as leave room for the whole list, where one head does; else rows of about 4 KB.
  const int64_t row = int64_t(1) << a.row_shift;
  int64_t slab = std::min<int64_t>(a.heads, kItemPieces / row / max_keep);
  const bool whole = max_keep <= kItemTokens && slab >= 1;
  if (!whole) slab = std::min<int64_t>(a.heads, 256 / row);
  a.slabs = static_cast<int>((a.heads + slab - 1) / slab);
  a.slab = static_cast<int>(slab);
  a.tokens = static_cast<int>(std::min<int64_t>({kItemTokens, kItemPieces / (slab * row), max_keep}));
  a.runs = static_cast<int>((max_keep + a.tokens - 1) / a.tokens);
  const int64_t items = batch->n_seqs * 2 * a.slabs * a.runs;
  if (items >= int64_t(1) << 31) return SAGE_ERR_UNSUPPORTED;
  a.items = static_cast<uint32_t>(items);
  const int smem = static_cast<int>(a.tokens * slab * row * 16);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(paged_compact_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kItemPieces * 16);
  if (e != cudaSuccess) return cuda_status(e);
  const int64_t most = std::min<int64_t>(sms * kMoveCtasPerSm, kPagedMoveRing);
  const unsigned grid = static_cast<unsigned>(a.runs == 1 ? items : std::min(items, most));
  paged_compact_kernel<<<grid, kMoveThreads, smem, static_cast<cudaStream_t>(stream)>>>(a);
  return cuda_status(cudaGetLastError());
}

}  // extern "C"
