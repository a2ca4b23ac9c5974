// paged_tree.cu -- drafted trees over the paged cache: the entry points of include/sage_paged_tree.h and the kernel that
// turns parents into ancestor bits.
//
// A thread takes a row.  Trees of up to 256 tokens: each row's bits and the ancestor that its bits reach up to are joined with those
// of that ancestor until all rows reach a root, log2 of the deepest row's steps (256 trees of 100-250 tokens: 5.1 us on the device, 10.9
// walking up one ancestor at a time).  Larger ones, and rows that a window cuts off, walk up: parents come before their children, so the
// walk goes down through the words of the row, each written once.  What bounds it: the launch and those chains.
#include "paged_batch.cuh"
#include "paged_check.h"
#include "sage_paged_tree.h"

namespace sage {
namespace {

constexpr int kTreeThreads = 256, kTreeShared = 4096;   // tokens whose parents are held in shared memory
constexpr int kTreeWords = kTreeThreads / 32;           // of the rows that are joined

__global__ void __launch_bounds__(kTreeThreads) paged_tree_kernel(const __grid_constant__ PagedTreeArgs a) {
  __shared__ int32_t up[kTreeShared];
  int start, end;
  seq_rows(a.b, blockIdx.x, start, end);
  const int n = end - start;
  if (n == 0) return;
  const int32_t* parents = a.parents + start;
  auto checked = [&](int i) {
    const int p = __ldg(parents + i);
    return p < i ? max(p, -1) : -1;
  };
  for (int i = threadIdx.x; i < n; i += kTreeThreads) {
    const int p = __ldg(parents + i);
    if (p < -1 || p >= i) record_bad_index(a.status, kWhereParent);
    if (i < kTreeShared) up[i] = checked(i);
  }
  if (threadIdx.x == 0 && n > 32ll * a.mask_words) record_bad_index(a.status, kWhereLength);
  __syncthreads();
  auto parent = [&](int i) { return i < kTreeShared ? up[i] : checked(i); };
  const int prefix = max(__ldg(a.b.kv_len + blockIdx.x), n) - n;   // (the least of lengths less n would wrap)
  const int window = a.window > 0 ? a.window : INT32_MAX;
  if (n <= kTreeThreads) {
    // ------------------------------------------------------------ rows joined
    __shared__ uint32_t bits[kTreeWords][kTreeThreads];
    __shared__ int32_t top[kTreeThreads], steps[kTreeThreads];   // the first ancestor not among the bits, how far up it is
    const int t = threadIdx.x;
    const bool live = t < n;
    uint32_t mine[kTreeWords];
    int at = live ? up[t] : -1, d = 1;
#pragma unroll
    for (int w = 0; w < kTreeWords; ++w) mine[w] = w == t >> 5 ? 1u << (t & 31) : 0u;
    while (__syncthreads_or(at >= 0)) {
#pragma unroll
      for (int w = 0; w < kTreeWords; ++w) bits[w][t] = mine[w];
      top[t] = at;
      steps[t] = d;
      __syncthreads();
      if (at >= 0) {
#pragma unroll
        for (int w = 0; w < kTreeWords; ++w) mine[w] |= bits[w][at];
        d += steps[at];
        at = top[at];
      }
    }
    if (!live) return;
    if (a.depth) a.depth[start + t] = d - 1;
    if (a.positions) a.positions[start + t] = prefix + d - 1;
    if (d <= window) {
      uint32_t* row = a.mask + static_cast<int64_t>(start + t) * a.mask_stride;
#pragma unroll
      for (int w = 0; w < kTreeWords; ++w)
        if (w < a.mask_words) row[w] = mine[w];
      for (int w = kTreeWords; w < a.mask_words; ++w) row[w] = 0;
      return;
    }
  }
  for (int t = threadIdx.x; t < n; t += kTreeThreads) {
    uint32_t* row = a.mask + static_cast<int64_t>(start + t) * a.mask_stride;
    int at = t, d = 0;   // an ancestor and how far up it is
    for (; at >= 0 && (at >> 5) >= a.mask_words; at = parent(at)) ++d;
    for (int w = a.mask_words - 1; w >= 0; --w) {
      uint32_t bits = 0;
      for (; at >= 0 && (at >> 5) == w; at = parent(at)) bits |= (d++ < window ? 1u : 0u) << (at & 31);
      row[w] = bits;
    }
    if (a.depth) a.depth[start + t] = d - 1;
    if (a.positions) a.positions[start + t] = prefix + d - 1;
  }
}

}  // namespace

cudaError_t launch_paged_tree(const PagedTreeArgs& a, cudaStream_t s) {
  paged_tree_kernel<<<a.b.n_seqs, kTreeThreads, 0, s>>>(a);
  return cudaGetLastError();
}

namespace {

sage_status check_tree(const sage_paged_tree_mask* t, int64_t n) {
  if (!t || t->mask_words <= 0 || t->mask_stride < 0 || (n > 1 && t->mask_stride < t->mask_words)) return SAGE_ERR_INVALID_ARG;
  if (n > 0 && !t->mask) return SAGE_ERR_INVALID_ARG;
  if (t->mask_words > 65536 || t->mask_stride > (int64_t(1) << 31)) return SAGE_ERR_UNSUPPORTED;
  if (!aligned(t->mask, 4) || !aligned(t->depth, 4)) return SAGE_ERR_ALIGNMENT;
  return SAGE_OK;
}

}  // namespace
}  // namespace sage

using namespace sage;

extern "C" {

sage_status sage_paged_tree(const sage_paged_batch* batch, int64_t n_tokens, const int32_t* parents, int64_t window,
                            const sage_paged_tree_mask* tree, int32_t* positions, void* status_block, void* stream) {
  sage_status st;
  if ((st = check_batch(batch, 1)) != SAGE_OK) return st;
  if (n_tokens < 0 || window < 0 || (n_tokens > 0 && !parents) || !status_block) return SAGE_ERR_INVALID_ARG;
  if (n_tokens > kMaxRows) return SAGE_ERR_UNSUPPORTED;
  if ((st = check_tree(tree, n_tokens)) != SAGE_OK) return st;
  if (!aligned(parents, 4) || !aligned(positions, 4) || !aligned(status_block, 4)) return SAGE_ERR_ALIGNMENT;
  if (n_tokens == 0 || batch->n_seqs == 0) return SAGE_OK;
  PagedTreeArgs a{};
  a.b.cu_q = batch->cu_q;
  a.b.kv_len = batch->kv_len;
  a.b.n_seqs = static_cast<int>(batch->n_seqs);
  a.b.n_tokens = static_cast<int>(n_tokens);
  a.parents = parents;
  a.window = window > INT32_MAX ? 0 : static_cast<int>(window);   // longer than any tree: none
  a.mask = tree->mask;
  a.mask_stride = tree->mask_stride;
  a.mask_words = static_cast<int>(tree->mask_words);
  a.depth = tree->depth;
  a.positions = positions;
  a.status = static_cast<int32_t*>(status_block);
  return cuda_status(launch_paged_tree(a, static_cast<cudaStream_t>(stream)));
}

sage_status sage_paged_attn_tree(const sage_view* q, const sage_paged_kv* cache, const sage_paged_batch* batch,
                                 const sage_paged_tree_mask* tree, float sm_scale, int64_t window, void* out,
                                 int64_t out_stride_token, int64_t out_stride_head, float* lse, void* ws, size_t ws_bytes,
                                 void* stream) {
  PagedAttnArgs a;
  sage_status st = attn_args(q, cache, batch, sm_scale, window, out, out_stride_token, out_stride_head, lse, ws, ws_bytes, a);
  if (st != SAGE_OK) return st;
  if ((st = check_tree(tree, q->n_tokens)) != SAGE_OK) return st;
  if (window > 0 && q->n_tokens > 0 && !tree->depth) return SAGE_ERR_INVALID_ARG;
  if (a.b.n_tokens == 0) return SAGE_OK;
  a.mask = tree->mask;
  a.mask_stride = tree->mask_stride;
  a.mask_words = static_cast<int>(tree->mask_words);
  a.depth = tree->depth;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int d = static_cast<int>(cache->head_dim);
  return cuda_status(few_rows(a) ? launch_paged_few_tree(a, *cache, d, s) : launch_paged_chunk_tree(a, *cache, d, s));
}

}  // extern "C"
