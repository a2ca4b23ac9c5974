// paged_check.h -- host side of the paged-cache entry points: argument checks, the batch as the kernels take it, and the
// workspace's layout.
#pragma once
#include <cmath>
#include <cstdint>

#include "paged_internal.h"

namespace sage {

constexpr size_t kPagedStatusBytes = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int64_t kMaxRows = int64_t(1) << 22, kMaxHeads = 4096, kMaxSeqs = 65536;

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline sage_status cuda_status(cudaError_t e) { return e == cudaSuccess ? SAGE_OK : SAGE_ERR_CUDA; }

// A [n, heads, d] bf16 view; n may be 0, and its data then null.
inline sage_status check_rows(const sage_view* v, int64_t n, int64_t d) {
  if (!v || v->n_tokens != n || v->n_heads <= 0 || v->head_dim != d) return SAGE_ERR_INVALID_ARG;
  if (n > 0 && !v->data) return SAGE_ERR_INVALID_ARG;
  if (v->n_heads > kMaxHeads) return SAGE_ERR_UNSUPPORTED;
  if (v->stride_token < 0 || v->stride_head < 0) return SAGE_ERR_INVALID_ARG;
  if (!aligned(v->data, 16) || (v->stride_token % 8) != 0 || (v->stride_head % 8) != 0) return SAGE_ERR_ALIGNMENT;
  return SAGE_OK;
}

inline sage_status check_cache(const sage_paged_kv* c) {
  if (!c || !c->k_pages || !c->v_pages || c->n_pages <= 0 || c->n_heads <= 0) return SAGE_ERR_INVALID_ARG;
  if (c->format != 0 && c->format != 1) return SAGE_ERR_INVALID_ARG;
  if (c->format == 1 && (!c->k_scale || !c->v_scale)) return SAGE_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return SAGE_ERR_UNSUPPORTED;
  if (c->n_heads > kMaxHeads || c->n_pages > INT32_MAX) return SAGE_ERR_UNSUPPORTED;
  if (c->page_size < 8 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)) != 0) return SAGE_ERR_UNSUPPORTED;
  if (!aligned(c->k_pages, 16) || !aligned(c->v_pages, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
    return SAGE_ERR_ALIGNMENT;
  const int64_t e = c->format == 1 ? 1 : 2;
  const int64_t strides[6] = {c->k_stride_page, c->k_stride_token, c->k_stride_head,
                              c->v_stride_page, c->v_stride_token, c->v_stride_head};
  const int64_t extents[3] = {c->n_pages, c->page_size, c->n_heads};
  for (int i = 0; i < 6; ++i) {
    if (extents[i % 3] == 1) continue;
    if (strides[i] <= 0) return SAGE_ERR_INVALID_ARG;
    if (strides[i] >= (int64_t(1) << 40) / e) return SAGE_ERR_UNSUPPORTED;
    if (strides[i] * e % 16 != 0) return SAGE_ERR_ALIGNMENT;
  }
  return SAGE_OK;
}

inline sage_status check_batch(const sage_paged_batch* b, int64_t page_size) {
  if (!b || b->n_seqs < 0) return SAGE_ERR_INVALID_ARG;
  if (b->n_seqs == 0) return SAGE_OK;
  if (!b->cu_q || !b->kv_len || !b->page_table || b->max_pages <= 0 || b->table_stride < 0) return SAGE_ERR_INVALID_ARG;
  if (b->n_seqs > 1 && b->table_stride < b->max_pages) return SAGE_ERR_INVALID_ARG;
  if (b->n_seqs > kMaxSeqs || b->max_pages > (int64_t(1) << 30) / page_size) return SAGE_ERR_UNSUPPORTED;
  if (!aligned(b->cu_q, 4) || !aligned(b->kv_len, 4) || !aligned(b->page_table, 4)) return SAGE_ERR_ALIGNMENT;
  return SAGE_OK;
}

// An output of the view's shape; rows that coincide (a zero stride) are refused.
inline sage_status check_target(const void* out, int64_t ost, int64_t osh, const sage_view* v) {
  if (!out || ost < 0 || osh < 0 || (ost == 0 && v->n_tokens > 1) || (osh == 0 && v->n_heads > 1)) return SAGE_ERR_INVALID_ARG;
  if (!aligned(out, 16) || (ost % 8) != 0 || (osh % 8) != 0) return SAGE_ERR_ALIGNMENT;
  return SAGE_OK;
}

inline PagedBatchDev batch_dev(const sage_paged_batch* b, const sage_paged_kv* c, int64_t n) {
  PagedBatchDev d;
  d.cu_q = b->cu_q;
  d.kv_len = b->kv_len;
  d.table = b->page_table;
  d.table_stride = b->table_stride;
  d.n_seqs = static_cast<int>(b->n_seqs);
  d.n_tokens = static_cast<int>(n);
  d.cap = static_cast<int>(b->max_pages * c->page_size);
  d.n_pages = static_cast<int>(c->n_pages);
  d.page_shift = 0;
  while ((int64_t(1) << d.page_shift) < c->page_size) ++d.page_shift;
  return d;
}

// Workspace: status block | counters | (maximum, sum) of each partial row | partial O.
constexpr size_t kCountersOff = kPagedStatusBytes;
constexpr size_t kMlOff = SAGE_PAGED_WS_HEADER;
static_assert(kCountersOff + sizeof(int32_t) * kPagedCounters <= kMlOff, "counters exceed the workspace header");
constexpr size_t kSlots = kPagedSlots;
constexpr size_t kPartOff = kMlOff + kSlots * kPagedChunkRows * sizeof(float2);

inline size_t paged_workspace_bytes(int64_t head_dim) {
  if (head_dim != 64 && head_dim != 128) return 0;
  return kPartOff + kSlots * kPagedChunkRows * static_cast<size_t>(head_dim) * sizeof(float);
}

// What the attention calls have in common: the checks, and the kernels' arguments (b.n_tokens is 0 where there is nothing
// to do).
inline sage_status attn_args(const sage_view* q, const sage_paged_kv* cache, const sage_paged_batch* batch, float sm_scale,
                             int64_t window, void* out, int64_t out_stride_token, int64_t out_stride_head, float* lse,
                             void* ws, size_t ws_bytes, PagedAttnArgs& a) {
  sage_status st;
  if ((st = check_cache(cache)) != SAGE_OK || (st = check_batch(batch, cache->page_size)) != SAGE_OK) return st;
  if (!q || q->n_tokens < 0) return SAGE_ERR_INVALID_ARG;
  const int64_t n = q->n_tokens, d = cache->head_dim;
  if (n > kMaxRows) return SAGE_ERR_UNSUPPORTED;
  if ((st = check_rows(q, n, d)) != SAGE_OK) return st;
  if (q->n_heads % cache->n_heads != 0) return SAGE_ERR_INVALID_ARG;
  if (q->n_heads / cache->n_heads > 128) return SAGE_ERR_UNSUPPORTED;
  if (window < 0) return SAGE_ERR_INVALID_ARG;
  if (!(sm_scale > 0.0f) || !(sm_scale * kLog2e < INFINITY)) return SAGE_ERR_INVALID_ARG;
  if (n > 0 && (st = check_target(out, out_stride_token, out_stride_head, q)) != SAGE_OK) return st;
  if (!aligned(lse, 4)) return SAGE_ERR_ALIGNMENT;
  if (!ws) return SAGE_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return SAGE_ERR_ALIGNMENT;
  if (ws_bytes < paged_workspace_bytes(d)) return SAGE_ERR_WORKSPACE;
  a = PagedAttnArgs{};
  if (n == 0 || batch->n_seqs == 0) return SAGE_OK;
  a.b = batch_dev(batch, cache, n);
  a.q = static_cast<const uint16_t*>(q->data);
  a.qst = q->stride_token;
  a.qsh = q->stride_head;
  a.hq = static_cast<int>(q->n_heads);
  a.hkv = static_cast<int>(cache->n_heads);
  a.window = window > (int64_t(1) << 30) ? 0 : static_cast<int>(window);   // longer than any sequence: none
  a.scale_log2 = sm_scale * kLog2e;
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.out = static_cast<uint16_t*>(out);
  a.ost = out_stride_token;
  a.osh = out_stride_head;
  a.lse = lse;
  char* w = static_cast<char*>(ws);
  a.status = reinterpret_cast<int32_t*>(w);
  a.counters = reinterpret_cast<int32_t*>(w + kCountersOff);
  a.part_ml = reinterpret_cast<float2*>(w + kMlOff);
  a.part_o = reinterpret_cast<float*>(w + kPartOff);
  return SAGE_OK;
}

// The mean query rows of a K/V head and sequence, times `seqs`, against 32.
inline bool few_rows(const PagedAttnArgs& a) {
  const int64_t rows = static_cast<int64_t>(a.b.n_tokens) * (a.hq / a.hkv);
  return rows <= 32 * static_cast<int64_t>(a.b.n_seqs < a.b.n_tokens ? a.b.n_seqs : a.b.n_tokens);
}

}  // namespace sage
