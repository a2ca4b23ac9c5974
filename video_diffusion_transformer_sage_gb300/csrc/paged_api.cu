// paged_api.cu -- the extern "C" entry points declared in include/sage_paged.h: argument checks and
// the launches.  No entry point allocates device memory.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "paged_internal.h"

namespace {

constexpr size_t kStatusBytes = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int64_t kMaxRows = int64_t(1) << 22, kMaxHeads = 4096, kMaxSeqs = 65536;

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline sage_status cuda_status(cudaError_t e) { return e == cudaSuccess ? SAGE_OK : SAGE_ERR_CUDA; }

// A [n, heads, d] bf16 view; n may be 0, and its data then null.
sage_status check_rows(const sage_view* v, int64_t n, int64_t d) {
  if (!v || v->n_tokens != n || v->n_heads <= 0 || v->head_dim != d) return SAGE_ERR_INVALID_ARG;
  if (n > 0 && !v->data) return SAGE_ERR_INVALID_ARG;
  if (v->n_heads > kMaxHeads) return SAGE_ERR_UNSUPPORTED;
  if (v->stride_token < 0 || v->stride_head < 0) return SAGE_ERR_INVALID_ARG;
  if (!aligned(v->data, 16) || (v->stride_token % 8) != 0 || (v->stride_head % 8) != 0) return SAGE_ERR_ALIGNMENT;
  return SAGE_OK;
}

sage_status check_cache(const sage_paged_kv* c) {
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

sage_status check_batch(const sage_paged_batch* b, int64_t page_size) {
  if (!b || b->n_seqs < 0) return SAGE_ERR_INVALID_ARG;
  if (b->n_seqs == 0) return SAGE_OK;
  if (!b->cu_q || !b->kv_len || !b->page_table || b->max_pages <= 0 || b->table_stride < 0) return SAGE_ERR_INVALID_ARG;
  if (b->n_seqs > 1 && b->table_stride < b->max_pages) return SAGE_ERR_INVALID_ARG;
  if (b->n_seqs > kMaxSeqs || b->max_pages > (int64_t(1) << 30) / page_size) return SAGE_ERR_UNSUPPORTED;
  if (!aligned(b->cu_q, 4) || !aligned(b->kv_len, 4) || !aligned(b->page_table, 4)) return SAGE_ERR_ALIGNMENT;
  return SAGE_OK;
}

// An output of the view's shape; rows that coincide (a zero stride) are refused.
sage_status check_target(const void* out, int64_t ost, int64_t osh, const sage_view* v) {
  if (!out || ost < 0 || osh < 0 || (ost == 0 && v->n_tokens > 1) || (osh == 0 && v->n_heads > 1)) return SAGE_ERR_INVALID_ARG;
  if (!aligned(out, 16) || (ost % 8) != 0 || (osh % 8) != 0) return SAGE_ERR_ALIGNMENT;
  return SAGE_OK;
}

sage::PagedBatchDev batch_dev(const sage_paged_batch* b, const sage_paged_kv* c, int64_t n) {
  sage::PagedBatchDev d;
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
constexpr size_t kCountersOff = kStatusBytes;
constexpr size_t kMlOff = SAGE_PAGED_WS_HEADER;
static_assert(kCountersOff + sizeof(int32_t) * (2 * sage::kPagedMaxCtas + 2) <= kMlOff, "counters exceed the workspace header");
constexpr size_t kSlots = sage::kPagedSlots;
constexpr size_t kPartOff = kMlOff + kSlots * sage::kPagedChunkRows * sizeof(float2);

}  // namespace

extern "C" {

sage_status sage_paged_append(const sage_view* q, const sage_view* k, const sage_view* v, const float* gamma_q,
                              const float* gamma_k, const float* rope_cos, const float* rope_sin, int64_t rope_rows,
                              const int32_t* positions, float eps, const sage_paged_kv* cache,
                              const sage_paged_batch* batch, void* q_out, int64_t q_out_stride_token,
                              int64_t q_out_stride_head, void* status_block, void* stream) {
  sage_status st;
  if ((st = check_cache(cache)) != SAGE_OK || (st = check_batch(batch, cache->page_size)) != SAGE_OK) return st;
  if (!k || !v || k->n_tokens < 0) return SAGE_ERR_INVALID_ARG;
  const int64_t n = k->n_tokens, d = cache->head_dim;
  if (n > kMaxRows) return SAGE_ERR_UNSUPPORTED;
  if ((st = check_rows(k, n, d)) != SAGE_OK || (st = check_rows(v, n, d)) != SAGE_OK) return st;
  if (k->n_heads != cache->n_heads || v->n_heads != cache->n_heads) return SAGE_ERR_INVALID_ARG;
  if (q) {
    if ((st = check_rows(q, n, d)) != SAGE_OK) return st;
    if (n > 0 && (st = check_target(q_out, q_out_stride_token, q_out_stride_head, q)) != SAGE_OK) return st;
    // In q's own memory each row may only go where it came from: another warp's row could be overwritten unread.
    if (n > 0 && q_out == q->data &&
        ((n > 1 && q_out_stride_token != q->stride_token) || (q->n_heads > 1 && q_out_stride_head != q->stride_head)))
      return SAGE_ERR_INVALID_ARG;
  }
  if ((rope_cos == nullptr) != (rope_sin == nullptr) || (rope_cos && rope_rows <= 0)) return SAGE_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !(eps < INFINITY)) return SAGE_ERR_INVALID_ARG;
  if (!aligned(gamma_q, 16) || !aligned(gamma_k, 16) || !aligned(rope_cos, 16) || !aligned(rope_sin, 16) ||
      !aligned(positions, 4) || !aligned(status_block, 4))
    return SAGE_ERR_ALIGNMENT;
  if (!status_block) return SAGE_ERR_INVALID_ARG;
  if (n * ((q ? q->n_heads : 0) + 2 * cache->n_heads) > (int64_t(1) << 31)) return SAGE_ERR_UNSUPPORTED;   // rows
  if (n == 0 || batch->n_seqs == 0) return SAGE_OK;
  const int64_t e = cache->format == 1 ? 1 : 2;
  sage::PagedAppendArgs a;
  a.b = batch_dev(batch, cache, n);
  a.q = q ? static_cast<const uint16_t*>(q->data) : nullptr;
  a.qst = q ? q->stride_token : 0;
  a.qsh = q ? q->stride_head : 0;
  a.k = static_cast<const uint16_t*>(k->data);
  a.kst = k->stride_token;
  a.ksh = k->stride_head;
  a.v = static_cast<const uint16_t*>(v->data);
  a.vst = v->stride_token;
  a.vsh = v->stride_head;
  a.hq = q ? static_cast<int>(q->n_heads) : 0;
  a.hkv = static_cast<int>(cache->n_heads);
  a.gamma_q = gamma_q;
  a.gamma_k = gamma_k;
  a.rope_cos = rope_cos;
  a.rope_sin = rope_sin;
  a.rope_rows = rope_rows;
  a.positions = positions;
  a.eps = eps;
  a.k_pages = static_cast<uint8_t*>(cache->k_pages);
  a.v_pages = static_cast<uint8_t*>(cache->v_pages);
  a.kp = cache->k_stride_page * e;
  a.kt = cache->k_stride_token * e;
  a.kh = cache->k_stride_head * e;
  a.vp = cache->v_stride_page * e;
  a.vt = cache->v_stride_token * e;
  a.vh = cache->v_stride_head * e;
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.ost = q_out_stride_token;
  a.osh = q_out_stride_head;
  a.status = static_cast<int32_t*>(status_block);
  return cuda_status(sage::launch_paged_append(a, static_cast<int>(d), cache->format == 1,
                                               static_cast<cudaStream_t>(stream)));
}

size_t sage_paged_workspace_bytes(int64_t head_dim) {
  if (head_dim != 64 && head_dim != 128) return 0;
  return kPartOff + kSlots * sage::kPagedChunkRows * static_cast<size_t>(head_dim) * sizeof(float);
}

sage_status sage_paged_attn(const sage_view* q, const sage_paged_kv* cache, const sage_paged_batch* batch,
                            float sm_scale, int64_t causal, int64_t window, void* out, int64_t out_stride_token,
                            int64_t out_stride_head, float* lse, void* ws, size_t ws_bytes, void* stream) {
  sage_status st;
  if ((st = check_cache(cache)) != SAGE_OK || (st = check_batch(batch, cache->page_size)) != SAGE_OK) return st;
  if (!q || q->n_tokens < 0) return SAGE_ERR_INVALID_ARG;
  const int64_t n = q->n_tokens, d = cache->head_dim;
  if (n > kMaxRows) return SAGE_ERR_UNSUPPORTED;
  if ((st = check_rows(q, n, d)) != SAGE_OK) return st;
  if (q->n_heads % cache->n_heads != 0) return SAGE_ERR_INVALID_ARG;
  if (q->n_heads / cache->n_heads > 128) return SAGE_ERR_UNSUPPORTED;
  if ((causal != 0 && causal != 1) || window < 0 || (window > 0 && !causal)) return SAGE_ERR_INVALID_ARG;
  if (!(sm_scale > 0.0f) || !(sm_scale * kLog2e < INFINITY)) return SAGE_ERR_INVALID_ARG;
  if (n > 0 && (st = check_target(out, out_stride_token, out_stride_head, q)) != SAGE_OK) return st;
  if (!aligned(lse, 4)) return SAGE_ERR_ALIGNMENT;
  if (!ws) return SAGE_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return SAGE_ERR_ALIGNMENT;
  if (ws_bytes < sage_paged_workspace_bytes(d)) return SAGE_ERR_WORKSPACE;
  if (n == 0 || batch->n_seqs == 0) return SAGE_OK;
  sage::PagedAttnArgs a;
  a.b = batch_dev(batch, cache, n);
  a.q = static_cast<const uint16_t*>(q->data);
  a.qst = q->stride_token;
  a.qsh = q->stride_head;
  a.hq = static_cast<int>(q->n_heads);
  a.hkv = static_cast<int>(cache->n_heads);
  a.causal = static_cast<int>(causal);
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
  // By the mean query rows of a K/V head and sequence: up to 32 the cache's bandwidth is the limit and the
  // warp-level kernel comes nearer to it, above the tensor cores' tiles pay (16 sequences of 4000 keys, 4 heads of 128
  // channels: 32 rows 39 us against 42, 40 rows 52 against 43; 8 sequences, 24 heads of 64 channels: 47 against 67,
  // 36 rows 76 against 67).
  const int64_t rows = n * (q->n_heads / cache->n_heads), seqs = batch->n_seqs < n ? batch->n_seqs : n;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(rows <= 32 * seqs ? sage::launch_paged_few(a, *cache, static_cast<int>(d), s)
                                       : sage::launch_paged_chunk(a, *cache, static_cast<int>(d), s));
}

}  // extern "C"
