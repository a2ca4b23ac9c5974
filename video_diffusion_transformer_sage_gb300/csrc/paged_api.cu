// paged_api.cu -- the extern "C" entry points declared in include/sage_paged.h: argument checks and
// the launches.  No entry point allocates device memory.
#include <cuda_runtime.h>

#include "paged_check.h"

using namespace sage;

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
  PagedAppendArgs a;
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
  return cuda_status(launch_paged_append(a, static_cast<int>(d), cache->format == 1,
                                         static_cast<cudaStream_t>(stream)));
}

size_t sage_paged_workspace_bytes(int64_t head_dim) { return paged_workspace_bytes(head_dim); }

sage_status sage_paged_attn(const sage_view* q, const sage_paged_kv* cache, const sage_paged_batch* batch,
                            float sm_scale, int64_t causal, int64_t window, void* out, int64_t out_stride_token,
                            int64_t out_stride_head, float* lse, void* ws, size_t ws_bytes, void* stream) {
  if ((causal != 0 && causal != 1) || (window > 0 && !causal)) return SAGE_ERR_INVALID_ARG;
  PagedAttnArgs a;
  const sage_status st = attn_args(q, cache, batch, sm_scale, window, out, out_stride_token, out_stride_head, lse, ws, ws_bytes, a);
  if (st != SAGE_OK || a.b.n_tokens == 0) return st;
  a.causal = static_cast<int>(causal);
  // By the mean query rows of a K/V head and sequence: up to 32 the cache's bandwidth is the limit and the
  // warp-level kernel comes nearer to it, above the tensor cores' tiles pay (16 sequences of 4000 keys, 4 heads of 128
  // channels: 32 rows 39 us against 42, 40 rows 52 against 43; 8 sequences, 24 heads of 64 channels: 47 against 67,
  // 36 rows 76 against 67).
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int d = static_cast<int>(cache->head_dim);
  return cuda_status(few_rows(a) ? launch_paged_few(a, *cache, d, s) : launch_paged_chunk(a, *cache, d, s));
}

}  // extern "C"
