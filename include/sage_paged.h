/*
 * sage_paged.h -- the paged K/V cache entry points of `libsage_gb300.so`: appending a batch's new
 * tokens to a cache that lies in pages, and attention of those tokens over it.
 *
 * sage.h computes attention over one packed sequence whose tokens are all there at once.  These
 * calls are for generation in pieces (a video chunk by chunk, a text token by token): K and V of
 * the tokens so far stay in the cache, and each call brings the new tokens of a batch of
 * sequences, one token or thousands of each.  The usual pair per layer is
 *   sage_paged_append(q, k, v, ...)   per-head RMSNorm and rotation of Q and K, K and V stored
 *   sage_paged_attn(q, ...)           the new tokens' attention over everything stored
 *
 * The general rules of sage.h hold: device pointers, caller-owned buffers, nothing allocated, work
 * enqueued on `stream` of the current device, arguments checked before anything is launched.  What
 * lies in device memory (lengths, page table, positions) cannot be checked there: the kernels
 * check every index before they use it.  An index that is out of range is never followed; the call
 * goes on with the rest as each entry point says, and the status block records SAGE_ERR_INVALID_ARG
 * with where = 16 (page table entry), 17 (length) or 18 (row of the rotary table), which
 * sage_check_device_status returns; the first one recorded stays until it is read.  A device wait that
 * expires is recorded as in sage.h (where = 19, 20 or 21), in the place of an index that was not read yet.  Since lengths are read on the device, a captured CUDA graph
 * may be replayed after they changed, as long as the buffers and n_tokens, n_seqs stay.
 */
#ifndef SAGE_GB300_PAGED_H
#define SAGE_GB300_PAGED_H

#include "sage.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A paged K/V cache.  Element (page, slot, head, c) of K lies at k_pages + page * k_stride_page +
 * slot * k_stride_token + head * k_stride_head + c, strides in elements; V likewise.
 *   format      0: bf16 values.
 *               1: FP8 E4M3 codes; a code c of head h stands for c * k_scale[h] (V: v_scale[h]).
 *                  k_scale, v_scale: device fp32 [n_heads], positive normal numbers below 2^126, fixed while
 *                  the cache is in use.
 *   page_size   tokens per page, a power of two from 8 to 1024.
 *   head_dim    64 or 128; n_heads 1 to 4096; n_pages 1 to 2^31 - 1.
 * Pages 16-byte aligned, strides positive multiples of 16 bytes below 2^40 bytes (a stride whose
 * dimension has one element is ignored).  E.g. [n_pages][page_size][n_heads][head_dim] or
 * [n_pages][n_heads][page_size][head_dim] contiguous; K and V may be slices of one buffer.
 * Slots that hold no token may hold anything, infinities and NaN included. */
typedef struct sage_paged_kv {
  void* k_pages;
  void* v_pages;
  int64_t n_pages;
  int64_t page_size;
  int64_t n_heads;
  int64_t head_dim;
  int64_t k_stride_page, k_stride_token, k_stride_head;
  int64_t v_stride_page, v_stride_token, v_stride_head;
  int64_t format;
  const float* k_scale;
  const float* v_scale;
} sage_paged_kv;

/* The sequences of a call and their new tokens.
 *   n_seqs      0 to 65536.
 *   cu_q        device int32 [n_seqs + 1], ascending: the new tokens of sequence b are rows
 *               cu_q[b] .. cu_q[b + 1] - 1 of the call's q, k, v (none where the two are equal).
 *               Rows from cu_q[n_seqs] on (a padded batch) are neither read for a result nor written.
 *   kv_len      device int32 [n_seqs]: tokens of sequence b in the cache, its new ones included: new
 *               token j of n has position kv_len[b] - n + j.  A position below 0 is left padding: the
 *               token is not stored and sees no key in causal attention.
 *   page_table  device int32, entry (b, i) at page_table[b * table_stride + i], i < max_pages: the
 *               page of positions i * page_size .. (i + 1) * page_size - 1 of sequence b.  Only entries of
 *               pages that a call stores to or sees a key of are read, so pages before a sliding
 *               window may be given back.  Sequences may share pages that are only read.
 *               max_pages * page_size is at most 2^30.  Of a kv_len above it sage_paged_append stores no
 *               position past the table, and sage_paged_attn takes it as max_pages * page_size. */
typedef struct sage_paged_batch {
  int64_t n_seqs;
  const int32_t* cu_q;
  const int32_t* kv_len;
  const int32_t* page_table;
  int64_t max_pages;
  int64_t table_stride;
} sage_paged_batch;

/* Appends the new tokens' K and V to the cache, with the qk_transform stage of
 * sage_qk_rmsnorm_rope on the way: per token and head, in fp32 with every product and sum rounded on
 * its own and in that entry point's order,
 *   y = (x / sqrt(mean x^2 + eps)) * gamma   where gamma is given,
 *   z_2i = y_2i cos_i - y_2i+1 sin_i,  z_2i+1 = y_2i sin_i + y_2i+1 cos_i   where the table is given
 *   (neighbouring channels are a pair; weights made for pairs (i, i + head_dim / 2) need their rows reordered first).
 *   K: stored as bf16_rn(z), or as the E4M3 code (round to nearest even, saturating) of
 *      fl32(z * fl32(1 / k_scale[h])), z itself not rounded to bf16 first.
 *   V: stored as it is, or as the E4M3 code of fl32(v * fl32(1 / v_scale[h])).
 *   Q: bf16_rn(z) to q_out.
 * With gamma, a table and a bf16 cache, the values are those of sage_qk_rmsnorm_rope bit for bit.
 *   q               bf16 [n_tokens, n_heads_q, head_dim] view, or NULL: K and V alone; its head
 *                   count is its own.  q_out has its own strides; it may be q itself, then with q's strides, and
 *                   otherwise overlaps none of the inputs.
 *   k, v            bf16 [n_tokens, cache n_heads, head_dim] views.
 *   gamma_q/_k      device fp32 [head_dim] or NULL (no norm of that operand).
 *   rope_cos/_sin   device fp32 [rope_rows][head_dim / 2], both or neither (no rotation).  For a rotation of
 *                   fewer channels, cos = 1 and sin = 0 in the rest.
 *   positions       device int32 [n_tokens]: the table row of each token; NULL: its position in
 *                   its sequence.
 *   status_block    as in sage.h (sage_status_block_bytes, zeroed once); a workspace of
 *                   sage_paged_attn begins with one.  The attention calls of sage.h do no work on a block
 *                   that holds an unread record: give them another.
 * A token with no place (left padding, a position past max_pages * page_size, a page or table row
 * out of range) is not stored and its q_out row becomes 0; left padding is no error.  No two tokens
 * of a call may have the same slot of the same page.  Views need 16-byte aligned data and strides of
 * multiples of 8 elements; n_tokens may be 0 (nothing is launched), n_tokens at most 2^22 and
 * n_tokens * (n_heads_q + 2 n_heads) at most 2^31.  One launch. */
sage_status sage_paged_append(const sage_view* q, const sage_view* k, const sage_view* v, const float* gamma_q,
                              const float* gamma_k, const float* rope_cos, const float* rope_sin, int64_t rope_rows,
                              const int32_t* positions, float eps, const sage_paged_kv* cache,
                              const sage_paged_batch* batch, void* q_out, int64_t q_out_stride_token,
                              int64_t q_out_stride_head, void* status_block, void* stream);

/* The part of the workspace that has to start as zeros: the status block and the join counters, which
 * every call leaves at zero. */
#define SAGE_PAGED_WS_HEADER 4096

/* Bytes of workspace sage_paged_attn needs for any batch with this head_dim: a status block, the join
 * counters and the partial results of a split key axis.  0 for a head_dim that is not taken. */
size_t sage_paged_workspace_bytes(int64_t head_dim);

/* Attention of the batch's new tokens over the cache:
 *   out[t][h] = bf16_rn( sum_j p_j v_j / sum_j p_j ),  p_j = exp(sm_scale * q[t][h] . k_j - max)
 * over the visible positions j of the token's sequence, K / V head h / (n_heads_q / n_heads):
 *   causal 0: all of [0, kv_len);   causal 1: those up to the token's own position pos;
 *   window > 0 (with causal 1 only): of those the last `window`, j > pos - window.
 * A row that sees no key becomes 0, its lse -infinity; any other whose q holds a NaN becomes NaN, and its lse too.
 * Scores, maxima, sums and accumulators are fp32; p is rounded to bf16 for the product with V, as in
 * sage_attn_dense_bf16_tc, or to fp16 with an E4M3 cache (whose codes fp16 holds exactly; q is then held as fp16
 * times a power of two per row).  Against a running maximum that may lag by 2^8, p lies in [0, 2^8] (fp16: times
 * 2^7).  Per element, |out - exact| <= 2^-7 sum_j w_j |v_j| + 2^-8 |out| plus fp32 rounding, w the exact weights; with
 * an E4M3 cache plus 2^-32 (sum_j |v_j| + n |out|) over the n visible keys, the steps of fp16's subnormals, which
 * p reaches at 2^-21 of the row's largest.  Stored K and V of a sequence's visible range must be finite (a NaN in a
 * value that only some of the rows see may reach the others).  Key positions whose page entry is
 * out of range are left out, as masked ones.
 *   q            bf16 [n_tokens, n_heads_q, head_dim] view; n_heads_q a multiple of the cache's
 *                n_heads, at most 128 times as many.
 *   out          bf16, element (t, h, c) at out[t * out_stride_token + h * out_stride_head + c],
 *                16-byte aligned, strides multiples of 8 elements and not 0 where there are several rows, not
 *                overlapping the inputs.
 *   lse          NULL, or device fp32 [n_tokens][n_heads_q] contiguous: ln sum_j exp(sm_scale q . k_j).
 *   sm_scale     positive, finite also when multiplied by log2 e.
 *   ws           256-byte aligned, >= sage_paged_workspace_bytes; its first SAGE_PAGED_WS_HEADER bytes
 *                zeroed once by the caller before its first use (and again after a recorded timeout);
 *                it begins with the status block.  Calls that may overlap on the GPU need workspaces of
 *                their own.
 * The result does not depend on what else runs: partial results are joined in a fixed order.
 * A batch whose mean query rows per K/V head and sequence (new tokens times n_heads_q / n_heads) are at most 32 takes
 * one launch of the kernel for few rows (a batch of 2^31 or more key tiles of 16 KB of K is recorded as where =
 * 17 and not computed), any other the tensor-core kernel for many rows, one launch or two. */
sage_status sage_paged_attn(const sage_view* q, const sage_paged_kv* cache, const sage_paged_batch* batch,
                            float sm_scale, int64_t causal, int64_t window, void* out, int64_t out_stride_token,
                            int64_t out_stride_head, float* lse, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SAGE_GB300_PAGED_H */
