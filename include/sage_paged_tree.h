/*
 * sage_paged_tree.h -- drafted trees over the paged K/V cache of sage_paged.h: the ancestor bits of a tree, and attention
 * of its tokens over the cache.
 *
 * In speculative decoding the new tokens of a sequence are guesses that branch: token i continues its parent, not the
 * token before it in the batch.  One step of a layer is
 *   sage_paged_tree(parents, ...)                once for all layers: who sees whom, and where each token stands
 *   sage_paged_append(..., positions, ...)       K and V stored one after the other, rotated by their places in the text
 *   sage_paged_attn_tree(q, ..., tree, ...)      each token sees the cached text and its own ancestors
 * and when the guesses have been verified, sage_paged_compact (sage_paged_pool.h) moves the accepted path's tokens
 * together.  The rules of sage.h and sage_paged.h hold: device pointers, caller-owned buffers, nothing allocated, arguments
 * checked before anything is launched, indices in device memory checked by the kernels and recorded in the status block.
 */
#ifndef SAGE_GB300_PAGED_TREE_H
#define SAGE_GB300_PAGED_TREE_H

#include "sage_paged.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Which new tokens of its sequence each row of a call sees.
 *   mask         device, row t at mask + t * mask_stride: bit i % 32 of word i / 32 is set where row t sees new token i
 *                (counted within t's sequence).  New tokens from 32 * mask_words on are seen by no row.  Any bits are
 *                allowed: forests, several texts packed into one sequence, tokens that nobody sees; not seeing itself too.
 *   mask_words   1 to 65536; mask_stride at least mask_words (with one row it does not count).
 *   depth        device int32 [n_tokens]: how many tokens stand between the cached text and the row's own.  Read by
 *                sage_paged_attn_tree only with a window, and there taken into [0, new tokens of the sequence - 1].
 *                May be NULL without one. */
typedef struct sage_paged_tree_mask {
  uint32_t* mask;
  int64_t mask_words;
  int64_t mask_stride;
  int32_t* depth;
} sage_paged_tree_mask;

/* The mask of a batch of trees given by their parents.
 *   parents      device int32 [n_tokens]: the row's parent, counted within its sequence and before the row itself, or -1 for
 *                one that continues the cached text.  Anything else is recorded as where = 22 and taken as -1.
 *   window       0, or the sliding window of the attention: an ancestor `window` or more steps up is not seen.
 *   tree         mask (all mask_words of a row are written) and depth, which may be NULL: bit i of row t is set where i is t
 *                or an ancestor of t; depth = the number of its ancestors.
 *   positions    NULL, or device int32 [n_tokens]: max(0, kv_len - new tokens) + depth, the `positions` of
 *                sage_paged_append.
 * Of the batch, cu_q and kv_len are read.  A sequence of more than 32 * mask_words new tokens is recorded as where = 17; the
 * bits that have no place are left out.  Rows behind the last sequence are left as they were.  The outputs overlap neither
 * each other nor the inputs.  One launch. */
sage_status sage_paged_tree(const sage_paged_batch* batch, int64_t n_tokens, const int32_t* parents, int64_t window,
                            const sage_paged_tree_mask* tree, int32_t* positions, void* status_block, void* stream);

/* Attention of a batch of trees over the cache: sage_paged_attn, with other visible keys.  Behind the P = kv_len - n cached
 * tokens of a sequence lie its n new ones, token i at position P + i, and row t sees
 *   the positions below P (window > 0: of those the ones above P + depth[t] - window), and
 *   position P + i of each new token i whose bit is set in its row of tree->mask, whatever the window.
 * With a window the page entries of positions from P + 1 - window on are read, whatever the depths.  A row that sees no key
 * becomes 0, its lse -infinity.  A new token that no row sees may hold anything, as slots without a token; the rest of
 * [0, kv_len) (with a window: of [P + 1 - window, kv_len)) must be finite.
 * All else as for sage_paged_attn: views, cache, batch, sm_scale, out, lse, ws, errors, and the choice of a kernel by the
 * batch's mean rows.  Whoever comes last, parts are joined in the order of their keys.  So is the precision: where
 * sage_paged_attn holds q as fp16, the kernel for many rows over an E4M3 cache holds it as the sum of three E5M2 values times a
 * power of two per row, exact but for values 2^-23 below the row's largest, which keep an absolute error of 2^-31 of it
 * (fp16: 2^-14 and 2^-25).  An infinite q counts as NaN there. */
sage_status sage_paged_attn_tree(const sage_view* q, const sage_paged_kv* cache, const sage_paged_batch* batch,
                                 const sage_paged_tree_mask* tree, float sm_scale, int64_t window, void* out,
                                 int64_t out_stride_token, int64_t out_stride_head, float* lse, void* ws, size_t ws_bytes,
                                 void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SAGE_GB300_PAGED_TREE_H */
