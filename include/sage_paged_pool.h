/*
 * sage_paged_pool.h -- the pages of the paged K/V cache of sage_paged.h: giving them out, sharing them between sequences
 * that begin alike, taking them back, copying them, and moving a sequence's kept tokens together.
 *
 * A page is a number; the same number stands for a page of K and of V in the cache of every layer, so the accounting
 * (reserve, fork, release) is one call for all layers, and copy and compact are one call for each layer's cache.
 *   a prompt or drafts       sage_paged_reserve: pages for the positions to come, before sage_paged_append
 *   beams, parallel samples  sage_paged_fork: the child shares the full pages of its parent and gets a page of its own for
 *                            the begun one, which sage_paged_copy fills
 *   verified drafts          sage_paged_compact moves the accepted tokens together, sage_paged_release gives back the pages
 *                            behind them; it also gives back those before a sliding window, or all of a finished sequence
 *
 * The rules of sage.h and sage_paged.h hold: device pointers, caller-owned buffers, nothing allocated, arguments checked
 * before anything is launched.  What lies in device memory is checked by the kernels: an index that is out of range is never
 * followed, the rest goes on, and the status block records SAGE_ERR_INVALID_ARG with `where` = 16 (page), 17 (length), 23 (kept
 * position), 24 (a page given back or shared that nobody holds) or 25 (row of the page table); an expired wait has where = 26.
 * Everything is read on the device, so a captured graph may be replayed after the numbers changed.  Results are
 * determined by the inputs, whatever runs when.
 */
#ifndef SAGE_GB300_PAGED_POOL_H
#define SAGE_GB300_PAGED_POOL_H

#include "sage_paged.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Pages and who holds them.
 *   refs          device int32 [n_pages]: how many entries of page tables hold the page; 0: free.  Negative counts are left
 *                 alone: such a page is never given out.
 *   page_table    device int32, entry (r, i) at page_table[r * table_stride + i], i < max_pages, as in sage_paged_batch.
 *                 An entry without a page is -1 (any negative number above -2^30 counts as it).
 *   page_size     a power of two from 8 to 1024; max_pages * page_size at most 2^30; n_rows 1 to 65536.
 * Counts and tables belong together: what other tables hold is counted too, by the caller or by calls with that table. */
typedef struct sage_paged_pool {
  int32_t* refs;
  int64_t n_pages;
  int32_t* page_table;
  int64_t n_rows;
  int64_t max_pages;
  int64_t table_stride;
  int64_t page_size;
} sage_paged_pool;

/* Bytes of workspace of the accounting calls: a status block first (sage_status_block_bytes, zeroed once by the caller),
 * then scratch.  0 for sizes that are not taken. */
size_t sage_paged_pool_workspace_bytes(int64_t n_rows, int64_t n_pages);

/* Gives back the pages of row r whose positions all lie outside [lo[r], hi[r]): each entry's page counts one less, the entry
 * becomes -1.  lo, hi: device int32 [n_rows]; lo NULL: 0.  Where hi <= lo the whole row goes.  An entry whose page does not
 * exist (where = 16) becomes -1 too, and so does one whose page nobody holds (24), which stays at 0.  One launch. */
sage_status sage_paged_release(const sage_paged_pool* pool, const int32_t* lo, const int32_t* hi, void* status_block,
                               void* stream);

/* Gives row r a page for each entry without one among those of the positions [lo[r], hi[r]).  The missing entries in
 * ascending order (row, entry) get the free pages in ascending order, whose counts become 1.
 *   lo, hi   device int32 [n_rows]; lo NULL: 0; taken into [0, max_pages * page_size], a larger hi is recorded (17).
 *   ok       NULL, or device int32 [n_rows]: 1 where the row has all its pages.  If the free pages do not last for the
 *            missing entries of the rows up to and with r, row r gets none: 0 (a row that misses none: 1).
 * One launch.  Calls on one pool come one after the other. */
sage_status sage_paged_reserve(const sage_paged_pool* pool, const int32_t* lo, const int32_t* hi, int32_t* ok, void* ws,
                               size_t ws_bytes, void* stream);

/* For each k < n_forks: row dst_rows[k], which holds no page, begins like row src_rows[k], n_tokens[k] positions long.  The
 * full pages are shared (the entries copied, the counts one more); a page begun gets a free one of the child's own, in
 * ascending order of k and page, and goes on the copy list:
 *   copy_src, copy_dst, copy_tokens   device int32 [n_forks]: the begun page, the child's, and how many tokens of it; -1, -1, 0
 *                                     where there is nothing to copy (sage_paged_copy takes the lists as they are).
 *   ok                                device int32 [n_forks]: 1 where the child was made.  0: the free pages did not last
 *                                     (as for sage_paged_reserve) and the child's row is empty, or the fork is not possible.
 * Not possible (where = 25): a row that does not exist, src = dst, a dst row that holds a page; and among the forks left, a dst
 * that an earlier one has, a src that is a dst of one of them.  (A fork not possible by itself changes no row and stands in no
 * other's way.)  n_tokens is taken into [0, max_pages * page_size] (17).  An entry of the source without a valid page (16), or
 * whose page nobody held before the call (24), is -1 in the child, or not copied.  n_forks at most n_rows.  One launch. */
sage_status sage_paged_fork(const sage_paged_pool* pool, const int32_t* src_rows, const int32_t* dst_rows,
                            const int32_t* n_tokens, int64_t n_forks, int32_t* copy_src, int32_t* copy_dst,
                            int32_t* copy_tokens, int32_t* ok, void* ws, size_t ws_bytes, void* stream);

/* K and V of the slots 0 .. n_tokens[i] - 1 of page src[i] to page dst[i], for each i < n_copies, as they are (codes of an
 * E4M3 cache too).
 *   src, dst   device int32 [n_copies].  An entry with a -1 on either side is left out; src = dst changes nothing.  A page
 *              may be the source of several copies; none may be the target of two, or target and source of two.
 *   n_tokens   device int32 [n_copies], or NULL: whole pages.  Taken into [0, page_size]; others are recorded (17).
 * n_copies at most 2^22.  One launch for each 65535 copies.  (Here and below K and V may be the same pages: they move once.) */
sage_status sage_paged_copy(const sage_paged_kv* cache, const int32_t* src, const int32_t* dst, const int32_t* n_tokens,
                            int64_t n_copies, void* status_block, void* stream);

/* Moves the kept tokens of each sequence together, in place: K and V of position keep[b * keep_stride + i] go to position
 * first[b] + i, for each i < n_keep[b], as if all were read before any is written.  The positions before first[b] stay; those
 * from first[b] + n_keep[b] on hold what is left (the caller sets kv_len, and may release their pages).
 *   first    device int32 [n_seqs].
 *   keep     device int32, n_keep[b] positions of sequence b, ascending, each from its new place on (keep[i] >= first + i)
 *            and below kv_len.  One that is not, or not above the one before it, is recorded (23) and its token not moved;
 *            what the new places of a list hold that does not ascend is not determined.  max_keep: the most a row may have;
 *            larger n_keep are cut (17), keep_stride >= max_keep.
 *   n_keep   device int32 [n_seqs].
 * Of the batch, kv_len (the tokens before the call) and page_table are read.  A token whose page, old or new, is out of range
 * is not moved (16).  Pages that are written belong to one sequence (a shared page would change for all).
 *   ws       256-byte aligned, >= SAGE_PAGED_WS_HEADER bytes, zeroed once (and again after a recorded timeout): a workspace of
 *            sage_paged_attn, or its header alone.  Calls that may overlap on the GPU need workspaces of their own.
 * One launch.  Lists longer than an item of 64 KB (256 tokens, or as many as one head's rows allow) are worked through in
 * pieces of 48 KB; more than 2^25 of them are refused (SAGE_ERR_UNSUPPORTED). */
sage_status sage_paged_compact(const sage_paged_kv* cache, const sage_paged_batch* batch, const int32_t* first,
                               const int32_t* keep, int64_t max_keep, int64_t keep_stride, const int32_t* n_keep, void* ws,
                               size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SAGE_GB300_PAGED_POOL_H */
