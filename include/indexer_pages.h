/*
 * Pages of the paged caches, kept on the GPU: copied, shared between requests
 * (forked), allotted to new tokens (grown), given back (freed) and moved
 * together (compacted), for AMD Instinct MI355X (gfx950).
 *
 * Conventions are those of indexer.h (device pointers owned by the caller,
 * work enqueued on `stream`, nothing allocated or kept, arguments checked on
 * the host before anything is enqueued, indexer_last_error()), with one
 * difference: values of device memory that name a place (pages, table rows)
 * are checked by the kernels, and what they name outside is skipped.
 *
 * The state of a pool of n_pages pages
 * ------------------------------------
 *   refs         i32 [n_pages]: how many table entries hold a page; a page
 *                with refs <= 0 is free.  Contiguous.
 *   block_table  i32 [n_rows][table_stride], n_cols of a row used: the pages
 *                of a request in the order of its tokens, -1 where it holds
 *                none.  As the indexer's decode calls and the attention take it.
 *   seq_lens     i32 [n_rows]: tokens of a request; it holds the pages
 *                ceil(seq_len / block_size) first entries of its row name.
 * Pages are given out lowest first, in the order of a call's list, so the same
 * calls give the same pages whatever ran beside them on other streams.  Calls
 * that change one state must follow each other (one stream, or events).
 *
 * A list of table rows may name a row that is not there (negative, or past
 * n_rows; padding of a batch), which is skipped, and name one twice: the
 * second and later ones are skipped.  Tables and lists have at most 8192 rows;
 * those of a call times its columns (rounded up to 256) fill a launch of fewer
 * than 2^32 threads, else it is INDEXER_EINVAL.
 */
#ifndef LIGHTNING_INDEXER_PAGES_H
#define LIGHTNING_INDEXER_PAGES_H

#include "indexer.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * One cache's pages: page p is the `bytes` bytes at base + p * stride.  A list
 * of them (host memory, read during the call) names every cache of a model: K
 * and V and their scales, the indexer's keys, of each layer.  bytes >= 1;
 * stride >= bytes where there is more than one page.  Copies are quickest
 * where base, stride and bytes are multiples of 16.
 */
typedef struct {
    void *base;
    int64_t stride, bytes;
} indexer_page_array;

/*
 * indexer_pages_copy -- page from[i] of every cache to page to[i], i < n.
 *
 *   from, to  i32 [n]; a pair with either outside the pool is skipped.  No
 *             page is named twice in `to`, or in both lists (but a pair of
 *             one page, which is skipped).
 */
typedef struct {
    const indexer_page_array *arrays;
    const int32_t *from, *to;
    void *stream;
    int32_t n_arrays, n, n_pages;
} indexer_pages_copy_args;

indexer_status indexer_pages_copy(const indexer_pages_copy_args *args);

/*
 * indexer_pages_fork -- request children[i] begins as request parents[i] is.
 *
 * With len = seq_lens[parent]: the child's row gets the parent's first
 * len / block_size entries, whose pages both hold from now on (refs + 1), and
 * where len is not a multiple of block_size a free page, with a copy of the
 * parent's last, partly filled page in every cache; the rest of its row is
 * -1, its seq_len len (at most n_cols * block_size).  Where no page is free
 * the child is left empty (row -1, seq_len 0).  Where the parent's last page is
 * not of the pool, the child has none there either: the page of its turn stays
 * free, and its last tokens are as little there as the parent's.  What a
 * child's row held is overwritten: free it first.  No row is both a child and a
 * parent.
 *
 *   fresh  i32 [n], out: the page a child got for its last tokens; -1 it got
 *          none (it needed none, or its parent's is not of the pool); -2 no
 *          page was free; -3 the pair was skipped
 *
 * arrays may be NULL (n_arrays 0): no page is copied.
 */
typedef struct {
    const indexer_page_array *arrays;
    int32_t *refs, *block_table;
    int64_t table_stride;
    int32_t *seq_lens;
    const int32_t *parents, *children;
    int32_t *fresh;
    void *stream;
    int32_t n_arrays, n, n_pages, n_rows, n_cols, block_size;
} indexer_pages_fork_args;

indexer_status indexer_pages_fork(const indexer_pages_fork_args *args);

/*
 * indexer_pages_grow -- room for new tokens of requests.
 *
 * Request rows[i] gets `tokens` more tokens (or new_tokens[i] of them, taken
 * as 0..tokens): its row the free pages that ceil((len + new) / block_size)
 * asks for, its seq_len len + new.  It must be the only holder of a partly
 * filled last page, as indexer_pages_fork leaves it.  A request whose row has
 * no column left is left as it is; so is one whose partly filled last page is
 * not of the pool, and one that needs pages where the pages needed by the list
 * up to it are more than were free.
 *
 *   slots  i64 [n][tokens], out: where the new tokens go in the caches, page *
 *          block_size + offset, as indexer_mx4_cache_write takes them; -1 for
 *          tokens past new_tokens[i], and all of a row that was left or skipped
 */
typedef struct {
    int32_t *refs, *block_table;
    int64_t table_stride;
    int32_t *seq_lens;
    const int32_t *rows, *new_tokens;
    int64_t *slots;
    void *stream;
    int32_t n, tokens, n_pages, n_rows, n_cols, block_size;
} indexer_pages_grow_args;

indexer_status indexer_pages_grow(const indexer_pages_grow_args *args);

/*
 * indexer_pages_free -- requests end: every page their rows name has one
 * holder less, the rows become -1 and the seq_lens 0.
 */
typedef struct {
    int32_t *refs, *block_table;
    int64_t table_stride;
    int32_t *seq_lens;
    const int32_t *rows;
    void *stream;
    int32_t n, n_pages, n_rows, n_cols;
} indexer_pages_free_args;

indexer_status indexer_pages_free(const indexer_pages_free_args *args);

/*
 * indexer_pages_compact -- the pages in use moved to the front.
 *
 * With L pages in use, the free pages below L are taken, in order, by the
 * pages in use from L on, in order: their bytes in every cache, their refs
 * (then 0 where they were), and the entries of block_table that name them.
 * Entries that name a free page become -1.  Other pages keep their bytes.
 *
 *   place  i32 [n_pages], out: where a page went (itself where it stayed); -1
 *          it was free.  For other tables of the same pool
 *   live   i32 [1], out: L
 */
typedef struct {
    const indexer_page_array *arrays;
    int32_t *refs, *block_table;
    int64_t table_stride;
    int32_t *place, *live;
    void *workspace;
    size_t workspace_bytes;
    void *stream;
    int32_t n_arrays, n_pages, n_rows, n_cols;
} indexer_pages_compact_args;

indexer_status indexer_pages_compact(const indexer_pages_compact_args *args);

/* Bytes of workspace a compaction needs (4-byte aligned). */
size_t indexer_pages_compact_workspace_bytes(int32_t n_pages);

#ifdef __cplusplus
}
#endif

#endif /* LIGHTNING_INDEXER_PAGES_H */
