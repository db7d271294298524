/*
 * A paged key/value cache held in 4 bits, and attention over it, for AMD
 * Instinct MI355X (gfx950): what follows the indexer's selection.  The
 * indexer (indexer.h) scores keys and selects, per query row, the top k; the
 * attention here reads the selected keys' K and V rows (or those of a sliding
 * window with a few first tokens) from a cache in microscaled 4-bit floats.
 *
 * Conventions are those of indexer.h (device pointers owned by the caller,
 * work enqueued on `stream`, nothing allocated or kept, arguments checked on
 * the host before anything is enqueued, indexer_last_error()), with two
 * differences: values of device memory that name a place (slots, block ids,
 * selected indices) are checked by the kernels, and what they name outside
 * the cache is skipped; and strides of the cache are in BYTES.
 *
 * The cache
 * ---------
 * Each of K and V is two byte arrays over the same pages,
 *   data   [n_blocks][block_size][n_heads][head_dim / 2]
 *   scale  [n_blocks][block_size][n_heads][head_dim / 32]
 * with any block, slot and head strides (so [block][head][slot] orders too);
 * a row's bytes are contiguous.  A slot is block * block_size + offset.  Data
 * pointers and strides are multiples of 16 bytes, and every stride is at least
 * a row; block_size and slot strides are below 2^24, block strides and a
 * block's extent below 2^32 (else INDEXER_ENOTSUP).  The cache as a whole may
 * be of any size.
 * Each 32 consecutive values of a row share a scale byte s, a factor
 * 2^(s - 127) (255: the 32 values are NaN), and hold 4 bits each: a sign and
 * a magnitude out of 0, .5, 1, 1.5, 2, 3, 4, 6 in code order; the even
 * dimension is a byte's low half.  These are the blocks of the OCP
 * microscaling format MXFP4.
 *
 * Writing a block of 32 values x of a source type (f16 or bf16):
 *   e = the least exponent with max|x| < 7 * 2^e, kept in -23..13 (f16) or
 *       -126..125 (bf16);  s = e + 127
 *   each value is x / 2^e rounded to the nearest magnitude, ties to the even
 *       code, at most 6 (a value in 6..7 is off by at most 1, which is half
 *       of the last step, 4 to 6)
 *   a block with a NaN or an infinity: s = 255, codes 0.
 * The exponent ranges are those whose every 4-bit value the source type holds
 * exactly, so a cache written from a type reads back in it without rounding;
 * blocks whose largest magnitude is at least 57344 (f16) or 7 * 2^125 (bf16)
 * saturate at 6 * 2^13 or 6 * 2^125.
 */
#ifndef LIGHTNING_INDEXER_MX4_H
#define LIGHTNING_INDEXER_MX4_H

#include "indexer.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    INDEXER_MX4_F16 = 0,
    INDEXER_MX4_BF16 = 1
} indexer_mx4_type;

/*
 * These entry points take their arguments in a structure (every member set; no
 * padding between members), which the call reads and does not keep.
 */

/* Byte strides of the cache's block, slot and head, for data and for scale. */
typedef struct {
    int64_t data_block, data_slot, data_head;
    int64_t scale_block, scale_slot, scale_head;
} indexer_mx4_strides;

/*
 * indexer_mx4_cache_write -- quantise rows into the cache as they come.
 *
 *   k, v         [n_tokens][n_heads][head_dim] of `type`, strides in elements
 *                (multiples of 8), 16-byte aligned; v NULL: k alone (then the
 *                v members are not used)
 *   slots        i64 [n_tokens], 8-byte aligned: token t goes to slot
 *                slots[t]; one that is negative or past the cache is skipped
 *                (padding of a batch).  Slots that are not skipped are
 *                distinct: a slot named twice holds undefined values.
 *   k_data ...   the cache; K and V have the same strides.  Other slots keep
 *                their bytes.
 *
 * n_heads in [1, 1024]; head_dim a multiple of 32 in [32, 1024].
 */
typedef struct {
    const void *k;
    int64_t k_stride_t, k_stride_h;
    const void *v;
    int64_t v_stride_t, v_stride_h;
    const int64_t *slots;
    void *k_data, *k_scale, *v_data, *v_scale;
    indexer_mx4_strides strides;
    void *stream;
    int32_t type, n_tokens, n_heads, head_dim, n_blocks, block_size;
} indexer_mx4_write_args;

indexer_status indexer_mx4_cache_write(const indexer_mx4_write_args *args);

/*
 * indexer_mx4_cache_read -- rows of one of the two caches as numbers.
 *
 *   slots  i64 [n_rows]: row i is slot slots[i] (the same slot may come
 *          again); zeros where that is negative or past the cache
 *   out    [n_rows][n_heads][head_dim] of `type`, strides in elements
 *          (multiples of 8), 16-byte aligned; each value is rounded once to
 *          the type (exact for a cache written from it)
 *
 * Shapes as in indexer_mx4_cache_write.
 */
typedef struct {
    const void *data, *scale;
    indexer_mx4_strides strides;
    const int64_t *slots;
    void *out;
    int64_t out_stride_t, out_stride_h;
    void *stream;
    int32_t type, n_rows, n_heads, head_dim, n_blocks, block_size;
} indexer_mx4_read_args;

indexer_status indexer_mx4_cache_read(const indexer_mx4_read_args *args);

/*
 * indexer_mx4_attend_selected -- attention of each query row to the keys its
 * selection names (the idx of indexer_topk and the fused calls).
 *
 * Query j of request r is row t = r*query_len + j, as in
 * indexer_score_decode, and sees positions p < seq_lens[r] - query_len + 1 + j
 * (and p < max_seq_len).  Of these it attends to the positions
 * p = idx[t][e] * pool_size + u, 0 <= u < pool_size (pool_size > 1: each
 * selected entry stands for that many consecutive keys, the windows of
 * indexer_pool_keys); a negative idx, a position it does not see and a page
 * outside the cache are skipped, and an entry named twice counts twice.
 * Query head h reads K/V head h / (n_heads / n_kv_heads):
 *
 *   z[p]    = sm_scale * q[t][h] . K[p]
 *   lse     = ln(sum_p exp(z[p]))          (natural logarithm)
 *   out     = sum_p exp(z[p] - lse) V[p]
 *
 * A row with no position has out 0 and lse -inf.
 *
 * indexer_mx4_attend_window -- the same attention to a sliding window and the
 * first tokens: with v = seq_lens[r] - query_len + 1 + j, row r*query_len + j
 * attends to the positions p < min(v, max_seq_len) that have
 *   p >= v - window  or  p < sinks        (window >= 1), or
 *   any p                                  (window = 0: plain causal).
 *
 *   q            [n_requests*query_len][n_heads][head_dim] of `type` (strides
 *                in elements, multiples of 8; 16-byte aligned).  The cached
 *                values enter the products in this type: exact for a cache
 *                written from it.  Of values that the type does not hold (a
 *                cache written from another) K's are infinite, and V's count
 *                as the largest that the type's own writer stores, 6 * 2^13
 *                or 6 * 2^125 in magnitude; neither reaches a row or head
 *                that does not attend to the key.  Products accumulate in
 *                f32; the softmax is f32 and its weights are rounded to
 *                `type` for the product with V.
 *   block_table  i32 [n_requests][bt_stride], pages of each request; entries
 *                of the first ceil(max_seq_len / block_size) columns are read
 *                where a position needs them (and the first of each row)
 *   out          like q (strides multiples of 8, 16-byte aligned), not
 *                overlapping any input
 *   lse          f32 [n_requests*query_len][n_heads], contiguous, or NULL
 *   workspace    indexer_mx4_attend_workspace_bytes(...) bytes, 256-byte
 *                aligned; NULL when that is 0.  Calls that may overlap (other
 *                streams, graphs replayed side by side) need one each
 *   idx          selected: i32 [n_requests*query_len][idx_stride], the first
 *                n_sel of a row used
 *
 * The members from idx to pool_size belong to the selected form, window and
 * sinks to the other; each form ignores the other's.
 *
 * head_dim 64, 96, 128, 192 or 256; n_heads (at most 1024) a multiple of
 * n_kv_heads; sm_scale positive and finite; pool_size in [1, 8192];
 * max_seq_len, n_sel * pool_size and n_requests * query_len * n_heads at most
 * 2^31 - 1024; window, sinks >= 0.  A launch holds fewer than 2^32 threads:
 * with up to 32 query heads a K/V head, any call of less than 8 million
 * n_requests * query_len * n_kv_heads (head_dim up to 128; 16 million above)
 * fits; one that does not is INDEXER_EINVAL.
 * n_requests = 0 enqueues nothing; n_sel = 0 writes the empty rows' values.
 */
typedef struct {
    const void *q;
    int64_t q_stride_t, q_stride_h;
    const void *k_data, *k_scale, *v_data, *v_scale;
    indexer_mx4_strides strides;
    const int32_t *block_table;
    int64_t bt_stride;
    const int32_t *seq_lens;
    void *out;
    int64_t out_stride_t, out_stride_h;
    float *lse;
    void *workspace;
    size_t workspace_bytes;
    void *stream;
    const int32_t *idx;
    int64_t idx_stride;
    int32_t n_sel, pool_size;
    int32_t window, sinks;
    int32_t type, n_blocks, block_size, n_requests, query_len, max_seq_len, n_heads, n_kv_heads, head_dim;
    float sm_scale;
} indexer_mx4_attend_args;

indexer_status indexer_mx4_attend_selected(const indexer_mx4_attend_args *args);
indexer_status indexer_mx4_attend_window(const indexer_mx4_attend_args *args);

/*
 * Bytes of workspace an attention call needs (0 if none): the partial results
 * of rows whose keys are shared out over several workgroups.  max_keys is the
 * most keys a row can attend to: n_sel * pool_size for the selected form; for
 * the window form max_seq_len where window = 0, else
 * min(max_seq_len, window + sinks) (a sum past 2^31 - 1 counts as that).
 * Depends on sizes alone.  Returns (size_t)-1 for sizes no call accepts.
 */
size_t indexer_mx4_attend_workspace_bytes(
    int32_t n_requests, int32_t query_len, int32_t max_keys, int32_t selected,
    int32_t n_heads, int32_t n_kv_heads, int32_t head_dim);

#ifdef __cplusplus
}
#endif

#endif /* LIGHTNING_INDEXER_MX4_H */
