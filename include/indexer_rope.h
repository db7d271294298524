/*
 * Queries and keys made ready for the indexer and the attention, for AMD
 * Instinct MI355X (gfx950): each head's RMS norm and the rotation by the
 * token's position, in one pass over the rows.
 *
 * Conventions are those of indexer.h (device pointers owned by the caller,
 * work enqueued on `stream`, nothing allocated or kept, arguments checked on
 * the host before anything is enqueued, indexer_last_error()).
 */
#ifndef LIGHTNING_INDEXER_ROPE_H
#define LIGHTNING_INDEXER_ROPE_H

#include "indexer.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    INDEXER_ROPE_F16 = 0,
    INDEXER_ROPE_BF16 = 1
} indexer_rope_type;

/*
 * indexer_norm_rope -- norm and rotation of every head's row of q and k.
 *
 * For a row x of head_dim values at token t, with n = n_freq:
 *
 *   y[i]  = x[i] * w[i] / sqrt(mean(x^2) + eps)     (the tensor's weight w; NULL: y = x)
 *   pair i < n:  (y[a], y[b]), a = i, b = i + n  (interleaved: a = 2 i, b = 2 i + 1)
 *   angle = positions[axis of i][t] * inv_freq[i]
 *   out[a] = rotary_scale * (y[a] cos(angle) - y[b] sin(angle))
 *   out[b] = rotary_scale * (y[b] cos(angle) + y[a] sin(angle))
 *   out[i] = y[i]  for i >= 2 n
 *
 *   q, k         [n_tokens][heads][head_dim] of `type`, strides in elements
 *                (multiples of 8), 16-byte aligned; k NULL: q alone (then the
 *                k members are not used)
 *   q_out, k_out like q and k; either the input itself with its strides, or
 *                memory that overlaps no input
 *   q_weight, k_weight   [head_dim] f32 (weight type 0) or of `type` (1),
 *                contiguous; NULL: that tensor is not normed
 *   positions    i32 (positions_64 = 0) or i64 [n_axes][n_tokens], tokens
 *                contiguous, axes pos_stride elements apart; any sign
 *   inv_freq     f32 [n_freq]
 *   axes         the axis of frequency i: bits 2 i and 2 i + 1 of the 256
 *
 * Values are f32 from the load to the one rounding of the result.  Angles are
 * reduced in f64: below 2^31 radians they are exact to 2^-20, whatever the
 * position.
 *
 * head_dim a multiple of 8 in [8, 256]; n_freq a multiple of 4 in
 * [0, head_dim / 2]; n_axes in [1, 4]; heads in [1, 1024] each; eps >= 0;
 * rotary_scale finite.  A launch holds fewer than 2^32 threads, 256 for four
 * tokens: more than 2^26 - 4 tokens are INDEXER_EINVAL.  n_tokens = 0 enqueues
 * nothing.
 */
typedef struct {
    const void *q;
    int64_t q_stride_t, q_stride_h;
    const void *k;
    int64_t k_stride_t, k_stride_h;
    void *q_out;
    int64_t q_out_stride_t, q_out_stride_h;
    void *k_out;
    int64_t k_out_stride_t, k_out_stride_h;
    const void *q_weight, *k_weight;
    const void *positions;
    int64_t pos_stride;
    const float *inv_freq;
    uint64_t axes[4];
    void *stream;
    int32_t type, n_tokens, n_q_heads, n_k_heads, head_dim, n_freq, n_axes, interleaved;
    int32_t positions_64, q_weight_type, k_weight_type;
    float eps, rotary_scale;
} indexer_norm_rope_args;

indexer_status indexer_norm_rope(const indexer_norm_rope_args *args);

#ifdef __cplusplus
}
#endif

#endif /* LIGHTNING_INDEXER_ROPE_H */
