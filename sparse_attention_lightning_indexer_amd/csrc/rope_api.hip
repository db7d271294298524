// C-ABI of the head norm and rotation (declared in include/indexer_rope.h).
// As in indexer_api.hip: every argument is checked on the host, without
// touching device memory or calling HIP, before anything is enqueued.
#include <math.h>

#include "../../include/indexer_rope.h"
#include "internal.h"
#include "rope_internal.h"

namespace {

using lidx::api_error;

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

static_assert(sizeof(indexer_norm_rope_args) == 22 * 8 + 14 * 4, "the binding packs the members");

#define ROPE_FAIL(st, ...) return (indexer_status)api_error(st, __VA_ARGS__)

indexer_status check_rows(const char *name, const void *p, int64_t st, int64_t sh, int32_t heads, int32_t head_dim) {
    if (!p) ROPE_FAIL(INDEXER_EINVAL, "%s is NULL", name);
    if (!aligned(p, 16)) ROPE_FAIL(INDEXER_EINVAL, "%s must be 16-byte aligned", name);
    if (sh % 8 || (heads > 1 && sh < head_dim))
        ROPE_FAIL(INDEXER_EINVAL, "%s's head stride %lld must be >= head_dim and a multiple of 8", name, (long long)sh);
    if (st % 8 || st < head_dim)
        ROPE_FAIL(INDEXER_EINVAL, "%s's row stride %lld must be >= head_dim and a multiple of 8", name, (long long)st);
    return INDEXER_OK;
}

indexer_status check_weight(const char *name, const void *p, int32_t type) {
    if (type != 0 && type != 1) ROPE_FAIL(INDEXER_EINVAL, "%s's type %d is neither 0 (f32) nor 1 (the rows')", name, type);
    if (!aligned(p, type ? 2 : 4)) ROPE_FAIL(INDEXER_EINVAL, "%s must be aligned to its values", name);
    return INDEXER_OK;
}

}  // namespace

extern "C" {

indexer_status indexer_norm_rope(const indexer_norm_rope_args *args) {
    if (!args) ROPE_FAIL(INDEXER_EINVAL, "args is NULL");
    const indexer_norm_rope_args &g = *args;
    if (g.type != INDEXER_ROPE_F16 && g.type != INDEXER_ROPE_BF16)
        ROPE_FAIL(INDEXER_EINVAL, "type=%d is neither INDEXER_ROPE_F16 nor INDEXER_ROPE_BF16", g.type);
    if (g.n_tokens < 0) ROPE_FAIL(INDEXER_EINVAL, "n_tokens=%d must be >= 0", g.n_tokens);
    const bool has_k = g.k != nullptr;
    if (g.n_q_heads < 1 || g.n_q_heads > lidx::kMaxHeads || (has_k && (g.n_k_heads < 1 || g.n_k_heads > lidx::kMaxHeads)))
        ROPE_FAIL(INDEXER_ENOTSUP, "n_q_heads=%d n_k_heads=%d not supported (1..%d)", g.n_q_heads, g.n_k_heads,
                  lidx::kMaxHeads);
    if (g.head_dim < 8 || g.head_dim > 256 || g.head_dim % 8)
        ROPE_FAIL(INDEXER_ENOTSUP, "head_dim=%d not supported (a multiple of 8 in 8..256)", g.head_dim);
    if (g.n_freq < 0 || g.n_freq > g.head_dim / 2 || g.n_freq % 4)
        ROPE_FAIL(INDEXER_ENOTSUP, "n_freq=%d not supported (a multiple of 4 in 0..head_dim/2)", g.n_freq);
    if (g.n_axes < 1 || g.n_axes > 4) ROPE_FAIL(INDEXER_ENOTSUP, "n_axes=%d not supported (1..4)", g.n_axes);
    if (!(g.eps >= 0.0f) || !isfinite(g.eps)) ROPE_FAIL(INDEXER_EINVAL, "eps=%g must be finite and >= 0", (double)g.eps);
    if (!isfinite(g.rotary_scale)) ROPE_FAIL(INDEXER_EINVAL, "rotary_scale=%g must be finite", (double)g.rotary_scale);
    indexer_status st = check_rows("q", g.q, g.q_stride_t, g.q_stride_h, g.n_q_heads, g.head_dim);
    if (st == INDEXER_OK)
        st = check_rows("q_out", g.q_out, g.q_out_stride_t, g.q_out_stride_h, g.n_q_heads, g.head_dim);
    if (st == INDEXER_OK) st = check_weight("q_weight", g.q_weight, g.q_weight_type);
    if (st == INDEXER_OK && has_k) {
        st = check_rows("k", g.k, g.k_stride_t, g.k_stride_h, g.n_k_heads, g.head_dim);
        if (st == INDEXER_OK)
            st = check_rows("k_out", g.k_out, g.k_out_stride_t, g.k_out_stride_h, g.n_k_heads, g.head_dim);
        if (st == INDEXER_OK) st = check_weight("k_weight", g.k_weight, g.k_weight_type);
    }
    if (st != INDEXER_OK) return st;
    if (g.n_freq > 0) {
        if (!g.positions) ROPE_FAIL(INDEXER_EINVAL, "positions is NULL");
        if (g.positions_64 != 0 && g.positions_64 != 1) ROPE_FAIL(INDEXER_EINVAL, "positions_64=%d is neither 0 nor 1", g.positions_64);
        if (!aligned(g.positions, g.positions_64 ? 8 : 4)) ROPE_FAIL(INDEXER_EINVAL, "positions must be aligned to its values");
        if (g.n_axes > 1 && g.pos_stride < g.n_tokens)
            ROPE_FAIL(INDEXER_EINVAL, "pos_stride=%lld < n_tokens=%d", (long long)g.pos_stride, g.n_tokens);
        if (!g.inv_freq || !aligned(g.inv_freq, 4)) ROPE_FAIL(INDEXER_EINVAL, "inv_freq is NULL or not 4-byte aligned");
        for (int i = 0; i < g.n_freq; ++i) {
            const int axis = (int)(g.axes[i >> 5] >> (2 * (i & 31))) & 3;
            if (axis >= g.n_axes) ROPE_FAIL(INDEXER_EINVAL, "axis %d of frequency %d is not one of n_axes=%d", axis, i, g.n_axes);
        }
    }
    if (g.n_tokens == 0) return (indexer_status)lidx::api_launch(hipSuccess, "");
    const lidx::RopePlan p = lidx::plan_rope(g.n_tokens, g.n_q_heads + (has_k ? g.n_k_heads : 0), g.head_dim, g.n_freq);
    if (!p.fits) ROPE_FAIL(INDEXER_EINVAL, "problem too large for one launch: %lld workgroups of %d threads",
                           (long long)p.workgroups, lidx::kRopeThreads);
    lidx::Rope a{};
    a.x[0] = g.q, a.st[0] = g.q_stride_t, a.sh[0] = g.q_stride_h;
    a.y[0] = g.q_out, a.yst[0] = g.q_out_stride_t, a.ysh[0] = g.q_out_stride_h;
    a.weight[0] = g.q_weight, a.weight_f32[0] = g.q_weight_type == 0, a.heads[0] = g.n_q_heads;
    if (has_k) {
        a.x[1] = g.k, a.st[1] = g.k_stride_t, a.sh[1] = g.k_stride_h;
        a.y[1] = g.k_out, a.yst[1] = g.k_out_stride_t, a.ysh[1] = g.k_out_stride_h;
        a.weight[1] = g.k_weight, a.weight_f32[1] = g.k_weight_type == 0, a.heads[1] = g.n_k_heads;
    }
    a.positions = g.positions;
    a.pos_stride = g.n_axes > 1 ? g.pos_stride : 0;
    a.pos64 = g.positions_64 != 0;
    a.inv_freq = g.inv_freq;
    for (int i = 0; i < 4; ++i) a.axes[i] = g.axes[i];
    a.n_tokens = g.n_tokens;
    a.head_dim = g.head_dim;
    a.n_freq = g.n_freq;
    a.eps = g.eps;
    a.inv_dim = 1.0f / (float)g.head_dim;
    a.rotary_scale = g.rotary_scale;
    a.bf16 = g.type == INDEXER_ROPE_BF16;
    a.neighbours = g.interleaved != 0;
    a.steps = p.steps;
    return (indexer_status)lidx::api_launch(lidx::launch_rope(a, p, (hipStream_t)g.stream), "norm and rotation launch");
}

// Whether a call of these sizes fits a launch, for the tests.  Not part of the interface.
int32_t lidx_rope_fits(int32_t n_tokens, int32_t heads, int32_t head_dim, int32_t n_freq) {
    return lidx::plan_rope(n_tokens, heads, head_dim, n_freq).fits;
}

}  // extern "C"
