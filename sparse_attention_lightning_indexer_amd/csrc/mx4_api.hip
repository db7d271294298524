// C-ABI of the 4-bit cache operators (declared in include/indexer_mx4.h).
// As in indexer_api.hip: every argument is checked on the host, without
// touching device memory or calling HIP, before anything is enqueued.
#include <math.h>

#include "../../include/indexer_mx4.h"
#include "internal.h"
#include "mx4_internal.h"

namespace {

using lidx::api_error;

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

static_assert(sizeof(indexer_mx4_write_args) == 18 * 8 + 6 * 4 && sizeof(indexer_mx4_read_args) == 13 * 8 + 6 * 4 &&
                  sizeof(indexer_mx4_attend_args) == 25 * 8 + 14 * 4,
              "members without padding: the binding packs them");

constexpr int32_t kMaxKeys = INT32_MAX - 1023;  // room for positions of a last, partly filled tile

#define MX4_FAIL(st, ...) return (indexer_status)api_error(st, __VA_ARGS__)
#define MX4_TRY(expr)                                \
    do {                                             \
        const indexer_status st_ = (expr);           \
        if (st_ != INDEXER_OK) return st_;           \
    } while (0)

indexer_status done(hipError_t e, const char *what) { return (indexer_status)lidx::api_launch(e, what); }

indexer_status check_type(int32_t type) {
    if (type != INDEXER_MX4_F16 && type != INDEXER_MX4_BF16)
        MX4_FAIL(INDEXER_EINVAL, "type=%d is neither INDEXER_MX4_F16 nor INDEXER_MX4_BF16", type);
    return INDEXER_OK;
}

indexer_status check_rows(const char *name, const void *p, int64_t st, int64_t sh, int32_t n_heads, int32_t head_dim) {
    if (!p) MX4_FAIL(INDEXER_EINVAL, "%s is NULL", name);
    if (!aligned(p, 16)) MX4_FAIL(INDEXER_EINVAL, "%s must be 16-byte aligned", name);
    if (sh % 8 || (n_heads > 1 && sh < head_dim))
        MX4_FAIL(INDEXER_EINVAL, "%s's head stride %lld must be >= head_dim and a multiple of 8", name, (long long)sh);
    if (st % 8 || st < head_dim)
        MX4_FAIL(INDEXER_EINVAL, "%s's row stride %lld must be >= head_dim and a multiple of 8", name, (long long)st);
    return INDEXER_OK;
}

// Strides of the pages: no two rows may share bytes along one dimension.
indexer_status check_pages(int32_t n_blocks, int32_t block_size, int32_t n_heads, int32_t head_dim,
                           const indexer_mx4_strides &st, lidx::Mx4Pages *out) {
    int64_t d_sb = st.data_block, d_ss = st.data_slot, d_sh = st.data_head;
    int64_t s_sb = st.scale_block, s_ss = st.scale_slot, s_sh = st.scale_head;
    if (n_blocks < 0) MX4_FAIL(INDEXER_EINVAL, "n_blocks=%d must be >= 0", n_blocks);
    if (block_size < 1) MX4_FAIL(INDEXER_EINVAL, "block_size=%d must be >= 1", block_size);
    const int64_t row = head_dim / 2, srow = head_dim / 32;
    if (d_sb % 16 || d_ss % 16 || d_sh % 16)
        MX4_FAIL(INDEXER_EINVAL, "data strides %lld, %lld, %lld must be multiples of 16 bytes", (long long)d_sb,
                 (long long)d_ss, (long long)d_sh);
    if ((n_blocks > 1 && d_sb < row) || (block_size > 1 && d_ss < row) || (n_heads > 1 && d_sh < row))
        MX4_FAIL(INDEXER_EINVAL, "data strides %lld, %lld, %lld must be >= head_dim/2 = %lld", (long long)d_sb,
                 (long long)d_ss, (long long)d_sh, (long long)row);
    if ((n_blocks > 1 && s_sb < srow) || (block_size > 1 && s_ss < srow) || (n_heads > 1 && s_sh < srow))
        MX4_FAIL(INDEXER_EINVAL, "scale strides %lld, %lld, %lld must be >= head_dim/32 = %lld", (long long)s_sb,
                 (long long)s_ss, (long long)s_sh, (long long)srow);
    if (n_blocks <= 1) d_sb = s_sb = 0;
    if (block_size == 1) d_ss = s_ss = 0;
    if (n_heads == 1) d_sh = s_sh = 0;
    // the kernels' address arithmetic: 32-bit block and head strides, 24-bit slot strides and sizes, 32 bits inside
    // a block; the extents are computed (in 64 bits) once the strides are known to be small
    bool ok = block_size < 1 << 24 && d_ss < 1 << 24 && s_ss < 1 << 24 && d_sb <= UINT32_MAX && s_sb <= UINT32_MAX &&
              d_sh <= UINT32_MAX && s_sh <= UINT32_MAX;
    ok = ok && (block_size - 1) * d_ss + (n_heads - 1) * d_sh + row <= UINT32_MAX;
    ok = ok && (block_size - 1) * s_ss + (n_heads - 1) * s_sh + srow <= UINT32_MAX;
    if (!ok)
        MX4_FAIL(INDEXER_ENOTSUP, "pages not supported (block_size and slot strides below 2^24, a block's bytes and "
                 "block strides below 2^32)");
    *out = lidx::Mx4Pages{d_sb, d_ss, d_sh, s_sb, s_ss, s_sh, n_blocks, block_size,
                          lidx::fast_div((uint32_t)block_size), (int64_t)n_blocks * block_size, d_sb == 16 * s_sb && d_ss == 16 * s_ss};
    return INDEXER_OK;
}

// `of`: what the members' names begin with
indexer_status check_cache(const char *of, const void *data, const void *scale) {
    if (!data) MX4_FAIL(INDEXER_EINVAL, "%sdata is NULL", of);
    if (!scale) MX4_FAIL(INDEXER_EINVAL, "%sscale is NULL", of);
    if (!aligned(data, 16)) MX4_FAIL(INDEXER_EINVAL, "%sdata must be 16-byte aligned", of);
    return INDEXER_OK;
}

indexer_status check_row_shape(int32_t n_heads, int32_t head_dim) {
    if (n_heads < 1 || n_heads > lidx::kMaxHeads || head_dim < 32 || head_dim > 1024 || head_dim % 32)
        MX4_FAIL(INDEXER_ENOTSUP, "n_heads=%d head_dim=%d not supported (n_heads in 1..%d, head_dim a multiple of 32 "
                 "in 32..1024)", n_heads, head_dim, lidx::kMaxHeads);
    return INDEXER_OK;
}

bool attend_dim(int32_t d) { return d == 64 || d == 96 || d == 128 || d == 192 || d == 256; }

// Everything the two attentions share; fills all of `a` but the selection or
// window, and the launch fields.
indexer_status check_attend(const indexer_mx4_attend_args &g, lidx::Mx4Attend *a) {
    MX4_TRY(check_type(g.type));
    if (g.n_requests < 0 || g.max_seq_len < 0)
        MX4_FAIL(INDEXER_EINVAL, "n_requests=%d max_seq_len=%d must be >= 0", g.n_requests, g.max_seq_len);
    if (g.query_len < 1) MX4_FAIL(INDEXER_EINVAL, "query_len=%d must be >= 1", g.query_len);
    if (g.max_seq_len > kMaxKeys) MX4_FAIL(INDEXER_ENOTSUP, "max_seq_len=%d exceeds %d", g.max_seq_len, kMaxKeys);
    if (g.n_heads < 1 || g.n_heads > lidx::kMaxHeads || g.n_kv_heads < 1 || g.n_heads % g.n_kv_heads ||
        !attend_dim(g.head_dim))
        MX4_FAIL(INDEXER_ENOTSUP, "n_heads=%d n_kv_heads=%d head_dim=%d not supported (n_heads in 1..%d, a multiple of "
                 "n_kv_heads; head_dim 64, 96, 128, 192 or 256)", g.n_heads, g.n_kv_heads, g.head_dim, lidx::kMaxHeads);
    if ((int64_t)g.n_requests * g.query_len > kMaxKeys / g.n_heads)
        MX4_FAIL(INDEXER_EINVAL, "n_requests*query_len*n_heads exceeds the int32 range (%d)", kMaxKeys);
    if (!(g.sm_scale > 0.0f) || !isfinite(g.sm_scale) || !isfinite(g.sm_scale * 1.44269504f))
        MX4_FAIL(INDEXER_EINVAL, "sm_scale=%g must be positive and finite", (double)g.sm_scale);
    lidx::Mx4Pages pages;
    MX4_TRY(check_pages(g.n_blocks, g.block_size, g.n_kv_heads, g.head_dim, g.strides, &pages));
    MX4_TRY(check_rows("q", g.q, g.q_stride_t, g.q_stride_h, g.n_heads, g.head_dim));
    MX4_TRY(check_rows("out", g.out, g.out_stride_t, g.out_stride_h, g.n_heads, g.head_dim));
    if (g.n_blocks > 0) {
        MX4_TRY(check_cache("k_", g.k_data, g.k_scale));
        MX4_TRY(check_cache("v_", g.v_data, g.v_scale));
    }
    if (!g.seq_lens) MX4_FAIL(INDEXER_EINVAL, "seq_lens is NULL");
    if (!aligned(g.seq_lens, 4) || !aligned(g.block_table, 4))
        MX4_FAIL(INDEXER_EINVAL, "block_table and seq_lens must be 4-byte aligned");
    if (g.lse && !aligned(g.lse, 4)) MX4_FAIL(INDEXER_EINVAL, "lse must be 4-byte aligned");
    if (g.max_seq_len > 0) {
        if (!g.block_table) MX4_FAIL(INDEXER_EINVAL, "block_table is NULL");
        const int64_t need = ((int64_t)g.max_seq_len + g.block_size - 1) / g.block_size;
        if (g.bt_stride < need)
            MX4_FAIL(INDEXER_EINVAL, "bt_stride=%lld < ceil(max_seq_len/block_size)=%lld", (long long)g.bt_stride,
                     (long long)need);
    }
    *a = lidx::Mx4Attend{};
    a->q = g.q;
    a->q_st = g.q_stride_t;
    a->q_sh = g.q_stride_h;
    a->kd = (const uint8_t *)g.k_data;
    a->ks = (const uint8_t *)g.k_scale;
    a->vd = (const uint8_t *)g.v_data;
    a->vs = (const uint8_t *)g.v_scale;
    a->pages = pages;
    a->block_table = g.block_table;
    a->bt_stride = g.bt_stride;
    a->seq_lens = g.seq_lens;
    a->n_requests = g.n_requests;
    a->q_len = g.query_len;
    a->max_seq_len = g.max_seq_len;
    a->n_heads = g.n_heads;
    a->n_kv = g.n_kv_heads;
    a->group = g.n_heads / g.n_kv_heads;
    a->scale_log2 = (float)((double)g.sm_scale * 1.4426950408889634);
    a->out = g.out;
    a->out_st = g.out_stride_t;
    a->out_sh = g.out_stride_h;
    a->lse = g.lse;
    a->rows = g.n_requests * g.query_len;
    a->div_group = lidx::fast_div((uint32_t)a->group);
    a->div_pool = lidx::fast_div(1);
    return INDEXER_OK;
}

indexer_status run_attend(lidx::Mx4Attend &a, const indexer_mx4_attend_args &g, int64_t max_keys) {
    const int head_dim = g.head_dim;
    void *workspace = g.workspace;
    hipStream_t stream = (hipStream_t)g.stream;
    const bool selected = a.idx != nullptr;
    lidx::Mx4Plan p =
        lidx::plan_mx4_attend(a.n_requests, a.q_len, max_keys, selected, a.n_heads, a.n_kv, head_dim);
    // shared scales are loaded in whole 16-byte parts, those of 8 heads one after
    // the other; the order of the sums is the same either way
    const lidx::Mx4Pages &pages = a.pages;
    p.share = p.share && pages.s_sh == head_dim / 32 && pages.s_ss % 16 == 0 && pages.s_sb % 16 == 0 &&
              aligned(a.ks, 16) && aligned(a.vs, 16);
    if (!p.fits)
        MX4_FAIL(INDEXER_EINVAL, "problem too large for one launch: %lld workgroups of %d threads",
                 (long long)p.workgroups, p.threads);
    if (p.workspace_bytes && (!workspace || g.workspace_bytes < p.workspace_bytes || !aligned(workspace, 256)))
        MX4_FAIL(INDEXER_EWORKSPACE, "attention needs %zu bytes of 256-byte aligned workspace, got %zu",
                 p.workspace_bytes, workspace ? g.workspace_bytes : (size_t)0);
    if (a.rows == 0) return done(hipSuccess, "");
    a.units = p.units;
    a.m_tiles = p.m_tiles;
    a.n_splits = p.n_splits;
    a.head_group = p.head_group;
    a.div_kv = lidx::fast_div((uint32_t)(a.n_kv / (p.hp * p.head_group)));
    a.div_items = lidx::fast_div((uint32_t)(p.m_tiles * p.n_splits));
    a.part_o = (float *)workspace;
    a.part_ml = (float *)((char *)workspace + p.part_o_bytes);
    return done(g.type == INDEXER_MX4_BF16 ? lidx::launch_mx4_attend_bf16(a, p, head_dim, stream)
                                         : lidx::launch_mx4_attend_f16(a, p, head_dim, stream),
                "attention kernel launch");
}

int64_t window_keys(int32_t max_seq_len, int32_t window, int32_t sinks) {
    const int64_t w = (int64_t)window + sinks;
    return window == 0 || w > max_seq_len ? max_seq_len : w;
}

}  // namespace

namespace lidx {

static bool one_launch(int64_t workgroups, int threads) { return workgroups <= (int64_t)UINT32_MAX / threads; }

// The launch size and workspace of a plan.
static Mx4Plan sized(Mx4Plan p, int64_t rows, int n_heads, int n_kv, int head_dim) {
    const int64_t pieces = (int64_t)p.units * p.m_tiles * p.n_splits;
    p.workgroups = (pieces + 7) / 8 * 8 * (n_kv / (p.hp * p.head_group));
    if (p.n_splits > 1) {
        const size_t parts = (size_t)rows * n_heads * p.n_splits;
        p.part_o_bytes = (parts * head_dim * 4 + 255) / 256 * 256;
        p.workspace_bytes = p.part_o_bytes + (parts * 8 + 255) / 256 * 256;
    }
    p.threads = p.prompt ? kMx4PromptThreads : mx4_wave_threads(head_dim, p.hp);
    p.fits = one_launch(p.workgroups, p.threads) && (p.n_splits == 1 || one_launch(rows * n_heads, kMx4JoinThreads));
    return p;
}

// A wave holds one tile of 16 query rows, or two where a unit has more rows, or
// one tile of two K/V heads where a head has at most 8 rows and the rows fill
// the chip (1024 rows x 2048 selected keys, 8 heads: 457 us a head at a time,
// 428 us in pairs; 128 rows 76 and 68 us; 32 rows x 512 keys 9.2 and 16.3 us).
//
// Where there are fewer workgroups than compute units, several share a row's
// keys, about one workgroup per compute unit: one row of 131072 keys on 8 K/V
// heads takes 123, 67, 41 and 43 us with 8, 16, 32 and 64 shares (32 is one a
// compute unit).  Joining the shares is a second launch, about 5 us, the time
// of about 4 tiles of a wave; 32 rows of 512 keys on 8 heads, two tiles a
// wave, take 9.3 us whole and 15.8 us in halves.  So keys are shared only
// where that takes at least 4 tiles from every wave.
//
// With one workgroup a compute unit there are registers for the codes of two
// tiles on the way instead of one: one row of 131072 keys 38.1 and 34.9 us, but
// 32 rows of 512 keys, two tiles a wave, 9.3 and 10.7 us (its first loads wait
// for those that no tile needs); so from 8 tiles a wave on.
//
// Many rows of a request under a window go through the keys 256 at a time and
// together (mx4_prompt_kernel) where that is the shorter of two estimates, fit
// to head dimension 128 and 8 K/V heads of 8 query heads (other dimensions are
// taken in proportion; which form is shorter was not measured there): 2.05 us for 64 keys
// and 256 rows a compute unit (1.8 us half full), rounds of one workgroup a
// compute unit and 10 us, the keys shared out where that fills the last round
// better, at the price of a second launch and of the shares' traffic; against
// 0.79 us a SIMD for 32 keys and 32 rows of a wave, and 7 us a round.  Measured,
// together and apart, 8 query heads a K/V head: 1024 tokens over 16384 keys 510
// and 783 us, 512 tokens 304 and 401, 1000 under a window of 4096 156 and 223,
// 1100 under one of 512 77 and 108, 128 under one of 1024 37 and 18, 256 over
// 2048 52 and 39, 16 tokens of 32 requests over 4096 115 and 128, 4 tokens of
// them 106 and 41.
//
// Where a row's pairs of heads make a multiple of four and the rows fill the
// chip, the four waves of a workgroup take the same keys of four pairs, instead
// of different keys of one: nothing has to be joined, and (where the cache's
// layout allows, see run_attend) the waves share the keys' scales.  Measured,
// same and different keys, head dimension 128: 1024 rows x 2048 keys, 8 heads
// 390 and 450 us, 512 rows 206 and 218, 448 rows 200 and 198, 256 rows 143 and
// 123; 640, 512 and 384 rows x 512 keys 80 and 86, 63 and 71, 57 and 56; 256
// rows x 64 keys 11.7 and 17.3, 192 rows 11.2 and 11.6.  Head dimension 64, 2048
// keys: 512 rows of 8 heads 135 and 127, 384 rows of 16 heads 179 and 195, 320
// rows of them 166 and 163; 256 rows of 8 heads x 64 keys 8.6 and 11.5.  Head
// dimension 96, which does not share: 1024 rows x 2048 keys 363 and 457.  So from
// two workgroups a compute unit on (three below head dimension 128), or one
// where a wave has at most four tiles.  Workgroups that would share the scales
// but cannot take 443 us where those that do take 390.  Under a window, whose
// keys lie side by side, only few keys are worth it: 512 rows over 64, 128, 512
// and 2048 keys 17, 24, 66 and 248 us with the same keys, 26, 30, 68 and 233 us
// with different ones.
//
// Otherwise the 8 waves of a workgroup take the same keys of
// several K/V heads where the workgroups that leaves still fill whole rounds of
// the compute units (one at a time fits one): 1000 rows over a window of 4096
// 264 us with one head, 239, 221 and 219 us with 2, 4 and 8; 1024 causal rows
// over 16384 keys 820, 787, 776 and 778 us.
Mx4Plan plan_mx4_attend(int n_requests, int q_len, int64_t max_keys, bool selected, int n_heads, int n_kv,
                        int head_dim) {
    constexpr int kCus = 256;
    Mx4Plan p{};
    const int group = n_heads / n_kv;
    const int64_t rows = (int64_t)n_requests * q_len;
    const int64_t n_m = selected ? group : (int64_t)q_len * group;
    p.units = selected ? (int)rows : n_requests;
    p.mt = n_m > 16 ? 2 : 1;
    p.m_tiles = (int)((n_m + 16 * p.mt - 1) / (16 * p.mt));
    p.hp = n_m <= 8 && n_kv % 2 == 0 && head_dim <= 128 && (int64_t)p.units * (n_kv / 2) >= 2 * kCus ? 2 : 1;
    p.head_group = 1;
    if (!selected && head_dim <= 128 && n_m > 32) {
        const int64_t tiles = (n_m + 255) / 256, items = (int64_t)p.units * tiles * n_kv;
        const double steps = (double)max_keys / 64, fill = (double)n_m / (double)(tiles * 256);
        const double a_step = 2.05 * (0.76 + 0.24 * fill) * head_dim / 128;
        const int64_t apart = (int64_t)p.units * ((n_m + 31) / 32) * n_kv;  // workgroups of 32 rows
        double best = 0.79 / (4 * kCus) * (double)apart * ((double)max_keys / 32) * head_dim / 128 +
                      7.0 * (double)((apart + kCus - 1) / kCus);
        if (!one_launch(apart, mx4_wave_threads(head_dim, 1))) best = HUGE_VAL;
        for (int s = 1; s <= 16; ++s) {
            if (!one_launch((items + 7 * n_kv) * s, kMx4PromptThreads) ||
                (s > 1 && !one_launch(rows * n_heads, kMx4JoinThreads)))
                break;
            const double rounds = (double)((items * s + kCus - 1) / kCus);
            double t = 10.0 + rounds * ceil(steps / s) * a_step;
            if (s > 1) t += 5.0 + (double)rows * n_heads * s * head_dim * 8 / 4.5e6;
            if (t >= best) continue;
            best = t;
            p.prompt = true;
            p.n_splits = s;
            p.m_tiles = (int)tiles;
        }
        if (p.prompt) return sized(p, rows, n_heads, n_kv, head_dim);
    }
    const int64_t wgs = (int64_t)p.units * (n_kv / 8);
    if (p.hp == 2 && n_kv % 8 == 0 &&
        (max_keys <= 128 ? wgs >= kCus : selected && wgs >= (head_dim == 128 ? 2 : 3) * kCus)) {
        p.head_group = 4;
        p.share = selected && (head_dim == 64 || head_dim == 128);
        p.n_splits = 1;
        p.ahead = 1;
        return sized(p, rows, n_heads, n_kv, head_dim);
    }
    const int waves = mx4_wave_threads(head_dim, p.hp) / 64;
    const int64_t items = (int64_t)p.units * p.m_tiles * (n_kv / p.hp);
    const int64_t most = (max_keys + 32 * waves - 1) / (32 * waves);
    int64_t splits = items > 0 ? kCus / items : 1;
    if (splits > most) splits = most;
    if (splits > kMx4MaxSplits) splits = kMx4MaxSplits;
    // most: tiles of a wave that has a row's keys to itself
    if (splits < 1 || most * (splits - 1) < 4 * splits) splits = 1;
    p.n_splits = (int)splits;
    p.ahead = p.mt == 1 && p.hp == 1 && head_dim <= 128 && items * splits <= kCus && most >= 8 * splits ? 2 : 1;
    if (!selected && p.mt == 2 && waves == 8 && splits == 1)
        for (int g = 8; g > 1 && p.head_group == 1; g /= 2) {
            const int64_t wgs = items / g, rounds = (wgs + kCus - 1) / kCus;
            if (n_kv % g == 0 && 10 * wgs >= 9 * rounds * kCus) p.head_group = g;
        }
    return sized(p, rows, n_heads, n_kv, head_dim);
}

}  // namespace lidx

extern "C" {

indexer_status indexer_mx4_cache_write(const indexer_mx4_write_args *args) {
    if (!args) MX4_FAIL(INDEXER_EINVAL, "args is NULL");
    const indexer_mx4_write_args &g = *args;
    MX4_TRY(check_type(g.type));
    if (g.n_tokens < 0) MX4_FAIL(INDEXER_EINVAL, "n_tokens=%d must be >= 0", g.n_tokens);
    MX4_TRY(check_row_shape(g.n_heads, g.head_dim));
    lidx::Mx4Write a{};
    MX4_TRY(check_pages(g.n_blocks, g.block_size, g.n_heads, g.head_dim, g.strides, &a.pages));
    MX4_TRY(check_rows("k", g.k, g.k_stride_t, g.k_stride_h, g.n_heads, g.head_dim));
    if (g.n_blocks > 0) MX4_TRY(check_cache("k_", g.k_data, g.k_scale));
    if (g.v) {
        MX4_TRY(check_rows("v", g.v, g.v_stride_t, g.v_stride_h, g.n_heads, g.head_dim));
        if (g.n_blocks > 0) MX4_TRY(check_cache("v_", g.v_data, g.v_scale));
    }
    if (!g.slots) MX4_FAIL(INDEXER_EINVAL, "slots is NULL");
    if (!aligned(g.slots, 8)) MX4_FAIL(INDEXER_EINVAL, "slots must be 8-byte aligned");
    if (g.n_tokens == 0 || g.n_blocks == 0) return done(hipSuccess, "");
    a.x[0] = g.k;
    a.x[1] = g.v;
    a.st[0] = g.k_stride_t;
    a.st[1] = g.v_stride_t;
    a.sh[0] = g.k_stride_h;
    a.sh[1] = g.v_stride_h;
    a.data[0] = (uint8_t *)g.k_data;
    a.data[1] = (uint8_t *)g.v_data;
    a.scale[0] = (uint8_t *)g.k_scale;
    a.scale[1] = (uint8_t *)g.v_scale;
    a.slots = g.slots;
    a.n_tokens = g.n_tokens;
    a.n_heads = g.n_heads;
    a.head_dim = g.head_dim;
    a.n_tensors = g.v ? 2 : 1;
    a.div_e = lidx::fast_div((uint32_t)(g.n_heads * (g.head_dim / 8)));
    a.div_c = lidx::fast_div((uint32_t)(g.head_dim / 8));
    a.bf16 = g.type == INDEXER_MX4_BF16;
    return done(lidx::launch_mx4_write(a, (hipStream_t)g.stream), "cache write launch");
}

indexer_status indexer_mx4_cache_read(const indexer_mx4_read_args *args) {
    if (!args) MX4_FAIL(INDEXER_EINVAL, "args is NULL");
    const indexer_mx4_read_args &g = *args;
    MX4_TRY(check_type(g.type));
    if (g.n_rows < 0) MX4_FAIL(INDEXER_EINVAL, "n_rows=%d must be >= 0", g.n_rows);
    MX4_TRY(check_row_shape(g.n_heads, g.head_dim));
    if (g.n_blocks < 1) MX4_FAIL(INDEXER_EINVAL, "n_blocks=%d must be >= 1 to read", g.n_blocks);
    lidx::Mx4Read a{};
    MX4_TRY(check_pages(g.n_blocks, g.block_size, g.n_heads, g.head_dim, g.strides, &a.pages));
    MX4_TRY(check_cache("", g.data, g.scale));
    MX4_TRY(check_rows("out", g.out, g.out_stride_t, g.out_stride_h, g.n_heads, g.head_dim));
    if (!g.slots) MX4_FAIL(INDEXER_EINVAL, "slots is NULL");
    if (!aligned(g.slots, 8)) MX4_FAIL(INDEXER_EINVAL, "slots must be 8-byte aligned");
    if (g.n_rows == 0) return done(hipSuccess, "");
    a.data = (const uint8_t *)g.data;
    a.scale = (const uint8_t *)g.scale;
    a.slots = g.slots;
    a.out = g.out;
    a.st = g.out_stride_t;
    a.sh = g.out_stride_h;
    a.n_rows = g.n_rows;
    a.n_heads = g.n_heads;
    a.head_dim = g.head_dim;
    a.div_e = lidx::fast_div((uint32_t)(g.n_heads * (g.head_dim / 8)));
    a.div_c = lidx::fast_div((uint32_t)(g.head_dim / 8));
    a.bf16 = g.type == INDEXER_MX4_BF16;
    return done(lidx::launch_mx4_read(a, (hipStream_t)g.stream), "cache read launch");
}

indexer_status indexer_mx4_attend_selected(const indexer_mx4_attend_args *args) {
    if (!args) MX4_FAIL(INDEXER_EINVAL, "args is NULL");
    const indexer_mx4_attend_args &g = *args;
    lidx::Mx4Attend a;
    MX4_TRY(check_attend(g, &a));
    if (g.n_sel < 0) MX4_FAIL(INDEXER_EINVAL, "n_sel=%d must be >= 0", g.n_sel);
    if (g.pool_size < 1) MX4_FAIL(INDEXER_EINVAL, "pool_size=%d must be >= 1", g.pool_size);
    if (g.pool_size > lidx::kMaxPool) MX4_FAIL(INDEXER_ENOTSUP, "pool_size=%d exceeds %d", g.pool_size, lidx::kMaxPool);
    if ((int64_t)g.n_sel * g.pool_size > kMaxKeys)
        MX4_FAIL(INDEXER_ENOTSUP, "n_sel*pool_size=%lld exceeds %d", (long long)g.n_sel * g.pool_size, kMaxKeys);
    if (!g.idx) MX4_FAIL(INDEXER_EINVAL, "idx is NULL");
    if (!aligned(g.idx, 4)) MX4_FAIL(INDEXER_EINVAL, "idx must be 4-byte aligned");
    if (g.idx_stride < g.n_sel)
        MX4_FAIL(INDEXER_EINVAL, "idx_stride=%lld < n_sel=%d", (long long)g.idx_stride, g.n_sel);
    a.idx = g.idx;
    a.idx_st = g.idx_stride;
    a.n_sel = g.n_sel;
    a.pool = g.pool_size;
    a.div_pool = lidx::fast_div((uint32_t)g.pool_size);
    return run_attend(a, g, (int64_t)g.n_sel * g.pool_size);
}

indexer_status indexer_mx4_attend_window(const indexer_mx4_attend_args *args) {
    if (!args) MX4_FAIL(INDEXER_EINVAL, "args is NULL");
    const indexer_mx4_attend_args &g = *args;
    lidx::Mx4Attend a;
    MX4_TRY(check_attend(g, &a));
    if (g.window < 0 || g.sinks < 0)
        MX4_FAIL(INDEXER_EINVAL, "window=%d sinks=%d must be >= 0", g.window, g.sinks);
    a.window = g.window;
    a.sinks = g.window ? g.sinks : 0;
    return run_attend(a, g, window_keys(g.max_seq_len, g.window, g.sinks));
}

size_t indexer_mx4_attend_workspace_bytes(int32_t n_requests, int32_t query_len, int32_t max_keys, int32_t selected,
                                          int32_t n_heads, int32_t n_kv_heads, int32_t head_dim) {
    if (n_requests < 0 || query_len < 1 || max_keys < 0 || n_heads < 1 || n_heads > lidx::kMaxHeads ||
        n_kv_heads < 1 || n_heads % n_kv_heads || !attend_dim(head_dim) ||
        (int64_t)n_requests * query_len > kMaxKeys / n_heads)
        return (size_t)-1;
    const lidx::Mx4Plan p =
        lidx::plan_mx4_attend(n_requests, query_len, max_keys, selected != 0, n_heads, n_kv_heads, head_dim);
    return p.fits ? p.workspace_bytes : (size_t)-1;
}

// The form an attention call takes, for tests that are meant for one of them:
// many rows, shared scales (where the layout allows), tiles ahead, row tiles and
// K/V heads of a wave, groups of heads of a workgroup, shares of a row's keys,
// threads.  Not part of the interface.
void lidx_mx4_attend_form(int32_t n_requests, int32_t query_len, int32_t max_keys, int32_t selected, int32_t n_heads,
                          int32_t n_kv_heads, int32_t head_dim, int32_t form[8]) {
    const lidx::Mx4Plan p =
        lidx::plan_mx4_attend(n_requests, query_len, max_keys, selected != 0, n_heads, n_kv_heads, head_dim);
    const int32_t fields[8] = {p.prompt, p.share, p.ahead, p.mt, p.hp, p.head_group, p.n_splits, p.threads};
    for (int i = 0; i < 8; ++i) form[i] = fields[i];
}

}  // extern "C"
