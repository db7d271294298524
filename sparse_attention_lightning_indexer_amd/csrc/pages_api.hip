// C-ABI of the page operators (declared in include/indexer_pages.h).  As in
// indexer_api.hip: every argument is checked on the host, without touching
// device memory or calling HIP, before anything is enqueued.
#include "../../include/indexer_pages.h"
#include "internal.h"
#include "pages_internal.h"

namespace {

using lidx::api_error;

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

static_assert(sizeof(indexer_page_array) == 3 * 8 && sizeof(indexer_pages_copy_args) == 4 * 8 + 4 * 4 &&
                  sizeof(indexer_pages_fork_args) == 9 * 8 + 6 * 4 && sizeof(indexer_pages_grow_args) == 8 * 8 + 6 * 4 &&
                  sizeof(indexer_pages_free_args) == 6 * 8 + 4 * 4 && sizeof(indexer_pages_compact_args) == 9 * 8 + 4 * 4,
              "the binding packs the members");

constexpr int32_t kMaxTokens = INT32_MAX - 1023;

#define PAGES_FAIL(st, ...) return (indexer_status)api_error(st, __VA_ARGS__)
#define PAGES_TRY(expr)                              \
    do {                                             \
        const indexer_status st_ = (expr);           \
        if (st_ != INDEXER_OK) return st_;           \
    } while (0)

indexer_status done(hipError_t e, const char *what) { return (indexer_status)lidx::api_launch(e, what); }

indexer_status check_list(const char *name, const void *p, size_t size) {
    if (!p) PAGES_FAIL(INDEXER_EINVAL, "%s is NULL", name);
    if (!aligned(p, size)) PAGES_FAIL(INDEXER_EINVAL, "%s must be %zu-byte aligned", name, size);
    return INDEXER_OK;
}

indexer_status check_arrays(const indexer_page_array *arrays, int32_t n, int32_t n_pages) {
    if (n < 0) PAGES_FAIL(INDEXER_EINVAL, "n_arrays=%d must be >= 0", n);
    if (n > 0 && !arrays) PAGES_FAIL(INDEXER_EINVAL, "arrays is NULL");
    for (int i = 0; i < n; ++i) {
        const indexer_page_array &a = arrays[i];
        if (!a.base) PAGES_FAIL(INDEXER_EINVAL, "array %d's base is NULL", i);
        if (a.bytes < 1 || a.bytes > INT32_MAX)
            PAGES_FAIL(INDEXER_EINVAL, "array %d's pages of %lld bytes are not supported (1..2^31-1)", i, (long long)a.bytes);
        if (n_pages > 1 && a.stride < a.bytes)
            PAGES_FAIL(INDEXER_EINVAL, "array %d's stride %lld must be >= its pages' %lld bytes", i, (long long)a.stride,
                       (long long)a.bytes);
        if (n_pages > 1 && a.stride > INT64_MAX / n_pages)
            PAGES_FAIL(INDEXER_EINVAL, "array %d's stride %lld is too large", i, (long long)a.stride);
    }
    return INDEXER_OK;
}

// The arrays of a launch, from `first` on.
lidx::PageArrays arrays_from(const indexer_page_array *arrays, int32_t n, int32_t first) {
    lidx::PageArrays r{};
    for (; r.n < lidx::kPageArrays && first + r.n < n; ++r.n) {
        const indexer_page_array &a = arrays[first + r.n];
        const uintptr_t all = (uintptr_t)a.base | (uintptr_t)a.stride | (uintptr_t)a.bytes;
        const int width = all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : 1;
        const uint32_t units = lidx::page_units(a.bytes, width);
        if (r.n && (int64_t)r.units + units > INT32_MAX) break;  // 2^31 bytes in units of a byte still fit one array
        r.a[r.n] = lidx::PageArray{(uint8_t *)a.base, a.stride, a.bytes, r.units, width};
        r.units += units;
    }
    r.div_units = lidx::fast_div(r.units ? r.units : 1);
    return r;
}

indexer_status check_pool(int32_t n_pages, int32_t n) {
    if (n_pages < 0) PAGES_FAIL(INDEXER_EINVAL, "n_pages=%d must be >= 0", n_pages);
    if (n_pages > kMaxTokens) PAGES_FAIL(INDEXER_ENOTSUP, "n_pages=%d exceeds %d", n_pages, kMaxTokens);
    if (n < 0) PAGES_FAIL(INDEXER_EINVAL, "n=%d must be >= 0", n);
    return INDEXER_OK;
}

// block_size 0: not used
indexer_status check_table(int32_t *refs, int32_t *table, int64_t stride, int32_t *seq_lens, int32_t n_pages, int32_t n_rows,
                           int32_t n_cols, int32_t block_size, lidx::PageTable *out) {
    if (n_rows < 0 || n_cols < 0) PAGES_FAIL(INDEXER_EINVAL, "n_rows=%d n_cols=%d must be >= 0", n_rows, n_cols);
    if (n_pages > 0) PAGES_TRY(check_list("refs", refs, 4));
    if (n_rows > 0 && n_cols > 0) PAGES_TRY(check_list("block_table", table, 4));
    if (n_rows > 1 && stride < n_cols)
        PAGES_FAIL(INDEXER_EINVAL, "table_stride=%lld < n_cols=%d", (long long)stride, n_cols);
    if (n_rows > 0 && seq_lens) PAGES_TRY(check_list("seq_lens", seq_lens, 4));
    *out = lidx::PageTable{refs, table, n_rows > 1 ? stride : 0, seq_lens, n_pages, n_rows, n_cols, block_size};
    return INDEXER_OK;
}

indexer_status check_rows(int32_t n, int32_t n_rows) {
    if (n > lidx::kPageRows || n_rows > lidx::kPageRows)
        PAGES_FAIL(INDEXER_ENOTSUP, "n=%d n_rows=%d not supported (lists and tables of at most %d rows)", n, n_rows,
                   lidx::kPageRows);
    return INDEXER_OK;
}

indexer_status check_launch(int32_t n_cols, int32_t n) {
    if (!lidx::page_rows_fit(n_cols, n))
        PAGES_FAIL(INDEXER_EINVAL, "problem too large for one launch: %d rows of %d columns", n, n_cols);
    return INDEXER_OK;
}

indexer_status check_block(int32_t block_size, int32_t n_cols) {
    if (block_size < 1) PAGES_FAIL(INDEXER_EINVAL, "block_size=%d must be >= 1", block_size);
    if ((int64_t)n_cols * block_size > kMaxTokens)
        PAGES_FAIL(INDEXER_ENOTSUP, "n_cols*block_size=%lld exceeds %d", (long long)n_cols * block_size, kMaxTokens);
    return INDEXER_OK;
}

}  // namespace

extern "C" {

indexer_status indexer_pages_copy(const indexer_pages_copy_args *args) {
    if (!args) PAGES_FAIL(INDEXER_EINVAL, "args is NULL");
    const indexer_pages_copy_args &g = *args;
    PAGES_TRY(check_pool(g.n_pages, g.n));
    PAGES_TRY(check_arrays(g.arrays, g.n_arrays, g.n_pages));
    if (g.n == 0 || g.n_pages == 0 || g.n_arrays == 0) return done(hipSuccess, "");
    PAGES_TRY(check_list("from", g.from, 4));
    PAGES_TRY(check_list("to", g.to, 4));
    for (int32_t first = 0; first < g.n_arrays;) {
        lidx::PageCopy a{arrays_from(g.arrays, g.n_arrays, first), g.from, g.to, g.n, g.n_pages};
        PAGES_TRY(done(lidx::launch_pages_copy(a, (hipStream_t)g.stream), "page copy launch"));
        first += a.arrays.n;
    }
    return INDEXER_OK;
}

indexer_status indexer_pages_fork(const indexer_pages_fork_args *args) {
    if (!args) PAGES_FAIL(INDEXER_EINVAL, "args is NULL");
    const indexer_pages_fork_args &g = *args;
    PAGES_TRY(check_pool(g.n_pages, g.n));
    PAGES_TRY(check_arrays(g.arrays, g.n_arrays, g.n_pages));
    PAGES_TRY(check_rows(g.n, g.n_rows));
    PAGES_TRY(check_block(g.block_size, g.n_cols));
    lidx::PageFork a{};
    PAGES_TRY(check_table(g.refs, g.block_table, g.table_stride, g.seq_lens, g.n_pages, g.n_rows, g.n_cols, g.block_size, &a.t));
    if (g.n == 0) return done(hipSuccess, "");
    if (g.n_rows > 0) PAGES_TRY(check_list("seq_lens", g.seq_lens, 4));
    PAGES_TRY(check_launch(g.n_cols, g.n));
    PAGES_TRY(check_list("parents", g.parents, 4));
    PAGES_TRY(check_list("children", g.children, 4));
    PAGES_TRY(check_list("fresh", g.fresh, 4));
    a.parents = g.parents;
    a.children = g.children;
    a.fresh = g.fresh;
    a.n = g.n;
    PAGES_TRY(done(lidx::launch_pages_fork_plan(a, (hipStream_t)g.stream), "page fork launch"));
    if (g.n_cols == 0) return INDEXER_OK;
    int32_t first = 0;
    do {  // the rows, and copies of the first list of arrays, if there is one
        lidx::PageArrays arrays = arrays_from(g.arrays, g.n_arrays, first);
        if (g.n_pages == 0) arrays.units = 0;
        PAGES_TRY(done(lidx::launch_pages_fork(a, arrays, first == 0, (hipStream_t)g.stream), "page fork launch"));
        first += arrays.n;
    } while (first < g.n_arrays);
    return INDEXER_OK;
}

indexer_status indexer_pages_grow(const indexer_pages_grow_args *args) {
    if (!args) PAGES_FAIL(INDEXER_EINVAL, "args is NULL");
    const indexer_pages_grow_args &g = *args;
    PAGES_TRY(check_pool(g.n_pages, g.n));
    if (g.tokens < 0) PAGES_FAIL(INDEXER_EINVAL, "tokens=%d must be >= 0", g.tokens);
    PAGES_TRY(check_rows(g.n, g.n_rows));
    PAGES_TRY(check_block(g.block_size, g.n_cols));
    if ((int64_t)g.n * g.tokens > kMaxTokens)
        PAGES_FAIL(INDEXER_ENOTSUP, "n*tokens=%lld exceeds %d", (long long)g.n * g.tokens, kMaxTokens);
    lidx::PageGrow a{};
    PAGES_TRY(check_table(g.refs, g.block_table, g.table_stride, g.seq_lens, g.n_pages, g.n_rows, g.n_cols, g.block_size, &a.t));
    if (g.n == 0 || g.tokens == 0) return done(hipSuccess, "");
    if (g.n_rows > 0) PAGES_TRY(check_list("seq_lens", g.seq_lens, 4));
    PAGES_TRY(check_list("rows", g.rows, 4));
    PAGES_TRY(check_list("slots", g.slots, 8));
    if (g.new_tokens) PAGES_TRY(check_list("new_tokens", g.new_tokens, 4));
    a.rows = g.rows;
    a.new_tokens = g.new_tokens;
    a.slots = g.slots;
    a.n = g.n;
    a.tokens = g.tokens;
    return done(lidx::launch_pages_grow(a, (hipStream_t)g.stream), "page grow launch");
}

indexer_status indexer_pages_free(const indexer_pages_free_args *args) {
    if (!args) PAGES_FAIL(INDEXER_EINVAL, "args is NULL");
    const indexer_pages_free_args &g = *args;
    PAGES_TRY(check_pool(g.n_pages, g.n));
    PAGES_TRY(check_rows(g.n, g.n_rows));
    lidx::PageFree a{};
    PAGES_TRY(check_table(g.refs, g.block_table, g.table_stride, g.seq_lens, g.n_pages, g.n_rows, g.n_cols, 0, &a.t));
    if (g.n == 0 || g.n_rows == 0) return done(hipSuccess, "");
    PAGES_TRY(check_launch(g.n_cols, g.n));
    PAGES_TRY(check_list("seq_lens", g.seq_lens, 4));
    PAGES_TRY(check_list("rows", g.rows, 4));
    a.rows = g.rows;
    a.n = g.n;
    return done(lidx::launch_pages_free(a, (hipStream_t)g.stream), "page free launch");
}

indexer_status indexer_pages_compact(const indexer_pages_compact_args *args) {
    if (!args) PAGES_FAIL(INDEXER_EINVAL, "args is NULL");
    const indexer_pages_compact_args &g = *args;
    PAGES_TRY(check_pool(g.n_pages, 0));
    PAGES_TRY(check_arrays(g.arrays, g.n_arrays, g.n_pages));
    PAGES_TRY(check_rows(0, g.n_rows));
    lidx::PageCompact a{};
    PAGES_TRY(check_table(g.refs, g.block_table, g.table_stride, nullptr, g.n_pages, g.n_rows, g.n_cols, 0, &a.t));
    PAGES_TRY(check_launch(g.n_cols, g.n_rows));
    PAGES_TRY(check_list("live", g.live, 4));
    if (g.n_pages > 0) PAGES_TRY(check_list("place", g.place, 4));
    const size_t need = indexer_pages_compact_workspace_bytes(g.n_pages);
    if (!g.workspace || g.workspace_bytes < need || !aligned(g.workspace, 4))
        PAGES_FAIL(INDEXER_EWORKSPACE, "compaction needs %zu bytes of 4-byte aligned workspace, got %zu", need,
                   g.workspace ? g.workspace_bytes : (size_t)0);
    a.place = g.place;
    a.live = g.live;
    a.moves = (int32_t *)g.workspace;
    a.from = a.moves + 1;
    a.to = a.from + g.n_pages / 2;
    PAGES_TRY(done(lidx::launch_pages_compact_plan(a, (hipStream_t)g.stream), "page compaction launch"));
    int32_t first = 0;
    do {
        const lidx::PageArrays arrays = arrays_from(g.arrays, g.n_arrays, first);
        PAGES_TRY(done(lidx::launch_pages_move(a, arrays, first == 0 && g.n_cols > 0, (hipStream_t)g.stream),
                       "page compaction launch"));
        first += arrays.n;
    } while (first < g.n_arrays);
    return INDEXER_OK;
}

size_t indexer_pages_compact_workspace_bytes(int32_t n_pages) {
    return n_pages < 0 ? (size_t)-1 : 4 * ((size_t)1 + 2 * (size_t)(n_pages / 2));
}

}  // extern "C"
