// Internal interface of the page operators (pages_api.hip, pages_kernel.hip).
// Not exported.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx4_internal.h"

namespace lidx {

// Caches of a launch; more are taken in several launches.
constexpr int kPageArrays = 64;
// Rows of a table, and entries of a list of them.
constexpr int kPageRows = 8192;

struct PageArray {
    uint8_t *base;
    int64_t stride, bytes;
    uint32_t first_unit;  // units of a page in the arrays before
    int32_t width;        // bytes of an access: 16, 4 or 1
};

struct PageArrays {
    PageArray a[kPageArrays];
    int32_t n;
    uint32_t units;  // of a page in all of them
    FastDiv div_units;
};

// Pairs of pages to copy: from[i] to to[i].
struct PageCopy {
    PageArrays arrays;
    const int32_t *from, *to;
    int32_t n, n_pages;
};

struct PageTable {
    int32_t *refs, *table;
    int64_t stride;
    int32_t *seq_lens;
    int32_t n_pages, n_rows, n_cols, block_size;
};

struct PageFork {
    PageTable t;
    const int32_t *parents, *children;
    int32_t *fresh;
    int32_t n;
};

struct PageGrow {
    PageTable t;
    const int32_t *rows, *new_tokens;
    int64_t *slots;
    int32_t n, tokens;
    bool all;  // every slot in the first launch
};

struct PageFree {
    PageTable t;
    const int32_t *rows;
    int32_t n;
};

struct PageCompact {
    PageTable t;
    int32_t *place, *live;
    int32_t *from, *to, *moves;  // workspace: the moves, and their number
};

hipError_t launch_pages_copy(const PageCopy &a, hipStream_t stream);
// Which pages go to whom; then (a list of arrays at a time) the copies and, with the first, the tables' rows.
hipError_t launch_pages_fork_plan(const PageFork &a, hipStream_t stream);
hipError_t launch_pages_fork(const PageFork &a, const PageArrays &arrays, bool rows, hipStream_t stream);
hipError_t launch_pages_grow(const PageGrow &a, hipStream_t stream);
hipError_t launch_pages_free(const PageFree &a, hipStream_t stream);
hipError_t launch_pages_compact_plan(const PageCompact &a, hipStream_t stream);
hipError_t launch_pages_move(const PageCompact &a, const PageArrays &arrays, bool rows, hipStream_t stream);
// A launch holds the rows of n entries, 256 columns a workgroup, and the copies.
bool page_rows_fit(int n_cols, int64_t n);
uint32_t page_units(int64_t bytes, int width);

}  // namespace lidx
