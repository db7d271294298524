// Pages of the paged caches for gfx950: copied, forked, grown, freed, compacted.
//
// Copies are memory-bound, two bytes moved for each copied.  A wave takes a
// unit of a page of one cache, kLoads accesses of 16 bytes a lane, all asked
// for before the first is stored.
//
// Which free page goes to whom depends on all entries of a list and on all
// pages before it, so one workgroup decides: it scans the list for what each
// entry needs, then the counts for as many free pages as that, lowest first,
// and stops there.  The result is the same in any run; only counts change by
// atomics, whose order does not matter.
#include "device_common.h"
#include "mx4_internal.h"
#include "pages_internal.h"

namespace lidx {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kLoads = 4;
constexpr int kPlanThreads = 1024, kPlanWaves = kPlanThreads / 64;
constexpr int kCounts = 16;  // counts of pages a thread looks at at a time
constexpr int kGroup = 8;    // children whose rows a workgroup writes

template <typename W>
__device__ __forceinline__ void copy_unit(const uint8_t *src, uint8_t *dst, int64_t left, int lane) {
    W v[kLoads];
    const int64_t n = left / (int64_t)sizeof(W);
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
        if (i * 64 + lane < n) v[i] = reinterpret_cast<const W *>(src)[i * 64 + lane];
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
        if (i * 64 + lane < n) reinterpret_cast<W *>(dst)[i * 64 + lane] = v[i];
}

// One unit of a page, by a wave.
__device__ __forceinline__ void copy_part(const PageArrays &arrays, uint32_t unit, int from, int to, int lane) {
    int lo = 0, hi = arrays.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (arrays.a[mid].first_unit <= unit) lo = mid;
        else hi = mid - 1;
    }
    const PageArray &a = arrays.a[lo];
    const int64_t at = (int64_t)(unit - a.first_unit) * (64 * kLoads) * a.width;
    const uint8_t *src = a.base + (int64_t)from * a.stride + at;
    uint8_t *dst = a.base + (int64_t)to * a.stride + at;
    if (a.width == 16) copy_unit<u32x4>(src, dst, a.bytes - at, lane);
    else if (a.width == 4) copy_unit<uint32_t>(src, dst, a.bytes - at, lane);
    else copy_unit<uint8_t>(src, dst, a.bytes - at, lane);
}

// The pair that an item, a unit of a pair's page, belongs to.
__device__ __forceinline__ int pair_of(int64_t item, const PageArrays &arrays) {
    return (int)(item <= INT32_MAX ? quotient((uint32_t)item, arrays.div_units) : item / arrays.units);
}

__global__ void __launch_bounds__(kThreads) pages_copy_kernel(PageCopy c) {
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
    const int n = c.count ? min(*c.count, c.n) : c.n;
    const int64_t items = (int64_t)n * c.arrays.units;
    for (int64_t item = (int64_t)blockIdx.x * kWaves + wave; item < items; item += (int64_t)gridDim.x * kWaves) {
        const int i = pair_of(item, c.arrays);
        const uint32_t unit = (uint32_t)(item - (int64_t)i * c.arrays.units);
        const int from = uni(c.from[i]), to = uni(c.to[i]);
        if ((uint32_t)from >= (uint32_t)c.n_pages || (uint32_t)to >= (uint32_t)c.n_pages || from == to) continue;
        copy_part(c.arrays, unit, from, to, lane);
    }
}

// The sum of the values of the threads before, and of all of them.  `scratch`
// holds a word a wave; two barriers.
__device__ __forceinline__ int plan_scan(int v, int *scratch, int &total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int upto = wave_incl_scan(v);
    __syncthreads();  // the words of the scan before are no longer read
    if (lane == 63) scratch[wave] = upto;
    __syncthreads();
    const int mine = lane < kPlanWaves ? scratch[lane] : 0;
    const int sums = row_incl_scan(mine);
    total = __builtin_amdgcn_readlane(sums, kPlanWaves - 1);
    const int w = uni(wave);
    const int before = w ? __builtin_amdgcn_readlane(sums, w - 1) : 0;
    return before + upto - v;
}

// Which of the kCounts pages from `first` on are held, a bit each.
__device__ __forceinline__ uint32_t held_bits(const PageTable &t, int64_t first) {
    int held[kCounts];
    uint32_t bits = 0;
    if (first + kCounts <= t.n_pages) {
        __builtin_memcpy(held, t.refs + first, sizeof held);
#pragma unroll
        for (int i = 0; i < kCounts; ++i) bits |= (uint32_t)(held[i] > 0) << i;
    } else {
        for (int i = 0; first + i < t.n_pages; ++i) bits |= (uint32_t)(t.refs[first + i] > 0) << i;
    }
    return bits;
}
// A bit for each of the kCounts pages from `first` on that lies below `end`.
__device__ __forceinline__ uint32_t bits_below(int64_t first, int64_t end) {
    const int64_t left = end - first;
    return left >= kCounts ? (1u << kCounts) - 1u : (left > 0 ? (1u << left) - 1u : 0u);
}

// Calls found(rank, page) for the lowest `want` free pages; how many there were.
template <typename F>
__device__ __forceinline__ int find_free(const PageTable &t, int want, int *scratch, F found) {
    int have = 0;
    for (int64_t base = 0; base < t.n_pages && have < want; base += kPlanThreads * kCounts) {
        const int64_t first = base + threadIdx.x * kCounts;
        uint32_t free = ~held_bits(t, first) & bits_below(first, t.n_pages);
        int total;
        int rank = have + plan_scan(__popc(free), scratch, total);
        while (free && rank < want) {
            const int i = __ffs(free) - 1;
            free &= free - 1;
            found(rank++, (int)(first + i));
        }
        have += total;
    }
    return min(have, want);
}

// Which entries of a list count: those that name a row for the first time.
// first: an int a row.
__device__ __forceinline__ void mark_first(int *first, const int32_t *rows, int n, int n_rows) {
    for (int i = threadIdx.x; i < n_rows; i += kPlanThreads) first[i] = INT32_MAX;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int r = rows[i];
        if ((uint32_t)r < (uint32_t)n_rows) atomicMin(&first[r], i);
    }
    __syncthreads();
}

// A request's tokens, as many as its row can hold.
__device__ __forceinline__ int length_of(const PageTable &t, int row) {
    return (int)min((int64_t)max(t.seq_lens[row], 0), (int64_t)t.n_cols * t.block_size);
}

__global__ void __launch_bounds__(kPlanThreads) pages_fork_plan_kernel(PageFork a) {
    __shared__ int first[kPageRows], rank_of[kPageRows], scratch[kPlanWaves];
    const PageTable &t = a.t;
    mark_first(first, a.children, a.n, t.n_rows);
    // what each pair needs: bit 31 of its rank says that it counts, bit 30 that it needs a page
    int wanted = 0;
    for (int base = 0; base < a.n; base += kPlanThreads) {
        const int i = base + threadIdx.x;
        bool counts = false, needs = false;
        if (i < a.n) {
            const int p = a.parents[i], c = a.children[i];
            counts = (uint32_t)p < (uint32_t)t.n_rows && (uint32_t)c < (uint32_t)t.n_rows && p != c && first[c] == i;
            needs = counts && length_of(t, p) % t.block_size != 0;
        }
        int total;
        const int rank = wanted + plan_scan(needs, scratch, total);
        if (i < a.n) rank_of[i] = rank | (int)((uint32_t)counts << 31) | needs << 30;
        wanted += total;
    }
    __syncthreads();
    int *pages = first;  // the pairs are known
    const int have = find_free(t, wanted, scratch, [&](int rank, int page) { pages[rank] = page; });
    __syncthreads();
    for (int i = threadIdx.x; i < a.n; i += kPlanThreads) {
        const int word = rank_of[i], rank = word & 0x3fffffff;
        int fresh = -3;
        if (word < 0) {
            const bool needs = word >> 30 & 1, ok = !needs || rank < have;
            fresh = needs ? (ok ? pages[rank] : -2) : -1;
            t.seq_lens[a.children[i]] = ok ? length_of(t, a.parents[i]) : 0;
            if (fresh >= 0) t.refs[fresh] = 1;
        }
        a.fresh[i] = fresh;
    }
}

// The rows of kGroup children, 256 columns of them: a thread a column, so the
// children of one parent in a row add to a page's count once.
__global__ void __launch_bounds__(kThreads) pages_fork_rows_kernel(PageFork a) {
    const PageTable &t = a.t;
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= t.n_cols) return;
    const int i0 = (int)blockIdx.y * kGroup, i1 = min(i0 + kGroup, a.n);
    int held = -1, times = 0;
    for (int i = i0; i < i1; ++i) {
        const int fresh = a.fresh[i];
        if (fresh == -3) continue;
        const int child = a.children[i];
        int page = -1;
        if (fresh != -2) {
            const int full = t.seq_lens[child] / t.block_size;
            if (c < full) {
                page = t.table[(int64_t)a.parents[i] * t.stride + c];
                if ((uint32_t)page >= (uint32_t)t.n_pages) page = -1;
                if (page != held) {
                    if (held >= 0) atomicAdd(&t.refs[held], times);
                    held = page;
                    times = 0;
                }
                ++times;
            } else if (c == full) {
                page = fresh;  // or -1
            }
        }
        t.table[(int64_t)child * t.stride + c] = page;
    }
    if (held >= 0) atomicAdd(&t.refs[held], times);
}

__global__ void __launch_bounds__(kThreads) pages_fork_copy_kernel(PageFork a, PageArrays arrays) {
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
    const PageTable &t = a.t;
    const int64_t items = (int64_t)a.n * arrays.units;
    for (int64_t item = (int64_t)blockIdx.x * kWaves + wave; item < items; item += (int64_t)gridDim.x * kWaves) {
        const int i = pair_of(item, arrays);
        const uint32_t unit = (uint32_t)(item - (int64_t)i * arrays.units);
        const int to = uni(a.fresh[i]);
        if (to < 0) continue;
        const int full = t.seq_lens[a.children[i]] / t.block_size;
        const int from = uni(t.table[(int64_t)a.parents[i] * t.stride + full]);
        if ((uint32_t)from >= (uint32_t)t.n_pages) continue;
        copy_part(arrays, unit, from, to, lane);
    }
}

// New tokens of entry i.
__device__ __forceinline__ int new_of(const PageGrow &a, int i) {
    return a.new_tokens ? min(max(a.new_tokens[i], 0), a.tokens) : a.tokens;
}

__device__ __forceinline__ int64_t pages_for(int64_t tokens, int block_size) {
    return (tokens + block_size - 1) / block_size;
}

// Where new token k of an entry whose row has grown goes.
__device__ __forceinline__ int64_t slot_of(const PageGrow &a, int i, int k) {
    const PageTable &t = a.t;
    const int r = a.rows[i], mine = new_of(a, i);
    if (k >= mine) return -1;
    const uint32_t p = (uint32_t)(t.seq_lens[r] - mine + k), c = p / (uint32_t)t.block_size;
    const int page = t.table[(int64_t)r * t.stride + c];
    if ((uint32_t)page >= (uint32_t)t.n_pages) return -1;
    return (int64_t)page * t.block_size + (p - c * (uint32_t)t.block_size);
}

__global__ void __launch_bounds__(kPlanThreads) pages_grow_kernel(PageGrow a) {
    __shared__ int first[kPageRows], upto_of[kPageRows], scratch[kPlanWaves];
    const PageTable &t = a.t;
    mark_first(first, a.rows, a.n, t.n_rows);
    // entry i needs pages upto_of[i - 1] .. upto_of[i] of the free ones; bit 31: it is left or skipped
    int wanted = 0;
    for (int base = 0; base < a.n; base += kPlanThreads) {
        const int i = base + threadIdx.x;
        bool counts = false;
        int need = 0;
        if (i < a.n) {
            const int r = a.rows[i];
            if ((uint32_t)r < (uint32_t)t.n_rows && first[r] == i) {
                const int len = length_of(t, r);
                const int64_t want = pages_for((int64_t)len + new_of(a, i), t.block_size);
                counts = want <= t.n_cols;
                if (counts) need = (int)(want - pages_for(len, t.block_size));
            }
        }
        int total;
        const int before = plan_scan(need, scratch, total);
        if (i < a.n) upto_of[i] = (wanted + before + need) | (int)((uint32_t)!counts << 31);
        wanted += total;
    }
    __syncthreads();
    // the pages, by rank, where the slots will be: a page holds a new token at least, so they fit
    const int have = find_free(t, wanted, scratch, [&](int rank, int page) { a.slots[rank] = page; });
    __syncthreads();
    for (int i = threadIdx.x; i < a.n; i += kPlanThreads) {
        const int word = upto_of[i], upto = word & 0x7fffffff;
        const int need = upto - (i ? upto_of[i - 1] & 0x7fffffff : 0);
        bool grows = word >= 0 && (need == 0 || upto <= have);
        if (grows) {
            const int r = a.rows[i], len = length_of(t, r), held = (int)pages_for(len, t.block_size);
            for (int k = 0; k < need; ++k) {
                const int page = (int)a.slots[upto - need + k];
                t.table[(int64_t)r * t.stride + held + k] = page;
                t.refs[page] = 1;
            }
            t.seq_lens[r] = len + new_of(a, i);
        }
        first[i] = grows;  // rows are known; i < kPageRows
    }
    __syncthreads();
    // the first slot of every entry, and in a short list the others
    for (int i = threadIdx.x; i < a.n; i += kPlanThreads)
        a.slots[(int64_t)i * a.tokens] = first[i] ? slot_of(a, i, 0) : -1;
    if (!a.all) return;
    const uint32_t all = (uint32_t)a.n * (uint32_t)a.tokens;
    for (uint32_t e = threadIdx.x; e < all; e += kPlanThreads) {
        const int i = (int)(e / (uint32_t)a.tokens), k = (int)(e - (uint32_t)i * (uint32_t)a.tokens);
        if (k) a.slots[e] = first[i] ? slot_of(a, i, k) : -1;
    }
}

// The slots after the first, of a long list: a first one of -1 says that the row has not grown.
__global__ void __launch_bounds__(kThreads) pages_slots_kernel(PageGrow a) {
    const uint32_t all = (uint32_t)a.n * (uint32_t)a.tokens;
    for (uint32_t e = blockIdx.x * kThreads + threadIdx.x; e < all; e += gridDim.x * kThreads) {
        const int i = (int)(e / (uint32_t)a.tokens), k = (int)(e - (uint32_t)i * (uint32_t)a.tokens);
        if (k) a.slots[e] = a.slots[e - k] >= 0 ? slot_of(a, i, k) : -1;
    }
}

// A row of the list a workgroup of blockIdx.y, 256 columns of it.  An entry is taken by
// exchanging it with -1, so a row named twice gives its pages back once.
__global__ void __launch_bounds__(kThreads) pages_free_kernel(PageFree a) {
    const PageTable &t = a.t;
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int r = a.rows[blockIdx.y];
    if ((uint32_t)r >= (uint32_t)t.n_rows) return;
    if (c == 0) t.seq_lens[r] = 0;
    if (c >= t.n_cols) return;
    int32_t *entry = t.table + (int64_t)r * t.stride + c;
    if (*entry == -1) return;
    const int page = atomicExch(entry, -1);
    if ((uint32_t)page < (uint32_t)t.n_pages) atomicSub(&t.refs[page], 1);
}

__global__ void __launch_bounds__(kPlanThreads) pages_compact_plan_kernel(PageCompact a) {
    __shared__ int scratch[kPlanWaves];
    const PageTable &t = a.t;
    constexpr int STEP = kPlanThreads * kCounts;
    int live = 0, below = 0, total;  // pages in use; those of them below `live`, which stay
    for (int64_t base = 0; base < t.n_pages; base += STEP) {
        plan_scan(__popc(held_bits(t, base + threadIdx.x * kCounts)), scratch, total);
        live += total;
    }
    for (int64_t base = 0; base < live; base += STEP) {
        const int64_t first = base + threadIdx.x * kCounts;
        plan_scan(first < live ? __popc(held_bits(t, first) & bits_below(first, live)) : 0, scratch, total);
        below += total;
    }
    // the free pages below `live` and the pages in use from there on, each in order: live - below of either
    int seen = 0;
    for (int64_t base = 0; base < t.n_pages; base += STEP) {
        const int64_t first = base + threadIdx.x * kCounts;
        const uint32_t bits = held_bits(t, first);
        int before = seen + plan_scan(__popc(bits), scratch, total);  // pages in use before this one
        seen += total;
        for (int i = 0; i < kCounts && first + i < t.n_pages; ++i) {
            const int p = (int)(first + i);
            const bool used = bits >> i & 1;
            a.place[p] = used ? p : -1;
            if (!used && p < live) a.to[p - before] = p;
            if (used && p >= live) a.from[before - below] = p;
            before += used;
        }
    }
    __syncthreads();
    for (int k = threadIdx.x; k < live - below; k += kPlanThreads) {
        const int from = a.from[k], to = a.to[k];
        a.place[from] = to;
        t.refs[to] = t.refs[from];
        t.refs[from] = 0;
    }
    if (threadIdx.x == 0) {
        *a.live = live;
        *a.moves = live - below;
    }
}

__global__ void __launch_bounds__(kThreads) pages_rename_kernel(PageCompact a) {
    const PageTable &t = a.t;
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= t.n_cols) return;
    for (int r = (int)blockIdx.y; r < t.n_rows; r += (int)gridDim.y) {
        int32_t *entry = t.table + (int64_t)r * t.stride + c;
        const int page = *entry;
        if (page != -1) *entry = (uint32_t)page < (uint32_t)t.n_pages ? a.place[page] : -1;
    }
}

// Workgroups of a copy: a wave a unit, up to 16 workgroups a compute unit, which then take several
unsigned copy_groups(int64_t items) {
    const int64_t groups = (items + kWaves - 1) / kWaves, most = 16 * 256;
    return (unsigned)(groups < most ? groups : most);
}

dim3 columns(int n_cols, int rows) { return dim3(n_cols ? (unsigned)((n_cols + kThreads - 1) / kThreads) : 1u, (unsigned)rows); }

}  // namespace

uint32_t page_units(int64_t bytes, int width) {
    const int64_t unit = (int64_t)64 * kLoads * width;
    return (uint32_t)((bytes + unit - 1) / unit);
}

hipError_t launch_pages_copy(const PageCopy &a, hipStream_t stream) {
    hipLaunchKernelGGL(pages_copy_kernel, dim3(copy_groups((int64_t)a.n * a.arrays.units)), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_pages_fork(const PageFork &a, hipStream_t stream) {
    hipLaunchKernelGGL(pages_fork_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a);
    if (a.t.n_cols > 0)
        hipLaunchKernelGGL(pages_fork_rows_kernel, columns(a.t.n_cols, (a.n + kGroup - 1) / kGroup), dim3(kThreads), 0, stream,
                           a);
    return hipGetLastError();
}

hipError_t launch_pages_fork_copy(const PageFork &a, const PageArrays &arrays, hipStream_t stream) {
    hipLaunchKernelGGL(pages_fork_copy_kernel, dim3(copy_groups((int64_t)a.n * arrays.units)), dim3(kThreads), 0, stream, a,
                       arrays);
    return hipGetLastError();
}

hipError_t launch_pages_grow(const PageGrow &grow, hipStream_t stream) {
    PageGrow a = grow;
    const int64_t all = (int64_t)a.n * a.tokens;
    a.all = all <= 16 * kPlanThreads;
    hipLaunchKernelGGL(pages_grow_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a);
    if (!a.all) {
        const int64_t groups = (all + kThreads - 1) / kThreads;
        hipLaunchKernelGGL(pages_slots_kernel, dim3((unsigned)(groups < 2048 ? groups : 2048)), dim3(kThreads), 0, stream, a);
    }
    return hipGetLastError();
}

hipError_t launch_pages_free(const PageFree &a, hipStream_t stream) {
    hipLaunchKernelGGL(pages_free_kernel, columns(a.t.n_cols, a.n), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_pages_compact(const PageCompact &a, hipStream_t stream) {
    hipLaunchKernelGGL(pages_compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a);
    if (a.t.n_rows > 0 && a.t.n_cols > 0)
        hipLaunchKernelGGL(pages_rename_kernel, columns(a.t.n_cols, a.t.n_rows), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace lidx
