// Pages of the paged caches for gfx950: copied, forked, grown, freed, compacted.
//
// Copies are memory-bound, two bytes moved for each copied.  A wave takes a
// unit of a page of one cache, kLoads accesses of 16 bytes a lane, all asked
// for before the first is stored.  512 pages of the 20 caches of four layers, 176 MB:
// 53 us back to back (6.6 TB/s there and back; a copy of 1 GiB reaches 5.1).
//
// Which free page goes to whom depends on all entries of a list and on all
// pages before it, so one workgroup decides: it scans the list for what each
// entry needs, then the counts for as many free pages as that, lowest first,
// and stops there (3 to 4 us).  The result is the same in any run; only counts
// change by atomics, whose order does not matter.  What follows the decision,
// tables and copies, is one launch, by workgroups of either kind: 64 requests that
// share four prompts of about 500 pages, 44 MB moved, 10 us.
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
constexpr int kOwnPages = 2; // new pages of a row that its thread writes itself

template <typename W, bool STREAM>
__device__ __forceinline__ void copy_unit(const uint8_t *src, uint8_t *dst, int64_t left, int lane) {
    W v[kLoads];
    const int64_t n = left / (int64_t)sizeof(W);
    const W *s = reinterpret_cast<const W *>(src) + lane;
    W *d = reinterpret_cast<W *>(dst) + lane;
    auto put = [&](int i) {
        if (STREAM) __builtin_nontemporal_store(v[i], d + i * 64);
        else d[i * 64] = v[i];
    };
    if (n >= 64 * kLoads) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) v[i] = s[i * 64];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) put(i);
        return;
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
        if (i * 64 + lane < n) v[i] = s[i * 64];
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
        if (i * 64 + lane < n) put(i);
}

// One unit of a page, by a wave.
template <bool STREAM>
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
    if (a.width == 16) copy_unit<u32x4, STREAM>(src, dst, a.bytes - at, lane);
    else if (a.width == 4) copy_unit<uint32_t, false>(src, dst, a.bytes - at, lane);
    else copy_unit<uint8_t, false>(src, dst, a.bytes - at, lane);
}

// The pair that an item, a unit of a pair's page, belongs to.
__device__ __forceinline__ int pair_of(int64_t item, const PageArrays &arrays) {
    return (int)(item <= INT32_MAX ? quotient((uint32_t)item, arrays.div_units) : item / arrays.units);
}

// The pairs of a list, shared out to the waves of `groups` workgroups, of which this is `group`.
template <bool STREAM>
__device__ __forceinline__ void copy_pairs(const PageArrays &arrays, const int32_t *list_from, const int32_t *list_to, int n,
                                           int n_pages, unsigned group, unsigned groups) {
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
    const int64_t items = (int64_t)n * arrays.units;
    for (int64_t item = (int64_t)group * kWaves + wave; item < items; item += (int64_t)groups * kWaves) {
        const int i = pair_of(item, arrays);
        const uint32_t unit = (uint32_t)(item - (int64_t)i * arrays.units);
        const int from = uni(list_from[i]), to = uni(list_to[i]);
        if ((uint32_t)from >= (uint32_t)n_pages || (uint32_t)to >= (uint32_t)n_pages || from == to) continue;
        copy_part<STREAM>(arrays, unit, from, to, lane);
    }
}

template <bool STREAM>
__global__ void __launch_bounds__(kThreads) pages_copy_kernel(PageCopy c) {
    copy_pairs<STREAM>(c.arrays, c.from, c.to, c.n, c.n_pages, blockIdx.x, gridDim.x);
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
__device__ __forceinline__ void fork_rows(const PageFork &a, unsigned group) {
    __shared__ int fresh_of[kGroup], child_of[kGroup], parent_of[kGroup], full_of[kGroup];
    const PageTable &t = a.t;
    const unsigned strips = ((unsigned)t.n_cols + kThreads - 1) / kThreads;
    const int i0 = (int)(group / strips) * kGroup;
    const int64_t c = (int64_t)(group % strips) * kThreads + threadIdx.x;
    if (threadIdx.x < kGroup) {
        const int i = i0 + (int)threadIdx.x;
        const int fresh = i < a.n ? a.fresh[i] : -3, child = i < a.n ? a.children[i] : 0, parent = i < a.n ? a.parents[i] : 0;
        const bool counts = fresh != -3;
        fresh_of[threadIdx.x] = fresh;
        child_of[threadIdx.x] = counts ? child : 0;
        parent_of[threadIdx.x] = counts ? parent : 0;
        full_of[threadIdx.x] = counts ? t.seq_lens[child] / t.block_size : 0;  // 0 where it was left empty
    }
    __syncthreads();
    if (c >= t.n_cols) return;
    int page[kGroup];
#pragma unroll
    for (int k = 0; k < kGroup; ++k)
        page[k] = c < full_of[k] || (c == full_of[k] && fresh_of[k] >= 0) ? t.table[(int64_t)parent_of[k] * t.stride + c] : -1;
    int held = -1, times = 0;
#pragma unroll
    for (int k = 0; k < kGroup; ++k) {
        if (fresh_of[k] == -3) continue;
        int mine = (uint32_t)page[k] < (uint32_t)t.n_pages ? page[k] : -1;
        if (c < full_of[k]) {
            if (mine != held) {
                if (held >= 0) atomicAdd(&t.refs[held], times);
                held = mine;
                times = 0;
            }
            ++times;
        } else if (mine >= 0) {
            mine = fresh_of[k];
        } else if (c == full_of[k] && fresh_of[k] >= 0) {
            // the parent's last page is none of the pool's, and the child has none either: the page
            // stays free, whose bytes are another's (copies of it read the same entry and leave it)
            t.refs[fresh_of[k]] = 0;
            a.fresh[i0 + k] = -1;
        }
        t.table[(int64_t)child_of[k] * t.stride + c] = mine;
    }
    if (held >= 0) atomicAdd(&t.refs[held], times);
}

// The copies of the parents' last pages, by the workgroups from first_group on.
__device__ __forceinline__ void fork_copies(const PageFork &a, const PageArrays &arrays, unsigned group, unsigned groups) {
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
    const PageTable &t = a.t;
    const int64_t items = (int64_t)a.n * arrays.units;
    for (int64_t item = (int64_t)group * kWaves + wave; item < items; item += (int64_t)groups * kWaves) {
        const int i = pair_of(item, arrays);
        const uint32_t unit = (uint32_t)(item - (int64_t)i * arrays.units);
        const int to = uni(a.fresh[i]), parent = uni(a.parents[i]);
        if (to < 0) continue;
        const int full = min(length_of(t, parent) / t.block_size, t.n_cols - 1);  // (its column exists, whatever the row)
        const int from = uni(t.table[(int64_t)parent * t.stride + full]);
        if ((uint32_t)from < (uint32_t)t.n_pages) copy_part<false>(arrays, unit, from, to, lane);
    }
}

// After the plan: the rows by the first row_groups workgroups, the copies by the others.
__global__ void __launch_bounds__(kThreads) pages_fork_kernel(PageFork a, PageArrays arrays, unsigned row_groups) {
    if (blockIdx.x < row_groups) fork_rows(a, blockIdx.x);
    else fork_copies(a, arrays, blockIdx.x - row_groups, gridDim.x - row_groups);
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
    return (int64_t)page * t.block_size + (p - c * (uint32_t)t.block_size);
}

__global__ void __launch_bounds__(kPlanThreads) pages_grow_kernel(PageGrow a) {
    __shared__ int first[kPageRows], upto_of[kPageRows], scratch[kPlanWaves], long_rows;
    const PageTable &t = a.t;
    if (threadIdx.x == 0) long_rows = 0;
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
                const int len = length_of(t, r), more = new_of(a, i);
                const int64_t want = pages_for((int64_t)len + more, t.block_size);
                counts = want <= t.n_cols;
                if (counts && more && len % t.block_size)  // the page that is not full yet
                    counts = (uint32_t)t.table[(int64_t)r * t.stride + len / t.block_size] < (uint32_t)t.n_pages;
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
            for (int k = 0; k < min(need, kOwnPages); ++k) {
                const int page = (int)a.slots[upto - need + k];
                t.table[(int64_t)r * t.stride + held + k] = page;
                t.refs[page] = 1;
            }
            if (need > kOwnPages) long_rows = 1;
            t.seq_lens[r] = len + new_of(a, i);
        }
        first[i] = grows;  // rows are known; i < kPageRows
    }
    __syncthreads();
    if (long_rows) {  // the other pages of long rows, a thread each
        for (int rank = threadIdx.x; rank < have; rank += kPlanThreads) {
            int lo = 0, hi = a.n - 1;  // whose it is: the first that asks for more up to there
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if ((upto_of[mid] & 0x7fffffff) > rank) hi = mid;
                else lo = mid + 1;
            }
            const int k = rank - (lo ? upto_of[lo - 1] & 0x7fffffff : 0);
            if (!first[lo] || k < kOwnPages) continue;
            const int r = a.rows[lo], held = (int)pages_for(t.seq_lens[r] - new_of(a, lo), t.block_size);
            const int page = (int)a.slots[rank];
            t.table[(int64_t)r * t.stride + held + k] = page;
            t.refs[page] = 1;
        }
        __syncthreads();
    }
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

// A row of the list a workgroup of blockIdx.y, 256 columns of it.  A row named
// before in the list is left to the workgroups of its first mention.
__global__ void __launch_bounds__(kThreads) pages_free_kernel(PageFree a) {
    const PageTable &t = a.t;
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int y = (int)blockIdx.y, r = a.rows[y];
    if ((uint32_t)r >= (uint32_t)t.n_rows) return;
    int32_t *entry = t.table + (int64_t)r * t.stride + min(c, (int64_t)t.n_cols - 1);
    const int page = c < t.n_cols ? *entry : -1;
    bool again = false;
    for (int i = (int)(threadIdx.x & 63); i < y; i += 64) again |= a.rows[i] == r;
    if (__ballot(again)) return;
    if (c == 0) t.seq_lens[r] = 0;
    if (page == -1) return;
    *entry = -1;
    if ((uint32_t)page < (uint32_t)t.n_pages) atomicSub(&t.refs[page], 1);
}

__global__ void __launch_bounds__(kPlanThreads) pages_compact_plan_kernel(PageCompact a) {
    __shared__ int scratch[kPlanWaves];
    const PageTable &t = a.t;
    constexpr int STEP = kPlanThreads * kCounts;
    int live = 0, below = 0, total;  // pages in use; those of them below `live`, which stay
    const uint32_t mine = held_bits(t, threadIdx.x * kCounts);
    const int mine_before = plan_scan(__popc(mine), scratch, total);
    live = total;
    for (int64_t base = STEP; base < t.n_pages; base += STEP) {
        plan_scan(__popc(held_bits(t, base + threadIdx.x * kCounts)), scratch, total);
        live += total;
    }
    for (int64_t base = 0; base < live; base += STEP) {
        const int64_t first = base + threadIdx.x * kCounts;
        const uint32_t bits = base ? (first < live ? held_bits(t, first) : 0u) : mine;
        plan_scan(__popc(bits & bits_below(first, live)), scratch, total);
        below += total;
    }
    // the free pages below `live` and the pages in use from there on, each in order: live - below of either
    int seen = 0;
    for (int64_t base = 0; base < t.n_pages; base += STEP) {
        const int64_t first = base + threadIdx.x * kCounts;
        const uint32_t bits = base ? held_bits(t, first) : mine;
        int before = mine_before;  // pages in use before this one
        if (t.n_pages > STEP) {
            before = seen + plan_scan(__popc(bits), scratch, total);
            seen += total;
        }
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

// After the plan: table entries renamed by the first row_groups workgroups, pages copied by the others.
template <bool STREAM>
__global__ void __launch_bounds__(kThreads) pages_move_kernel(PageCompact a, PageArrays arrays, unsigned row_groups) {
    const PageTable &t = a.t;
    if (blockIdx.x >= row_groups) {
        copy_pairs<STREAM>(arrays, a.from, a.to, min(*a.moves, t.n_pages / 2), t.n_pages, blockIdx.x - row_groups,
                           gridDim.x - row_groups);
        return;
    }
    const unsigned strips = ((unsigned)t.n_cols + kThreads - 1) / kThreads;
    const int64_t c = (int64_t)(blockIdx.x % strips) * kThreads + threadIdx.x;
    if (c >= t.n_cols) return;
    int32_t *entry = t.table + (int64_t)(blockIdx.x / strips) * t.stride + c;
    const int page = *entry;
    if (page != -1) *entry = (uint32_t)page < (uint32_t)t.n_pages ? a.place[page] : -1;
}

unsigned strips_of(int n_cols) { return ((unsigned)n_cols + kThreads - 1) / kThreads; }

// Workgroups of a copy: a wave a unit, up to 32 workgroups a compute unit, whose
// waves then take several (8, 16 and 32 a compute unit: 512 pages of 344 KB in 77,
// 55 and 53 us).
unsigned copy_groups(int64_t items) {
    const int64_t groups = (items + kWaves - 1) / kWaves, most = 32 * 256;
    return (unsigned)(groups < most ? groups : most);
}


// More bytes than the eight L2s hold on either side of the copy: what is written
// passes through once.  512 pages of 344 KB, streaming accesses for nothing, what is
// written, what is read and both: 70, 55, 60 and 70 us.
bool streams(int64_t items) { return items * 64 * kLoads * 16 > (int64_t)32 << 20; }

}  // namespace

bool page_rows_fit(int n_cols, int64_t n) {
    return ((int64_t)strips_of(n_cols) * n + 32 * 256) * kThreads <= (int64_t)UINT32_MAX;
}

uint32_t page_units(int64_t bytes, int width) {
    const int64_t unit = (int64_t)64 * kLoads * width;
    return (uint32_t)((bytes + unit - 1) / unit);
}

hipError_t launch_pages_copy(const PageCopy &a, hipStream_t stream) {
    const int64_t items = (int64_t)a.n * a.arrays.units;
    if (streams(items))
        hipLaunchKernelGGL((pages_copy_kernel<true>), dim3(copy_groups(items)), dim3(kThreads), 0, stream, a);
    else
        hipLaunchKernelGGL((pages_copy_kernel<false>), dim3(copy_groups(items)), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_pages_fork_plan(const PageFork &a, hipStream_t stream) {
    hipLaunchKernelGGL(pages_fork_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_pages_fork(const PageFork &a, const PageArrays &arrays, bool rows, hipStream_t stream) {
    const unsigned row_groups = rows ? strips_of(a.t.n_cols) * (((unsigned)a.n + kGroup - 1) / kGroup) : 0u;
    const unsigned groups = row_groups + (arrays.units ? copy_groups((int64_t)a.n * arrays.units) : 0u);
    if (groups) hipLaunchKernelGGL(pages_fork_kernel, dim3(groups), dim3(kThreads), 0, stream, a, arrays, row_groups);
    return hipGetLastError();
}

hipError_t launch_pages_grow(const PageGrow &grow, hipStream_t stream) {
    PageGrow a = grow;
    const int64_t all = (int64_t)a.n * a.tokens;
    // few slots are written by the workgroup that decides: 4096 of one request in 7.8 us,
    // 8192 in 10.3 where two launches take 7.5, and 16384 in 15.5 where they take 7.7
    a.all = all <= 4 * kPlanThreads;
    hipLaunchKernelGGL(pages_grow_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a);
    if (!a.all) {
        const int64_t groups = (all + kThreads - 1) / kThreads;
        hipLaunchKernelGGL(pages_slots_kernel, dim3((unsigned)(groups < 2048 ? groups : 2048)), dim3(kThreads), 0, stream, a);
    }
    return hipGetLastError();
}

hipError_t launch_pages_free(const PageFree &a, hipStream_t stream) {
    const unsigned strips = a.t.n_cols ? strips_of(a.t.n_cols) : 1u;
    hipLaunchKernelGGL(pages_free_kernel, dim3(strips, (unsigned)a.n), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_pages_compact_plan(const PageCompact &a, hipStream_t stream) {
    hipLaunchKernelGGL(pages_compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_pages_move(const PageCompact &a, const PageArrays &arrays, bool rows, hipStream_t stream) {
    const unsigned row_groups = rows ? strips_of(a.t.n_cols) * (unsigned)a.t.n_rows : 0u;
    const int64_t items = (int64_t)(a.t.n_pages / 2) * arrays.units;
    const unsigned groups = row_groups + (items ? copy_groups(items) : 0u);
    if (!groups) return hipSuccess;
    if (streams(items))
        hipLaunchKernelGGL((pages_move_kernel<true>), dim3(groups), dim3(kThreads), 0, stream, a, arrays, row_groups);
    else
        hipLaunchKernelGGL((pages_move_kernel<false>), dim3(groups), dim3(kThreads), 0, stream, a, arrays, row_groups);
    return hipGetLastError();
}

}  // namespace lidx
