// Internal interface of the 4-bit cache operators (mx4_api.hip, mx4_cache.hip
// and the attention kernels).  Not exported.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace lidx {

// Division of a number below 2^31 by a fixed divisor d in [1, 2^31): with
// l = ceil(log2 d) and m = ceil(2^(31 + l) / d), m fits 32 bits and
// floor(n / d) = floor(n * m / 2^(31 + l)) for every n < 2^31 (Granlund and
// Montgomery, "Division by invariant integers using multiplication", with
// N = 31).
struct FastDiv {
    uint32_t d, m, s;
};

inline FastDiv fast_div(uint32_t d) {
    uint32_t l = 0;
    while ((1ull << l) < d) ++l;
    // d = 1: m = 2^31, one shift short of 32: floor(n * 2^31 / 2^31)
    const uint64_t m = ((1ull << (31 + l)) + d - 1) / d;
    return FastDiv{d, (uint32_t)m, l};
}

__device__ __forceinline__ uint32_t quotient(uint32_t n, const FastDiv &f) {
    return __umulhi(n << 1, f.m) >> f.s;
}

// The pages of one cache: strides in bytes, block ids below n_blocks.
struct Mx4Pages {
    int64_t d_sb, d_ss, d_sh;  // data: block, slot, head
    int64_t s_sb, s_ss, s_sh;  // scale
    int32_t n_blocks;
    int32_t block_size;
    FastDiv div_bs;
    int64_t n_slots;
    bool congruent;  // every scale stride is a sixteenth of the data stride
};

struct Mx4Write {
    const void *x[2];
    int64_t st[2], sh[2];
    uint8_t *data[2];
    uint8_t *scale[2];
    Mx4Pages pages;
    const int64_t *slots;
    int32_t n_tokens, n_heads, head_dim;
    int32_t n_tensors;
    FastDiv div_e, div_c;  // 8-value chunks of a token, and of a row
    bool bf16;
};

struct Mx4Read {
    const uint8_t *data, *scale;
    Mx4Pages pages;
    const int64_t *slots;
    void *out;
    int64_t st, sh;
    int32_t n_rows, n_heads, head_dim;
    FastDiv div_e, div_c;
    bool bf16;
};

hipError_t launch_mx4_write(const Mx4Write &a, hipStream_t stream);
hipError_t launch_mx4_read(const Mx4Read &a, hipStream_t stream);

struct Mx4Attend {
    const void *q;
    int64_t q_st, q_sh;
    const uint8_t *kd, *ks, *vd, *vs;
    Mx4Pages pages;
    const int32_t *block_table;
    int64_t bt_stride;
    const int32_t *seq_lens;
    int32_t n_requests, q_len, max_seq_len;
    int32_t n_heads, n_kv, group;
    float scale_log2;  // sm_scale * log2(e)
    // selected: idx != nullptr
    const int32_t *idx;
    int64_t idx_st;
    int32_t n_sel, pool;
    FastDiv div_pool, div_group, div_items, div_kv;
    // window
    int32_t window, sinks;
    void *out;
    int64_t out_st, out_sh;
    float *lse;
    // launch
    int32_t rows;       // n_requests * q_len
    int32_t units;      // row units: rows (selected) or requests (window)
    int32_t m_tiles;    // tiles of query rows per unit and K/V head
    int32_t n_splits;   // workgroups that share a tile's keys
    int32_t head_group; // groups of hp K/V heads a workgroup's waves are shared out to
    float *part_o;      // [rows][n_heads][n_splits][head_dim]
    float *part_ml;     // [rows][n_heads][n_splits][2]
};

constexpr int kMx4MaxSplits = 64;

// Threads of a workgroup of the wave-at-a-time form (hp K/V heads a wave), of
// the many-rows form and of the join.
constexpr int mx4_wave_threads(int head_dim, int hp) { return head_dim <= 128 && hp == 1 ? 512 : 256; }
constexpr int kMx4PromptThreads = 512, kMx4JoinThreads = 256;

// Launch geometry: how many 16-row tiles a wave holds and how many workgroups
// share a row's keys; a function of sizes alone.
struct Mx4Plan {
    bool prompt;  // 256 rows of a request a workgroup, going through the keys together
    bool share;   // the waves of a workgroup, on 8 K/V heads of a row, share their keys' scales (if the layout allows)
    int ahead;    // tiles whose codes a wave has on the way
    int mt, hp, m_tiles, n_splits, head_group, units;
    int threads;        // of a workgroup
    int64_t workgroups;
    size_t part_o_bytes, workspace_bytes;
    bool fits;          // both launches hold fewer than 2^32 threads, as a launch must
};
Mx4Plan plan_mx4_attend(int n_requests, int q_len, int64_t max_keys, bool selected, int n_heads, int n_kv,
                        int head_dim);
hipError_t launch_mx4_attend_f16(const Mx4Attend &a, const Mx4Plan &p, int head_dim, hipStream_t stream);
hipError_t launch_mx4_attend_bf16(const Mx4Attend &a, const Mx4Plan &p, int head_dim, hipStream_t stream);

}  // namespace lidx
