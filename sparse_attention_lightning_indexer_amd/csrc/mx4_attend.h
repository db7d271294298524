// Attention over the 4-bit cache for gfx950: the kernel, shared by its f16 and
// bf16 instances (mx4_attend_f16.hip, mx4_attend_bf16.hip).
//
// For a query row (token, head) and the positions p it attends to,
//   z[p] = c * q . K[p]   (c = sm_scale * log2 e),  out = sum 2^(z[p] - L) V[p],
//   L = log2 sum 2^z[p];  one pass with the running maximum m and sum l of a
// softmax, the accumulated product rescaled by 2^(m_old - m_new).
//
// A wave holds MT tiles of 16 query rows that share a K/V head and walks tiles
// of 32 keys of its own; the waves of a workgroup take the tiles of a row's
// keys in turn and join their (m, l, product) through LDS at the end, and rows
// with too few workgroups share their keys among several, joined by a second
// kernel.  Nothing in the loop waits for another wave, but for the barrier of a
// pair of tiles where waves share scales (below).
//
//  - Scores: S^T = K Q^T on 16x16x32 MFMAs.  The contraction runs over the
//    head dimension in any order both operands agree on, so a lane takes
//    head_dim / 4 consecutive values of its key (l & 15): one wide load of
//    codes and one scale byte (at head dimension 128, exactly one block).
//  - The conversion from 4 bits applies the scale and gives the query's type
//    exactly (caches written from it), two values an instruction.
//  - A lane then holds 8 scores of one query row, (l & 15), which is the
//    layout the product's P operand wants: P never leaves its lane, and
//    neither do m, l and the rescaling of O^T = V^T P^T.
//    The weights are rounded to the query's type there: the product takes both
//    operands in one type, and a second product with what the rounding left
//    would be half as many matrix instructions again.  Half a step of the type
//    each, averaged over the keys, is no more than the output's own rounding:
//    against 64 bits outputs are 1.1 to 1.4 times as far off as 32-bit sums
//    rounded once.  The weights' sum and everything else stays f32.
//  - V's rows are converted like K's, stored to the wave's own LDS rows and
//    read back transposed (ds_read_b64_tr_b16), 16 dimensions by 4 keys each.
//    Rows are padded by 32 bytes: the 8 consecutive rows that half a wave reads
//    32 bytes of, or writes 16 bytes of, then lie in different banks.  Conflicts
//    are still 0.39 of the cycles that LDS is active (shared scales, selected
//    keys; 0.16 in the many-rows kernel); which accesses they belong to was not
//    found out.
//  - Keys picked one by one come from beyond the L2s, in lines of 128 bytes: a
//    row of 4 bytes of scales costs what two rows of codes do.  Where the four
//    waves of a workgroup take the same keys of 8 K/V heads (SHARE), the scales
//    of all heads come in one load for 64 keys at a time, through LDS, one
//    barrier for them: 10 lines a key instead of up to 16.  1024 rows x 2048 of
//    131072 keys, 8 heads of 128: 450 us apart, 390-410 us shared, when 2.6 GB
//    pass the L2s at 6.4 TB/s; a plain read of 143 MB, the cache's size, which
//    the Infinity Cache holds, reaches 6.75, one of 4 GiB 6.3.
//  - Loads run ahead: a tile's codes from when the one before (PF = 2: two
//    before) is converted, the page ids a pair of tiles further, the selected
//    indices one more.
//
// Measured, 64 query heads on 8 K/V heads of 128: one row over 131072 keys 31 us
// (bf16, 4.6 TB/s: memory); 128 rows x 2048 keys of 32 requests 62 us (bf16, 4.7
// TB/s in gathered rows); 32 rows under a window of 1024 12.5 us and 32 rows x 512
// keys 9.5 us (f16: the latency of dependent loads and few tiles a wave).  What is
// loaded ahead is used as loaded, in a later tile (scale bytes as bytes), and q is
// known to have arrived before the loop: a value widened at once, or first used
// in the loop, has the compiler wait there for every load on the way
// (windows of head dimension 192 and 256 apart, see below).
//
// Masked positions: their scores become -inf by selection, so K's NaN there
// never spreads; V's blocks of NaN are replaced by zeros in the product, and
// the rows that do attend to such a key get their NaN by a mask of blocks
// (0 * NaN would otherwise reach rows that must not see the key).  Nor may V be
// infinite there: where a block's scale makes values that the type does not
// hold, its codes are written anew under the largest scale that does not, at
// most 6 times it.
#pragma once

#include <math.h>

#include <type_traits>

#include "device_common.h"
#include "mx4_internal.h"

namespace lidx {
namespace mx4 {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <bool BF16>
struct Type;
template <>
struct Type<false> {
    typedef half8 vec8;
    typedef _Float16 one;
    static constexpr uint32_t kTopScale = 140;  // 6 * 2^13 is the largest of this form the type holds
    static constexpr float kLift = 7.0f;
    static __device__ __forceinline__ f32x4 mfma(vec8 a, vec8 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    // 8 codes of one word under a scale
    static __device__ __forceinline__ vec8 from4(uint32_t w, float f) {
        u32x4 r;
        r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, f, 0));
        r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, f, 1));
        r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, f, 2));
        r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, f, 3));
        return __builtin_bit_cast(vec8, r);
    }
};
template <>
struct Type<true> {
    typedef bf8 vec8;
    typedef __bf16 one;
    static constexpr uint32_t kTopScale = 252;  // 6 * 2^125
    static constexpr float kLift = 0.0f;
    static __device__ __forceinline__ f32x4 mfma(vec8 a, vec8 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ vec8 from4(uint32_t w, float f) {
        u32x4 r;
        r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 0));
        r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 1));
        r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 2));
        r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 3));
        return __builtin_bit_cast(vec8, r);
    }
};

// The larger of two numbers (a NaN is passed over): the middle of them and
// infinity, one instruction where fmaxf takes three to quiet its operands.
__device__ __forceinline__ float larger(float a, float b) {
    return __builtin_amdgcn_fmed3f(a, b, __builtin_huge_valf());
}

// The codes of 8 values under a scale 2^steps times smaller, at most 6 times
// it.  A step takes the magnitudes 0, .5, 1, 1.5, 2, 3 to 0, 1, 2, 3, 4, 6, which
// is code + 2 from code 2 on and code 2 for 1, and the larger ones to 6, code 7.
__device__ __forceinline__ uint32_t larger_codes(uint32_t w, uint32_t steps) {
    uint32_t m = w & 0x77777777u;
    for (uint32_t i = min(steps, 4u); i; --i) {  // .5 passes 6 in four
        const uint32_t two = (m >> 1 | m >> 2) & 0x11111111u;  // code 2 on
        m += 2u * two + (m & ~two & 0x11111111u);
        m = (m | (m >> 3 & 0x11111111u) * 7u) & 0x77777777u;
    }
    return m | (w & 0x88888888u);
}

// Over the four lanes that share l & 15.
__device__ __forceinline__ float quarter_max(float v) {
    const unsigned u = __builtin_bit_cast(unsigned, v);
    auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const unsigned w = __builtin_bit_cast(
        unsigned, fmaxf(__builtin_bit_cast(float, (unsigned)a[0]), __builtin_bit_cast(float, (unsigned)a[1])));
    auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    return fmaxf(__builtin_bit_cast(float, (unsigned)b[0]), __builtin_bit_cast(float, (unsigned)b[1]));
}
__device__ __forceinline__ float quarter_sum(float v) {
    const unsigned u = __builtin_bit_cast(unsigned, v);
    auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const unsigned w = __builtin_bit_cast(
        unsigned, __builtin_bit_cast(float, (unsigned)a[0]) + __builtin_bit_cast(float, (unsigned)a[1]));
    auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    return __builtin_bit_cast(float, (unsigned)b[0]) + __builtin_bit_cast(float, (unsigned)b[1]);
}

// N (1 to 4) consecutive words to and from LDS, 16-byte aligned.
template <int N>
__device__ __forceinline__ void put_words(lds_u8 *dst, const uint32_t (&w)[N]) {
    typedef __attribute__((address_space(3))) u32x4 v4;
    typedef __attribute__((address_space(3))) u32x2 v2;
    typedef __attribute__((address_space(3))) uint32_t v1;
    if constexpr (N == 4) {
        *(v4 *)dst = u32x4{w[0], w[1], w[2], w[3]};
    } else {
        if constexpr (N >= 2) *(v2 *)dst = u32x2{w[0], w[1]};
        if constexpr (N % 2 == 1) *(v1 *)(dst + (N - 1) * 4) = w[N - 1];
    }
}
template <int N>
__device__ __forceinline__ void get_words(const lds_u8 *src, uint32_t (&w)[N]) {
    typedef const __attribute__((address_space(3))) u32x4 v4;
    typedef const __attribute__((address_space(3))) u32x2 v2;
    typedef const __attribute__((address_space(3))) uint32_t v1;
    if constexpr (N == 4) {
        const u32x4 v = *(v4 *)src;
        w[0] = v[0], w[1] = v[1], w[2] = v[2], w[3] = v[3];
    } else {
        if constexpr (N >= 2) {
            const u32x2 v = *(v2 *)src;
            w[0] = v[0], w[1] = v[1];
        }
        if constexpr (N % 2 == 1) w[N - 1] = *(v1 *)(src + (N - 1) * 4);
    }
}

constexpr float kNegInf = -__builtin_huge_valf();

// Weights stand against 2^kLift for the reference, of which their sum takes
// 2^kLift off again.  They stay below 2^8 of it, so f16, which ends at 2^16 and
// 2^-24, has room for 2^7: a weight is then lost below 2^-32 of the largest, not
// 2^-25.  (One key that leads 131071 others by 17.5 leaves them 0.33% of the
// weight, each 2^-25: as f16 against 1 all of them were 0.)  bf16 has f32's range.
//
// Weights are 2^(s c - m) with one rounding, m the rounded product of a largest
// score: the largest weight is then 2^r, r the rounding of m, which any sum of
// weights takes along.  From this |m| on, where r may pass an eighth (and at
// 2^32 a float's range), the product is rounded before m is taken off it, as it
// was for m.
constexpr float kFar = 2097152.0f;  // 2^21

template <int D, int HP>
struct Shape {
    static constexpr int KS = D / 32;               // MFMA steps over the head dimension
    static constexpr int NT = D / 16;               // 16-dimension tiles of the product
    static constexpr int UNITS = D <= 128 ? 4 : 8;  // 16-byte units of a key's codes in LDS
    static constexpr int ROW = 2 * D + 32;          // bytes of a V row in LDS
    static constexpr int WAVES = mx4_wave_threads(D, HP) / 64;
    static constexpr int KPL = 16 / HP, NU = 2 * HP;  // keys of a load, loads of a tile
    static constexpr int OROW = D + 4;              // floats of a row of the join (padded)
    static constexpr int JOIN = WAVES * 16 * OROW * 4;
    // a wave's rows; the second head's (HP = 2) begin 32 bytes later, in other banks
    static constexpr int SECOND = 16 * ROW + (HP == 2 ? 32 : 0);
    static constexpr int WSTAGE = 16 * ROW + SECOND;
    static constexpr int STAGE = WAVES * WSTAGE;
    static constexpr int LDS = (STAGE > JOIN ? STAGE : JOIN) + WAVES * 16 * 8;
};

// One workgroup's share of the work.
struct Item {
    int unit, kv, split, m0;  // row unit, K/V head, key share, first query row of its tile
};

__device__ __forceinline__ Item item_of(const Mx4Attend &a, int mt, int hp) {
    // Workgroups b, b + 8, b + 16, ... run on one XCD.  Piece w = (unit, row
    // tile, key share) runs on XCD w mod 8 for all its K/V heads, one after the
    // other, so the 128-byte lines the heads of a token share are fetched into
    // one L2.
    Item it;
    const uint32_t b = blockIdx.x >> 3;
    const uint32_t r = quotient(b, a.div_kv);  // groups of K/V heads
    it.kv = (int)(b - r * a.div_kv.d) * a.head_group * hp;
    const uint32_t w = r * 8u + (blockIdx.x & 7u);
    it.unit = (int)quotient(w, a.div_items);  // row tiles * key shares of a unit
    const uint32_t rest = w - (uint32_t)it.unit * a.div_items.d;
    const uint32_t tile = rest / (uint32_t)a.n_splits;
    it.split = (int)(rest - tile * (uint32_t)a.n_splits);
    it.m0 = (int)tile * 16 * mt;
    return it;
}

// What a row attends to: a window (or everything), selected keys, selected
// runs of `pool` keys; of requests that share a prefix, their own keys behind
// it, or the prefix's (a unit is then a group of requests).
enum Mode { kWindow = 0, kKeys = 1, kPools = 2, kOwn = 3, kPrefix = 4 };

// The requests of a group that share a prefix, and the prefix's length.
struct Group {
    int first, count, prefix;
};
__device__ __forceinline__ Group group_at(const Mx4Attend &a, int g) {
    Group r{0, a.n_requests, min(max(a.prefix_lens[g], 0), a.max_prefix)};
    if (a.group_starts) {
        r.first = min(max(a.group_starts[g], 0), a.n_requests);
        r.count = min(max(a.group_starts[g + 1], r.first), a.n_requests) - r.first;
    }
    return r;
}
// The group of a request: the last that begins at or before it; of no request
// and no prefix if there is none or it ends before.  Lanes look at a start
// each, with the length and the end that may be wanted, so this is one round
// trip to memory.  All lanes are active.
__device__ __forceinline__ Group group_of(const Mx4Attend &a, int request) {
    if (!a.group_starts) return a.n_groups ? group_at(a, 0) : Group{request, 0, 0};
    Group r{request, 0, 0};
    const int lane = threadIdx.x & 63;
    for (int base = 0; base < a.n_groups; base += 64) {
        const int g = min(base + lane, a.n_groups - 1);
        const int start = a.group_starts[g], end = a.group_starts[g + 1], prefix = a.prefix_lens[g];
        const int upto = __popcll(__ballot(base + lane < a.n_groups && start <= request));
        if (upto) {
            r.first = max(__builtin_amdgcn_readlane(start, upto - 1), 0);
            r.count = min(__builtin_amdgcn_readlane(end, upto - 1), a.n_requests) - r.first;
            r.prefix = min(max(__builtin_amdgcn_readlane(prefix, upto - 1), 0), a.max_prefix);
        }
        if (upto < 64) break;
    }
    // (of starts that do not ascend the first one may lie past the request)
    if (r.count <= 0 || request < r.first || request - r.first >= r.count) r = Group{request, 0, 0};
    return r;
}

// Waves per SIMD the registers have to leave room for.  Three (168 registers) are
// not quite enough for two K/V heads a wave at head dimension 128 with selected
// keys of their own in f16 (8 bytes a lane in scratch) and at 96 (8 to 16 bytes).
template <int D, int MT, int HP, int PF>
constexpr int waves_per_simd() {
    if (PF == 2) return 2;
    return HP == 2 ? 3 : (MT == 1 && D <= 128 ? 4 : (MT == 2 && D == 256 ? 1 : 2));
}

template <int N>
struct Set {
    static constexpr int value = N;
};

template <bool BF16, int D, int MT, int HP, int PF, int MODE, bool SHARE>
__global__ void __launch_bounds__((Shape<D, HP>::WAVES * 64), (waves_per_simd<D, MT, HP, PF>())) mx4_attend_kernel(Mx4Attend a) {
    static_assert(HP == 1 || MT == 1, "pairs of heads have one tile of rows");
    static_assert(HP == 1 || PF == 1, "a pair's second 16 keys are asked for late");
    static_assert(!SHARE || (HP == 2 && (MODE == kKeys || MODE == kPools) && (D == 64 || D == 128)), "shared scales: pairs of heads of selected rows");
    using T = Type<BF16>;
    using S = Shape<D, HP>;
    typedef typename T::vec8 vec8;
    constexpr int KS = S::KS, NT = S::NT, W = S::WAVES, NU = S::NU, KPL = S::KPL;
    constexpr bool SELECTED = MODE == kKeys || MODE == kPools;
    __shared__ __attribute__((aligned(16))) unsigned char smem[S::LDS];
    // SHARE: the scales of a pair of tiles and of the one after, of all the
    // workgroup's heads: 16-byte parts of K's, then of V's, each for the 64 keys
    constexpr int PARTS = D / 64;
    __shared__ u32x4 scales[SHARE ? 2 : 1][SHARE ? 2 * PARTS : 1][64];

    Item it = item_of(a, MT, HP);
    if (it.unit >= a.units) return;
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
    // the waves: head_group groups of HP K/V heads, and for each of them
    // `stride` waves that take its tiles in turn
    const int stride = W / a.head_group, turn = wave / a.head_group;
    const int first_kv = it.kv;
    it.kv += (wave - turn * a.head_group) * HP;
    const int col = lane & 15, qd = lane >> 4;
    // HP = 2: columns 0-7 are query rows of the first head, 8-15 of the second
    const int hcol = HP == 2 ? col >> 3 : 0, mcol = HP == 2 ? col & 7 : col;

    // the unit's request, query rows and visible keys
    Group group{};
    if (MODE == kPrefix) group = group_at(a, it.unit);
    if (MODE == kPrefix && it.m0 >= group.count * a.q_len * a.group) return;
    const int req = SELECTED ? it.unit / a.q_len : (MODE == kPrefix ? group.first : it.unit);
    const int seq = a.seq_lens[req];
    // query rows of the unit at this K/V head
    const int n_m = SELECTED ? a.group : (MODE == kPrefix ? group.count * a.q_len * a.group : a.q_len * a.group);
    if (MODE == kOwn) group = group_of(a, req);
    const int prefix = group.prefix;
    const int own_from = MODE == kOwn && !a.whole ? prefix : 0;  // where the row's keys begin
    auto token_of = [&](int m) { return SELECTED ? it.unit : req * a.q_len + (int)quotient((uint32_t)m, a.div_group); };
    auto head_in = [&](int kv, int m) {
        return kv * a.group + (SELECTED ? m : m - (int)quotient((uint32_t)m, a.div_group) * a.group);
    };
    // keys a token sees, before the cap by max_seq_len
    auto seen_of = [&](int token) -> int64_t {
        if (MODE != kPrefix) return (int64_t)seq - a.q_len + 1 + (token - req * a.q_len);
        const int r = (int)quotient((uint32_t)token, a.div_q);
        return min((int64_t)a.seq_lens[r] - a.q_len + 1 + (token - r * a.q_len), (int64_t)prefix);
    };
    const int64_t first_seen = MODE == kPrefix ? 0 : seen_of(token_of(it.m0));
    const int64_t last_seen = MODE == kPrefix ? prefix : seen_of(token_of(min(it.m0 + 16 * MT, n_m) - 1));
    int cap_first = (int)max((int64_t)0, min(first_seen, (int64_t)a.max_seq_len));  // kPrefix: known below
    const int cap_last = (int)max((int64_t)0, min(last_seen, (int64_t)a.max_seq_len));

    // tiles of 32 keys: selected entries in order; or the first tokens, then the window
    int n_tiles, sink_tiles = 0, base = 0;
    if (SELECTED) {
        n_tiles = cap_last > 0 ? (int)(((int64_t)a.n_sel * a.pool + 31) / 32) : 0;
    } else if (MODE >= kOwn) {
        if (MODE == kOwn) base = min(own_from, cap_last) & ~31;
        n_tiles = (cap_last - base + 31) / 32;
    } else {
        int64_t lo = a.window ? first_seen - a.window : 0;
        base = lo > 0 ? (int)min(lo, (int64_t)cap_last) & ~31 : 0;
        sink_tiles = (min(a.sinks, base) + 31) / 32;
        if (!a.window) sink_tiles = 0;
        n_tiles = sink_tiles + (cap_last - base + 31) / 32;
    }
    if (a.pages.n_blocks == 0) n_tiles = 0;
    const int per = (n_tiles + a.n_splits - 1) / a.n_splits;
    const int t_end = min(n_tiles, (it.split + 1) * per);
    const int t_begin = it.split * per + turn;

    // per query-row tile: this lane's column of Q (its row's values in the
    // order of the lane's part of the contraction), and the row's window
    vec8 q[MT][KS];
    int row_end[MT], row_start[MT];
    float mx[MT], ls[MT];
    float limit[MT];  // the score past which the reference is looked at again
    f32x4 o[MT][NT];
    uint32_t nan_blocks[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        limit[mt] = kNegInf;
        const int mc = min(it.m0 + mt * 16 + mcol, n_m - 1);
        const int token = token_of(mc);
        const uint4 *src = reinterpret_cast<const uint4 *>((const uint16_t *)a.q + (int64_t)token * a.q_st +
                                                           (int64_t)head_in(it.kv + hcol, mc) * a.q_sh + qd * (KS * 8));
#pragma unroll
        for (int s = 0; s < KS; ++s) q[mt][s] = __builtin_bit_cast(vec8, src[s]);
        const int64_t seen = seen_of(token);
        row_end[mt] = (int)max((int64_t)0, min(seen, (int64_t)a.max_seq_len));
        row_start[mt] = a.window ? (int)min(max((int64_t)0, seen - a.window), (int64_t)row_end[mt]) : 0;
        if (MODE >= kOwn) row_start[mt] = own_from;
        mx[mt] = kNegInf;
        ls[mt] = 0.0f;
        nan_blocks[mt] = 0u;
#pragma unroll
        for (int n = 0; n < NT; ++n) o[mt][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    if (MODE == kOwn && a.finish && group.count) {
        // the prefix's shares of a row, computed before: the waves that take its keys begin with
        // some of them each, instead of with nothing
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int mc = min(it.m0 + mt * 16 + mcol, n_m - 1);
            const int64_t th = (int64_t)token_of(mc) * a.n_heads + head_in(it.kv + hcol, mc);
            const float *ml = a.part_ml + th * a.shares * 2, *po = a.part_o + th * a.shares * D + qd * 4;
            for (int s = turn; s < a.prefix_shares; s += stride) {
                const float m = ml[s * 2], l = ml[s * 2 + 1];
                f32x4 x[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) x[n] = *reinterpret_cast<const f32x4 *>(po + (int64_t)s * D + n * 16);
                const float top = fmaxf(mx[mt], m), sub = top == kNegInf ? 0.0f : top;
                const float f = __builtin_amdgcn_exp2f(mx[mt] - sub), g = __builtin_amdgcn_exp2f(m - sub);
                mx[mt] = top;
                ls[mt] = ls[mt] * f + (qd == 0 ? l * g : 0.0f);  // the lanes' sums are added at the end
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[mt][n][i] = o[mt][n][i] * f + x[n][i] * g;
            }
            if (mx[mt] != kNegInf && fabsf(mx[mt]) < kFar) limit[mt] = mx[mt] + 8.0f;
        }
    }
    if (MODE == kPrefix) {
        uint32_t least = (uint32_t)row_end[0];
        if (MT == 2) least = min(least, (uint32_t)row_end[MT - 1]);
        cap_first = (int)wave_min_u32(least);
    }

    // A tile's 32 keys are the rows of score tiles 0 and 1 (keys `row` and 16 +
    // row of the tile).  Four neighbouring lanes load a key's row, a quarter
    // each (HP = 2: eight lanes the rows of both heads), so that their 16-byte
    // loads fall into one line; where the lanes of one row were 16 apart, as the
    // products want them, a load instruction took four times the line lookups.
    // Load u takes keys u * KPL + krow.  Finding the rows is shared: of the 64
    // keys of two tiles (this one and the wave's next) each lane finds one, and
    // the others ask it for the offset.
    const int krow = lane >> (HP + 1), ch = lane & 3, hsel = HP == 2 ? (lane >> 2) & 1 : 0;
    const uint64_t head_d = (uint64_t)((uint32_t)it.kv * (uint32_t)a.pages.d_sh);
    const uint32_t head_s = (uint32_t)it.kv * (uint32_t)a.pages.s_sh;
    const uint8_t *kd = a.kd + head_d, *vd = a.vd + head_d, *ks = a.ks + head_s, *vs = a.vs + head_s;
    const int32_t *table = a.block_table + (int64_t)req * a.bt_stride;
    const int32_t *sel = SELECTED ? a.idx + (int64_t)it.unit * a.idx_st : nullptr;
    const uint32_t end_entry = SELECTED ? min((uint32_t)a.n_sel * (uint32_t)a.pool, (uint32_t)t_end * 32u) : 0u;
    const uint32_t end_unit = MODE == kPools ? (uint32_t)(cap_last + a.pool - 1) / (uint32_t)a.pool : 0u;
    const uint32_t own_tile = (uint32_t)((qd >> 1) * stride), own_key = (uint32_t)((qd & 1) * 16 + col);

    // The steps from a pair of tiles to its offsets.  Each loads from a place
    // that exists whatever the lane's key (a clamped entry, page 0 of the table,
    // slot 0 of the cache), so none branches on a key and the loads of a step
    // overlap (`congruent` is one branch of the whole wave); a position of -1 and
    // the bits of `found` say what counts.
    // 1: the entry's selected index
    auto load_index = [&](int tile) -> int {
        const uint32_t e = ((uint32_t)tile + own_tile) * 32u + own_key;
        return sel[min(MODE == kPools ? quotient(min(e, 0x7fffffffu), a.div_pool) : e, (uint32_t)a.n_sel - 1u)];
    };
    // 2: the position
    auto position = [&](int tile, int id) -> int {
        const uint32_t mine = (uint32_t)tile + own_tile;
        const uint32_t e = mine * 32u + own_key;
        if (MODE == kKeys) return e < end_entry && (uint32_t)id < (uint32_t)cap_last ? id : -1;
        if (MODE == kPools) {
            const uint32_t u = e - quotient(min(e, 0x7fffffffu), a.div_pool) * (uint32_t)a.pool;
            const uint32_t p = (uint32_t)id * (uint32_t)a.pool + u;
            return e < end_entry && (uint32_t)id < end_unit && p < (uint32_t)cap_last ? (int)p : -1;
        }
        const uint32_t p = (mine < (uint32_t)sink_tiles ? 0u : (uint32_t)(base - sink_tiles * 32)) + e;
        return mine < (uint32_t)t_end && p < (uint32_t)cap_last ? (int)p : -1;
    };
    // 3: its page's id
    const int32_t *shared_table = a.block_table + (int64_t)group.first * a.bt_stride;
    auto load_page = [&](int p) -> int {
        if (MODE == kOwn) return (p < prefix ? shared_table : table)[quotient((uint32_t)max(p, 0), a.pages.div_bs)];
        return table[quotient((uint32_t)max(p, 0), a.pages.div_bs)];
    };
    // 4: where its row begins, in data and (unless that is a sixteenth of it) scale bytes
    uint64_t at = 0, sat = 0, found = 0;
    auto locate = [&](int p, int page) {
        const bool ok = p >= 0 && (uint32_t)page < (uint32_t)a.pages.n_blocks;
        const uint32_t q = (uint32_t)max(p, 0);
        const uint32_t off = q - __umul24(quotient(q, a.pages.div_bs), (uint32_t)a.pages.block_size);
        const uint32_t o = ok ? off : 0u, pg = ok ? (uint32_t)page : 0u;
        at = (uint64_t)pg * (uint32_t)a.pages.d_sb + __umul24(o, (uint32_t)a.pages.d_ss);
        if (!a.pages.congruent) sat = (uint64_t)pg * (uint32_t)a.pages.s_sb + __umul24(o, (uint32_t)a.pages.s_ss);
        found = __ballot(ok);
    };
    auto ask_lane = [&](uint64_t v, int from) -> uint64_t {
        const uint32_t lo = (uint32_t)__builtin_amdgcn_ds_bpermute(from * 4, (int)(uint32_t)v);
        const uint32_t hi = (uint32_t)__builtin_amdgcn_ds_bpermute(from * 4, (int)(uint32_t)(v >> 32));
        return ((uint64_t)hi << 32) | lo;
    };
    // from the lane that found this lane's key of load u of tile `b` of the pair
    auto ask = [&](uint64_t v, int b, int u) -> uint64_t { return ask_lane(v, b * 32 + u * KPL + krow); };
    // 5: the codes and scales.  The KS words (8 values each) of quarter c lie in
    // blocks (c * KS + s) / 4: at most NB of them
    constexpr int NB = KS % 4 == 0 ? KS / 4 : (KS == 2 ? 1 : 2);
    constexpr int ALIGN = KS % 4 == 0 ? 16 : (KS % 2 == 0 ? 8 : 4);
    // Scales stay bytes until they are used: widening them at once would wait for them
    // there.  Windows of head dimension 192 and 256 are quicker with words and without
    // the wait for q below: full attention of 126 x 2 tokens over 4584 keys at 192 218 us
    // for 247, 36 x 4 over 21189 at 256 201 for 223, 16 x 100 over 20088 at 256 2449 for
    // 2559 (selected keys at 192 are 2% slower so in f16).
    constexpr bool WIDEN = D >= 192 && MODE == kWindow;
    struct Raw {
        uint32_t k[KS], v[KS];
        typename std::conditional<WIDEN, uint32_t, uint8_t>::type sk[NB], sv[NB];
    };
    const int blk0 = ch * KS / 4;
    const uint64_t chunk = (uint64_t)((uint32_t)hsel * (uint32_t)a.pages.d_sh) + (uint32_t)(ch * KS * 4);
    const uint64_t schunk = (uint64_t)((uint32_t)hsel * (uint32_t)a.pages.s_sh) + (uint32_t)blk0;
    Raw raw[PF][NU];    // PF = 2: of the wave's even and odd tiles
    uint32_t have[PF];  // the keys that count: bit k is key k of the tile
    // K's part of load u, V's, or both, of tile b of the pair
    auto load_rows = [&](Raw (&raw)[NU], int b, int u, bool k, bool v) {
        const uint64_t row = ask(at, b, u), d = row + chunk;
        if (k) __builtin_memcpy(raw[u].k, __builtin_assume_aligned(kd + d, ALIGN), KS * 4);
        if (v) __builtin_memcpy(raw[u].v, __builtin_assume_aligned(vd + d, ALIGN), KS * 4);
        if (SHARE) return;
        const uint64_t sc = (a.pages.congruent ? row >> 4 : ask(sat, b, u)) + schunk;
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            // the last block of a row again where the lane has fewer than NB
            const uint32_t more = NB * 4 == KS || NB == 1 ? (uint32_t)n : (uint32_t)(min(blk0 + n, D / 32 - 1) - blk0);
            if (k) raw[u].sk[n] = ks[sc + more];
            if (v) raw[u].sv[n] = vs[sc + more];
        }
    };
    // SHARE: thread (key, part) of the workgroup asks for its part of the
    // scales of the pair that was located last, and puts it into LDS
    u32x4 part = {0u, 0u, 0u, 0u};
    const int part_key = (int)threadIdx.x / (2 * PARTS), part_of = (int)threadIdx.x % (2 * PARTS);
    auto load_part = [&]() {
        const uint64_t row = ask_lane(a.pages.congruent ? at >> 4 : sat, part_key & 63);
        const uint8_t *src = (part_of < PARTS ? a.ks : a.vs) + (uint32_t)first_kv * (uint32_t)a.pages.s_sh;
        part = *reinterpret_cast<const u32x4 *>(src + row + (part_of & (PARTS - 1)) * 16);
    };
    auto store_part = [&](int buffer) {
        if (2 * PARTS * 64 == W * 64 || part_key < 64) scales[buffer][part_of][part_key & 63] = part;
    };
    // the byte of block `blk` of the workgroup's head `hd` (tensor 0: K, 1: V)
    auto shared_scale = [&](int buffer, int tensor, int key, int hd, int blk) -> uint32_t {
        const int byte = hd * (D / 32) + blk;
        return ((const __attribute__((address_space(3))) uint8_t *)&scales[buffer][tensor * PARTS + (byte >> 4)][key])[byte & 15];
    };
    int buffer = 0;
    // which of the blocks of quarter c its word s belongs to
    auto block_of = [&](int c, int s) { return KS % 4 == 0 ? s / 4 : (KS == 2 ? 0 : (c * KS + s) / 4 - c * KS / 4); };

    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
    lds_u8 *stage = (lds_u8 *)smem + wave * S::WSTAGE;
    // K's codes change lanes through the same LDS rows before V needs them:
    // units of 16 bytes, swapped inside a row so that the 8 lanes of an access
    // meet different banks
    auto unit_at = [&](int row, int unit) {
        return S::UNITS == 4 ? row * 64 + ((unit ^ ((row >> 2) & 3)) * 16) : row * 128 + ((unit ^ ((row >> 1) & 7)) * 16);
    };

    // four keys of 16 dimensions, transposed, and the four 16 rows on
    auto two_reads = [&](lds_u8 *src) -> vec8 {
        union {
            s16x4 h[2];
            vec8 v;
        } vt;
        vt.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)src);
        vt.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(src + S::SECOND));
        return vt.v;
    };

    int id = -1, pos = -1, page = -1;
    const bool any_tile = t_begin < t_end;
    if (any_tile) {
        if (SELECTED) id = load_index(t_begin);
        pos = position(t_begin, id);
        page = load_page(pos);
    }
    // q, asked for before, has arrived when the first page's id has.  Said here,
    // else its first use, which is in the loop, waits there for all loads on the
    // way in every tile
    if (!WIDEN) wait_vmem_all_known();
    if (any_tile) {
        locate(pos, page);
        if (SHARE) load_part();
#pragma unroll
        for (int b = 0; b < PF; ++b) {
            have[b] = (uint32_t)(found >> (b * 32));
#pragma unroll
            for (int u = 0; u < NU; ++u) load_rows(raw[b], b, u, true, true);
        }
        auto following = [&](int tile) {
            if (SELECTED) id = load_index(tile);
            pos = position(tile, id);
            page = load_page(pos);
        };
        following(t_begin + 2 * stride);
        if (PF == 2) {
            locate(pos, page);
            following(t_begin + 4 * stride);
        }
        if (SELECTED) id = load_index(t_begin + (PF == 2 ? 6 : 4) * stride);
        if (SHARE) {
            store_part(0);
            __syncthreads();
        }
    }

    // one tile: `b` is its place in its pair, SET where its codes are
    auto multiply = [&](auto set, int b, int tile) __attribute__((always_inline)) {
        constexpr int SET = decltype(set)::value;
        Raw(&raw_)[NU] = raw[SET];
        const uint32_t valid = have[SET];
        const int p0 = SELECTED ? 0 : (tile < sink_tiles ? tile * 32 : base + (tile - sink_tiles) * 32);
        bool whole = valid == 0xffffffffu;
        if (MODE >= kOwn) {
            whole = whole && p0 + 32 <= cap_first && p0 >= own_from;
        } else if (!SELECTED) {
            whole = whole && p0 + 32 <= cap_first &&
                    (!a.window || p0 + 32 <= a.sinks || (int64_t)p0 >= last_seen - a.window);
        }
        // whether key k of the tile counts for this lane's query row
        auto counts = [&](int mt, int k) -> bool {
            bool in = (valid >> k) & 1u;
            if (!SELECTED) {
                const int p = p0 + k;
                in = in && p < row_end[mt] && (p >= row_start[mt] || p < a.sinks);
            }
            return in;
        };

        uint32_t sv[NU][NB];
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
            for (int n = 0; n < NB; ++n) sv[u][n] = SHARE ? 0u : raw_[u].sv[n];
        if (SHARE) {
#pragma unroll
            for (int u = 0; u < NU; ++u)
                sv[u][0] = shared_scale(buffer, 1, b * 32 + u * KPL + krow, it.kv - first_kv + hsel, blk0);
        }
        // V's scales: 0 for keys that do not count; rarely, 0 for blocks of NaN,
        // with a mark for the rows that do attend to such a block, and at most
        // the type's largest
        bool bad = false;
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
            for (int n = 0; n < NB; ++n) bad |= sv[u][n] > T::kTopScale;
        if (valid != 0xffffffffu) {
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                const bool in = (valid >> (u * KPL + krow)) & 1u;
#pragma unroll
                for (int n = 0; n < NB; ++n) sv[u][n] = in ? sv[u][n] : 0u;
            }
        }
        if (__ballot(bad)) {
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                uint32_t mine = 0;  // blocks of NaN in this lane's part of its key
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    if (sv[u][n] == 255u) {
                        mine |= 1u << min(blk0 + n, D / 32 - 1);
                        sv[u][n] = 0u;
                    }
                    if (sv[u][n] > T::kTopScale) {
#pragma unroll
                        for (int st = 0; st < KS; ++st)
                            if (block_of(ch, st) == n)
                                raw_[u].v[st] = larger_codes(raw_[u].v[st], sv[u][n] - T::kTopScale);
                        sv[u][n] = T::kTopScale;
                    }
                }
                if (__ballot(mine != 0u)) {
                    for (int row = 0; row < KPL; ++row) {
                        uint32_t blocks[2] = {0u, 0u};
#pragma unroll
                        for (int g = 0; g < 4 * HP; ++g)
                            blocks[g >> 2] |= (uint32_t)__builtin_amdgcn_readlane((int)mine, row * 4 * HP + g);
                        if (!(blocks[0] | blocks[1])) continue;
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
                            if (counts(mt, u * KPL + row)) nan_blocks[mt] |= hcol ? blocks[1] : blocks[0];
                    }
                }
            }
        }

        // K's codes and scales to the lanes that multiply them: quarter qd of row
        // col (a quarter of more than 4 words is two units)
        constexpr int K1 = KS < 4 ? KS : 4, K2 = KS > 4 ? KS - 4 : 1, U = S::UNITS, TILE = 16 * 16 * U, HEAD = 2 * TILE + 128;
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            const int key = u * KPL + krow;  // key >> 4 is the same in all lanes
            lds_u8 *dst = stage + hsel * HEAD + (u * KPL >> 4) * TILE;
            uint32_t w1[K1], w2[K2];
#pragma unroll
            for (int i = 0; i < K1; ++i) w1[i] = raw_[u].k[i];
            put_words<K1>(dst + unit_at(key & 15, U == 4 ? ch : ch * 2), w1);
            if constexpr (KS > 4) {
#pragma unroll
                for (int i = 0; i < K2; ++i) w2[i] = raw_[u].k[4 + i];
                put_words<K2>(dst + unit_at(key & 15, ch * 2 + 1), w2);
            }
        }
        // scales, a byte per load in one word: lane (row, head, quarter) has them
        uint32_t pack[NB];
#pragma unroll
        for (int n = 0; n < (SHARE ? 0 : NB); ++n) {
            pack[n] = raw_[0].sk[n];
#pragma unroll
            for (int u = 1; u < NU; ++u) pack[n] |= (uint32_t)raw_[u].sk[n] << (8 * u);
        }

        // scores: of each head with all columns, then each column its head's
        f32x4 s[MT][2];
#pragma unroll
        for (int hh = 0; hh < HP; ++hh) {
            uint32_t sk[NB];
#pragma unroll
            for (int n = 0; n < (SHARE ? 0 : NB); ++n) {
                const int who = ((col & (KPL - 1)) * 4 * HP + hh * 4 + qd) * 4;
                sk[n] = (uint32_t)__builtin_amdgcn_ds_bpermute(who, (int)pack[n]) >> (HP == 2 ? 8 * hcol : 0);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                uint32_t kc[KS], w1[K1], w2[K2], shared_k = 0;
                if (SHARE) shared_k = shared_scale(buffer, 0, b * 32 + u * 16 + col, it.kv - first_kv + hh, qd * KS / 4);
                const lds_u8 *src = stage + hh * HEAD + u * TILE;
                get_words<K1>(src + unit_at(col, U == 4 ? qd : qd * 2), w1);
#pragma unroll
                for (int i = 0; i < K1; ++i) kc[i] = w1[i];
                if constexpr (KS > 4) {
                    get_words<K2>(src + unit_at(col, qd * 2 + 1), w2);
#pragma unroll
                    for (int i = 0; i < K2; ++i) kc[4 + i] = w2[i];
                }
                f32x4 sum[MT];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) sum[mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int st = 0; st < KS; ++st) {
                    uint32_t sb;
                    if constexpr (SHARE) {
                        sb = shared_k;
                    } else {
                        sb = sk[0];
#pragma unroll
                        for (int b = 1; b < NB; ++b) sb = block_of(qd, st) == b ? sk[b] : sb;
                        sb = (sb >> (8 * HP * u)) & 255u;
                    }
                    const vec8 kv = T::from4(kc[st], __builtin_bit_cast(float, sb << 23));
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) sum[mt] = T::mfma(kv, q[mt][st], sum[mt]);
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[mt][u][i] = hh == 0 || hcol ? sum[mt][i] : s[mt][u][i];
            }
        }

        // V's rows into the wave's LDS: all of them, or (HP = 2) 16 keys of both
        // heads, the other 16 when these are used up
        auto store_v = [&](int u) {
#pragma unroll
            for (int st = 0; st < KS; ++st) {
                uint32_t sb = sv[u][0];
#pragma unroll
                for (int b = 1; b < NB; ++b) sb = block_of(ch, st) == b ? sv[u][b] : sb;
                const vec8 vv = T::from4(raw_[u].v[st], __builtin_bit_cast(float, sb << 23));
                lds_u8 *row = stage + (HP == 2 ? hsel * S::SECOND + ((u & 1) * KPL + krow) * S::ROW
                                               : (u * KPL + krow) * S::ROW);
                *(lds_u32x4 *)(row + (ch * KS + st) * 16) = __builtin_bit_cast(u32x4, vv);
            }
        };
        store_v(0);
        store_v(1);

        // the codes of the tile PF on, into the registers this one's came from;
        // after the pair's last of these the offsets of the pair after, and the
        // page ids of the one after that, and the indices of the next
        const int nb = PF == 2 ? b : b ^ 1;
        have[SET] = (uint32_t)(found >> (nb * 32));
#pragma unroll
        for (int u = 0; u < NU; ++u) load_rows(raw_, nb, u, true, u < 2);
        auto advance = [&]() {
            if (nb == 0) return;
            const int first = tile - b * stride;  // of this pair
            locate(pos, page);
            if (SHARE) load_part();
            pos = position(first + (PF == 2 ? 6 : 4) * stride, id);
            page = load_page(pos);
            if (SELECTED) id = load_index(first + (PF == 2 ? 8 : 6) * stride);
        };
        if (HP == 1) advance();

        if (!whole) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s[mt][u][i] = counts(mt, u * 16 + 4 * qd + i) ? s[mt][u][i] : kNegInf;
        }

        // softmax.  The reference m of a row is a maximum so far, the same in its
        // four lanes; it moves only when a score passes it by 2^8, so weights
        // stay below 2^(8 + kLift) (kFar: and an eighth) and the rescaling is rare
        vec8 p[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma clang fp contract(off)
            float top = larger(s[mt][0][0], s[mt][0][1]);
            top = larger(larger(top, s[mt][0][2]), s[mt][0][3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) top = larger(top, s[mt][1][i]);
            top *= a.scale_log2;
            float times = a.scale_log2, plus = T::kLift - (mx[mt] == kNegInf ? 0.0f : mx[mt]);
            if (__ballot(top > limit[mt])) {
                const float m_new = larger(mx[mt], quarter_max(top));
                const float f = m_new > mx[mt] ? __builtin_amdgcn_exp2f(mx[mt] - m_new) : 1.0f;
                mx[mt] = m_new;
                ls[mt] *= f;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[mt][n][i] *= f;
                const bool near = fabsf(m_new) < kFar;
                limit[mt] = near ? m_new + 8.0f : kNegInf;
                const float sub = m_new == kNegInf ? 0.0f : m_new;
                plus = T::kLift - sub;
                if (__ballot(!near && m_new != kNegInf)) {
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[mt][u][i] = s[mt][u][i] * times - sub;
                    times = 1.0f;
                    plus = T::kLift;
                }
            }
            float sum = 0.0f;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[mt][u][i], times, plus));
                    sum += e;
                    p[mt][u * 4 + i] = (typename T::one)e;
                }
            ls[mt] += sum;
        }

        // O^T += V^T P^T.  HP = 2: a product over 16 keys of both heads, with
        // zeros for P where a column is the other head's
        if constexpr (HP == 1) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const vec8 vt = two_reads(stage + (4 * qd + (col >> 2)) * S::ROW + n * 32 + (col & 3) * 8);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) o[mt][n] = T::mfma(vt, p[mt], o[mt][n]);
            }
        } else {
            const u32x4 pw = __builtin_bit_cast(u32x4, p[0]);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (t) {
                    store_v(2);
                    store_v(3);
                    load_rows(raw_, nb, 2, false, true);
                    load_rows(raw_, nb, 3, false, true);
                    advance();
                }
                const vec8 pt = __builtin_bit_cast(vec8, u32x4{hcol ? 0u : pw[2 * t], hcol ? 0u : pw[2 * t + 1],
                                                               hcol ? pw[2 * t] : 0u, hcol ? pw[2 * t + 1] : 0u});
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const vec8 vt = two_reads(stage + (4 * qd + (col >> 2)) * S::ROW + n * 32 + (col & 3) * 8);
                    o[0][n] = T::mfma(vt, pt, o[0][n]);
                }
            }
        }
    };
    if constexpr (PF == 2) {
        for (int tile = t_begin; tile < t_end; tile += 2 * stride) {
            multiply(Set<0>{}, 0, tile);
            if (tile + stride < t_end) multiply(Set<1>{}, 1, tile + stride);
        }
    } else {
        int odd = 0;
        for (int tile = t_begin; tile < t_end; tile += stride, odd ^= 1) {
            multiply(Set<0>{}, odd, tile);
            if (SHARE && odd) {  // the same tiles in every wave; nobody reads the other buffer any more
                store_part(buffer ^= 1);
                __syncthreads();
            }
        }
    }

    // join the waves: each writes its product, m and l; every thread then adds
    // up a share of the outputs
    float *jo = reinterpret_cast<float *>(smem);
    float *jml = reinterpret_cast<float *>(smem + (S::STAGE > S::JOIN ? S::STAGE : S::JOIN));
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const float l = quarter_sum(ls[mt]);
        __syncthreads();  // the staging rows, or the last tile's join, are no longer read
        float *dst = jo + (wave * 16 + col) * S::OROW;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            f32x4 v = o[mt][n];
            if ((nan_blocks[mt] >> (n / 2)) & 1u) v = f32x4{NAN, NAN, NAN, NAN};
            *reinterpret_cast<f32x4 *>(dst + n * 16 + qd * 4) = v;
        }
        if (qd == 0) {
            jml[(wave * 16 + col) * 2] = mx[mt];
            jml[(wave * 16 + col) * 2 + 1] = l;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < a.head_group * 16 * (D / 8); e += W * 64) {
            const int hrow = e / (D / 8), c = e - hrow * (D / 8);
            const int hg = hrow >> 4, row = hrow & 15;
            const int m = HP == 2 ? row & 7 : it.m0 + mt * 16 + row;
            if (m >= n_m) continue;
            const float *ml = jml + (hg * 16 + row) * 2, *src = jo + (hg * 16 + row) * S::OROW + c * 8;
            const int step = a.head_group * 16;  // to the next wave of this head
            float m_all = kNegInf;
            for (int w = 0; w < stride; ++w) m_all = fmaxf(m_all, ml[w * step * 2]);
            const int token = token_of(m), head = head_in(first_kv + hg * HP + (HP == 2 ? row >> 3 : 0), m);
            const int64_t th = (int64_t)token * a.n_heads + head;
            const float sub = m_all == kNegInf ? 0.0f : m_all;
            float l_all = 0.0f, acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
            for (int w = 0; w < stride; ++w) {
                const float f = __builtin_amdgcn_exp2f(ml[w * step * 2] - sub);
                l_all += f * ml[w * step * 2 + 1];
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] += f * src[w * step * S::OROW + i];
            }
            if (MODE == kPrefix || (MODE == kOwn ? !a.finish : a.n_splits > 1)) {
                const int64_t share = MODE >= kOwn ? th * a.shares + a.first_share + it.split : th * a.n_splits + it.split;
                float *dst2 = a.part_o + share * D + c * 8;
                *reinterpret_cast<f32x4 *>(dst2) = f32x4{acc[0], acc[1], acc[2], acc[3]};
                *reinterpret_cast<f32x4 *>(dst2 + 4) = f32x4{acc[4], acc[5], acc[6], acc[7]};
                if (c == 0) {
                    a.part_ml[share * 2] = m_all;
                    a.part_ml[share * 2 + 1] = l_all;
                }
            } else {
                const float inv = l_all == 0.0f ? 0.0f : 1.0f / l_all;
                vec8 r;
#pragma unroll
                for (int i = 0; i < 8; ++i) r[i] = (typename T::one)(acc[i] * inv);
                *reinterpret_cast<vec8 *>((uint16_t *)a.out + (int64_t)token * a.out_st + (int64_t)head * a.out_sh +
                                          c * 8) = r;
                if (c == 0 && a.lse)
                    a.lse[th] = l_all == 0.0f ? kNegInf : (m_all + (log2f(l_all) - T::kLift)) * 0.69314718055994530942f;
            }
        }
    }
}

// Many query rows of a request at one K/V head (a prompt's, or a chunk's) under
// a window: 256 rows a workgroup, 32 a wave, and the workgroup goes through the
// keys together, 64 at a time.  Each key is converted once for the 256 rows: a
// thread converts 32 values of K or of V and stores them to LDS in the query's
// type, where every wave reads the tile as the products' operand (V transposed,
// as above).  Converting in every wave was 64 of the about 200 vector
// instructions a wave spent on 32 rows and 32 keys, against 32 products.
//
// Two buffers, one barrier a step: after it a thread converts its part of the
// next step into the other buffer, asks for the codes of the step after and the
// page id of the one after that, and the wave multiplies.  A wave passes over
// steps that none of its rows sees.  The maximum is looked for only where the
// weights' sum says that the reference is too low (a weight past about 2^8 of
// it), or no key was seen yet, or the reference is past kFar; otherwise weights
// cost one multiply-add, one exponential and one addition each.
//
// Per key of a buffer a word says what is unusual: bit 31 a page outside the
// cache, bits 0-7 blocks of V that are NaN (stored as zeros; the rows that see
// the key get their NaN at the end).
//
// Measured, 64 query heads on 8 K/V heads of 128: 1024 causal tokens over 16384
// keys 482 us (f16, 1.11 PFLOP/s, where an 8192-cubed library product reaches
// 1.14), 1000 tokens under a window of 4096 141 us a call with other inputs between
// (bf16, 0.96 PFLOP/s).  Before the loads of a step ran through the step (see
// above) and K's rows were read 16 keys ahead of their products: 511 and 149 us.
// 32 requests of 64 heads over 131072 keys that they share: 64 steps in 130 us,
// 1.95 GHz, the matrix units busy for 44% of the cycles and the vector units for
// 40 to 50%, with two waves a SIMD to overlap them; half of the waves a product
// behind the others, so that they would meet different units, is slower (155 us
// where all together take 150).
template <int D>
struct PromptShape {
    static constexpr int MT = 2, W = kMx4PromptThreads / 64, KEYS = 64, ROWS = W * 16 * MT;
    static constexpr int ROW = 2 * D + 32;
    static constexpr int BUFFER = 2 * KEYS * ROW;  // K, then V
};

template <bool BF16, int D, int MODE = kWindow>
__global__ void __launch_bounds__(kMx4PromptThreads, 2) mx4_prompt_kernel(Mx4Attend a) {
    using T = Type<BF16>;
    using P = PromptShape<D>;
    typedef typename T::vec8 vec8;
    constexpr int KS = D / 32, NT = D / 16, MT = P::MT, KEYS = P::KEYS, ROW = P::ROW;
    constexpr float kMostSum = BF16 ? 0x1p8f : 0x1p15f;  // 2^(8 + kLift)
    __shared__ __attribute__((aligned(16))) unsigned char smem[2 * P::BUFFER];
    __shared__ uint32_t unusual[2][KEYS];
    __shared__ __attribute__((aligned(16))) uint32_t any[2][4];

    Item it = item_of(a, P::ROWS / 16, 1);
    if (it.unit >= a.units) return;
    it.m0 = (a.m_tiles - 1) * P::ROWS - it.m0;  // the rows with the most keys first
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
    const int col = lane & 15, qd = lane >> 4;
    Group group{};
    if (MODE == kPrefix) group = group_at(a, it.unit);
    const int req = MODE == kPrefix ? group.first : it.unit;
    const int n_m = MODE == kPrefix ? group.count * a.q_len * a.group : a.q_len * a.group;
    if (MODE == kPrefix && it.m0 >= n_m) return;
    const int seq = a.seq_lens[req];
    if (MODE == kOwn) group = group_of(a, req);
    const int prefix = group.prefix;
    const int own_from = MODE == kOwn && !a.whole ? prefix : 0;
    auto token_in = [&](int m) { return (int)quotient((uint32_t)m, a.div_group); };  // of the request, or its group
    auto seen_of = [&](int m) -> int64_t {
        if (MODE != kPrefix) return (int64_t)seq - a.q_len + 1 + token_in(min(m, n_m - 1));
        const int t = token_in(min(m, n_m - 1)), r = (int)quotient((uint32_t)t, a.div_q);
        return min((int64_t)a.seq_lens[req + r] - a.q_len + 1 + (t - r * a.q_len), (int64_t)prefix);
    };
    auto capped = [&](int64_t v) { return (int)max((int64_t)0, min(v, (int64_t)a.max_seq_len)); };

    // the workgroup's keys: steps of 64, the first tokens and then the window
    const int64_t first_seen = MODE >= kOwn ? 0 : seen_of(it.m0);
    const int cap_last = capped(MODE == kPrefix ? prefix : seen_of(it.m0 + P::ROWS - 1));
    const int64_t lo = MODE >= kOwn ? own_from : (a.window ? first_seen - a.window : 0);
    const int base = lo > 0 ? (int)min(lo, (int64_t)cap_last) & ~(KEYS - 1) : 0;
    const int sink_steps = MODE < kOwn && a.window ? (min(a.sinks, base) + KEYS - 1) / KEYS : 0;
    int n_steps = sink_steps + (cap_last - base + KEYS - 1) / KEYS;
    if (a.pages.n_blocks == 0) n_steps = 0;
    const int per = (n_steps + a.n_splits - 1) / a.n_splits;
    const int s_begin = it.split * per, s_end = min(n_steps, s_begin + per);
    auto start_of = [&](int step) { return step < sink_steps ? step * KEYS : base + (step - sink_steps) * KEYS; };

    // the wave's rows
    const int m0 = it.m0 + wave * 16 * MT;
    int cap_first_w = MODE == kPrefix ? 0 : capped(seen_of(m0));  // kPrefix: known below
    const int cap_last_w = m0 < n_m ? capped(MODE == kPrefix ? prefix : seen_of(m0 + 16 * MT - 1)) : 0;
    const int64_t first_w = MODE >= kOwn ? 0 : seen_of(m0) - a.window;
    const int64_t last_w = MODE >= kOwn ? 0 : seen_of(m0 + 16 * MT - 1) - a.window;
    vec8 q[MT][KS];
    int row_end[MT], row_start[MT];
    float mx[MT], ls[MT];
    float limit[MT];  // weights' sum past which the reference is looked at again; -1: always (none yet, or past kFar)
    f32x4 o[MT][NT];
    uint32_t nan_blocks[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        limit[mt] = -1.0f;
        const int m = min(m0 + mt * 16 + col, n_m - 1), t = token_in(m);
        const uint4 *src = reinterpret_cast<const uint4 *>(
            (const uint16_t *)a.q + (int64_t)(req * a.q_len + t) * a.q_st +
            (int64_t)(it.kv * a.group + m - t * a.group) * a.q_sh + qd * 8);
#pragma unroll
        for (int st = 0; st < KS; ++st) q[mt][st] = __builtin_bit_cast(vec8, src[st * 4]);
        const int64_t seen = seen_of(m);
        row_end[mt] = capped(seen);
        row_start[mt] = a.window ? (int)min(max((int64_t)0, seen - a.window), (int64_t)row_end[mt]) : 0;
        if (MODE >= kOwn) row_start[mt] = own_from;
        mx[mt] = kNegInf;
        ls[mt] = 0.0f;
        nan_blocks[mt] = 0u;
#pragma unroll
        for (int n = 0; n < NT; ++n) o[mt][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    if (MODE == kPrefix) cap_first_w = (int)wave_min_u32((uint32_t)min(row_end[0], row_end[1]));

    // the thread's part of a step: quarter ch of one key's K (waves 0-3) or V
    const bool is_v = wave >= 4;
    const int key = (threadIdx.x & 255) >> 2, ch = lane & 3;
    constexpr int NB = KS % 4 == 0 ? KS / 4 : (KS == 2 ? 1 : 2);
    constexpr int ALIGN = KS % 4 == 0 ? 16 : (KS % 2 == 0 ? 8 : 4);
    const int blk0 = ch * KS / 4;
    const uint8_t *src_d = (is_v ? a.vd : a.kd) + (uint64_t)((uint32_t)it.kv * (uint32_t)a.pages.d_sh);
    const uint8_t *src_s = (is_v ? a.vs : a.ks) + (uint64_t)((uint32_t)it.kv * (uint32_t)a.pages.s_sh);
    const int32_t *table = a.block_table + (int64_t)req * a.bt_stride;
    uint32_t code[KS];
    uint8_t loaded_sc[NB];  // bytes until they are used: widening them at once would wait for them there
    bool seen_key = false, bad_page = false;
    // position of the thread's key in a step; -1 past the end
    auto position = [&](int step) {
        const int64_t p = (int64_t)start_of(step) + key;
        return step < s_end && p < cap_last ? (int)p : -1;
    };
    const int32_t *shared_table = a.block_table + (int64_t)group.first * a.bt_stride;
    auto load_page = [&](int p) -> int {
        if (MODE == kOwn) return (p < prefix ? shared_table : table)[quotient((uint32_t)max(p, 0), a.pages.div_bs)];
        return table[quotient((uint32_t)max(p, 0), a.pages.div_bs)];
    };
    auto load_codes = [&](int p, int page) {
        const bool in = (uint32_t)page < (uint32_t)a.pages.n_blocks;
        seen_key = p >= 0 && in;
        bad_page = p >= 0 && !in;
        const uint32_t r = (uint32_t)max(p, 0);
        const uint32_t off = r - __umul24(quotient(r, a.pages.div_bs), (uint32_t)a.pages.block_size);
        const uint32_t at = seen_key ? off : 0u, pg = seen_key ? (uint32_t)page : 0u;
        const uint64_t d = (uint64_t)pg * (uint32_t)a.pages.d_sb + __umul24(at, (uint32_t)a.pages.d_ss) + ch * KS * 4;
        const uint64_t sb = (uint64_t)pg * (uint32_t)a.pages.s_sb + __umul24(at, (uint32_t)a.pages.s_ss);
        __builtin_memcpy(code, __builtin_assume_aligned(src_d + d, ALIGN), KS * 4);
#pragma unroll
        for (int n = 0; n < NB; ++n) loaded_sc[n] = src_s[sb + (uint32_t)min(blk0 + n, D / 32 - 1)];
    };
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
    auto store_step = [&](int buf) {
        uint32_t word = bad_page ? 0x80000000u : 0u, sc[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n) sc[n] = loaded_sc[n];
        if (is_v) {
            bool bad = false;
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                sc[n] = seen_key ? sc[n] : 0u;
                bad |= sc[n] > T::kTopScale;
            }
            if (__ballot(bad)) {
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    if (sc[n] == 255u) {
                        word |= 1u << min(blk0 + n, D / 32 - 1);
                        sc[n] = 0u;
                    }
                    if (sc[n] > T::kTopScale) {
#pragma unroll
                        for (int st = 0; st < KS; ++st)
                            if ((ch * KS + st) / 4 - blk0 == n) code[st] = larger_codes(code[st], sc[n] - T::kTopScale);
                        sc[n] = T::kTopScale;
                    }
                }
            }
            word |= (uint32_t)dpp_move<0xb1>(0, (int)word);
            word |= (uint32_t)dpp_move<0x4e>(0, (int)word);
            if (ch == 0) unusual[buf][key] = word;
            const bool some = __ballot(word != 0u) != 0;
            if (lane == 0) any[buf][wave - 4] = some;
        }
        lds_u8 *dst = (lds_u8 *)smem + buf * P::BUFFER + (is_v ? KEYS * ROW : 0) + key * ROW;
#pragma unroll
        for (int st = 0; st < KS; ++st) {
            uint32_t b = sc[0];
#pragma unroll
            for (int n = 1; n < NB; ++n) b = (ch * KS + st) / 4 - blk0 == n ? sc[n] : b;
            const vec8 v = T::from4(code[st], __builtin_bit_cast(float, b << 23));
            *(lds_u32x4 *)(dst + (ch * KS + st) * 16) = __builtin_bit_cast(u32x4, v);
        }
    };

    // q, asked for before the first page's id, has arrived when that has.  Said
    // here, else its first use, which is in the loop, waits there in every step
    // for all loads on the way, the codes of the next among them
    int pos = -1, page = -1;
    const bool any_step = s_begin < s_end;
    if (any_step) {
        pos = position(s_begin);
        page = load_page(pos);
    }
    wait_vmem_all_known();
    if (any_step) {
        load_codes(pos, page);
        pos = position(s_begin + 1);
        page = load_page(pos);
        store_step(0);
        load_codes(pos, page);
        pos = position(s_begin + 2);
        page = load_page(pos);
    }
    for (int step = s_begin; step < s_end; ++step) {
        const int buf = (step - s_begin) & 1;
        lds_barrier();
        if (step + 1 < s_end) {
            store_step(buf ^ 1);
            load_codes(pos, page);
            pos = position(step + 3);
            page = load_page(pos);
        }
        const int p0 = start_of(step);
        // none of the wave's rows sees a key of this step
        if (p0 >= cap_last_w || (MODE < kOwn && a.window && p0 + KEYS <= first_w && p0 >= a.sinks)) continue;
        const lds_u8 *kb = (const lds_u8 *)smem + buf * P::BUFFER;
        // scores, the operands of 16 keys read while the products of the 16 before run
        f32x4 s[MT][4];
        u32x4 kf[2][KS];
        auto read_keys = [&](int u) {
#pragma unroll
            for (int st = 0; st < KS; ++st)
                kf[u & 1][st] = *(const lds_u32x4 *)(kb + (u * 16 + col) * ROW + (st * 4 + qd) * 16);
        };
        read_keys(0);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (u < 3) read_keys(u + 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) s[mt][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int st = 0; st < KS; ++st)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    s[mt][u] = T::mfma(__builtin_bit_cast(vec8, kf[u & 1][st]), q[mt][st], s[mt][u]);
            __builtin_amdgcn_sched_barrier(0);
        }
        const uint32_t odd = any[buf][0] | any[buf][1] | any[buf][2] | any[buf][3];
        const bool strange = uni((int)odd) != 0;
        const bool whole = !strange && p0 + KEYS <= cap_first_w &&
                           (MODE >= kOwn ? p0 >= own_from
                                         : !a.window || p0 + KEYS <= a.sinks || (int64_t)p0 >= last_w);
        auto counts = [&](int mt, int k) -> bool {
            const int p = p0 + k;
            return p < row_end[mt] && (p >= row_start[mt] || p < a.sinks) && !(unusual[buf][k] >> 31);
        };
        if (strange) {
            for (int k = 0; k < KEYS; ++k) {
                const uint32_t word = unusual[buf][k];
                if (!(word & 0xffu)) continue;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    if (counts(mt, k)) nan_blocks[mt] |= word & 0xffu;
            }
        }

        if (!whole) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s[mt][u][i] = counts(mt, u * 16 + 4 * qd + i) ? s[mt][u][i] : kNegInf;
        }

        // softmax
        vec8 p[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma clang fp contract(off)
            auto weigh = [&](auto rounded) {
                const float sub = mx[mt] == kNegInf ? 0.0f : mx[mt], plus = T::kLift - sub;
                float sum = 0.0f;
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float e = __builtin_amdgcn_exp2f(
                            decltype(rounded)::value ? s[mt][u][i] * a.scale_log2 - sub + T::kLift
                                                     : __builtin_fmaf(s[mt][u][i], a.scale_log2, plus));
                        sum += e;
                        p[mt][u >> 1][(u & 1) * 4 + i] = (typename T::one)e;
                    }
                return sum;
            };
            float sum = weigh(Set<0>{});
            if (__ballot(sum > limit[mt])) {
                float top = s[mt][0][0];
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) top = larger(top, s[mt][u][i]);
                const float m_new = larger(mx[mt], quarter_max(top) * a.scale_log2);
                const float f = m_new > mx[mt] ? __builtin_amdgcn_exp2f(mx[mt] - m_new) : 1.0f;
                mx[mt] = m_new;
                ls[mt] *= f;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[mt][n][i] *= f;
                const bool near = fabsf(m_new) < kFar;
                limit[mt] = near ? kMostSum : -1.0f;
                if (__ballot(!near && m_new != kNegInf))
                    sum = weigh(Set<1>{});
                else
                    sum = weigh(Set<0>{});
            }
            ls[mt] += sum;
        }

        // O^T += V^T P^T
        const lds_u8 *vb = kb + KEYS * ROW + (4 * qd + (col >> 2)) * ROW + (col & 3) * 8;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                union {
                    s16x4 h[2];
                    vec8 v;
                } vt;
                vt.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(vb + h * 32 * ROW + n * 32));
                vt.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(vb + (h * 32 + 16) * ROW + n * 32));
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) o[mt][n] = T::mfma(vt.v, p[mt][h], o[mt][n]);
            }
    }

    // a lane has 4 consecutive outputs of its row in each 16
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int m = m0 + mt * 16 + col;
        const float l = quarter_sum(ls[mt]);
        if (m >= n_m) continue;
        const int t = token_in(m), token = req * a.q_len + t, head = it.kv * a.group + m - t * a.group;
        const int64_t th = (int64_t)token * a.n_heads + head;
        const int64_t share = MODE >= kOwn ? th * a.shares + a.first_share + it.split : th * a.n_splits + it.split;
        const bool partial = MODE == kPrefix || (MODE == kOwn ? !a.finish : a.n_splits > 1);
        const float inv = partial ? 1.0f : (l == 0.0f ? 0.0f : 1.0f / l);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            f32x4 v = o[mt][n];
            if ((nan_blocks[mt] >> (n / 2)) & 1u) v = f32x4{NAN, NAN, NAN, NAN};
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] *= inv;
            if (partial) {
                *reinterpret_cast<f32x4 *>(a.part_o + share * D + n * 16 + qd * 4) = v;
            } else {
                typename T::one r[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) r[i] = (typename T::one)v[i];
                uint2 w;
                __builtin_memcpy(&w, r, 8);
                *reinterpret_cast<uint2 *>((uint16_t *)a.out + (int64_t)token * a.out_st + (int64_t)head * a.out_sh +
                                           n * 16 + qd * 4) = w;
            }
        }
        if (qd) continue;
        if (partial) {
            a.part_ml[share * 2] = mx[mt];
            a.part_ml[share * 2 + 1] = l;
        } else if (a.lse) {
            a.lse[th] = l == 0.0f ? kNegInf : (mx[mt] + (log2f(l) - T::kLift)) * 0.69314718055994530942f;
        }
    }
}

// Joins the shares of rows whose keys were split (at most kMx4MaxSplits): a workgroup per
// query row and head.  Threads take 4 outputs of every 1024 / D-th share, so
// the loads of a row's shares overlap, and add up through LDS.  Latency: 32
// shares of 64 heads of 128 take 4.7 us, most of it the launch and two dependent
// rounds of loads.
template <bool BF16, int D, bool SHARED = false>
__global__ void __launch_bounds__(kMx4JoinThreads) mx4_join_kernel(Mx4Attend a) {
    using T = Type<BF16>;
    typedef typename T::vec8 vec8;
    constexpr int C = D / 4, G = kMx4JoinThreads / C;  // chunks of 4 outputs, shares in flight
    __shared__ float weight[kMx4MaxSplits], total[1];
    static_assert(kMx4MaxSplits <= 64, "a lane per share");
    __shared__ __attribute__((aligned(16))) float part[G][D];
    const int64_t th = blockIdx.x;
    // SHARED: the prefix's shares, of a row whose request has one, then its own keys'
    int n_shares = a.n_splits, skip = 0;
    if (SHARED) {
        n_shares = a.shares;
        if (a.prefix_shares && !group_of(a, (int)(th / a.n_heads / a.q_len)).count) skip = a.prefix_shares;
    }
    const int c = threadIdx.x % C, g = threadIdx.x / C;
    const float *po = a.part_o + th * n_shares * D + c * 4;
    if (threadIdx.x < 64) {
        const float *ml = a.part_ml + th * n_shares * 2;
        const bool has = (int)threadIdx.x < n_shares && (int)threadIdx.x >= skip;
        const float m = has ? ml[2 * threadIdx.x] : kNegInf;
        float l = has ? ml[2 * threadIdx.x + 1] : 0.0f;
        float m_all = m;
        for (int d = 32; d; d >>= 1) m_all = fmaxf(m_all, __shfl_xor(m_all, d));
        const float f = __builtin_amdgcn_exp2f(m - (m_all == kNegInf ? 0.0f : m_all));
        l *= f;
        for (int d = 32; d; d >>= 1) l += __shfl_xor(l, d);
        weight[threadIdx.x] = f;
        if (threadIdx.x == 0) {
            total[0] = l;
            if (a.lse) a.lse[th] = l == 0.0f ? kNegInf : (m_all + (log2f(l) - T::kLift)) * 0.69314718055994530942f;
        }
    }
    __syncthreads();
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    if (g < G) {
#pragma unroll 4
        for (int s = skip + g; s < n_shares; s += G) {
            const f32x4 x = *reinterpret_cast<const f32x4 *>(po + (int64_t)s * D);
            const float f = weight[s];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] += f * x[i];
        }
        *reinterpret_cast<f32x4 *>(&part[g][c * 4]) = acc;
    }
    __syncthreads();
    if (threadIdx.x >= D / 8) return;
    const float inv = total[0] == 0.0f ? 0.0f : 1.0f / total[0];
    vec8 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < G; ++k) v += part[k][threadIdx.x * 8 + i];
        r[i] = (typename T::one)(v * inv);
    }
    const int64_t token = th / a.n_heads;
    const int head = (int)(th - token * a.n_heads);
    *reinterpret_cast<vec8 *>((uint16_t *)a.out + token * a.out_st + (int64_t)head * a.out_sh + threadIdx.x * 8) = r;
}

template <bool BF16, int D, int MT, int HP, int PF, bool SHARE = false>
hipError_t launch_tiles(const Mx4Attend &a, const Mx4Plan &p, hipStream_t stream) {
    const dim3 grid((unsigned)p.workgroups), block(Shape<D, HP>::WAVES * 64);
    if (!a.idx)
        hipLaunchKernelGGL((mx4_attend_kernel<BF16, D, MT, HP, PF, kWindow, false>), grid, block, 0, stream, a);
    else if (a.pool == 1)
        hipLaunchKernelGGL((mx4_attend_kernel<BF16, D, MT, HP, PF, kKeys, SHARE>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((mx4_attend_kernel<BF16, D, MT, HP, PF, kPools, SHARE>), grid, block, 0, stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.n_splits == 1) return e;
    hipLaunchKernelGGL((mx4_join_kernel<BF16, D>), dim3((unsigned)(a.rows * a.n_heads)), dim3(kMx4JoinThreads), 0, stream, a);
    return hipGetLastError();
}

template <bool BF16, int D>
hipError_t launch_dim(const Mx4Attend &a, const Mx4Plan &p, hipStream_t stream) {
    if constexpr (D <= 128) {
        if (p.prompt) {
            hipLaunchKernelGGL((mx4_prompt_kernel<BF16, D>), dim3((unsigned)p.workgroups), dim3(kMx4PromptThreads), 0, stream, a);
            hipError_t e = hipGetLastError();
            if (e != hipSuccess || a.n_splits == 1) return e;
            hipLaunchKernelGGL((mx4_join_kernel<BF16, D>), dim3((unsigned)(a.rows * a.n_heads)), dim3(kMx4JoinThreads), 0, stream,
                               a);
            return hipGetLastError();
        }
        if constexpr (D != 96) {
            if (p.share) return launch_tiles<BF16, D, 1, 2, 1, true>(a, p, stream);
        }
        if (p.hp == 2) return launch_tiles<BF16, D, 1, 2, 1>(a, p, stream);
    }
    if constexpr (D <= 128) {
        if (p.ahead == 2) return launch_tiles<BF16, D, 1, 1, 2>(a, p, stream);
    }
    if (p.mt == 1) return launch_tiles<BF16, D, 1, 1, 1>(a, p, stream);
    return launch_tiles<BF16, D, 2, 1, 1>(a, p, stream);
}

// Requests that share a prefix: the keys of one of the two parts of a row.
template <bool BF16, int D, int MODE>
hipError_t launch_part(const Mx4Attend &a, const Mx4Plan &p, hipStream_t stream) {
    const dim3 grid((unsigned)p.workgroups);
    if constexpr (D <= 128) {
        if (p.prompt) {
            hipLaunchKernelGGL((mx4_prompt_kernel<BF16, D, MODE>), grid, dim3(kMx4PromptThreads), 0, stream, a);
            return hipGetLastError();
        }
        if (p.hp == 2) {
            hipLaunchKernelGGL((mx4_attend_kernel<BF16, D, 1, 2, 1, MODE, false>), grid, dim3(Shape<D, 2>::WAVES * 64), 0,
                               stream, a);
            return hipGetLastError();
        }
        if (p.ahead == 2) {
            hipLaunchKernelGGL((mx4_attend_kernel<BF16, D, 1, 1, 2, MODE, false>), grid, dim3(Shape<D, 1>::WAVES * 64), 0,
                               stream, a);
            return hipGetLastError();
        }
    }
    if (p.mt == 1)
        hipLaunchKernelGGL((mx4_attend_kernel<BF16, D, 1, 1, 1, MODE, false>), grid, dim3(Shape<D, 1>::WAVES * 64), 0, stream, a);
    else
        hipLaunchKernelGGL((mx4_attend_kernel<BF16, D, 2, 1, 1, MODE, false>), grid, dim3(Shape<D, 1>::WAVES * 64), 0, stream, a);
    return hipGetLastError();
}

// The launch fields of one part.
inline Mx4Attend part_of(Mx4Attend a, const Mx4Plan &p, int first_share) {
    a.units = p.units;
    a.m_tiles = p.m_tiles;
    a.n_splits = p.n_splits;
    a.head_group = p.head_group;
    a.div_kv = fast_div((uint32_t)(a.n_kv / (p.hp * p.head_group)));
    a.div_items = fast_div((uint32_t)(p.m_tiles * p.n_splits));
    a.first_share = first_share;
    return a;
}

template <bool BF16, int D>
hipError_t launch_shared_dim(const Mx4Attend &a, const Mx4SharedPlan &p, hipStream_t stream) {
    if (a.prefix_shares) {
        const hipError_t e = launch_part<BF16, D, kPrefix>(part_of(a, p.prefix, 0), p.prefix, stream);
        if (e != hipSuccess) return e;
    }
    const hipError_t e = launch_part<BF16, D, kOwn>(part_of(a, p.own, a.prefix_shares), p.own, stream);
    if (e != hipSuccess || a.finish) return e;
    hipLaunchKernelGGL((mx4_join_kernel<BF16, D, true>), dim3((unsigned)(a.rows * a.n_heads)), dim3(kMx4JoinThreads), 0, stream,
                       a);
    return hipGetLastError();
}

template <bool BF16>
hipError_t launch_shared(const Mx4Attend &a, const Mx4SharedPlan &p, int head_dim, hipStream_t stream) {
    switch (head_dim) {
        case 64: return launch_shared_dim<BF16, 64>(a, p, stream);
        case 96: return launch_shared_dim<BF16, 96>(a, p, stream);
        case 128: return launch_shared_dim<BF16, 128>(a, p, stream);
        case 192: return launch_shared_dim<BF16, 192>(a, p, stream);
        case 256: return launch_shared_dim<BF16, 256>(a, p, stream);
        default: return hipErrorInvalidValue;
    }
}

template <bool BF16>
hipError_t launch_attend(const Mx4Attend &a, const Mx4Plan &p, int head_dim, hipStream_t stream) {
    switch (head_dim) {
        case 64: return launch_dim<BF16, 64>(a, p, stream);
        case 96: return launch_dim<BF16, 96>(a, p, stream);
        case 128: return launch_dim<BF16, 128>(a, p, stream);
        case 192: return launch_dim<BF16, 192>(a, p, stream);
        case 256: return launch_dim<BF16, 256>(a, p, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace mx4
}  // namespace lidx
