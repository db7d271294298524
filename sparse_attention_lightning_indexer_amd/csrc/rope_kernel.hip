// Head norms and rotation by position for gfx950: queries and keys as the
// indexer, the cache's writer and the attention take them.
//
// A row (a token's head) is read once and written once, so this is
// memory-bound: 4 bytes a value.  `lanes` neighbouring lanes hold a row, each
// VEC pairs as one wide load of first and one of second values (for pairs of
// neighbours one of whole pairs from each half of the row), so a rotation never
// leaves its lane and the norm is a sum over `lanes` lanes by lane moves (4096
// tokens of 128 + 16 heads of 128: 49 us either way; neighbours as two consecutive
// loads 62).  A wave takes a token (or
// with few tokens some of its rows) and has kBatch steps of 64 / lanes rows on
// the way; rows, weights, positions and frequencies are asked for together.
//
// The angles depend on the token and the pair alone: a wave computes its
// token's sines and cosines once, one or two pairs a lane, and its rows read
// them from LDS.  angle = position * frequency is formed in f64 as turns and
// reduced to half a turn there; position 131071 at frequency 1 in f32 would be
// off by 2^-8 radians, and a table of sines would be read again for every token.
//
// Measured: 16384 tokens of 64 + 8 heads of 128 in bf16 102 us (5.9 TB/s; a copy of
// 1 GiB reaches 5.1), 4001 tokens of 16 + 16 heads of 80 with three axes 12.6 us, 32
// tokens of 64 + 8 heads 3.7 us.  With weights loaded value by value and the choice
// between q's and k's arguments left to a load 162, 24 and 6 us.
#include "device_common.h"
#include "rope_internal.h"

namespace lidx {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = kRopeThreads / 64;
constexpr int kBatch = 4;  // steps whose rows a wave has on the way

template <int VEC>
struct Words {
    typedef u32x4 type;
};
template <>
struct Words<4> {
    typedef u32x2 type;
};

template <bool BF16>
__device__ __forceinline__ float widen(uint32_t word, int half) {
    if (BF16) return __builtin_bit_cast(float, half ? word & 0xffff0000u : word << 16);
    const uint16_t h = (uint16_t)(half ? word >> 16 : word);
    return (float)__builtin_bit_cast(_Float16, h);
}
template <bool BF16>
__device__ __forceinline__ uint32_t narrow(float lo, float hi) {
    if (BF16) {
        const __bf16 a = (__bf16)lo, b = (__bf16)hi;
        return (uint32_t)__builtin_bit_cast(uint16_t, a) | (uint32_t)__builtin_bit_cast(uint16_t, b) << 16;
    }
    const _Float16 a = (_Float16)lo, b = (_Float16)hi;
    return (uint32_t)__builtin_bit_cast(uint16_t, a) | (uint32_t)__builtin_bit_cast(uint16_t, b) << 16;
}

// A kernel argument in scalar registers.  Of a choice between two arguments by
// the lane the compiler would otherwise make a load from the arguments' memory
// at an address of the lane's, and wait for it.
__device__ __forceinline__ int64_t held(int64_t v) {
    asm("" : "+s"(v));
    return v;
}
__device__ __forceinline__ const void *held(const void *p) { return (const void *)held((int64_t)p); }

// The sum over the LANES lanes of a row, in every one of them.
template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
    auto add = [](float a, int b) { return a + __builtin_bit_cast(float, b); };
    auto bits = [](float a) { return __builtin_bit_cast(int, a); };
    if (LANES >= 2) v = add(v, dpp_move<0xb1>(0, bits(v)));
    if (LANES >= 4) v = add(v, dpp_move<0x4e>(0, bits(v)));
    if (LANES >= 8) v = add(v, dpp_move<0x141>(0, bits(v)));   // row_half_mirror
    if (LANES >= 16) v = add(v, dpp_move<0x140>(0, bits(v)));  // row_mirror
    if (LANES >= 32) v += __shfl_xor(v, 16);
    return v;
}

template <bool BF16, int VEC, int LANES, bool NEIGHBOURS, bool STREAM>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(Rope a) {
    typedef typename Words<VEC>::type words;
    constexpr int ROWS = 64 / LANES;  // rows of a step
    __shared__ __attribute__((aligned(16))) float turn[kWaves][2][128];
    __shared__ __attribute__((aligned(16))) float weight[2][256];
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
    const int64_t token = min((int64_t)blockIdx.x * kWaves + wave, (int64_t)a.n_tokens - 1);
    const int first = (int)blockIdx.y * a.steps;  // the wave's first step
    const int all = a.heads[0] + a.heads[1];
    const int end = (int64_t)blockIdx.x * kWaves + wave < a.n_tokens ? min(first + a.steps, (all + ROWS - 1) / ROWS) : first;

    // the lane's pairs: i0 .. i0 + VEC, or of neighbours half of them from either
    // half of the row (first0, first1), and where their values lie in a row
    const int i0 = (lane & (LANES - 1)) * VEC, first0 = NEIGHBOURS ? i0 / 2 : i0, first1 = a.head_dim / 4 + i0 / 2;
    const bool inside = i0 < a.head_dim / 2, turns = first0 < a.n_freq, turns1 = NEIGHBOURS ? first1 < a.n_freq : turns;
    const int at0 = !inside ? 0 : (NEIGHBOURS || turns ? i0 : i0 + a.n_freq);
    const int at1 = !inside ? 0 : (!NEIGHBOURS && turns ? i0 + a.n_freq : i0 + a.head_dim / 2);

    struct Row {
        words x0, x1;
    };
    Row rows[kBatch];
    const int row = lane / LANES;
    const int64_t q_sh = held(a.sh[0]), k_sh = held(a.sh[1]);
    const uint16_t *q = (const uint16_t *)held(a.x[0]) + token * a.st[0];
    const uint16_t *k = (const uint16_t *)held(a.x[1]) + token * a.st[1];
    auto load = [&](Row &r, int step) {
        const int h = min(step * ROWS + row, all - 1);  // past the last head: the last one again, not stored
        const uint16_t *src = h < a.heads[0] ? q + h * q_sh : k + (h - a.heads[0]) * k_sh;
        const words *s0 = reinterpret_cast<const words *>(src + at0), *s1 = reinterpret_cast<const words *>(src + at1);
        r.x0 = *s0;
        r.x1 = *s1;
    };
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
        if (first + b < end) load(rows[b], first + b);

    // the weights, for all of the workgroup's waves
    {
        const int i = min((int)threadIdx.x, a.head_dim - 1);
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int t = 0; t < 2; ++t)
            if (a.weight[t]) {
                if (a.weight_f32[t]) w[t] = ((const uint32_t *)a.weight[t])[i];
                else w[t] = ((const uint16_t *)a.weight[t])[i];
            }
#pragma unroll
        for (int t = 0; t < 2; ++t)
            weight[t][threadIdx.x] = a.weight_f32[t] ? __builtin_bit_cast(float, w[t]) : widen<BF16>(w[t], 0);
    }
    // sines and cosines of the token's pairs, two at most a lane
    double pos[2];
    float freq[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int i = min(lane + u * 64, a.n_freq - 1);
        pos[u] = 0.0;
        freq[u] = 0.0f;
        if (u * 64 < a.n_freq) {
            const uint64_t w0 = i & 32 ? held((int64_t)a.axes[1]) : held((int64_t)a.axes[0]);
            const uint64_t w1 = i & 32 ? held((int64_t)a.axes[3]) : held((int64_t)a.axes[2]);
            const int axis = (int)((u ? w1 : w0) >> (2 * (i & 31))) & 3;
            const int64_t at = axis * a.pos_stride + token;
            if (a.pos64) pos[u] = (double)((const int64_t *)a.positions)[at];
            else pos[u] = (double)((const int32_t *)a.positions)[at];
            freq[u] = a.inv_freq[i];
        }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        if (u * 64 >= a.n_freq) break;
        const double t = pos[u] * ((double)freq[u] * 0.15915494309189533577);
        float s, c;
        sincospif((float)(2.0 * (t - rint(t))), &s, &c);
        turn[wave][0][lane + u * 64] = c * a.rotary_scale;
        turn[wave][1][lane + u * 64] = s * a.rotary_scale;
    }
    lds_barrier();
    float c[VEC], s[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        const int i = NEIGHBOURS && j >= VEC / 2 ? (turns1 ? first1 - VEC / 2 : 0) : (turns ? first0 : 0);
        c[j] = turn[wave][0][i + j];
        s[j] = turn[wave][1][i + j];
    }

    const int64_t q_osh = held(a.ysh[0]), k_osh = held(a.ysh[1]);
    uint16_t *q_out = (uint16_t *)held(a.y[0]) + token * a.yst[0], *k_out = (uint16_t *)held(a.y[1]) + token * a.yst[1];
    const bool q_normed = a.weight[0], k_normed = a.weight[1];
    for (int step = first; step < end; step += kBatch) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (step + b >= end) break;
            const int h = (step + b) * ROWS + row;
            const bool is_q = h < a.heads[0];
            float x[2 * VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                x[j] = widen<BF16>(rows[b].x0[j / 2], j & 1);
                x[VEC + j] = widen<BF16>(rows[b].x1[j / 2], j & 1);
            }
            if (step + b + kBatch < end) load(rows[b], step + b + kBatch);
            if (is_q ? q_normed : k_normed) {
                float sum = 0.0f;
#pragma unroll
                for (int j = 0; j < 2 * VEC; ++j) sum = __builtin_fmaf(x[j], x[j], sum);
                sum = row_sum<LANES>(inside ? sum : 0.0f);
                const float mean = __builtin_fmaf(sum, a.inv_dim, a.eps);
                float r = __builtin_amdgcn_rsqf(mean);
                // squares of bf16 values pass f32's range on both sides: such rows are scaled and summed again
                const bool range = mean >= 0x1p-100f && mean < __builtin_huge_valf();
                if (BF16 && __ballot(!range)) {
                    const float by = range ? 1.0f : (mean < 0x1p-100f ? 0x1p100f : 0x1p-70f);
                    sum = 0.0f;
#pragma unroll
                    for (int j = 0; j < 2 * VEC; ++j) {
                        x[j] *= by;
                        sum = __builtin_fmaf(x[j], x[j], sum);
                    }
                    sum = row_sum<LANES>(inside ? sum : 0.0f);
                    r = __builtin_amdgcn_rsqf(__builtin_fmaf(sum, a.inv_dim, a.eps * by * by));
                }
                const float *w = weight[is_q ? 0 : 1];
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    x[j] = x[j] * r * w[at0 + j];  // (r times a weight may leave the range)
                    x[VEC + j] = x[VEC + j] * r * w[at1 + j];
                }
            }
            if (turns || turns1) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    if (NEIGHBOURS && !(j < VEC / 2 ? turns : turns1)) continue;
                    float &u = x[NEIGHBOURS ? 2 * j : j], &v = x[NEIGHBOURS ? 2 * j + 1 : VEC + j];
                    const float p = u * c[j] - v * s[j], q = v * c[j] + u * s[j];
                    u = p;
                    v = q;
                }
            }
            if (h >= all || !inside) continue;
            words y0, y1;
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) {
                y0[j] = narrow<BF16>(x[2 * j], x[2 * j + 1]);
                y1[j] = narrow<BF16>(x[VEC + 2 * j], x[VEC + 2 * j + 1]);
            }
            uint16_t *dst = is_q ? q_out + h * q_osh : k_out + (h - a.heads[0]) * k_osh;
            words *d0 = reinterpret_cast<words *>(dst + at0), *d1 = reinterpret_cast<words *>(dst + at1);
            if (STREAM) {
                __builtin_nontemporal_store(y0, d0);
                __builtin_nontemporal_store(y1, d1);
            } else {
                *d0 = y0;
                *d1 = y1;
            }
        }
    }
}

template <bool BF16, int VEC, int LANES>
hipError_t launch_lanes(const Rope &a, const RopePlan &p, hipStream_t stream) {
    const dim3 grid((unsigned)((a.n_tokens + (int64_t)kWaves - 1) / kWaves), (unsigned)p.parts), block(kRopeThreads);
    // more than the eight L2s hold: what is written passes through once (104 us with streaming loads too, 102 without)
    const bool stream_rows = (int64_t)a.n_tokens * (a.heads[0] + a.heads[1]) * a.head_dim * 2 > (int64_t)32 << 20;
    if (a.neighbours)
        if (stream_rows)
            hipLaunchKernelGGL((norm_rope_kernel<BF16, VEC, LANES, true, true>), grid, block, 0, stream, a);
        else
            hipLaunchKernelGGL((norm_rope_kernel<BF16, VEC, LANES, true, false>), grid, block, 0, stream, a);
    else if (stream_rows)
        hipLaunchKernelGGL((norm_rope_kernel<BF16, VEC, LANES, false, true>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((norm_rope_kernel<BF16, VEC, LANES, false, false>), grid, block, 0, stream, a);
    return hipGetLastError();
}

template <bool BF16>
hipError_t launch_type(const Rope &a, const RopePlan &p, hipStream_t stream) {
    if (p.vec == 8) {
        switch (p.lanes) {
            case 2: return launch_lanes<BF16, 8, 2>(a, p, stream);
            case 4: return launch_lanes<BF16, 8, 4>(a, p, stream);
            case 8: return launch_lanes<BF16, 8, 8>(a, p, stream);
            default: return launch_lanes<BF16, 8, 16>(a, p, stream);
        }
    }
    switch (p.lanes) {
        case 8: return launch_lanes<BF16, 4, 8>(a, p, stream);
        case 16: return launch_lanes<BF16, 4, 16>(a, p, stream);
        default: return launch_lanes<BF16, 4, 32>(a, p, stream);
    }
}

}  // namespace

RopePlan plan_rope(int64_t n_tokens, int heads, int head_dim, int n_freq) {
    RopePlan p{};
    // 16-byte loads need halves and the rotated part to be multiples of 8 values
    p.vec = head_dim % 16 == 0 && n_freq % 8 == 0 ? 8 : 4;
    p.lanes = p.vec == 8 ? 2 : 8;
    while (p.lanes * p.vec * 2 < head_dim) p.lanes *= 2;
    const int rows = 64 / p.lanes, steps = (heads + rows - 1) / rows;
    p.steps = steps;
    while (p.steps > 1 && n_tokens * ((steps + p.steps - 1) / p.steps) < 4096) p.steps = (p.steps + 1) / 2;
    p.parts = (steps + p.steps - 1) / p.steps;
    p.workgroups = (n_tokens + kWaves - 1) / kWaves * p.parts;
    p.fits = p.workgroups <= (int64_t)UINT32_MAX / kRopeThreads;
    return p;
}

hipError_t launch_rope(const Rope &a, const RopePlan &p, hipStream_t stream) {
    return a.bf16 ? launch_type<true>(a, p, stream) : launch_type<false>(a, p, stream);
}

}  // namespace lidx
