// Head norms and rotation by position for gfx950: queries and keys as the
// indexer, the cache's writer and the attention take them.
//
// A row (a token's head) is read once and written once, so this is
// memory-bound: 4 bytes a value.  `lanes` neighbouring lanes hold a row, each
// VEC pairs as one wide load of first and one of second values (for pairs of
// neighbours two consecutive loads), so a rotation never leaves its lane and
// the norm is a sum over `lanes` lanes by lane moves.
//
// The angles depend on the token and the pair alone: a wave computes its
// token's sines and cosines once, one pair a lane, and its rows read them
// from LDS.  angle = position * frequency is formed in f64 as turns and reduced
// to half a turn there; position 131071 at frequency 1 in f32 would be off by
// 2^-8 radians, and a table of sines would be read again for every token.
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

template <bool BF16, int VEC, int LANES, bool NEIGHBOURS>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(Rope a) {
    typedef typename Words<VEC>::type words;
    constexpr int ROWS = 64 / LANES;  // rows of a step
    __shared__ float turn[kWaves][2][128];
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
    const int64_t token = (int64_t)blockIdx.x * kWaves + wave;
    if (token >= a.n_tokens) return;
    const int first = (int)blockIdx.y * a.steps;  // the wave's first step
    const int all = a.heads[0] + a.heads[1];

    // the lane's pairs: i0 .. i0 + VEC, and where their values lie in a row
    const int i0 = (lane & (LANES - 1)) * VEC;
    const bool inside = i0 < a.head_dim / 2, turns = i0 < a.n_freq;
    const int at0 = NEIGHBOURS ? 2 * i0 : (turns ? i0 : i0 + a.n_freq);
    const int at1 = NEIGHBOURS ? 2 * i0 + VEC : (turns ? i0 + a.n_freq : i0 + a.head_dim / 2);

    struct Row {
        words x0, x1;
    };
    Row rows[kBatch];
    const int row = lane / LANES;
    auto load = [&](Row &r, int step) {
        // past the last head: the last one again, not stored
        const int h = min(step * ROWS + row, all - 1);
        const int which = h >= a.heads[0];
        const uint16_t *src = (const uint16_t *)a.x[which] + token * a.st[which] +
                              (int64_t)(h - (which ? a.heads[0] : 0)) * a.sh[which];
        r.x0 = *reinterpret_cast<const words *>(src + (inside ? at0 : 0));
        r.x1 = *reinterpret_cast<const words *>(src + (inside ? at1 : 0));
    };
    const int end = min(first + a.steps, (all + ROWS - 1) / ROWS);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) load(rows[b], min(first + b, end - 1));

    // sines and cosines of the token's pairs
    for (int i = lane; i < a.n_freq; i += 64) {
        const int axis = (int)(a.axes[i >> 5] >> (2 * (i & 31))) & 3;
        const int64_t at = axis * a.pos_stride + token;
        const double p = a.pos64 ? (double)((const int64_t *)a.positions)[at] : (double)((const int32_t *)a.positions)[at];
        const double t = p * ((double)a.inv_freq[i] * 0.15915494309189533577);
        float s, c;
        sincospif((float)(2.0 * (t - rint(t))), &s, &c);
        turn[wave][0][i] = c * a.rotary_scale;
        turn[wave][1][i] = s * a.rotary_scale;
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    float c[VEC], s[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        c[j] = turn[wave][0][turns ? i0 + j : 0];
        s[j] = turn[wave][1][turns ? i0 + j : 0];
    }
    // the weights of the lane's values, of q and k
    float w[2][2 * VEC];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            w[t][j] = w[t][VEC + j] = 1.0f;
            if (!a.weight[t] || !inside) continue;
            const int p = at0 + j, q = at1 + j;
            if (a.weight_f32[t]) {
                w[t][j] = ((const float *)a.weight[t])[p];
                w[t][VEC + j] = ((const float *)a.weight[t])[q];
            } else {
                w[t][j] = widen<BF16>(((const uint16_t *)a.weight[t])[p], 0);
                w[t][VEC + j] = widen<BF16>(((const uint16_t *)a.weight[t])[q], 0);
            }
        }

    for (int step = first; step < end; step += kBatch) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (step + b >= end) break;
            const int h = (step + b) * ROWS + row;
            const int which = h >= a.heads[0];
            float x[2 * VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                x[j] = widen<BF16>(rows[b].x0[j / 2], j & 1);
                x[VEC + j] = widen<BF16>(rows[b].x1[j / 2], j & 1);
            }
            load(rows[b], min(step + b + kBatch, end - 1));
            // the norm's sum; bf16 squares may pass f32's range, and are then summed of smaller values
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 2 * VEC; ++j) sum = __builtin_fmaf(x[j], x[j], sum);
            sum = row_sum<LANES>(inside ? sum : 0.0f);
            float r = 1.0f / sqrtf(sum / (float)a.head_dim + a.eps);
            if (BF16 && __ballot(sum == __builtin_huge_valf())) {
                float small = 0.0f;
#pragma unroll
                for (int j = 0; j < 2 * VEC; ++j) {
                    const float v = x[j] * 0x1p-70f;
                    small = __builtin_fmaf(v, v, small);
                }
                small = row_sum<LANES>(inside ? small : 0.0f);
                if (sum == __builtin_huge_valf()) r = 0x1p-70f / sqrtf(small / (float)a.head_dim);
            }
            if (a.weight[which]) {
#pragma unroll
                for (int j = 0; j < 2 * VEC; ++j) x[j] = x[j] * r * (which ? w[1][j] : w[0][j]);
            }
            if (turns) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
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
            uint16_t *dst = (uint16_t *)a.y[which] + token * a.yst[which] +
                            (int64_t)(h - (which ? a.heads[0] : 0)) * a.ysh[which];
            *reinterpret_cast<words *>(dst + at0) = y0;
            *reinterpret_cast<words *>(dst + at1) = y1;
        }
    }
}

template <bool BF16, int VEC, int LANES>
hipError_t launch_lanes(const Rope &a, const RopePlan &p, hipStream_t stream) {
    const dim3 grid((unsigned)((a.n_tokens + (int64_t)kWaves - 1) / kWaves), (unsigned)p.parts), block(kRopeThreads);
    if (a.neighbours)
        hipLaunchKernelGGL((norm_rope_kernel<BF16, VEC, LANES, true>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((norm_rope_kernel<BF16, VEC, LANES, false>), grid, block, 0, stream, a);
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
