// Writing rows into the 4-bit cache and reading them back (gfx950).
//
// A block of 32 values x becomes a scale 2^e, e the least exponent with
// max|x| < 7 * 2^e inside the source type's range, and 32 codes of the nearest
// magnitude to |x| / 2^e out of 0, .5, 1, 1.5, 2, 3, 4, 6 (ties to the even
// code, at most 6).  With max|x| = 1.m * 2^k that e is k - 2, or k - 1 where
// 1.m >= 1.75, so it comes from the bits of the largest magnitude alone.
// The conversions take the scale as an operand and round once, to nearest
// even, saturating; the scale is a power of two, so nothing else rounds and
// every result is exact to the bit.
//
// Four neighbouring lanes hold a block, 8 values (16 bytes) each: every global
// access of a wave is contiguous, the block's maximum is two lane swaps inside
// quads, each lane stores its 8 codes as one word, and the first lane of the
// four the scale byte.  Memory-bound: 2 bytes in and 0.53 out per value (the
// reader the other way round), one pass.
#include "device_common.h"
#include "mx4_internal.h"

namespace lidx {
namespace {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf2_t __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;

// Page and offset of a slot; false if it is not one of the cache.
__device__ __forceinline__ bool place(const Mx4Pages &p, int64_t slot, int64_t &block, int64_t &off) {
    if (slot < 0 || slot >= p.n_slots) return false;
    if (p.n_slots <= 0x7fffffffll) {
        const uint32_t b = quotient((uint32_t)slot, p.div_bs);
        block = b;
        off = (uint32_t)slot - b * (uint32_t)p.block_size;
    } else {
        block = slot / p.block_size;
        off = slot - block * p.block_size;
    }
    return true;
}

// The larger of this lane's and its quad neighbours' values.
__device__ __forceinline__ uint32_t quad_max(uint32_t u) {
    u = max(u, (uint32_t)dpp_move<0xb1>(0, (int)u));  // quad_perm [1,0,3,2]
    u = max(u, (uint32_t)dpp_move<0x4e>(0, (int)u));  // quad_perm [2,3,0,1]
    return u;
}

// The scale byte of a block from the largest magnitude's bits (sign cleared).
// 255 for infinities and NaN.
template <bool BF16>
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
    if (BF16) {
        if (top >= 0x7f80u) return 255u;
        // exponent field k + 127 (0: subnormal, below the range's start), then
        // + 1 where the fraction's two leading bits are set; e + 127 = field - 2 + that
        const int s = (int)(top >> 7) - 2 + (int)((top & 0x60u) == 0x60u);
        return (uint32_t)min(max(s, 1), 252);
    }
    if (top >= 0x7c00u) return 255u;
    // f16 exponent field is k + 15; the range's start, e = -23, covers
    // magnitudes below 7 * 2^-23 and with them k <= -22: subnormals (k <= -15)
    // need their leading bit
    int k, frac;
    if (top >= 0x400u) {
        k = (int)(top >> 10) - 15;
        frac = (int)((top & 0x300u) == 0x300u);
    } else {
        const int lead = 31 - __clz((int)(top | 1u));     // top = 1.m * 2^lead units of 2^-24
        k = lead - 24;
        frac = (int)(((top << (10 - lead)) & 0x300u) == 0x300u);
    }
    return (uint32_t)(min(max(k - 2 + frac, -23), 13) + 127);
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) mx4_write_kernel(Mx4Write a, int tokens_per_wg) {
    const int which = blockIdx.y;
    const uint16_t *x = (const uint16_t *)(which ? a.x[1] : a.x[0]);
    const int64_t st = which ? a.st[1] : a.st[0], sh = which ? a.sh[1] : a.sh[0];
    uint8_t *data = which ? a.data[1] : a.data[0];
    uint8_t *scale = which ? a.scale[1] : a.scale[0];
    const uint32_t t0 = blockIdx.x * (uint32_t)tokens_per_wg;
    const uint32_t nt = min((uint32_t)tokens_per_wg, (uint32_t)a.n_tokens - t0);
    const uint32_t units = nt * a.div_e.d;
    // 8-value chunks; units and the step are multiples of 4, so the lanes of a
    // quad stay together
    for (uint32_t u = threadIdx.x; u < units; u += kThreads) {
        const uint32_t t = quotient(u, a.div_e), r = u - t * a.div_e.d;
        const uint32_t h = quotient(r, a.div_c), c = r - h * a.div_c.d;
        const uint4 v = *reinterpret_cast<const uint4 *>(x + (int64_t)(t0 + t) * st + (int64_t)h * sh + c * 8);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
        const uint32_t s = scale_byte<BF16>(quad_max(top));
        const float f = __builtin_bit_cast(float, s << 23);
        uint32_t code = 0;
        if (s != 255u) {
            if constexpr (BF16) {
                code = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(code, __builtin_bit_cast(bf2_t, w[0]), f, 0);
                code = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(code, __builtin_bit_cast(bf2_t, w[1]), f, 1);
                code = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(code, __builtin_bit_cast(bf2_t, w[2]), f, 2);
                code = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(code, __builtin_bit_cast(bf2_t, w[3]), f, 3);
            } else {
                code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(code, __builtin_bit_cast(half2_t, w[0]), f, 0);
                code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(code, __builtin_bit_cast(half2_t, w[1]), f, 1);
                code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(code, __builtin_bit_cast(half2_t, w[2]), f, 2);
                code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(code, __builtin_bit_cast(half2_t, w[3]), f, 3);
            }
        }
        int64_t block, off;
        if (!place(a.pages, a.slots[t0 + t], block, off)) continue;
        *reinterpret_cast<uint32_t *>(data + block * a.pages.d_sb + off * a.pages.d_ss + h * a.pages.d_sh + c * 4) = code;
        if (!(c & 3u)) scale[block * a.pages.s_sb + off * a.pages.s_ss + h * a.pages.s_sh + (c >> 2)] = (uint8_t)s;
    }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) mx4_read_kernel(Mx4Read a, int rows_per_wg) {
    const uint32_t t0 = blockIdx.x * (uint32_t)rows_per_wg;
    const uint32_t nt = min((uint32_t)rows_per_wg, (uint32_t)a.n_rows - t0);
    const uint32_t units = nt * a.div_e.d;
    uint16_t *out = (uint16_t *)a.out;
    for (uint32_t u = threadIdx.x; u < units; u += kThreads) {
        const uint32_t t = quotient(u, a.div_e), r = u - t * a.div_e.d;
        const uint32_t h = quotient(r, a.div_c), c = r - h * a.div_c.d;
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        int64_t block, off;
        if (place(a.pages, a.slots[t0 + t], block, off)) {
            const uint32_t code = *reinterpret_cast<const uint32_t *>(a.data + block * a.pages.d_sb +
                                                                      off * a.pages.d_ss + h * a.pages.d_sh + c * 4);
            const uint32_t s = a.scale[block * a.pages.s_sb + off * a.pages.s_ss + h * a.pages.s_sh + (c >> 2)];
            const float f = __builtin_bit_cast(float, s << 23);  // 255: the conversion gives NaN
            if constexpr (BF16) {
                w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, f, 0));
                w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, f, 1));
                w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, f, 2));
                w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, f, 3));
            } else {
                w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(code, f, 0));
                w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(code, f, 1));
                w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(code, f, 2));
                w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(code, f, 3));
            }
        }
        *reinterpret_cast<uint4 *>(out + (int64_t)(t0 + t) * a.st + (int64_t)h * a.sh + c * 8) =
            make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Tokens a workgroup takes: about four chunks a thread, at least one token.
int tokens_per_wg(int chunks_per_token) {
    const int n = 4 * kThreads / chunks_per_token;
    return n < 1 ? 1 : n;
}

}  // namespace

hipError_t launch_mx4_write(const Mx4Write &a, hipStream_t stream) {
    const int per = tokens_per_wg((int)a.div_e.d);
    const dim3 grid((unsigned)(((int64_t)a.n_tokens + per - 1) / per), (unsigned)a.n_tensors);
    if (a.bf16)
        hipLaunchKernelGGL(mx4_write_kernel<true>, grid, dim3(kThreads), 0, stream, a, per);
    else
        hipLaunchKernelGGL(mx4_write_kernel<false>, grid, dim3(kThreads), 0, stream, a, per);
    return hipGetLastError();
}

hipError_t launch_mx4_read(const Mx4Read &a, hipStream_t stream) {
    const int per = tokens_per_wg((int)a.div_e.d);
    const dim3 grid((unsigned)(((int64_t)a.n_rows + per - 1) / per));
    if (a.bf16)
        hipLaunchKernelGGL(mx4_read_kernel<true>, grid, dim3(kThreads), 0, stream, a, per);
    else
        hipLaunchKernelGGL(mx4_read_kernel<false>, grid, dim3(kThreads), 0, stream, a, per);
    return hipGetLastError();
}

}  // namespace lidx
