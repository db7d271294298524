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
// reader the other way round), one pass.  A thread issues the loads of kBatch
// chunks before it uses the first: with one at a time, writing 131072 tokens of
// 8 x 128, K and V, took 145 us and reading K back 89 us; with four 132 us
// (5.1 TB/s) and 67 us, with eight 146 and 69 us.
#include "device_common.h"
#include "mx4_internal.h"

namespace lidx {
namespace {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kBatch = 4;

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

template <bool BF16, bool STREAM>
__global__ void __launch_bounds__(kThreads) mx4_write_kernel(Mx4Write a, int tokens_per_wg) {
    const int which = blockIdx.y;
    const uint16_t *x = (const uint16_t *)(which ? a.x[1] : a.x[0]);
    const int64_t st = which ? a.st[1] : a.st[0], sh = which ? a.sh[1] : a.sh[0];
    uint8_t *data = which ? a.data[1] : a.data[0];
    uint8_t *scale = which ? a.scale[1] : a.scale[0];
    const uint32_t t0 = blockIdx.x * (uint32_t)tokens_per_wg;
    const uint32_t nt = min((uint32_t)tokens_per_wg, (uint32_t)a.n_tokens - t0);
    const uint32_t units = nt * a.div_e.d;
    // 8-value chunks, kBatch of a thread's at a time: their loads are all issued
    // before the first is used.  units and the steps are multiples of 4, so the
    // lanes of a quad stay together
    for (uint32_t u0 = threadIdx.x; u0 < units; u0 += kBatch * kThreads) {
        u32x4 v[kBatch];
        int64_t slot[kBatch];
        uint32_t head[kBatch], chunk[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const uint32_t u = min(u0 + i * kThreads, units - 4u + (threadIdx.x & 3u));
            const uint32_t t = quotient(u, a.div_e), r = u - t * a.div_e.d;
            head[i] = quotient(r, a.div_c);
            chunk[i] = r - head[i] * a.div_c.d;
            const u32x4 *src = reinterpret_cast<const u32x4 *>(x + (int64_t)(t0 + t) * st + (int64_t)head[i] * sh +
                                                               chunk[i] * 8);
            v[i] = STREAM ? __builtin_nontemporal_load(src) : *src;
            slot[i] = a.slots[t0 + t];
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const uint32_t w[4] = {v[i][0], v[i][1], v[i][2], v[i][3]};
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) top = max(top, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
            const uint32_t s = scale_byte<BF16>(quad_max(top));
            const float f = __builtin_bit_cast(float, s << 23);
            uint32_t code = 0;
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
            if (s == 255u) code = 0u;
            int64_t block, off;
            if (u0 + i * kThreads >= units || !place(a.pages, slot[i], block, off)) continue;
            const uint32_t h = head[i], c = chunk[i];
            *reinterpret_cast<uint32_t *>(data + block * a.pages.d_sb + off * a.pages.d_ss + h * a.pages.d_sh + c * 4) =
                code;
            if (!(c & 3u))
                scale[block * a.pages.s_sb + off * a.pages.s_ss + h * a.pages.s_sh + (c >> 2)] = (uint8_t)s;
        }
    }
}

template <bool BF16, bool STREAM>
__global__ void __launch_bounds__(kThreads) mx4_read_kernel(Mx4Read a, int rows_per_wg) {
    const uint32_t t0 = blockIdx.x * (uint32_t)rows_per_wg;
    const uint32_t nt = min((uint32_t)rows_per_wg, (uint32_t)a.n_rows - t0);
    const uint32_t units = nt * a.div_e.d;
    uint16_t *out = (uint16_t *)a.out;
    for (uint32_t u0 = threadIdx.x; u0 < units; u0 += kBatch * kThreads) {
        uint32_t code[kBatch], s[kBatch], row[kBatch], head[kBatch], chunk[kBatch];
        int64_t slot[kBatch];
        bool ok[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const uint32_t u = min(u0 + i * kThreads, units - 1u);
            row[i] = quotient(u, a.div_e);
            const uint32_t r = u - row[i] * a.div_e.d;
            head[i] = quotient(r, a.div_c);
            chunk[i] = r - head[i] * a.div_c.d;
            slot[i] = a.slots[t0 + row[i]];
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            int64_t block = 0, off = 0;  // slot 0 exists; it is read and not used where the row's does not
            ok[i] = place(a.pages, slot[i], block, off);
            code[i] = *reinterpret_cast<const uint32_t *>(a.data + block * a.pages.d_sb + off * a.pages.d_ss +
                                                          head[i] * a.pages.d_sh + chunk[i] * 4);
            s[i] = a.scale[block * a.pages.s_sb + off * a.pages.s_ss + head[i] * a.pages.s_sh + (chunk[i] >> 2)];
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const float f = __builtin_bit_cast(float, s[i] << 23);  // 255: the conversion gives NaN
            uint32_t w[4];
            if constexpr (BF16) {
                w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code[i], f, 0));
                w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code[i], f, 1));
                w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code[i], f, 2));
                w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code[i], f, 3));
            } else {
                w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(code[i], f, 0));
                w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(code[i], f, 1));
                w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(code[i], f, 2));
                w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(code[i], f, 3));
            }
            if (u0 + i * kThreads >= units) continue;
            const u32x4 v = ok[i] ? u32x4{w[0], w[1], w[2], w[3]} : u32x4{0u, 0u, 0u, 0u};
            u32x4 *dst = reinterpret_cast<u32x4 *>(out + (int64_t)(t0 + row[i]) * a.st + (int64_t)head[i] * a.sh +
                                                   chunk[i] * 8);
            if (STREAM) __builtin_nontemporal_store(v, dst);
            else *dst = v;
        }
    }
}

// Tokens a workgroup takes: about kBatch chunks a thread, at least one token,
// and as many as keep the launch below 2^32 threads.
int tokens_per_wg(int64_t tokens, int chunks_per_token) {
    const int64_t most = (int64_t)UINT32_MAX / kThreads, least = (tokens + most - 1) / most;
    const int64_t n = kBatch * kThreads / chunks_per_token;
    return (int)(n < least ? least : n);
}

// More values on the 16-bit side than the eight L2s hold (32 MiB): they pass
// through once, so keeping them would only push out the codes.  131072 rows of
// 8 x 128: read back 67 us with ordinary stores, 50.5 us (6.75 TB/s) with
// streaming ones; written one tensor 66 and 60 us.  Smaller results stay for
// whoever reads them next.
bool streams(int64_t rows, int heads, int head_dim) { return rows * heads * head_dim * 2 > (int64_t)32 << 20; }

template <bool BF16>
void write_launch(const Mx4Write &a, bool stream_x, dim3 grid, int per, hipStream_t stream) {
    if (stream_x)
        hipLaunchKernelGGL((mx4_write_kernel<BF16, true>), grid, dim3(kThreads), 0, stream, a, per);
    else
        hipLaunchKernelGGL((mx4_write_kernel<BF16, false>), grid, dim3(kThreads), 0, stream, a, per);
}

template <bool BF16>
void read_launch(const Mx4Read &a, bool stream_out, dim3 grid, int per, hipStream_t stream) {
    if (stream_out)
        hipLaunchKernelGGL((mx4_read_kernel<BF16, true>), grid, dim3(kThreads), 0, stream, a, per);
    else
        hipLaunchKernelGGL((mx4_read_kernel<BF16, false>), grid, dim3(kThreads), 0, stream, a, per);
}

}  // namespace

hipError_t launch_mx4_write(const Mx4Write &a, hipStream_t stream) {
    const int per = tokens_per_wg(a.n_tokens, (int)a.div_e.d);
    const dim3 grid((unsigned)(((int64_t)a.n_tokens + per - 1) / per), (unsigned)a.n_tensors);
    const bool big = streams(a.n_tokens, a.n_heads, a.head_dim);
    a.bf16 ? write_launch<true>(a, big, grid, per, stream) : write_launch<false>(a, big, grid, per, stream);
    return hipGetLastError();
}

hipError_t launch_mx4_read(const Mx4Read &a, hipStream_t stream) {
    const int per = tokens_per_wg(a.n_rows, (int)a.div_e.d);
    const dim3 grid((unsigned)(((int64_t)a.n_rows + per - 1) / per));
    const bool big = streams(a.n_rows, a.n_heads, a.head_dim);
    a.bf16 ? read_launch<true>(a, big, grid, per, stream) : read_launch<false>(a, big, grid, per, stream);
    return hipGetLastError();
}

}  // namespace lidx
