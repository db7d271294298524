// Internal interface of the head norm and rotation (rope_api.hip,
// rope_kernel.hip).  Not exported.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lidx {

struct Rope {
    const void *x[2];  // q, k
    int64_t st[2], sh[2];
    void *y[2];
    int64_t yst[2], ysh[2];
    const void *weight[2];  // nullptr: not normed
    bool weight_f32[2];
    const void *positions;
    int64_t pos_stride;
    bool pos64;
    const float *inv_freq;
    uint64_t axes[4];  // two bits a frequency
    int32_t n_tokens, head_dim, n_freq;
    int32_t heads[2];
    float eps, rotary_scale, inv_dim;
    bool bf16, neighbours;
    int32_t steps;  // of rows of its token that a wave takes
};

struct RopePlan {
    int vec;           // pairs of a lane
    int lanes;         // of a row, a power of two
    int parts, steps;  // waves of a token, and the steps of 64 / lanes rows each of them takes
    int64_t workgroups;
    bool fits;  // fewer than 2^32 threads
};
RopePlan plan_rope(int64_t n_tokens, int heads, int head_dim, int n_freq);
constexpr int kRopeThreads = 256;

hipError_t launch_rope(const Rope &a, const RopePlan &p, hipStream_t stream);

}  // namespace lidx
