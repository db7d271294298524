// Attention of requests that share a prefix, bf16 queries (see mx4_attend.h).
#include "mx4_attend.h"

namespace lidx {

hipError_t launch_mx4_shared_bf16(const Mx4Attend &a, const Mx4SharedPlan &p, int head_dim, hipStream_t stream) {
    return mx4::launch_shared<true>(a, p, head_dim, stream);
}

}  // namespace lidx
