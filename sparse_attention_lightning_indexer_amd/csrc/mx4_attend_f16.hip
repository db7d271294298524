// The f16 instances of the attention over the 4-bit cache.
#include "mx4_attend.h"

namespace lidx {

hipError_t launch_mx4_attend_f16(const Mx4Attend &a, const Mx4Plan &p, int head_dim, hipStream_t stream) {
    return mx4::launch_attend<false>(a, p, head_dim, stream);
}

}  // namespace lidx
