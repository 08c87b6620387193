// Matrix products of the 16-bit expert layer, forward: y = W x.
#include "gemm_launch.h"

namespace bm_host {

int launch_experts_fwd(int dtype, const GemmArgs &g, const GemmPlan &p, hipStream_t s) {
    return bm::launch_layout<kForward>(dtype, g, p, s);
}

}  // namespace bm_host
