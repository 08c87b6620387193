// Matrix products of the 16-bit expert layer, rows' gradient: dx = W^T dy.
#include "gemm_launch.h"

namespace bm_host {

int launch_experts_dx(int dtype, const GemmArgs &g, const GemmPlan &p, hipStream_t s) {
    return bm::launch_layout<kGradRows>(dtype, g, p, s);
}

}  // namespace bm_host
