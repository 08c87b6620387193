// Matrix products of the 16-bit expert layer, weights' gradient: dW = dy x^T.
#include "gemm_launch.h"

namespace bm_host {

int launch_experts_dw(int dtype, const GemmArgs &g, const GemmPlan &p, hipStream_t s) {
    return bm::launch_layout<kGradWeights>(dtype, g, p, s);
}

}  // namespace bm_host
