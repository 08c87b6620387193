// The norms around a block: launches in bfloat16, and by type.
#include "norm_kernels.h"

namespace bm_host {

int launch_block_norm(const NormArgs &a, int dtype, hipStream_t st) {
    return dtype == BITMOE_BF16 ? bm::launch_norm<BITMOE_BF16>(a, st) : launch_block_norm_f16(a, st);
}
int launch_block_norm_backward(const NormBackArgs &a, int dtype, hipStream_t st) {
    return dtype == BITMOE_BF16 ? bm::launch_norm_backward<BITMOE_BF16>(a, st) : launch_block_norm_backward_f16(a, st);
}

}  // namespace bm_host
