// The norms around a block: launches in float16.
#include "norm_kernels.h"

namespace bm_host {

int launch_block_norm_f16(const NormArgs &a, hipStream_t st) { return bm::launch_norm<BITMOE_F16>(a, st); }
int launch_block_norm_backward_f16(const NormBackArgs &a, hipStream_t st) { return bm::launch_norm_backward<BITMOE_F16>(a, st); }

}  // namespace bm_host
