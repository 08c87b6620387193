// C ABI: the output rows of a product over a share of the experts that none of
// the share's rows goes to.
#include "experts_check.h"

extern "C" int moe_expert_clear_ungrouped(const int32_t *offsets, int E, int R, const bitmoe_rows *y, void *stream) {
    using namespace bm_host;
    if (!y) return BITMOE_EINVAL;
    int rc = check_sizes(E, R, y->cols, 1);
    if (rc || (rc = check_rows(y, R, y->cols, true))) return rc;
    if (R == 0) return BITMOE_OK;
    if (!offsets || !aligned(offsets, 4)) return BITMOE_EINVAL;
    return launch_clear_ungrouped(offsets, E, R, rows_arg(y), y->cols, y->dtype == BITMOE_F32,
                                  reinterpret_cast<hipStream_t>(stream));
}
