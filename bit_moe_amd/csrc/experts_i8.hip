// Products grouped by expert in 8 bits: launches.
#include <algorithm>

#include "gemm_i8.h"
#include "rows8.h"

namespace {

using namespace bm;

template <int DT>
int launch_of(const GemmArgs &args, hipStream_t s) {
    GemmArgs g = args;
    g.splits = 1;
    const int mt = g.R / 128 + std::min(g.E, g.R), nt = (g.N + 127) / 128;
    const int64_t grid = ((int64_t)mt * nt + 7) / 8 * 8;
    if (grid * 256 >= (int64_t)1 << 32) return BITMOE_EUNSUPPORTED;
    k_i8_any<DT><<<(int)grid, 256, 0, s>>>(g, mt, nt);
    BM_LAUNCH_CHECK();
    return BITMOE_OK;
}

}  // namespace

namespace bm_host {

size_t i8_ws_bytes(int, int, int, int) { return 0; }

int launch_gemm_i8(int out, const GemmArgs &g, void *, hipStream_t s) {
    return out == BITMOE_BF16 ? launch_of<kI8 + BITMOE_BF16>(g, s) : launch_of<kI8 + BITMOE_F16>(g, s);
}

}  // namespace bm_host
