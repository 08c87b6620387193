// Launches of the matrix products of one layout.
#pragma once

#include <algorithm>
#include <atomic>

#include "gemm_any.h"
#include "gemm_few.h"
#include "gemm_tile.h"

namespace bm {

template <int LAY, int DT, int BM, int BN, int WM, int WN, bool MAPS = false, bool PARTS = false>
int launch_tile(const GemmArgs &g, const bm_host::GemmPlan &p, hipStream_t s) {
    constexpr int lds = TileLds<LAY, BM, BN, WM, WN, MAPS>::bytes;
    // LDS above 64 KiB must be opted into per kernel and device
    static std::atomic<uint64_t> opted{0};
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return BITMOE_EHIP;
    if (dev > 63 || !(opted.load(std::memory_order_relaxed) >> dev & 1)) {
        if (hipFuncSetAttribute(reinterpret_cast<const void *>(k_gemm_tile<LAY, DT, BM, BN, WM, WN, MAPS, PARTS>),
                                hipFuncAttributeMaxDynamicSharedMemorySize, lds) != hipSuccess)
            return BITMOE_EHIP;
        if (dev <= 63) opted.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
    }
    // as many workgroups as fit the GPU together, each for several tiles
    const int64_t most = std::max<int64_t>((int64_t)bm_host::cu_count() * (160 * 1024 / lds) / 8 * 8, 8);
    k_gemm_tile<LAY, DT, BM, BN, WM, WN, MAPS, PARTS><<<(int)std::min<int64_t>(p.grid, most), 64 * WM * WN, lds, s>>>(g, p.mt, p.nt);
    BM_LAUNCH_CHECK();
    return BITMOE_OK;
}

template <int DT, int P>
void launch_few(const GemmArgs &g, const bm_host::GemmPlan &p, hipStream_t s) {
    if (p.chunks == 1) k_gemm_few<DT, P, 1><<<(int)p.grid, 256, 0, s>>>(g, p.mt, p.nt);
    else k_gemm_few<DT, P, 4><<<(int)p.grid, 256, 0, s>>>(g, p.mt, p.nt);
}

template <int LAY, int DT>
int launch_layout_of(const GemmArgs &g, const bm_host::GemmPlan &p, hipStream_t s) {
    if constexpr (LAY == kGradWeights) {
        if (g.arows) switch (p.kind) {
            case bm_host::kTile256: return launch_tile<LAY, DT, 256, 256, 2, 4, true>(g, p, s);
            case bm_host::kTile128: return launch_tile<LAY, DT, 128, 128, 2, 2, true>(g, p, s);
        }
    }
    if constexpr (LAY != kForward) {
        if (g.a_low) switch (p.kind) {
            case bm_host::kTile256: return launch_tile<LAY, DT, 256, 256, 2, 4, false, true>(g, p, s);
            case bm_host::kTile128: return launch_tile<LAY, DT, 128, 128, 2, 2, false, true>(g, p, s);
            case bm_host::kTile128x256:
                if constexpr (LAY == kGradRows) return launch_tile<LAY, DT, 128, 256, 2, 4, false, true>(g, p, s);
                return BITMOE_EINVAL;
            case bm_host::kTile64x128:
                if constexpr (LAY == kGradRows) return launch_tile<LAY, DT, 64, 128, 2, 2, false, true>(g, p, s);
                return BITMOE_EINVAL;
        }
    }
    switch (p.kind) {
        case bm_host::kTile256: return launch_tile<LAY, DT, 256, 256, 2, 4>(g, p, s);
        case bm_host::kTile128: return launch_tile<LAY, DT, 128, 128, 2, 2>(g, p, s);
        case bm_host::kTile128x256:
            if constexpr (LAY != kGradWeights) return launch_tile<LAY, DT, 128, 256, 2, 4>(g, p, s);
            return BITMOE_EINVAL;
        case bm_host::kTile64x128:
            if constexpr (LAY != kGradWeights) return launch_tile<LAY, DT, 64, 128, 2, 2>(g, p, s);
            return BITMOE_EINVAL;
    }
    if (p.grid * 256 >= (int64_t)1 << 32) return BITMOE_EUNSUPPORTED;
    if constexpr (LAY == kForward) {
        if (p.kind == bm_host::kFew) {
            if (p.parts == 1) launch_few<DT, 1>(g, p, s);
            else if (p.parts == 2) launch_few<DT, 2>(g, p, s);
            else launch_few<DT, 4>(g, p, s);
            BM_LAUNCH_CHECK();
            return BITMOE_OK;
        }
    }
    if constexpr (LAY != kForward) {
        if (g.a_low) {
            k_gemm<LAY, DT, 128, 128, 2, 2, true><<<(int)p.grid, 256, 0, s>>>(g, p.mt, p.nt);
            BM_LAUNCH_CHECK();
            return BITMOE_OK;
        }
    }
    k_gemm<LAY, DT, 128, 128, 2, 2, false><<<(int)p.grid, 256, 0, s>>>(g, p.mt, p.nt);
    BM_LAUNCH_CHECK();
    return BITMOE_OK;
}

template <int LAY>
int launch_layout(int dtype, const GemmArgs &g, const bm_host::GemmPlan &p, hipStream_t s) {
    return dtype == BITMOE_BF16 ? launch_layout_of<LAY, BITMOE_BF16>(g, p, s) : launch_layout_of<LAY, BITMOE_F16>(g, p, s);
}

}  // namespace bm
