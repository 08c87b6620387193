// Products grouped by expert in 8 bits: y = W x over codes, on
// v_mfma_i32_16x16x64_i8 with int32 sums (kernels: gemm_tile.h for rows on 16
// bytes, gemm_i8.h for the others; which one: experts_i8_plan.cpp).
#include "gemm_launch.h"
#include "rows8.h"

namespace {

using namespace bm;
using bm_host::GemmPlan;

template <int DT, int P>
void few(const GemmArgs &g, const GemmPlan &p, hipStream_t s) {
    if (p.chunks == 1) k_i8_few<DT, P, 1><<<(int)p.grid, 256, 0, s>>>(g, p.mt, p.nt);
    else k_i8_few<DT, P, 4><<<(int)p.grid, 256, 0, s>>>(g, p.mt, p.nt);
}

template <int DT>
int product(const GemmArgs &args, const GemmPlan &p, hipStream_t s) {
    if (p.kind == bm_host::kAny || p.kind == bm_host::kFew) {
        if (p.grid * 256 >= (int64_t)1 << 32) return BITMOE_EUNSUPPORTED;
        GemmArgs g = args;
        g.kper = 2 * p.kper;                     // codes
        if (p.kind == bm_host::kAny) k_i8_any<DT><<<(int)p.grid, 256, 0, s>>>(g, p.mt, p.nt);
        else if (p.parts == 1) few<DT, 1>(g, p, s);
        else if (p.parts == 2) few<DT, 2>(g, p, s);
        else few<DT, 4>(g, p, s);
        BM_LAUNCH_CHECK();
        return BITMOE_OK;
    }
    GemmArgs g = args;                           // pairs of codes
    g.a.ld /= 2;
    g.a.span32 = bm_host::span32(g.a.map ? g.a.rows : 256, g.a.ld);
    g.b.ld /= 2;
    g.b.span32 = bm_host::span32(256, g.b.ld);
    g.b_stride /= 2;
    g.K /= 2;
    switch (p.kind) {
        case bm_host::kTile256: return launch_tile<kForward, DT, 256, 256, 2, 4>(g, p, s);
        case bm_host::kTile128x256: return launch_tile<kForward, DT, 128, 256, 2, 4>(g, p, s);
        case bm_host::kTile128: return launch_tile<kForward, DT, 128, 128, 2, 2>(g, p, s);
        default: return launch_tile<kForward, DT, 64, 128, 2, 2>(g, p, s);
    }
}

template <int DT>
int launch_of(const GemmArgs &args, void *ws, hipStream_t s) {
    const GemmPlan p = bm_host::i8_plan(args, bm_host::i8_whole(args));
    GemmArgs g = args;
    g.splits = p.splits;
    g.kper = p.kper;
    if (p.splits == 1) return product<DT>(g, p, s);
    // the parts: plain int32 rows, joined by a second launch
    GemmArgs part = g;
    part.c = GemmRows{ws, nullptr, g.N, g.R, 0, 0, false};
    part.c_f32 = true;
    part.c_split = (int64_t)g.R * g.N;
    part.raw = true;
    const int rc = product<DT>(part, p, s);
    if (rc) return rc;
    const int per = (g.N + 7) / 8;
    int cs = 0;
    while (cs < 8 && (1 << cs) < per) cs++;
    const int rpb = 256 >> cs;
    const dim3 grid((per + (1 << cs) - 1) >> cs, std::min((g.R + rpb - 1) / rpb, 65535));
    const float *parts = static_cast<const float *>(ws);
    if (g.splits == 2) k_i8_join<DT, 2><<<grid, 256, 0, s>>>(g, parts, cs);
    else if (g.splits == 4) k_i8_join<DT, 4><<<grid, 256, 0, s>>>(g, parts, cs);
    else k_i8_join<DT, 8><<<grid, 256, 0, s>>>(g, parts, cs);
    BM_LAUNCH_CHECK();
    return BITMOE_OK;
}

}  // namespace

namespace bm_host {

int launch_gemm_i8(int out, const GemmArgs &g, void *ws, hipStream_t s) {
    return out == BITMOE_BF16 ? launch_of<kI8 + BITMOE_BF16>(g, ws, s) : launch_of<kI8 + BITMOE_F16>(g, ws, s);
}

}  // namespace bm_host
