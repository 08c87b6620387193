// Matrix products of the 16-bit expert layer: forward, rows' gradient and
// weights' gradient over groups of rows of any size, C = A B^T on
// v_mfma_f32_16x16x32 with fp32 accumulation (kernels: gemm_tile.h,
// gemm_any.h; which one: experts_plan.cpp), and the join of a split contraction.
#include <algorithm>
#include <type_traits>

#include "gemm_util.h"

namespace {

using namespace bm;

// C = the parts' sum (in order), with the epilogue.  Parts are float32 [splits]
// [rows][N]; rows are the call's (those of a group), or the experts' rows one
// after another.  Bound by the parts' bytes, which the caches hold where it is
// worth splitting at all.  NS parts' loads are issued together (16 parts one
// after another took 9 us), and no more than there are: 2 parts of 2048 x 2048
// with bias, residual and pre took 12.6 us where each was loaded four times.
template <int LAY, int DT, int NS>
__global__ void __launch_bounds__(256)
k_join(GemmArgs g, const float *part, int rows, int cshift) {
    const int per = 256 >> cshift, n = ((blockIdx.x << cshift) + (threadIdx.x & ((1 << cshift) - 1))) * 8;
    const int left = g.N - n;
    if (left <= 0) return;
    const int r0 = LAY == kGradWeights ? 0 : group_start(g, 0), r1 = LAY == kGradWeights ? rows : group_start(g, g.E);
    const int64_t step = (int64_t)rows * g.N;
    for (int r = r0 + blockIdx.y * per + (threadIdx.x >> cshift); r < r1; r += gridDim.y * per) {
        const int e = LAY == kGradWeights ? r / g.M : 0, row = LAY == kGradWeights ? r - e * g.M : row_of(g.c, r);
        if (row < 0) continue;
        const float *p = part + (int64_t)r * g.N + n;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        float bias[8], res[8];
        if (left >= 8) {
            if (LAY == kForward && g.bias) load_row<DT>(g.bias, n, false, bias);
            if (LAY == kForward && g.res) load_row<DT>(g.res, (int64_t)row * g.ld_res + n, g.res_f32, res);
        }
        for (int s0 = 0; s0 < g.splits; s0 += NS) {              // (splits is a multiple of NS)
            float o[NS][8];
            if (left >= 8) {
#pragma unroll
                for (int s = 0; s < NS; s++) load8<DT>(p, (s0 + s) * step, 8, true, o[s]);
            } else {
                for (int s = 0; s < NS; s++) load8<DT>(p, (s0 + s) * step, left, true, o[s]);
            }
#pragma unroll
            for (int s = 0; s < NS; s++)
#pragma unroll
                for (int j = 0; j < 8; j++) v[j] += o[s][j];
        }
        if (left >= 8) {
            finish<LAY, DT>(g, e, 0, row, n, v, bias, res);
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++)
                if (j < left) {
                    float one[1] = {v[j]}, bias[1] = {0.f}, res[1] = {0.f};
                    if (LAY == kForward && g.bias) load_row<DT>(g.bias, n + j, false, bias);
                    if (LAY == kForward && g.res) load_row<DT>(g.res, (int64_t)row * g.ld_res + n + j, g.res_f32, res);
                    finish<LAY, DT>(g, e, 0, row, n + j, one, bias, res);
                }
        }
    }
}

// The rows that two operands' maps give the weights' gradient; one that either
// lacks adds nothing, whatever the other holds (0 times an infinity would).
__global__ void __launch_bounds__(256)
k_rows(GemmRows a, GemmRows b, int R, int32_t *arows, int32_t *brows) {
    const int r = blockIdx.x * 256 + threadIdx.x;
    if (r >= R) return;
    const int ra = row_of(a, r), rb = row_of(b, r);
    arows[r] = rb < 0 ? -1 : ra;
    brows[r] = ra < 0 ? -1 : rb;
}

template <int LAY>
int join(int dtype, const GemmArgs &g, const float *part, int rows, hipStream_t s) {
    const int per = (g.N + 7) / 8;
    int cs = 0;
    while (cs < 8 && (1 << cs) < per) cs++;
    const int rpb = 256 >> cs;
    const dim3 grid((per + (1 << cs) - 1) >> cs, std::min((rows + rpb - 1) / rpb, 65535));
    auto go = [&](auto dt, auto ns) {
        k_join<LAY, dt.value, ns.value><<<grid, 256, 0, s>>>(g, part, rows, cs);
        BM_LAUNCH_CHECK();
        return BITMOE_OK;
    };
    auto typed = [&](auto dt) {
        if (g.splits == 2) return go(dt, std::integral_constant<int, 2>{});
        if (g.splits == 4) return go(dt, std::integral_constant<int, 4>{});
        return go(dt, std::integral_constant<int, 8>{});
    };
    return dtype == BITMOE_BF16 ? typed(std::integral_constant<int, BITMOE_BF16>{})
                                : typed(std::integral_constant<int, BITMOE_F16>{});
}

int launch(int layout, int dtype, const GemmArgs &g, const bm_host::GemmPlan &p, hipStream_t s) {
    switch (layout) {
        case kForward: return bm_host::launch_experts_fwd(dtype, g, p, s);
        case kGradRows: return bm_host::launch_experts_dx(dtype, g, p, s);
        default: return bm_host::launch_experts_dw(dtype, g, p, s);
    }
}

}  // namespace

namespace bm_host {

int launch_gemm(int layout, int dtype, const GemmArgs &args, void *ws, hipStream_t s) {
    const GemmPlan p = gemm_plan(layout, args, gemm_whole(layout, args));
    GemmArgs g = args;
    g.splits = p.splits;
    g.kper = p.kper;
    if (layout == kGradWeights && (g.a.map || g.b.map) && p.kind != kAny && g.R > 0) {
        const size_t each = ((size_t)g.R * 4 + 255) / 256 * 256;
        int32_t *rows = reinterpret_cast<int32_t *>(static_cast<char *>(ws) + p.ws - 2 * each);
        k_rows<<<(g.R + 255) / 256, 256, 0, s>>>(g.a, g.b, g.R, rows, rows + each / 4);
        BM_LAUNCH_CHECK();
        g.arows = rows;
        g.brows = rows + each / 4;
        g.a.span32 = span32(g.a.rows, g.a.ld);
        g.b.span32 = span32(g.b.rows, g.b.ld);
    }
    if (p.splits == 1) return launch(layout, dtype, g, p, s);
    // the parts: plain float32 rows, joined by a second launch
    const int rows = layout == kGradWeights ? g.E * g.M : g.R;
    GemmArgs part = g;
    part.c = GemmRows{ws, nullptr, g.N, layout == kGradWeights ? g.M : g.R, 0, 0, false};
    part.c_stride = (int64_t)g.M * g.N;
    part.c_f32 = true;
    part.c_split = (int64_t)rows * g.N;
    part.accumulate = false;
    part.act = BITMOE_ACT_NONE;
    part.bias = part.res = nullptr;
    part.pre = nullptr;
    const int rc = launch(layout, dtype, part, p, s);
    if (rc) return rc;
    switch (layout) {
        case kForward: return join<kForward>(dtype, g, static_cast<float *>(ws), rows, s);
        case kGradRows: return join<kGradRows>(dtype, g, static_cast<float *>(ws), rows, s);
        default: return join<kGradWeights>(dtype, g, static_cast<float *>(ws), rows, s);
    }
}

}  // namespace bm_host
