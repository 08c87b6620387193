// Products grouped by expert in 8 bits: y = W x over codes, on
// v_mfma_i32_16x16x64_i8 with int32 sums (kernels: gemm_tile.h for rows on 16
// bytes, gemm_i8.h for the others; which one: experts_i8_plan.cpp).
#include "gemm_launch.h"
#include "rows8.h"

namespace {

using namespace bm;
using bm_host::GemmPlan;

// Rows of K codes at any address to rows of ld, whole 16-byte pieces with zeros
// behind K, at `to`: the call's rows of x (with their scales) that lie in a group,
// and the rows of W of the experts that have some.  A wave a row, a word a lane: the
// word of memory that holds its first code and, where it is not all of them, the
// next one (neighbouring lanes' words are one access; 16 bytes a lane at an odd
// address take several times an even one's).  No word without a code is read.
__global__ void __launch_bounds__(256)
k_i8_pack(GemmArgs g, uint8_t *x, float *scale, uint8_t *w, int ld) {
    const int lane = threadIdx.x & 63, r0 = group_start(g, 0), r1 = group_start(g, g.E);
    const int64_t last = g.R + (int64_t)g.E * g.N, step = (int64_t)gridDim.x * 4;
    for (int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); i < last; i += step) {
        const uint8_t *from;
        uint8_t *to;
        if (i < g.R) {
            const int r = (int)i;
            if (r < r0 || r >= r1) continue;
            const int row = row_of(g.a, r);
            from = row >= 0 ? static_cast<const uint8_t *>(g.a.p) + (int64_t)row * g.a.ld : nullptr;
            to = x + (int64_t)r * ld;
            if (lane == 0) scale[r] = row >= 0 ? g.a_scale[row * g.a_ld_scale] : 0.f;
        } else {
            const int e = (int)((i - g.R) / g.N), n = (int)(i - g.R - (int64_t)e * g.N);
            if (group_start(g, e + 1) <= group_start(g, e)) continue;
            from = static_cast<const uint8_t *>(g.b.p) + (int64_t)e * g.b_stride + (int64_t)n * g.b.ld;
            to = w + (i - g.R) * ld;
        }
        const int off = (int)(reinterpret_cast<uintptr_t>(from) & 3), K = from ? g.K : 0;
        const uint32_t *words = reinterpret_cast<const uint32_t *>(from - off);
        for (int j0 = 0; j0 < ld / 4; j0 += 256) {
            uint32_t lo[4], hi[4];
#pragma unroll
            for (int u = 0; u < 4; u++) {
                const int j = j0 + 64 * u + lane;
                lo[u] = 4 * j < K ? words[j] : 0;
                hi[u] = off && 4 * j + 4 - off < K ? words[j + 1] : 0;
            }
#pragma unroll
            for (int u = 0; u < 4; u++) {
                const int j = j0 + 64 * u + lane, left = K - 4 * j;
                uint32_t v = __builtin_amdgcn_alignbyte(hi[u], lo[u], off);
                if (left < 4) v = left > 0 ? v & ((1u << (8 * left)) - 1) : 0;
                if (j < ld / 4) *reinterpret_cast<uint32_t *>(to + 4 * j) = v;
            }
        }
    }
}

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
    if (p.pack) {
        const bm_host::I8Pack k = bm_host::i8_pack(g.E, g.R, g.N, g.K);
        char *at = static_cast<char *>(ws) + p.ws - k.bytes;
        uint8_t *x = reinterpret_cast<uint8_t *>(at + k.x), *w = reinterpret_cast<uint8_t *>(at + k.w);
        float *scale = reinterpret_cast<float *>(at + k.scale);
        const int64_t rows = g.R + (int64_t)g.E * g.N;
        k_i8_pack<<<(int)std::min<int64_t>((rows + 3) / 4, 1 << 16), 256, 0, s>>>(g, x, scale, w, (int)k.ld);
        BM_LAUNCH_CHECK();
        g.a = GemmRows{x, nullptr, k.ld, g.R, 0, 0, false};
        g.b = GemmRows{w, nullptr, k.ld, g.N, 0, 0, false};
        g.b_stride = (int64_t)g.N * k.ld;
        g.a_scale = scale;
        g.a_ld_scale = 1;
        g.K = (int)k.ld;
    }
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
