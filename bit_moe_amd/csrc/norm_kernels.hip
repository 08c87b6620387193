// The norms around a block, fused with its gate and the residual stream:
//   s = scale r + g (o a w_a),  a = 1 / rms(o);   n = s b w_b,  b = 1 / rms(s)
// and their gradients.  With p = w_b dn, t = ds + b (p - s b^2 <p, s> / H) and
// v = g t w_a:  dr = scale t,  do = a (v - o a^2 <v, o> / H),
//   dw_a = sum t g o a,  dg = t o a w_a,  dw_b = sum dn s b.
// One workgroup takes a row, each thread 8 of its columns (P times), which stay
// in registers from the sums to the outputs.  The backward pass needs all its sums
// in one step: <v, o> is taken apart into <g w_a o, ds>, <g w_a o, p> and
// <g w_a o, s>, which do not need t.  Bound by memory.
#include "norm.h"
#include "rows_util.h"

namespace {

using namespace bm;
using bm_host::NormArgs;
using bm_host::NormBackArgs;
using bm_host::NormMat;

constexpr int kMost = 16;           // waves of a workgroup

// Sums of N values over a workgroup's row, the lanes by a tree, the waves in
// order; every thread has them.  part: LDS that no other reduction uses between
// the same two barriers.
template <int N>
BM_DEV void row_sums(float (&v)[N], float (*part)[N]) {
    const int nw = blockDim.x >> 6;
#pragma unroll
    for (int i = 0; i < N; i++) v[i] = wave_sum(v[i]);
    if (nw == 1) return;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int i = 0; i < N; i++) part[threadIdx.x >> 6][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; i++) v[i] = part[0][i];
    for (int w = 1; w < nw; w++)
#pragma unroll
        for (int i = 0; i < N; i++) v[i] += part[w][i];
}

// 1 / rms of a row whose values are taken times f
constexpr float kDown = 0x1p-80f;   // f where the squares' sum leaves fp32
BM_DEV float inv_rms(float sum, int H, float eps, float f) { return rsqrtf(sum / (float)H + eps * f * f); }

template <int DT>
BM_DEV void load_w(const void *w, int c, int n, float (&v)[8]) {
    if (w) load8<DT>(w, c, n, false, v);
    else
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = 1.f;
}
template <int DT>
BM_DEV void load_m(const NormMat &m, int64_t r, int c, int n, float missing, float (&v)[8]) {
    if (m.p) load8<DT>(m.p, r * m.ld + c, n, m.f32, v);
    else
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = missing;
}

template <int DT, int P>
__global__ void __launch_bounds__(1024)
k_block_norm(NormArgs a) {
    __shared__ float part[4][kMost][1];
    const int64_t r = blockIdx.x;
    const int step = blockDim.x * 8;
    float v[P][8], o[P][8];
    auto col = [&](int p) { return (int)threadIdx.x * 8 + p * step; };
    auto left = [&](int p) { return min(max(a.H - col(p), 0), 8); };
    auto at = [&](int p) { return min(col(p), a.H - 1); };          // (an address inside the row, of which `left` are read)
#pragma unroll
    for (int p = 0; p < P; p++) {
        load_m<DT>(a.o, r, at(p), left(p), 0.f, o[p]);
        load_m<DT>(a.res, r, at(p), left(p), 0.f, v[p]);
    }
    auto squares = [&](const float (&x)[P][8], float f, int k) {
        float s[1] = {0.f};
#pragma unroll
        for (int p = 0; p < P; p++)
#pragma unroll
            for (int j = 0; j < 8; j++) s[0] = fmaf(x[p][j] * f, x[p][j] * f, s[0]);
        row_sums<1>(s, part[k]);
        return s[0];
    };
#pragma unroll
    for (int p = 0; p < P; p++)
#pragma unroll
        for (int j = 0; j < 8; j++) v[p][j] *= a.scale;
    if (a.o.p) {
        float f = 1.f, sum = squares(o, f, 0);
        if (!(sum < INFINITY)) sum = squares(o, f = kDown, 1);
        const float ra = inv_rms(sum, a.H, a.eps, f);
#pragma unroll
        for (int p = 0; p < P; p++) {
            float w[8], g[8];
            load_w<DT>(a.wa, at(p), left(p), w);
            load_m<DT>(a.gate, r, at(p), left(p), 1.f, g);
#pragma unroll
            for (int j = 0; j < 8; j++) v[p][j] = fmaf(g[j], o[p][j] * f * ra * w[j], v[p][j]);
        }
    }
    if (a.s.p) {
#pragma unroll
        for (int p = 0; p < P; p++)
            if (left(p) > 0) store8<DT>(a.s.p, r * a.s.ld + col(p), left(p), a.s.f32, v[p]);
    }
    if (!a.n.p) return;
    float f = 1.f, sum = squares(v, f, 2);
    if (!(sum < INFINITY)) sum = squares(v, f = kDown, 3);
    const float rb = inv_rms(sum, a.H, a.eps, f);
#pragma unroll
    for (int p = 0; p < P; p++) {
        float w[8];
        load_w<DT>(a.wb, at(p), left(p), w);
#pragma unroll
        for (int j = 0; j < 8; j++) v[p][j] = v[p][j] * f * rb * w[j];
        if (left(p) > 0) store8<DT>(a.n.p, r * a.n.ld + col(p), left(p), false, v[p]);
    }
}

// A workgroup's rows one after another; the sums over tokens stay in its
// registers and end as one slice of the partial sums.
template <int DT, int P>
__global__ void __launch_bounds__(1024)
k_block_norm_backward(NormBackArgs a) {
    __shared__ float part[2][kMost][6];
    const int step = blockDim.x * 8;
    auto col = [&](int p) { return (int)threadIdx.x * 8 + p * step; };
    auto left = [&](int p) { return min(max(a.H - col(p), 0), 8); };
    auto at = [&](int p) { return min(col(p), a.H - 1); };
    float wa[P][8], wb[P][8], da[P][8], dg[P][8], db[P][8];
#pragma unroll
    for (int p = 0; p < P; p++)
#pragma unroll
        for (int j = 0; j < 8; j++) da[p][j] = dg[p][j] = db[p][j] = 0.f;
    for (int64_t r = blockIdx.x; r < a.T; r += gridDim.x) {
        float dn[P][8], ds[P][8], s[P][8], o[P][8], g[P][8];
#pragma unroll
        for (int p = 0; p < P; p++) {
            load_m<DT>(a.dn, r, at(p), left(p), 0.f, dn[p]);
            load_m<DT>(a.ds, r, at(p), left(p), 0.f, ds[p]);
            load_m<DT>(a.s, r, at(p), left(p), 0.f, s[p]);
            load_m<DT>(a.o, r, at(p), left(p), 0.f, o[p]);
            load_m<DT>(a.gate, r, at(p), left(p), 1.f, g[p]);
            load_w<DT>(a.wa, at(p), left(p), wa[p]);
            load_w<DT>(a.wb, at(p), left(p), wb[p]);
        }
        // s and o times fs and fo
        float q[6], fs = 1.f, fo = 1.f;
        auto sums = [&](int k) {
#pragma unroll
            for (int i = 0; i < 6; i++) q[i] = 0.f;
#pragma unroll
            for (int p = 0; p < P; p++)
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const float x = s[p][j], y = o[p][j], d = wb[p][j] * dn[p][j], u = g[p][j] * wa[p][j] * y;
                    q[0] = fmaf(x, x, q[0]);
                    q[1] = fmaf(d, x, q[1]);
                    q[2] = fmaf(y, y, q[2]);
                    q[3] = fmaf(u, ds[p][j], q[3]);
                    q[4] = fmaf(u, d, q[4]);
                    q[5] = fmaf(u, x, q[5]);
                }
            row_sums<6>(q, part[k]);
        };
        sums(0);
        if (!(q[0] < INFINITY && q[2] < INFINITY)) {
            fs = q[0] < INFINITY ? 1.f : kDown;
            fo = q[2] < INFINITY ? 1.f : kDown;
#pragma unroll
            for (int p = 0; p < P; p++)
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    s[p][j] *= fs;
                    o[p][j] *= fo;
                }
            sums(1);
        }
        // (with the factors: s and o by their own, b and a are fs b', fo a')
        const float b1 = inv_rms(q[0], a.H, a.eps, fs), a1 = inv_rms(q[2], a.H, a.eps, fo);
        const float b = a.dn.p ? fs * b1 : 0.f, mean = b1 * q[1] / (float)a.H;             // of p and s b
        const float vo = q[3] + b * (q[4] - b1 * mean * q[5]), ra = fo * a1, mo = a1 * vo / (float)a.H;
#pragma unroll
        for (int p = 0; p < P; p++) {
            float t[8], d_o[8], u[8];
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float sn = s[p][j] * b1, on = o[p][j] * a1;
                t[j] = a.dn.p ? fmaf(b, wb[p][j] * dn[p][j] - sn * mean, ds[p][j]) : ds[p][j];
                const float gt = g[p][j] * t[j];
                d_o[j] = ra * (gt * wa[p][j] - on * mo);
                u[j] = t[j] * on * wa[p][j];
                if (a.dn.p) db[p][j] = fmaf(dn[p][j], sn, db[p][j]);
                da[p][j] = fmaf(gt, on, da[p][j]);
                dg[p][j] += u[j];
                t[j] *= a.scale;
            }
            if (left(p) > 0) {
                if (a.d_o.p) store8<DT>(a.d_o.p, r * a.d_o.ld + col(p), left(p), false, d_o);
                if (a.dres.p) store8<DT>(a.dres.p, r * a.dres.ld + col(p), left(p), a.dres.f32, t);
                if (a.dgate.p) store8<DT>(a.dgate.p, r * a.dgate.ld + col(p), left(p), false, u);
            }
        }
        if (blockDim.x > 64) __syncthreads();       // part
    }
    float *out = a.partial + (int64_t)blockIdx.x * 3 * a.H;
#pragma unroll
    for (int p = 0; p < P; p++)
        if (left(p) > 0) {
            if (a.dwa) store8<DT>(out, col(p), left(p), true, da[p]);
            if (a.dwb) store8<DT>(out, a.H + col(p), left(p), true, db[p]);
            if (a.dg) store8<DT>(out, 2 * a.H + col(p), left(p), true, dg[p]);
        }
}

// The slices' sums in order: 64 columns a block, four threads over the slices.
__global__ void __launch_bounds__(256)
k_norm_sums(const float *partial, int slices, int H, void *dwa, void *dwb, void *dg, int dw_dtype, int dg_dtype) {
    __shared__ float red[4][64];
    void *out = blockIdx.y == 0 ? dwa : blockIdx.y == 1 ? dwb : dg;
    const int dtype = blockIdx.y == 2 ? dg_dtype : dw_dtype;
    if (!out) return;
    const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6, c = blockIdx.x * 64 + tx;
    float s = 0.f;
    if (c < H)
        for (int i = ty; i < slices; i += 4) s += partial[((int64_t)i * 3 + blockIdx.y) * H + c];
    red[ty][tx] = s;
    __syncthreads();
    if (ty || c >= H) return;
    s = red[0][tx] + red[1][tx] + red[2][tx] + red[3][tx];
    if (dtype == BITMOE_F32) static_cast<float *>(out)[c] = s;
    else static_cast<uint16_t *>(out)[c] = (uint16_t)(dtype == BITMOE_BF16 ? elem_pair<BITMOE_BF16>(s, 0.f)
                                                                          : elem_pair<BITMOE_F16>(s, 0.f));
}

// threads of a row, and pieces of each
int row_threads(int H) { return std::min(((H + 7) / 8 + 63) / 64 * 64, 1024); }
template <class F>
int with(int dtype, int H, F f) {
    auto typed = [&](auto dt) {
        if (H <= 8192) return f(dt, std::integral_constant<int, 1>{});
        return f(dt, std::integral_constant<int, 2>{});
    };
    return dtype == BITMOE_BF16 ? typed(std::integral_constant<int, BITMOE_BF16>{})
                                : typed(std::integral_constant<int, BITMOE_F16>{});
}

}  // namespace

namespace bm_host {

int launch_block_norm(const NormArgs &args, int dtype, hipStream_t st) {
    return with(dtype, args.H, [&](auto dt, auto p) {
        k_block_norm<dt.value, p.value><<<args.T, row_threads(args.H), 0, st>>>(args);
        BM_LAUNCH_CHECK();
        return BITMOE_OK;
    });
}

int norm_slices(int T, int H) {
    (void)H;
    return std::min(T, 512);
}

int launch_block_norm_backward(const NormBackArgs &a, int dtype, hipStream_t st) {
    const int slices = norm_slices(a.T, a.H);
    if (slices > 0) {
        const int rc = with(dtype, a.H, [&](auto dt, auto p) {
            k_block_norm_backward<dt.value, p.value><<<slices, row_threads(a.H), 0, st>>>(a);
            BM_LAUNCH_CHECK();
            return BITMOE_OK;
        });
        if (rc) return rc;
    }
    if (a.dwa || a.dwb || a.dg) {
        k_norm_sums<<<dim3((a.H + 63) / 64, 3), 256, 0, st>>>(a.partial, slices, a.H, a.dwa, a.dwb, a.dg, a.dw_dtype, a.dg_dtype);
        BM_LAUNCH_CHECK();
    }
    return BITMOE_OK;
}

}  // namespace bm_host
