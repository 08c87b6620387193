// Row-wise kernels of the 16-bit expert layer: the gated activation, the
// weighted combine and the dense product's activation, with their gradients.
// All are bound by memory: each thread takes 8 consecutive values (16 bytes)
// of a row, reads every operand once and computes in fp32.
#include <algorithm>

#include "gemm_util.h"

namespace {

using namespace bm;

// A block's 256 threads over the rows' 8-value pieces: 2^cshift of them along
// a row (at least one row's pieces, or 256), the rest over further rows.
struct Grid2 {
    dim3 grid;
    int cshift;
};
Grid2 pieces_grid(int rows, int cols) {
    const int per = (cols + 7) / 8;
    int cs = 0;
    while (cs < 8 && (1 << cs) < per) cs++;
    const int rpb = 256 >> cs;
    return {dim3((per + (1 << cs) - 1) >> cs, std::min((rows + rpb - 1) / rpb, 65535)), cs};
}
#define BM_FOR_PIECES(r, c, rows, cols, cshift)                                                   \
    const int c = ((blockIdx.x << cshift) + (threadIdx.x & ((1 << cshift) - 1))) * 8;             \
    if (c < cols)                                                                                 \
        for (int r = blockIdx.y * (256 >> cshift) + (threadIdx.x >> cshift); r < rows; r += gridDim.y * (256 >> cshift))

struct Mat {
    void *p;
    int64_t ld;
};

// h = silu(gate) up
template <int DT>
__global__ void __launch_bounds__(256)
k_swiglu(Mat gate, Mat up, Mat h, int R, int I, int cshift) {
    BM_FOR_PIECES(r, c, R, I, cshift) {
        float a[8], b[8];
        load8<DT>(gate.p, (int64_t)r * gate.ld + c, I - c, false, a);
        load8<DT>(up.p, (int64_t)r * up.ld + c, I - c, false, b);
#pragma unroll
        for (int j = 0; j < 8; j++) a[j] = silu(a[j]) * b[j];
        store8<DT>(h.p, (int64_t)r * h.ld + c, I - c, false, a);
    }
}

// with p = 1 / (1 + e^-gate): dgate = dh up p (1 + gate (1 - p)), dup = dh gate p
template <int DT>
__global__ void __launch_bounds__(256)
k_swiglu_backward(Mat dh, Mat gate, Mat up, Mat dgate, Mat dup, int R, int I, int cshift) {
    BM_FOR_PIECES(r, c, R, I, cshift) {
        float d[8], a[8], b[8];
        load8<DT>(dh.p, (int64_t)r * dh.ld + c, I - c, false, d);
        load8<DT>(gate.p, (int64_t)r * gate.ld + c, I - c, false, a);
        load8<DT>(up.p, (int64_t)r * up.ld + c, I - c, false, b);
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const float p = 1.f / (1.f + __expf(-a[j])), g = a[j];
            a[j] = d[j] * b[j] * p * (1.f + g * (1.f - p));
            b[j] = d[j] * g * p;
        }
        store8<DT>(dgate.p, (int64_t)r * dgate.ld + c, I - c, false, a);
        store8<DT>(dup.p, (int64_t)r * dup.ld + c, I - c, false, b);
    }
}

// y[t] = sum_j w[t][j] o[t k + j] + residual[t], j ascending; KM >= k rows are
// loaded together
template <int DT, int KM>
__global__ void __launch_bounds__(256)
k_combine(Mat o, const float *w, int T, int k, int H, Mat res, bool res_f32, Mat y, bool y_f32, int cshift) {
    BM_FOR_PIECES(t, c, T, H, cshift) {
        float v[KM][8], acc[8];
#pragma unroll
        for (int j = 0; j < KM; j++)
            if (j < k) load8<DT>(o.p, ((int64_t)t * k + j) * o.ld + c, H - c, false, v[j]);
#pragma unroll
        for (int i = 0; i < 8; i++) acc[i] = 0.f;
#pragma unroll
        for (int j = 0; j < KM; j++)
            if (j < k) {
                const float wj = w ? w[(int64_t)t * k + j] : 1.f;
#pragma unroll
                for (int i = 0; i < 8; i++) acc[i] = fmaf(wj, v[j][i], acc[i]);
            }
        if (res.p) {
            float q[8];
            load8<DT>(res.p, (int64_t)t * res.ld + c, H - c, res_f32, q);
#pragma unroll
            for (int i = 0; i < 8; i++) acc[i] += q[i];
        }
        store8<DT>(y.p, (int64_t)t * y.ld + c, H - c, y_f32, acc);
    }
}

// One workgroup per token: d_o[t k + j] = w[t][j] dy[t] and, summed over the
// row, dw[t][j] = <dy[t], o[t k + j]>: a thread's pieces in order, the lanes
// by a tree, the waves in order.
template <int DT, int KM>
__global__ void __launch_bounds__(256)
k_combine_backward(Mat dy, bool dy_f32, Mat o, const float *w, int T, int k, int H, Mat d_o, float *dw) {
    __shared__ float part[KM][4];
    const int t = blockIdx.x, tid = threadIdx.x, nw = blockDim.x >> 6;
    float wt[KM], dot[KM];
#pragma unroll
    for (int j = 0; j < KM; j++) {
        wt[j] = w && j < k ? w[(int64_t)t * k + j] : 1.f;
        dot[j] = 0.f;
    }
    for (int c = tid * 8; c < H; c += blockDim.x * 8) {
        float d[8], v[KM][8];
        load8<DT>(dy.p, (int64_t)t * dy.ld + c, H - c, dy_f32, d);
        if (dw) {
#pragma unroll
            for (int j = 0; j < KM; j++)
                if (j < k) load8<DT>(o.p, ((int64_t)t * k + j) * o.ld + c, H - c, false, v[j]);
#pragma unroll
            for (int j = 0; j < KM; j++)
                if (j < k)
#pragma unroll
                    for (int i = 0; i < 8; i++) dot[j] = fmaf(d[i], v[j][i], dot[j]);
        }
        if (d_o.p) {
#pragma unroll
            for (int j = 0; j < KM; j++)
                if (j < k) {
                    float q[8];
#pragma unroll
                    for (int i = 0; i < 8; i++) q[i] = wt[j] * d[i];
                    store8<DT>(d_o.p, ((int64_t)t * k + j) * d_o.ld + c, H - c, false, q);
                }
        }
    }
    if (!dw) return;
#pragma unroll
    for (int j = 0; j < KM; j++)
        if (j < k) {
            const float s = wave_sum(dot[j]);
            if ((tid & 63) == 0) part[j][tid >> 6] = s;
        }
    __syncthreads();
    if (tid < k) {
        float s = 0.f;
        for (int i = 0; i < nw; i++) s += part[tid][i];
        dw[(int64_t)t * k + tid] = s;
    }
}

// dz = dy act'(pre), and the slice's column sums of dz before its rounding:
// 32 threads over 256 columns, 8 over the slice's rows.
template <int DT>
__global__ void __launch_bounds__(256)
k_act_backward(bm_host::ActBackward p, int rows_per, int want_sum) {
    __shared__ float red[8][256];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 256 + tx * 8;
    const int r0 = blockIdx.y * rows_per, r1 = min(r0 + rows_per, p.T);
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (c < p.N)
        for (int r = r0 + ty; r < r1; r += 8) {
            float d[8];
            load8<DT>(p.dy, (int64_t)r * p.ld_dy + c, p.N - c, false, d);
            if (p.pre) {
                float z[8];
                load8<DT>(p.pre, (int64_t)r * p.ld_pre + c, p.N - c, false, z);
#pragma unroll
                for (int j = 0; j < 8; j++) d[j] *= act_slope(z[j], p.act);
            }
            if (p.dz) store8<DT>(p.dz, (int64_t)r * p.ld_dz + c, p.N - c, false, d);
#pragma unroll
            for (int j = 0; j < 8; j++) sum[j] += d[j];
        }
    if (!want_sum) return;
#pragma unroll
    for (int j = 0; j < 8; j++) red[ty][tx * 8 + j] = sum[j];
    __syncthreads();
    const int col = blockIdx.x * 256 + threadIdx.x;
    if (col < p.N) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; i++) s += red[i][threadIdx.x];
        p.partial[(int64_t)blockIdx.y * p.N + col] = s;
    }
}
// db from the slices' sums: 16 columns a block, 16 threads over the slices
__global__ void __launch_bounds__(256)
k_bias_grad(const float *partial, int slices, int N, void *db, int db_dtype) {
    __shared__ float red[16][16];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, c = blockIdx.x * 16 + tx;
    float s = 0.f;
    if (c < N)
        for (int i = ty; i < slices; i += 16) s += partial[(int64_t)i * N + c];
    red[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && c < N) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < 16; i++) s += red[i][tx];
        if (db_dtype == BITMOE_F32) static_cast<float *>(db)[c] = s;
        else static_cast<uint16_t *>(db)[c] = (uint16_t)(db_dtype == BITMOE_BF16 ? elem_pair<BITMOE_BF16>(s, 0.f)
                                                                              : elem_pair<BITMOE_F16>(s, 0.f));
    }
}

Mat mat(const bitmoe_rows *m) { return m ? Mat{m->data, m->ld} : Mat{nullptr, 0}; }

template <int KM>
int combine_k(const bitmoe_rows &o, const float *w, int T, int k, const bitmoe_rows *res, const bitmoe_rows &y,
              hipStream_t s) {
    const Grid2 g = pieces_grid(T, o.cols);
    const bool rt = res && res->dtype == BITMOE_F32, yt = y.dtype == BITMOE_F32;
    if (o.dtype == BITMOE_BF16)
        k_combine<BITMOE_BF16, KM><<<g.grid, 256, 0, s>>>(mat(&o), w, T, k, o.cols, mat(res), rt, mat(&y), yt, g.cshift);
    else
        k_combine<BITMOE_F16, KM><<<g.grid, 256, 0, s>>>(mat(&o), w, T, k, o.cols, mat(res), rt, mat(&y), yt, g.cshift);
    BM_LAUNCH_CHECK();
    return BITMOE_OK;
}
template <int KM>
int combine_backward_k(const bitmoe_rows &dy, const bitmoe_rows *o, const float *w, int T, int k,
                       const bitmoe_rows *d_o, float *dw, int dtype, hipStream_t s) {
    const int block = dy.cols <= 512 ? 64 : 256;
    if (dtype == BITMOE_BF16)
        k_combine_backward<BITMOE_BF16, KM><<<T, block, 0, s>>>(mat(&dy), dy.dtype == BITMOE_F32, mat(o), w, T, k, dy.cols, mat(d_o), dw);
    else
        k_combine_backward<BITMOE_F16, KM><<<T, block, 0, s>>>(mat(&dy), dy.dtype == BITMOE_F32, mat(o), w, T, k, dy.cols, mat(d_o), dw);
    BM_LAUNCH_CHECK();
    return BITMOE_OK;
}

}  // namespace

namespace bm_host {

int launch_swiglu(const bitmoe_rows &gate, const bitmoe_rows &up, const bitmoe_rows &h, int dtype, hipStream_t s) {
    const Grid2 g = pieces_grid(gate.rows, gate.cols);
    if (dtype == BITMOE_BF16)
        k_swiglu<BITMOE_BF16><<<g.grid, 256, 0, s>>>(mat(&gate), mat(&up), mat(&h), gate.rows, gate.cols, g.cshift);
    else
        k_swiglu<BITMOE_F16><<<g.grid, 256, 0, s>>>(mat(&gate), mat(&up), mat(&h), gate.rows, gate.cols, g.cshift);
    BM_LAUNCH_CHECK();
    return BITMOE_OK;
}

int launch_swiglu_backward(const bitmoe_rows &dh, const bitmoe_rows &gate, const bitmoe_rows &up,
                           const bitmoe_rows &dgate, const bitmoe_rows &dup, int dtype, hipStream_t s) {
    const Grid2 g = pieces_grid(gate.rows, gate.cols);
    if (dtype == BITMOE_BF16)
        k_swiglu_backward<BITMOE_BF16><<<g.grid, 256, 0, s>>>(mat(&dh), mat(&gate), mat(&up), mat(&dgate), mat(&dup),
                                                              gate.rows, gate.cols, g.cshift);
    else
        k_swiglu_backward<BITMOE_F16><<<g.grid, 256, 0, s>>>(mat(&dh), mat(&gate), mat(&up), mat(&dgate), mat(&dup),
                                                             gate.rows, gate.cols, g.cshift);
    BM_LAUNCH_CHECK();
    return BITMOE_OK;
}

int launch_combine(const bitmoe_rows &o, const float *w, int T, int k, const bitmoe_rows *residual,
                   const bitmoe_rows &y, hipStream_t s) {
    if (k <= 2) return combine_k<2>(o, w, T, k, residual, y, s);
    if (k <= 8) return combine_k<8>(o, w, T, k, residual, y, s);
    return combine_k<16>(o, w, T, k, residual, y, s);
}

int launch_combine_backward(const bitmoe_rows &dy, const bitmoe_rows *o, const float *w, int T, int k,
                            const bitmoe_rows *d_o, float *dw, int dtype, hipStream_t s) {
    if (k <= 2) return combine_backward_k<2>(dy, o, w, T, k, d_o, dw, dtype, s);
    if (k <= 8) return combine_backward_k<8>(dy, o, w, T, k, d_o, dw, dtype, s);
    return combine_backward_k<16>(dy, o, w, T, k, d_o, dw, dtype, s);
}

// about 8 blocks a compute unit, at least 16 rows each
int act_backward_slices(int T, int N) {
    const int cols = (N + 255) / 256;
    return std::min((T + 15) / 16, std::min(std::max(2048 / cols, 1), 65535));
}

int launch_act_backward(const ActBackward &p, int dtype, hipStream_t s) {
    const int slices = act_backward_slices(p.T, p.N);
    if (slices > 0) {
        const dim3 grid((p.N + 255) / 256, slices);
        const int rows_per = (p.T + slices - 1) / slices;
        if (dtype == BITMOE_BF16) k_act_backward<BITMOE_BF16><<<grid, 256, 0, s>>>(p, rows_per, p.db != nullptr);
        else k_act_backward<BITMOE_F16><<<grid, 256, 0, s>>>(p, rows_per, p.db != nullptr);
        BM_LAUNCH_CHECK();
    }
    if (p.db) {
        k_bias_grad<<<(p.N + 15) / 16, 256, 0, s>>>(p.partial, slices, p.N, p.db, p.db_dtype);
        BM_LAUNCH_CHECK();
    }
    return BITMOE_OK;
}

}  // namespace bm_host
