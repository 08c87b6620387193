// Row-wise kernels of the 16-bit expert layer: the gated activation, the
// weighted combine and the dense product's activation, with their gradients.
// All are bound by memory: each thread takes 8 consecutive values (16 bytes)
// of a row, reads every operand once and computes in fp32.  In bfloat16, cold:
// SwiGLU's backward of 65536 x 2048 213 us (1.34 GB, 6.3 TB/s), combine of 8192 x 8
// x 7168 onto a residual 195 (1.17 GB, 6.0), its backward 386 (2.0 GB, 5.2; half of
// it writes), dz of 8192 x 2048 in two parts with db 30 + 4 us.  A plain copy runs at 5.0, so
// what is left is the launch and the last blocks' end.  8 rows of 2048 take 2.7
// us, a launch.
#include <algorithm>
#include <type_traits>

#include "gemm_util.h"

namespace {

using namespace bm;

// A block's 256 threads over the rows' 8-value pieces: 2^cshift of them along
// a row, the rest over further rows.  Of 256, 128 and 64 the widest that leaves
// no more than a sixteenth of the threads without a piece (7168 values are 3.5
// times 256 pieces, 7 times 128: combine of 8192 x 8 x 7168 173 against 179 us;
// x 2560, 64 against 256: 63 and 72).
struct Grid2 {
    dim3 grid;
    int cshift;
};
Grid2 pieces_grid(int rows, int cols) {
    const int per = (cols + 7) / 8;
    int cs = 0;
    while (cs < 8 && (1 << cs) < per) cs++;
    auto idle = [&](int c) { return (((per + (1 << c) - 1) >> c) << c) - per; };
    int best = cs;
    for (int c = cs; c >= 6 && idle(best) * 16 > per; c--)
        if (idle(c) < idle(best)) best = c;
    cs = best;
    const int rpb = 256 >> cs;
    return {dim3((per + (1 << cs) - 1) >> cs, std::min((rows + rpb - 1) / rpb, 65535)), cs};
}
// body(full, row, column) for each piece: full is a constant, true where all 8
// values are there, so that a piece's loads are issued together, not each
// behind a test (which cost the combine a quarter of its rate).
template <class F>
BM_DEV void for_pieces(int rows, int cols, int cshift, F body) {
    const int c = ((blockIdx.x << cshift) + (threadIdx.x & ((1 << cshift) - 1))) * 8;
    const int step = gridDim.y * (256 >> cshift);
    int r = blockIdx.y * (256 >> cshift) + (threadIdx.x >> cshift);
    if (c + 8 <= cols) {
        for (; r < rows; r += step) body(std::true_type{}, r, c);
    } else if (c < cols) {
        for (; r < rows; r += step) body(std::false_type{}, r, c);
    }
}

struct Mat {
    void *p;
    int64_t ld;
};
// Whether a call's operands go through the memory-side cache (256 MiB), as
// they should where the kernel before left them there or the next will read
// them, or past it: loads past it from 288 MiB moved (combine of k 8, H 7168:
// 44.2 us, 45.9 past it, at 280 MiB; 109 and 88 at 560; swiglu 29.1 and 32.9 at
// 192 MiB, 138 and 116 at 768), stores too from 768 MiB (combine's backward 86
// us with stores through it, 102 past it, at 448 MiB moved; 203 and 187 at 896).
enum { kCached, kLoadsPast, kAllPast };
int past_cache(int64_t bytes) {
    return bytes >= (int64_t)768 << 20 ? kAllPast : bytes >= (int64_t)288 << 20 ? kLoadsPast : kCached;
}
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// a piece as it is in memory, and its values
template <bool FULL, int PAST>
BM_DEV uint4 piece(const Mat &m, int64_t r, int c, int cols) {
    const uint16_t *p = static_cast<const uint16_t *>(m.p) + r * m.ld + c;
    if (!FULL) return load16_part(p, cols - c);
    if (PAST == kCached) return load16(p);
    const u32x4_any u = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any *>(p));
    return make_uint4(u[0], u[1], u[2], u[3]);
}
template <int DT>
BM_DEV void values(const uint4 &u, float *v) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] = elem_f32<DT>(w[j >> 1] >> (16 * (j & 1)) & 0xFFFFu);
}
template <int DT, bool FULL, int PAST>
BM_DEV void put(const Mat &m, int64_t r, int c, int cols, bool f32, const float *v) {
    if (FULL && PAST == kAllPast && !f32) {
        u32x4_any u;
#pragma unroll
        for (int j = 0; j < 4; j++) u[j] = elem_pair<DT>(v[2 * j], v[2 * j + 1]);
        __builtin_nontemporal_store(u, reinterpret_cast<u32x4_any *>(static_cast<uint16_t *>(m.p) + r * m.ld + c));
        return;
    }
    store8<DT>(m.p, r * m.ld + c, FULL ? 8 : cols - c, f32, v);
}

// h = silu(gate) up
template <int DT, int PAST>
__global__ void __launch_bounds__(256)
k_swiglu(Mat gate, Mat up, Mat h, int R, int I, int cshift) {
    for_pieces(R, I, cshift, [&](auto whole, int r, int c) {
        constexpr bool full = decltype(whole)::value;
        float a[8], b[8];
        const uint4 ua = piece<full, PAST>(gate, r, c, I), ub = piece<full, PAST>(up, r, c, I);
        values<DT>(ua, a);
        values<DT>(ub, b);
#pragma unroll
        for (int j = 0; j < 8; j++) a[j] = silu(a[j]) * b[j];
        put<DT, full, PAST>(h, r, c, I, false, a);
    });
}

// with p = 1 / (1 + e^-gate): dgate = dh up p (1 + gate (1 - p)), dup = dh gate p
template <int DT, int PAST>
__global__ void __launch_bounds__(256)
k_swiglu_backward(Mat dh, Mat gate, Mat up, Mat dgate, Mat dup, int R, int I, int cshift) {
    for_pieces(R, I, cshift, [&](auto whole, int r, int c) {
        constexpr bool full = decltype(whole)::value;
        float d[8], a[8], b[8];
        const uint4 ud = piece<full, PAST>(dh, r, c, I), ua = piece<full, PAST>(gate, r, c, I), ub = piece<full, PAST>(up, r, c, I);
        values<DT>(ud, d);
        values<DT>(ua, a);
        values<DT>(ub, b);
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const float p = 1.f / (1.f + __expf(-a[j])), g = a[j];
            a[j] = d[j] * b[j] * p * (1.f + g * (1.f - p));
            b[j] = d[j] * g * p;
        }
        put<DT, full, PAST>(dgate, r, c, I, false, a);
        put<DT, full, PAST>(dup, r, c, I, false, b);
    });
}

// y[t] = sum_j w[t][j] o[t k + j] + residual[t], j ascending; KM >= k rows are
// loaded together
template <int DT, int KM, int PAST>
__global__ void __launch_bounds__(256)
k_combine(Mat o, const float *w, int T, int k, int H, Mat res, bool res_f32, Mat y, bool y_f32, int cshift) {
    for_pieces(T, H, cshift, [&](auto whole, int t, int c) {
        constexpr bool full = decltype(whole)::value;
        uint4 u[KM];
        float wt[KM], acc[8], q[8];
#pragma unroll
        for (int j = 0; j < KM; j++)
            if (j < k) u[j] = piece<full, PAST>(o, (int64_t)t * k + j, c, H);
#pragma unroll
        for (int j = 0; j < KM; j++) wt[j] = w && j < k ? w[(int64_t)t * k + j] : 1.f;
        if (res.p) load8<DT>(res.p, (int64_t)t * res.ld + c, full ? 8 : H - c, res_f32, q);
#pragma unroll
        for (int i = 0; i < 8; i++) acc[i] = 0.f;
#pragma unroll
        for (int j = 0; j < KM; j++)
            if (j < k) {
                float v[8];
                values<DT>(u[j], v);
#pragma unroll
                for (int i = 0; i < 8; i++) acc[i] = fmaf(wt[j], v[i], acc[i]);
            }
        if (res.p) {
#pragma unroll
            for (int i = 0; i < 8; i++) acc[i] += q[i];
        }
        put<DT, full, PAST>(y, t, c, H, y_f32, acc);
    });
}

// One workgroup per token: d_o[t k + j] = w[t][j] dy[t] and, summed over the
// row, dw[t][j] = <dy[t], o[t k + j]>: a thread's pieces in order, the lanes
// by a tree, the waves in order.
template <int DT, int KM, int PAST>
__global__ void __launch_bounds__(256)
k_combine_backward(Mat dy, bool dy_f32, Mat o, const float *w, int t0, int k, int H, Mat d_o, float *dw) {
    __shared__ float part[KM][4];
    const int t = t0 + blockIdx.x, tid = threadIdx.x, nw = blockDim.x >> 6;
    float wt[KM], dot[KM];
#pragma unroll
    for (int j = 0; j < KM; j++) {
        wt[j] = w && j < k ? w[(int64_t)t * k + j] : 1.f;
        dot[j] = 0.f;
    }
    auto at = [&](auto whole, int c) {
        constexpr bool full = decltype(whole)::value;
        float d[8];
        uint4 u[KM];
        if (dw) {
#pragma unroll
            for (int j = 0; j < KM; j++)
                if (j < k) u[j] = piece<full, PAST>(o, (int64_t)t * k + j, c, H);
        }
        load8<DT>(dy.p, (int64_t)t * dy.ld + c, full ? 8 : H - c, dy_f32, d);
        if (d_o.p) {
            // (o is read: d_o may be o)
#pragma unroll
            for (int j = 0; j < KM; j++)
                if (j < k) {
                    float q[8];
#pragma unroll
                    for (int i = 0; i < 8; i++) q[i] = wt[j] * d[i];
                    put<DT, full, PAST>(d_o, (int64_t)t * k + j, c, H, false, q);
                }
        }
        if (dw) {
#pragma unroll
            for (int j = 0; j < KM; j++)
                if (j < k) {
                    float v[8];
                    values<DT>(u[j], v);
#pragma unroll
                    for (int i = 0; i < 8; i++) dot[j] = fmaf(d[i], v[i], dot[j]);
                }
        }
    };
    for (int c = tid * 8; c < H; c += blockDim.x * 8) {
        if (c + 8 <= H) at(std::true_type{}, c);
        else at(std::false_type{}, c);
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

// dz = dy act'(pre) in the operands' type, because the matrix cores take no
// other: in two parts (split16), or rounded to one where the caller wants the
// products in half the time or where one holds it all (relu).  With it the
// slice's column sums of dz itself:
// 32 threads over 256 columns, 8 over the slice's rows.
template <int DT>
__global__ void __launch_bounds__(256)
k_act_backward(bm_host::ActBackward p, int rows_per, int want_sum) {
    __shared__ float red[8][256];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 256 + tx * 8;
    const int r0 = blockIdx.y * rows_per, r1 = min(r0 + rows_per, p.T);
    const Mat dy{const_cast<void *>(p.dy), p.ld_dy}, pre{const_cast<void *>(p.pre), p.ld_pre}, dz{p.dz, p.ld_dz};
    const Mat low_part{static_cast<uint16_t *>(p.dz) + p.low, p.ld_dz};
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    auto at = [&](auto whole, int r) {
        constexpr bool full = decltype(whole)::value;
        float d[8], z[8];
        const uint4 ud = piece<full, kCached>(dy, r, c, p.N), uz = p.pre ? piece<full, kCached>(pre, r, c, p.N) : make_uint4(0, 0, 0, 0);
        values<DT>(ud, d);
        if (p.pre) {
            values<DT>(uz, z);
            slope_row(d, z, p.act);
        }
        if (p.dz && p.low) {
            float high[8], low[8];
            split16<DT>(d, high, low);
            put<DT, full, kCached>(dz, r, c, p.N, false, high);
            put<DT, full, kCached>(low_part, r, c, p.N, false, low);
        } else if (p.dz) {
            put<DT, full, kCached>(dz, r, c, p.N, false, d);
        }
#pragma unroll
        for (int j = 0; j < 8; j++) sum[j] += d[j];
    };
    if (c + 8 <= p.N) {
#pragma unroll 2
        for (int r = r0 + ty; r < r1; r += 8) at(std::true_type{}, r);
    } else if (c < p.N) {
        for (int r = r0 + ty; r < r1; r += 8) at(std::false_type{}, r);
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
    if (c < N) {
        // eight at a time: one round trip to memory for 128 slices
        for (int i0 = ty; i0 < slices; i0 += 128) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] = i0 + 16 * j < slices ? partial[(int64_t)(i0 + 16 * j) * N + c] : 0.f;
#pragma unroll
            for (int j = 0; j < 8; j++) s += v[j];
        }
    }
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

// A row of c at a time for each of the call's rows outside the groups; where
// there are none, a launch (3 to 6 us) and two loads a block.
__global__ void __launch_bounds__(256)
k_clear_ungrouped(const int32_t *offsets, int E, int R, GemmRows c, int cols, bool f32) {
    const int first = min(max(offsets[0], 0), R), behind = max(min(max(offsets[E], 0), R), first);
    for (int i = blockIdx.x; i < first + R - behind; i += gridDim.x) {
        const int row = row_of(c, i < first ? i : behind + i - first);
        if (row < 0) continue;
        for (int n = threadIdx.x * 8; n < cols; n += 256 * 8) {
            const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            store8<BITMOE_BF16>(const_cast<void *>(c.p), (int64_t)row * c.ld + n, cols - n, f32, zero);
        }
    }
}

Mat mat(const bitmoe_rows *m) { return m ? Mat{m->data, m->ld} : Mat{nullptr, 0}; }

// f(type, past) with both as constants
template <class F>
int with(int dtype, int64_t bytes, F f) {
    auto typed = [&](auto dt) {
        switch (past_cache(bytes)) {
            case kCached: return f(dt, std::integral_constant<int, kCached>{});
            case kLoadsPast: return f(dt, std::integral_constant<int, kLoadsPast>{});
            default: return f(dt, std::integral_constant<int, kAllPast>{});
        }
    };
    return dtype == BITMOE_BF16 ? typed(std::integral_constant<int, BITMOE_BF16>{})
                                : typed(std::integral_constant<int, BITMOE_F16>{});
}
// f(at least k) as a constant
template <class F>
int with_k(int k, F f) {
    if (k <= 2) return f(std::integral_constant<int, 2>{});
    if (k <= 4) return f(std::integral_constant<int, 4>{});
    if (k <= 8) return f(std::integral_constant<int, 8>{});
    return f(std::integral_constant<int, 16>{});
}

}  // namespace

namespace bm_host {

int launch_clear_ungrouped(const int32_t *offsets, int E, int R, const GemmRows &c, int cols, bool f32, hipStream_t s) {
    k_clear_ungrouped<<<std::min(R, 1024), 256, 0, s>>>(offsets, E, R, c, cols, f32);
    BM_LAUNCH_CHECK();
    return BITMOE_OK;
}

int launch_swiglu(const bitmoe_rows &gate, const bitmoe_rows &up, const bitmoe_rows &h, int dtype, hipStream_t s) {
    const Grid2 g = pieces_grid(gate.rows, gate.cols);
    return with(dtype, (int64_t)gate.rows * gate.cols * 6, [&](auto dt, auto past) {
        k_swiglu<dt.value, past.value><<<g.grid, 256, 0, s>>>(mat(&gate), mat(&up), mat(&h), gate.rows, gate.cols, g.cshift);
        BM_LAUNCH_CHECK();
        return BITMOE_OK;
    });
}

int launch_swiglu_backward(const bitmoe_rows &dh, const bitmoe_rows &gate, const bitmoe_rows &up,
                           const bitmoe_rows &dgate, const bitmoe_rows &dup, int dtype, hipStream_t s) {
    const Grid2 g = pieces_grid(gate.rows, gate.cols);
    return with(dtype, (int64_t)gate.rows * gate.cols * 10, [&](auto dt, auto past) {
        k_swiglu_backward<dt.value, past.value><<<g.grid, 256, 0, s>>>(mat(&dh), mat(&gate), mat(&up), mat(&dgate),
                                                                       mat(&dup), gate.rows, gate.cols, g.cshift);
        BM_LAUNCH_CHECK();
        return BITMOE_OK;
    });
}

int launch_combine(const bitmoe_rows &o, const float *w, int T, int k, const bitmoe_rows *residual,
                   const bitmoe_rows &y, hipStream_t s) {
    const Grid2 g = pieces_grid(T, o.cols);
    const bool rt = residual && residual->dtype == BITMOE_F32, yt = y.dtype == BITMOE_F32;
    return with_k(k, [&](auto km) {
        return with(o.dtype, (int64_t)T * o.cols * 2 * (k + 2), [&](auto dt, auto past) {
            k_combine<dt.value, km.value, past.value>
                <<<g.grid, 256, 0, s>>>(mat(&o), w, T, k, o.cols, mat(residual), rt, mat(&y), yt, g.cshift);
            BM_LAUNCH_CHECK();
            return BITMOE_OK;
        });
    });
}

int launch_combine_backward(const bitmoe_rows &dy, const bitmoe_rows *o, const float *w, int T, int k,
                            const bitmoe_rows *d_o, float *dw, int dtype, hipStream_t s) {
    // a thread has a piece or more (8192 tokens of k 8, 64 / 128 / 256 threads:
    // H 512 25.7 / - / 39.8 us, 1024 53.8 / 53.0 / 57.6, 2048 128 / 113 / 100)
    const int block = dy.cols <= 512 ? 64 : dy.cols <= 1024 ? 128 : 256;
    const int64_t bytes = (int64_t)T * dy.cols * 2 * (1 + k * ((dw != nullptr) + (d_o != nullptr)));
    return with_k(k, [&](auto km) {
        return with(dtype, bytes, [&](auto dt, auto past) {
            constexpr int most = 1 << 23;               // (a launch holds less than 2^32 threads)
            for (int t0 = 0; t0 < T; t0 += most) {
                k_combine_backward<dt.value, km.value, past.value><<<std::min(T - t0, most), block, 0, s>>>(
                    mat(&dy), dy.dtype == BITMOE_F32, mat(o), w, t0, k, dy.cols, mat(d_o), dw);
                BM_LAUNCH_CHECK();
            }
            return BITMOE_OK;
        });
    });
}

// about 8 blocks a compute unit, at least 16 rows each (512, 1024, 2048, 4096
// blocks: 8192 x 2048 with db 29.0, 25.6, 24.3, 24.7 us, 65536 x 512 50.1, 44.8,
// 44.0, 46.5; more blocks are more partial sums to read again)
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
