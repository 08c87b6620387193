// Rows in 8 bits: activations and weights into int8 codes with a scale for 32,
// 64 or 128 columns or for the whole row, and back; the gated activation into
// them, and with its inputs kept in them.
//
// A code is rint(127 x / m) for the block's largest magnitude m.  The quotient
// t / m has to be right where it is a tie (x = m / 2 gives 63.5, which is common in
// 16 bits) and within a few steps elsewhere, where no 16-bit x comes near one.  An
// estimate q = t inv with inv = 1 / m to a step, and one move by its exact remainder
// (an fma), q + (t - q m) inv, is: the move's own error is 2^-22 of two steps, so a
// quotient that float32 holds comes out as it is.  m and x are first taken to m's own
// power of two, so nothing overflows on the way.
// Bound by memory, and close behind it by the arithmetic of a code (9 operations) and
// of silu: 65536 x 2048 with its inputs kept forward 192 us, backward 182, one after the
// other 345 to 349 (6.3 TB/s); 16384 x 7168 to codes 67 us and back 61, one after the other 117,
// by rows 66, 8192 x 7168 by rows 33; silu into codes 65536 x 2048 by rows 115 us, in
// blocks 114.  (us a call, calls one after another on changing inputs.)  8 columns
// a thread: 16 make a store past the cache half a line (the backward pass 299 us against
// 219 before its other steps).  The codes are stored through the cache, where what reads
// them next finds them.
#include "rows8.h"
#include "rows_util.h"

namespace {

using namespace bm;

// ---- codes ----------------------------------------------------------------
struct Coder {
    float f, m, inv;        // x f = 127 x 2^-e, m 2^-e, its reciprocal
    uint32_t keep;          // 0: the block's codes are 0
};
// of a block's largest magnitude (its bits, above infinity's for a NaN)
BM_DEV Coder coder(uint32_t bits, float *scale) {
    Coder k;
    // 2^-e, at most 2^100 (what is smaller than 2^-100 need not reach 1)
    const float to1 = __uint_as_float((uint32_t)min(max(254 - (int)(bits >> 23), 1), 227) << 23);
    const float m = __uint_as_float(bits);
    k.m = m * to1;
    k.f = 127.f * to1;
    k.inv = __builtin_amdgcn_rcpf(k.m);
    k.keep = bits != 0 && bits < 0x7F800000u ? 0xFFFFFFFFu : 0u;
    // m / 127, correctly rounded: an estimate by 1 / 127 rounded, and its remainder;
    // at most what 127 times stays finite (fp32's largest value / 127, rounded down)
    const float c = 1.f / 127.f, q = k.m * c, s = fmaf(fmaf(-127.f, q, k.m), c, q);
    const float from1 = __uint_as_float((254u << 23) - __float_as_uint(to1));
    *scale = bits < 0x7F800000u ? fminf(s * from1, 0x1.0204060000000p+121f) : __uint_as_float(0x7FC00000u);
    return k;
}
BM_DEV uint32_t max_bits(uint32_t m, float v) { return max(m, __float_as_uint(v) & 0x7FFFFFFFu); }
BM_DEV uint32_t code_bits(const Coder &k, float x) {
    const float t = x * k.f, q = t * k.inv;
    // (the low byte of a value near 1.5 2^23 is that of the integer nearest to what was added)
    return __float_as_uint(fmaf(fmaf(-q, k.m, t), k.inv, q) + 12582912.f);
}
BM_DEV uint32_t code4(const Coder &k, const float *x) {
    const uint32_t lo = __builtin_amdgcn_perm(code_bits(k, x[1]), code_bits(k, x[0]), 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(code_bits(k, x[3]), code_bits(k, x[2]), 0x04000C0Cu);
    return (lo | hi) & k.keep;
}
// the values of four codes
BM_DEV void value4(uint32_t w, float scale, float *v) {
    w ^= 0x80808080u;
#pragma unroll
    for (int j = 0; j < 4; j++) v[j] = ((float)(w >> (8 * j) & 0xFFu) - 128.f) * scale;
}

typedef uint32_t u32x2_b __attribute__((ext_vector_type(2), aligned(1)));
// the first n of eight codes
BM_DEV void put_codes(int8_t *p, int n, const uint32_t (&w)[2]) {
    if (n >= 8) {
        *reinterpret_cast<u32x2_b *>(p) = u32x2_b{w[0], w[1]};
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (j < n) p[j] = (int8_t)(w[j >> 2] >> (8 * (j & 3)));
    }
}
template <int PAST>
BM_DEV uint2 get_codes(const int8_t *p, int n) {
    if (n >= 8) {
        const u32x2_b *q = reinterpret_cast<const u32x2_b *>(p);
        const u32x2_b u = PAST == kCached ? *q : __builtin_nontemporal_load(q);
        return make_uint2(u[0], u[1]);
    }
    uint32_t w[2] = {0, 0};
    if (n > 0) {
        // (all loads at once: load_part)
        uint32_t e[8];
#pragma unroll
        for (int j = 0; j < 8; j++) e[j] = (uint8_t)p[min(j, n - 1)];
#pragma unroll
        for (int j = 0; j < 8; j++) w[j >> 2] |= j < n ? e[j] << (8 * (j & 3)) : 0;
    }
    return make_uint2(w[0], w[1]);
}
BM_DEV void values8(const uint2 &u, float scale, float (&v)[8]) {
    value4(u.x, scale, v);
    value4(u.y, scale, v + 4);
}

// p = 1 / (1 + e^-z) and 1 - p, each to a few steps of its own and |z| for the exponent's
// rounding, by t = e^-|z|, so that the reciprocal is of 1 .. 2, where the one instruction is
// good to a step (a division's ten, of values that a kernel needs once each, would bound
// these kernels).  t is the square of e^-|z|/2: the exponential instruction gives 0 below
// float32's smallest normal value, from |z| = 87.3, where z p is still 10^-36
// (the multiplication takes the forward pass of 65536 x 2048 from 187.8 to 188.7 us, the
// backward 214.7 to 215.0, one call after another).
BM_DEV void logistic(float z, float *p, float *not_p) {
    const float e = __builtin_amdgcn_exp2f(fabsf(z) * -0.72134752044448170f);      // (log2(e) / 2)
    const float t = e * e, r = __builtin_amdgcn_rcpf(1.f + t), s = t * r;
    *p = z < 0.f ? s : r;
    *not_p = z < 0.f ? r : s;
}
BM_DEV float silu_of(float z) {
    float p, q;
    logistic(z, &p, &q);
    return z * p;
}

struct Rows8 {
    int8_t *q;
    float *scale;
    int64_t ld, ld_scale;
    int shift;              // log2 of the block, or 31: the row
};

// ---- blocks of columns ----------------------------------------------------
// A thread takes 8 columns, so that each access of a wave is one run of memory (of
// 16 a thread, stores past the cache would be halves of lines); the 4, 8 or 16 lanes
// of a block exchange their largest magnitudes (all of them are there: a row's
// threads are a multiple of 16).
template <int CTRL>
BM_DEV uint32_t dpp_max(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true));
}
template <int SHIFT>
BM_DEV uint32_t block_max(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; j++) m = max_bits(m, v[j]);
    m = dpp_max<0x4E>(dpp_max<0xB1>(m));         // lanes ^ 1, ^ 2
    if (SHIFT >= 6) m = dpp_max<0x141>(m);       // the other four of eight
    if (SHIFT >= 7) m = dpp_max<0x140>(m);       // the other eight of sixteen
    return m;
}
template <int SHIFT>
BM_DEV void put_block(const Rows8 &q, int64_t r, int c, int n, const float (&v)[8]) {
    float scale;
    const Coder k = coder(block_max<SHIFT>(v), &scale);
    const uint32_t w[2] = {code4(k, v), code4(k, v + 4)};
    if (n > 0) put_codes(q.q + r * q.ld + c, n, w);
    if ((c & ((1 << SHIFT) - 1)) == 0 && n > 0) q.scale[r * q.ld_scale + (c >> SHIFT)] = scale;
}
// body(row, column, how many of its 8 are there) for every thread of every
// block of columns that has any
template <int SHIFT, class F>
BM_DEV void for_blocks(int rows, int cols, int cshift, F body) {
    const int c = ((blockIdx.x << cshift) + (threadIdx.x & ((1 << cshift) - 1))) * 8;
    const int step = gridDim.y * (256 >> cshift);
    int r = blockIdx.y * (256 >> cshift) + (threadIdx.x >> cshift);
    const int first = c & ~((1 << SHIFT) - 1);
    if (first + (1 << SHIFT) <= cols) {
        for (; r < rows; r += step) body(r, c, std::integral_constant<int, 8>{});
    } else if (first < cols) {
        for (; r < rows; r += step) body(r, c, min(max(cols - c, 0), 8));
    }
}

template <int DT, bool F32, int SHIFT, int PAST>
__global__ void __launch_bounds__(256)
k_quantize_blocks(Mat x, Rows8 q, int R, int C, int cshift) {
    for_blocks<SHIFT>(R, C, cshift, [&](int r, int c, auto n) {
        float v[8];
        load_values<DT, PAST>(x.p, r * x.ld + c, n, F32, v);
        put_block<SHIFT>(q, r, c, n, v);
    });
}

template <int DT, int SHIFT, int PAST>
__global__ void __launch_bounds__(256)
k_swiglu_blocks(Mat gate, Mat up, Rows8 q, int R, int I, int cshift) {
    for_blocks<SHIFT>(R, I, cshift, [&](int r, int c, auto n) {
        float g[8], u[8];
        load_values<DT, PAST>(gate.p, r * gate.ld + c, n, false, g);
        load_values<DT, PAST>(up.p, r * up.ld + c, n, false, u);
#pragma unroll
        for (int j = 0; j < 8; j++) g[j] = silu_of(g[j]) * u[j];
        put_block<SHIFT>(q, r, c, n, g);
    });
}

template <int DT, int SHIFT, int PAST>
__global__ void __launch_bounds__(256)
k_swiglu_checkpoint(Mat gate, Mat up, Mat h, Rows8 gate8, Rows8 up8, int R, int I, int cshift) {
    for_blocks<SHIFT>(R, I, cshift, [&](int r, int c, auto n) {
        float g[8], u[8];
        load_values<DT, PAST>(gate.p, r * gate.ld + c, n, false, g);
        load_values<DT, PAST>(up.p, r * up.ld + c, n, false, u);
        put_block<SHIFT>(gate8, r, c, n, g);
        put_block<SHIFT>(up8, r, c, n, u);
#pragma unroll
        for (int j = 0; j < 8; j++) g[j] = silu_of(g[j]) * u[j];
        if (n > 0) store_values<DT, PAST>(h.p, r * h.ld + c, n, false, g);
    });
}

template <int DT, int PAST>
__global__ void __launch_bounds__(256)
k_swiglu_checkpoint_backward(Mat dh, Rows8 gate8, Rows8 up8, Mat dgate, Mat dup, Mat h, int R, int I, int cshift) {
    for_blocks<3>(R, I, cshift, [&](int r, int c, auto n) {
        float d[8], g[8], u[8];
        const uint2 cg = get_codes<PAST>(gate8.q + r * gate8.ld + c, n), cu = get_codes<PAST>(up8.q + r * up8.ld + c, n);
        const float sg = gate8.scale[r * gate8.ld_scale + (c >> gate8.shift)];
        const float su = up8.scale[r * up8.ld_scale + (c >> up8.shift)];
        load_values<DT, PAST>(dh.p, r * dh.ld + c, n, false, d);
        values8(cg, sg, g);
        values8(cu, su, u);
        // with p = 1 / (1 + e^-gate): dgate = dh up p (1 + gate (1 - p)), dup = dh gate p, h = gate p up
#pragma unroll
        for (int j = 0; j < 8; j++) {
            float p, q;
            logistic(g[j], &p, &q);
            const float v = g[j] * p;
            g[j] = d[j] * u[j] * p * (1.f + g[j] * q);
            u[j] *= v;
            d[j] *= v;
        }
        if (n > 0) store_values<DT, PAST>(dgate.p, r * dgate.ld + c, n, false, g);
        if (n > 0) store_values<DT, PAST>(dup.p, r * dup.ld + c, n, false, d);
        if (h.p && n > 0) store_values<DT, PAST>(h.p, r * h.ld + c, n, false, u);
    });
}

template <int DT, int PAST>
__global__ void __launch_bounds__(256)
k_dequantize(Rows8 q, Mat y, bool f32, int R, int C, int cshift) {
    for_blocks<3>(R, C, cshift, [&](int r, int c, auto n) {
        float v[8];
        values8(get_codes<PAST>(q.q + r * q.ld + c, n), q.scale[r * q.ld_scale + (c >> q.shift)], v);
        if (n > 0) store_values<DT, PAST>(y.p, r * y.ld + c, n, f32, v);
    });
}

// ---- a scale for the row --------------------------------------------------
// NT threads a row, 8 columns each and P times, kept in registers between the
// maximum and the codes (P = 0: any number, made twice).
template <int DT, bool F32, int PAST>
struct RowOf {
    Mat x;
    BM_DEV void get(int64_t r, int c, int n, float (&v)[8]) const { load_values<DT, PAST>(x.p, r * x.ld + c, n, F32, v); }
};
template <int DT, int PAST>
struct SwigluOf {
    Mat gate, up;
    BM_DEV void get(int64_t r, int c, int n, float (&v)[8]) const {
        float u[8];
        load_values<DT, PAST>(gate.p, r * gate.ld + c, n, false, v);
        load_values<DT, PAST>(up.p, r * up.ld + c, n, false, u);
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = silu_of(v[j]) * u[j];
    }
};

template <int NT, int P, class S>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT)
k_rows8(S src, Rows8 q, int r0, int R, int C) {
    constexpr int RPB = NT < 256 ? 256 / NT : 1, NW = NT / 64;
    __shared__ uint32_t part[NW];
    const int tid = threadIdx.x % NT;
    const int64_t r = r0 + (int64_t)blockIdx.x * RPB + threadIdx.x / NT;
    if (r >= R) return;                          // (whole waves; NT > 64: never)
    constexpr int H = P ? P : 1;
    float v[H][8];
    uint32_t m = 0;
    auto largest = [&](const float (&a)[8]) {
#pragma unroll
        for (int j = 0; j < 8; j++) m = max_bits(m, a[j]);
    };
    if (P) {
#pragma unroll
        for (int p = 0; p < P; p++) {
            const int c = (p * NT + tid) * 8;
            if (c + 8 <= C) src.get(r, c, 8, v[p]);
            else src.get(r, min(c, C - 1), max(C - c, 0), v[p]);
        }
#pragma unroll
        for (int p = 0; p < P; p++) largest(v[p]);
    } else {
        for (int c = tid * 8; c < C; c += NT * 8) {
            src.get(r, c, C - c, v[0]);
            largest(v[0]);
        }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, kWave));
    if (NW > 1) {
        if ((tid & 63) == 0) part[tid >> 6] = m;
        __syncthreads();
        m = part[0];
#pragma unroll
        for (int w = 1; w < NW; w++) m = max(m, part[w]);
    }
    float scale;
    const Coder k = coder(m, &scale);
    auto codes = [&](int c, const float (&a)[8]) {
        const uint32_t w[2] = {code4(k, a), code4(k, a + 4)};
        put_codes(q.q + r * q.ld + c, C - c, w);
    };
    if (P) {
#pragma unroll
        for (int p = 0; p < P; p++) {
            const int c = (p * NT + tid) * 8;
            if (c < C) codes(c, v[p]);
        }
    } else {
        for (int c = tid * 8; c < C; c += NT * 8) {
            src.get(r, c, C - c, v[0]);
            codes(c, v[0]);
        }
    }
    if (tid == 0) q.scale[r * q.ld_scale] = scale;
}

// ---- launches -------------------------------------------------------------
Mat mat(const bitmoe_rows *m) { return m ? Mat{m->data, m->ld} : Mat{nullptr, 0}; }
Rows8 rows8(const bitmoe_rows8 &m) {
    const int shift = m.block == 32 ? 5 : m.block == 64 ? 6 : m.block == 128 ? 7 : 31;
    return Rows8{static_cast<int8_t *>(m.q.data), m.scale, m.q.ld, m.ld_scale, shift};
}

template <int NT, int P, class S>
int rows8_by(const S &src, const Rows8 &q, int R, int C, hipStream_t s) {
    constexpr int RPB = NT < 256 ? 256 / NT : 1;
    constexpr int most = 1 << 21;               // (a launch holds less than 2^32 threads)
    for (int r0 = 0; r0 < R; r0 += most) {
        k_rows8<NT, P, S><<<(std::min(R - r0, most) + RPB - 1) / RPB, NT < 256 ? 256 : NT, 0, s>>>(src, q, r0, std::min(R, r0 + most), C);
        BM_LAUNCH_CHECK();
    }
    return BITMOE_OK;
}
// Threads of a row and pieces of 8 columns of each, which registers hold (none: the
// row is read twice).  us, the one taken first: rows of 1024 columns, 16384 of them,
// 64 x 2 12.3, 256 x 1 16.6, 64 x 4 12.9; of 2048, 32768 rows, 256 x 1 41.9, 64 x 4 40.5,
// 64 x 8 42.7, 1024 x 1 96, from gate and up 55.5, 58.5, 71.2, 138; of 4096, 16384 rows,
// 256 x 4 37.5, 64 x 8 45.1, 1024 x 1 56.9; of 7168, 16384 rows, 256 x 4 60, 1024 x 1 72.5,
// 1024 x 4 92.6, 256 rows 1024 x 1 3.5, 256 x 4 4.4; of 16384, 2048 rows, 1024 x 4 23.1,
// read twice 25.2.
template <class S>
int rows8_of(const S &src, const Rows8 &q, int R, int C, hipStream_t s) {
    if (C > 32768) return rows8_by<1024, 0>(src, q, R, C, s);
    if (C > 8192) return rows8_by<1024, 4>(src, q, R, C, s);
    if (C > 2048) return R < 1024 ? rows8_by<1024, 1>(src, q, R, C, s) : rows8_by<256, 4>(src, q, R, C, s);
    if (C > 1024) return rows8_by<256, 1>(src, q, R, C, s);
    return rows8_by<64, 2>(src, q, R, C, s);
}

// f(SHIFT) of the block
template <class F>
int with_shift(int block, F f) {
    if (block == 32) return f(std::integral_constant<int, 5>{});
    if (block == 64) return f(std::integral_constant<int, 6>{});
    return f(std::integral_constant<int, 7>{});
}
template <class F>
int with_type(int dtype, F f) {
    return dtype == BITMOE_BF16 ? f(std::integral_constant<int, BITMOE_BF16>{}) : f(std::integral_constant<int, BITMOE_F16>{});
}

}  // namespace

namespace bm_host {

int launch_quantize_rows(const bitmoe_rows &x, const bitmoe_rows8 &q, hipStream_t s) {
    const Rows8 out = rows8(q);
    return with_type(x.dtype, [&](auto dt) {
        constexpr int DT = dt.value;
        auto go = [&](auto f32) {
            constexpr bool F = decltype(f32)::value;
            const int64_t bytes = (int64_t)x.rows * x.cols * (F ? 5 : 3);
            if (q.block == 0) {
                if (past_cache(bytes) == kCached) return rows8_of(RowOf<DT, F, kCached>{mat(&x)}, out, x.rows, x.cols, s);
                return rows8_of(RowOf<DT, F, kLoadsPast>{mat(&x)}, out, x.rows, x.cols, s);
            }
            const Grid2 g = pieces_grid(x.rows, x.cols, 8, 4);
            return with_shift(q.block, [&](auto sh) {
                return with_past(bytes, [&](auto past) {
                    k_quantize_blocks<DT, F, sh.value, past.value><<<g.grid, 256, 0, s>>>(mat(&x), out, x.rows, x.cols, g.cshift);
                    BM_LAUNCH_CHECK();
                    return BITMOE_OK;
                });
            });
        };
        if constexpr (DT == BITMOE_F16) {                      // (float32 is neither 16-bit type's)
            if (x.dtype == BITMOE_F32) return go(std::true_type{});
        }
        return go(std::false_type{});
    });
}

int launch_dequantize_rows(const bitmoe_rows8 &q, const bitmoe_rows &y, hipStream_t s) {
    return with_type(y.dtype, [&](auto dt) {
        const Grid2 g = pieces_grid(q.q.rows, q.q.cols, 8, 4);
        return with_past((int64_t)y.cols * q.q.rows * (y.dtype == BITMOE_F32 ? 5 : 3), [&](auto past) {
            k_dequantize<dt.value, past.value><<<g.grid, 256, 0, s>>>(rows8(q), mat(&y), y.dtype == BITMOE_F32, q.q.rows, q.q.cols, g.cshift);
            BM_LAUNCH_CHECK();
            return BITMOE_OK;
        });
    });
}

int launch_swiglu_rows8(const bitmoe_rows &gate, const bitmoe_rows &up, const bitmoe_rows8 &q, hipStream_t s) {
    return with_type(gate.dtype, [&](auto dt) {
        if (q.block == 0) {
            if (past_cache((int64_t)gate.rows * gate.cols * 5) == kCached)
                return rows8_of(SwigluOf<dt.value, kCached>{mat(&gate), mat(&up)}, rows8(q), gate.rows, gate.cols, s);
            return rows8_of(SwigluOf<dt.value, kLoadsPast>{mat(&gate), mat(&up)}, rows8(q), gate.rows, gate.cols, s);
        }
        // (through the cache at any size.  Past it, us: 16384 x 2048 33.3 and 33.3, 32768 rows
        // 56.1, 61.6 through it, 65536 rows 115 and 118, 16384 x 7168 108 and 108)
        const Grid2 g = pieces_grid(gate.rows, gate.cols, 8, 4);
        return with_shift(q.block, [&](auto sh) {
            k_swiglu_blocks<dt.value, sh.value, kCached><<<g.grid, 256, 0, s>>>(mat(&gate), mat(&up), rows8(q), gate.rows, gate.cols, g.cshift);
            BM_LAUNCH_CHECK();
            return BITMOE_OK;
        });
    });
}

int launch_swiglu_checkpoint(const bitmoe_rows &gate, const bitmoe_rows &up, const bitmoe_rows &h,
                             const bitmoe_rows8 &gate8, const bitmoe_rows8 &up8, hipStream_t s) {
    const Grid2 g = pieces_grid(gate.rows, gate.cols, 8, 4);
    return with_type(gate.dtype, [&](auto dt) {
        return with_shift(gate8.block, [&](auto sh) {
            return with_past((int64_t)gate.rows * gate.cols * 8, [&](auto past) {
                k_swiglu_checkpoint<dt.value, sh.value, past.value><<<g.grid, 256, 0, s>>>(
                    mat(&gate), mat(&up), mat(&h), rows8(gate8), rows8(up8), gate.rows, gate.cols, g.cshift);
                BM_LAUNCH_CHECK();
                return BITMOE_OK;
            });
        });
    });
}

int launch_swiglu_checkpoint_backward(const bitmoe_rows &dh, const bitmoe_rows8 &gate8, const bitmoe_rows8 &up8,
                                      const bitmoe_rows &dgate, const bitmoe_rows &dup, const bitmoe_rows *h,
                                      hipStream_t s) {
    const Grid2 g = pieces_grid(dh.rows, dh.cols, 8, 4);
    return with_type(dh.dtype, [&](auto dt) {
        return with_past((int64_t)dh.rows * dh.cols * (h ? 10 : 8), [&](auto past) {
            k_swiglu_checkpoint_backward<dt.value, past.value><<<g.grid, 256, 0, s>>>(
                mat(&dh), rows8(gate8), rows8(up8), mat(&dgate), mat(&dup), mat(h), dh.rows, dh.cols, g.cshift);
            BM_LAUNCH_CHECK();
            return BITMOE_OK;
        });
    });
}

}  // namespace bm_host
