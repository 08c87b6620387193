// The norms around a block, fused with its gate and the residual stream:
//   s = scale r + g (o a w_a),  a = 1 / rms(o);   n = s b w_b,  b = 1 / rms(s)
// and their gradients.  With p = w_b dn, t = ds + b (p - s b^2 <p, s> / H) and
// v = g t w_a:  dr = scale t,  do = a (v - o a^2 <v, o> / H),
//   dw_a = sum t g o a,  dg = t o a w_a,  dw_b = sum dn s b.
// A row is taken by a workgroup's threads (or several rows by a part of them each),
// 8 columns a piece, and stays in their registers from the sums to the outputs.  The
// backward pass needs all its sums in one step: <v, o> is taken apart into
// <g w_a o, ds>, <g w_a o, p> and <g w_a o, s>, which do not need t.
// Bound by memory: 8192 x 7168 with a gate by channel forward 106 us (4.5 TB/s), with a
// float32 stream 140 (5.0), backward 145 (4.9) and 250 (4.2), with a gate by token 192 (4.9)
// and 342 (3.8: 25 registers spill).  3001 x 2047, rows that are not on 16 bytes, forward 15
// to 20 us (3.2 to 4.2 TB/s), backward 35 to 42 (2.1 to 2.6), with a float32 stream and a
// gate by token 69.  (us a call, calls one after another on changing inputs.)  Above 8192
// columns the backward pass spills 380 to 498 registers: 2048 x 16384 560 to 810 us (0.7 to
// 1.0 TB/s).  The forward pass goes through the memory-side cache (134 to 140 us against
// 147 past it), the backward pass reads past it where a call moves more than it holds (158
// us against 171).
#pragma once

#include <algorithm>
#include <initializer_list>

#include "norm.h"
#include "rows_util.h"

namespace bm {

using bm_host::NormArgs;
using bm_host::NormBackArgs;
using bm_host::NormMat;

constexpr int kMost = 16;           // waves of a workgroup

// A wave's sum by lane moves alone (shuffles go through LDS), in every lane: rows
// of 16 lanes, then 15 and 47 onto the next row, 31 onto the upper half.
template <int CTRL, int ROWS>
BM_DEV float dpp_add(float v) {
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xF, ROWS == 0xF));
}
BM_DEV float lane_of(float v, int lane) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane)); }
BM_DEV float wave_total(float v) {
    v = dpp_add<0x142, 0xA>(row16_sum(v));
    return lane_of(dpp_add<0x143, 0xC>(v), 63);
}
// Sums of N values over the `nw` waves of a row, the waves' by a tree too; every
// thread has them.  put before a barrier, get behind it.
template <int N>
BM_DEV void put_sums(float (&v)[N], float (*part)[8], int wave) {
#pragma unroll
    for (int i = 0; i < N; i++) v[i] = wave_total(v[i]);
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int i = 0; i < N; i++) part[wave][i] = v[i];
    }
}
template <int N>
BM_DEV void get_sums(float (&v)[N], const float (*part)[8], int nw) {
    const int w = threadIdx.x & 15;
#pragma unroll
    for (int i = 0; i < N; i++) v[i] = w < nw ? part[w][i] : 0.f;
#pragma unroll
    for (int i = 0; i < N; i++) v[i] = lane_of(row16_sum(v[i]), 15);
}

// 1 / rms of a row whose values are taken times f
constexpr float kDown = 0x1p-80f;   // f where the squares' sum leaves fp32
BM_DEV float inv_rms(float sum, int H, float eps, float f) { return rsqrtf(sum / (float)H + eps * f * f); }

// the first n (<= 0: none) of eight columns from c of row r, `missing` for a matrix
// that is not there
template <int DT, int PAST>
BM_DEV void load_cols(const NormMat &m, int64_t r, int c, int n, float missing, float (&v)[8]) {
    if (m.p) load_values<DT, PAST>(m.p, r * m.ld + c, n, m.f32, v);
    else
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = missing;
}
template <int DT>
BM_DEV void load_w(const void *w, int c, int n, float (&v)[8]) {
    load_cols<DT, kCached>(NormMat{const_cast<void *>(w), 0, false}, 0, c, n, 1.f, v);
}
template <int DT, int PAST>
BM_DEV void store_cols(const NormMat &m, int64_t r, int c, int n, const float (&v)[8]) {
    store_values<DT, PAST>(m.p, r * m.ld + c, n, m.f32, v);
}

template <int DT, int P>
__global__ void __launch_bounds__(1024)
k_block_norm(NormArgs a, int r0) {
    __shared__ float part[4][kMost][8];
    const int64_t r = r0 + (int64_t)blockIdx.x;
    float v[P][8], o[P][8];
    auto col = [&](int p) { return (int)(threadIdx.x + p * blockDim.x) * 8; };
    auto left = [&](int p) { return a.H - col(p); };
#pragma unroll
    for (int p = 0; p < P; p++) {
        load_cols<DT, kCached>(a.o, r, col(p), left(p), 0.f, o[p]);
        load_cols<DT, kCached>(a.res, r, col(p), left(p), 0.f, v[p]);
    }
    auto squares = [&](const float (&x)[P][8], float f, int k) {
        float s[1] = {0.f};
#pragma unroll
        for (int p = 0; p < P; p++)
#pragma unroll
            for (int j = 0; j < 8; j++) s[0] = fmaf(x[p][j] * f, x[p][j] * f, s[0]);
        put_sums<1>(s, part[k], threadIdx.x >> 6);
        if (blockDim.x > 64) __syncthreads();
        get_sums<1>(s, part[k], blockDim.x >> 6);
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
            load_w<DT>(a.wa, col(p), left(p), w);
            load_cols<DT, kCached>(a.gate, r, col(p), left(p), 1.f, g);
#pragma unroll
            for (int j = 0; j < 8; j++) v[p][j] = fmaf(g[j], o[p][j] * f * ra * w[j], v[p][j]);
        }
    }
    if (a.s.p) {
#pragma unroll
        for (int p = 0; p < P; p++)
            if (left(p) > 0) store_cols<DT, kCached>(a.s, r, col(p), left(p), v[p]);
    }
    if (!a.n.p) return;
    float f = 1.f, sum = squares(v, f, 2);
    if (!(sum < INFINITY)) sum = squares(v, f = kDown, 3);
    const float rb = inv_rms(sum, a.H, a.eps, f);
#pragma unroll
    for (int p = 0; p < P; p++) {
        float w[8];
        load_w<DT>(a.wb, col(p), left(p), w);
#pragma unroll
        for (int j = 0; j < 8; j++) v[p][j] = v[p][j] * f * rb * w[j];
        if (left(p) > 0) store_cols<DT, kCached>(a.n, r, col(p), left(p), v[p]);
    }
}

// ---- backward -------------------------------------------------------------
// eight values of a row as they are in memory; WIDE: the row may be float32
template <bool WIDE>
struct Piece {
    uint4 lo, hi;
};
template <int DT, int PAST, bool WIDE>
BM_DEV void fetch(const NormMat &m, int64_t r, int c, int n, Piece<WIDE> &q) {
    q.lo = make_uint4(0, 0, 0, 0);
    if (WIDE) q.hi = make_uint4(0, 0, 0, 0);
    if (!m.p || n <= 0) return;
    if (WIDE && m.f32) {
        float v[8];
        load_values<DT, PAST>(m.p, r * m.ld + c, n, true, v);
        q.lo = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        q.hi = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
    } else {
        q.lo = n >= 8 ? piece<true, PAST>(Mat{m.p, m.ld}, r, c, 0)
                      : load_part(static_cast<const uint16_t *>(m.p) + r * m.ld + c, n);
    }
}
template <int DT, bool WIDE>
BM_DEV void unpack(const Piece<WIDE> &q, bool f32, float (&v)[8]) {
    if (WIDE && f32) {
        const uint32_t w[8] = {q.lo.x, q.lo.y, q.lo.z, q.lo.w, q.hi.x, q.hi.y, q.hi.z, q.hi.w};
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = __uint_as_float(w[j]);
    } else {
        values<DT>(q.lo, v);
    }
}

// a value that the compiler takes for a new one
BM_DEV void hold(uint4 &q) { asm volatile("" : "+v"(q.x), "+v"(q.y), "+v"(q.z), "+v"(q.w)); }

// A workgroup is `groups` rows of `nt` threads each, and takes its rows one after
// another, the next ones' values on their way meanwhile.  What is summed over
// tokens stays in registers (a gate of one row and w_a leave one sum, of t o a: dw_a
// is it times g, dg it times w_a) and ends as one slice of the partial sums.  One
// barrier a row: what it separates alternates between two places (three for
// `far`, which also has to be cleared).
template <int DT, int P, int MOST, int PAST, bool WIDE, bool TOKEN>
__global__ void __launch_bounds__(MOST)
k_block_norm_backward(NormBackArgs a, int nt, int groups) {
    __shared__ float part[3][kMost][8];
    __shared__ int far[3];
    extern __shared__ float joined[];
    const int group = __builtin_amdgcn_readfirstlane(threadIdx.x / nt), tid = threadIdx.x - group * nt;   // (nt: whole waves)
    const int nw = nt >> 6, wave = threadIdx.x >> 6, first = group * nw;
    auto col = [&](int p) { return (tid + p * nt) * 8; };
    auto left = [&](int p) { return a.H - col(p); };
    // g w_a (w_a alone for a gate by token); w_b stays as it is in memory
    float wa[P][8], sa[P][8], sb[P][8];
    uint4 wb[P];
#pragma unroll
    for (int p = 0; p < P; p++) {
        float g[8];
        load_w<DT>(a.wa, col(p), left(p), wa[p]);
        load_w<DT>(TOKEN ? nullptr : a.gate.p, col(p), left(p), g);
        const uint32_t one = elem_pair<DT>(1.f, 1.f);
        wb[p] = make_uint4(one, one, one, one);
        if (a.wb) {
            Piece<false> w;
            fetch<DT, kCached>(NormMat{const_cast<void *>(a.wb), 0, false}, 0, col(p), left(p), w);
            wb[p] = w.lo;
        }
#pragma unroll
        for (int j = 0; j < 8; j++) {
            wa[p][j] *= g[j];
            sa[p][j] = sb[p][j] = 0.f;
        }
    }
    if (threadIdx.x < 3) far[threadIdx.x] = 0;
    __syncthreads();
    struct Row {
        Piece<false> dn, o, g;
        Piece<WIDE> ds, s;
    };
    Row ahead[P];
    const int64_t step = (int64_t)gridDim.x * groups;
    auto load = [&](int64_t r) __attribute__((always_inline)) {
#pragma unroll
        for (int p = 0; p < P; p++) {
            const int n = r < a.T ? left(p) : 0;
            fetch<DT, PAST>(a.dn, r, col(p), n, ahead[p].dn);
            fetch<DT, PAST>(a.o, r, col(p), n, ahead[p].o);
            fetch<DT, PAST>(a.s, r, col(p), n, ahead[p].s);
            fetch<DT, PAST>(a.ds, r, col(p), n, ahead[p].ds);
            if (TOKEN) fetch<DT, PAST>(a.gate, r, col(p), n, ahead[p].g);
        }
    };
    load((int64_t)blockIdx.x * groups + group);
    int turn = 0, three = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * groups; r0 < a.T; r0 += step) {
        const int64_t r = r0 + group;
        Row row[P];
#pragma unroll
        for (int p = 0; p < P; p++) row[p] = ahead[p];
        load(r + step);
        // (the row's values stay as they are in memory, half the registers, and are unpacked
        // for each pass anew, which the compiler would not do by itself)
        float q[6], fs = 1.f, fo = 1.f;
        auto sums = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < 6; i++) q[i] = 0.f;
#pragma unroll
            for (int p = 0; p < P; p++) {
                float dn[8], ds[8], s[8], o[8], g[8], w[8];
                unpack<DT>(row[p].dn, false, dn);
                unpack<DT>(row[p].o, false, o);
                unpack<DT>(row[p].s, a.s.f32, s);
                unpack<DT>(row[p].ds, a.ds.f32, ds);
                if (TOKEN) unpack<DT>(row[p].g, false, g);
                values<DT>(wb[p], w);
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const float x = s[j] * fs, y = o[j] * fo, d = w[j] * dn[j];
                    const float u = (TOKEN ? g[j] * wa[p][j] : wa[p][j]) * y;
                    q[0] = fmaf(x, x, q[0]);
                    q[1] = fmaf(d, x, q[1]);
                    q[2] = fmaf(y, y, q[2]);
                    q[3] = fmaf(u, ds[j], q[3]);
                    q[4] = fmaf(u, d, q[4]);
                    q[5] = fmaf(u, x, q[5]);
                }
                __builtin_amdgcn_sched_barrier(0);         // (one piece's values at a time in registers)
            }
        };
        auto anew = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int p = 0; p < P; p++) {
                hold(row[p].dn.lo);
                hold(row[p].o.lo);
                hold(row[p].s.lo);
                hold(row[p].ds.lo);
                if (WIDE) hold(row[p].s.hi);
                if (WIDE) hold(row[p].ds.hi);
                if (TOKEN) hold(row[p].g.lo);
                hold(wb[p]);
#pragma unroll
                for (int j = 0; j < 8; j++) asm volatile("" : "+v"(wa[p][j]));
            }
        };
        sums();
        put_sums<6>(q, part[turn], wave);
        // squares' sums that may leave fp32 (16 waves' stay below 2^120)
        if (!(q[0] < 0x1p116f && q[2] < 0x1p116f)) far[three] = 1;
        const int next = three == 2 ? 0 : three + 1;
        if (threadIdx.x == 0) far[next] = 0;
        __syncthreads();
        get_sums<6>(q, part[turn] + first, nw);
        if (far[three]) {
            fs = q[0] < 0x1p120f ? 1.f : kDown;
            fo = q[2] < 0x1p120f ? 1.f : kDown;
            anew();
            sums();
            put_sums<6>(q, part[2], wave);
            __syncthreads();
            get_sums<6>(q, part[2] + first, nw);
            __syncthreads();
        }
        turn ^= 1;
        three = next;
        // (with the factors: s and o by their own, b and a are fs b', fo a')
        const float b1 = inv_rms(q[0], a.H, a.eps, fs), a1 = inv_rms(q[2], a.H, a.eps, fo);
        const float b = a.dn.p ? fs * b1 : 0.f, mean = b1 * q[1] / (float)a.H;             // of p and s b
        const float vo = q[3] + b * (q[4] - b1 * mean * q[5]), ra = fo * a1, mo = a1 * vo / (float)a.H;
        if (r >= a.T) continue;
        anew();
#pragma unroll
        for (int p = 0; p < P; p++) {
            float dn[8], ds[8], s[8], o[8], g[8], w[8];
            unpack<DT>(row[p].dn, false, dn);
            unpack<DT>(row[p].o, false, o);
            unpack<DT>(row[p].s, a.s.f32, s);
            unpack<DT>(row[p].ds, a.ds.f32, ds);
            if (TOKEN) unpack<DT>(row[p].g, false, g);
            values<DT>(wb[p], w);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float sn = s[j] * fs * b1, on = o[j] * fo * a1;
                // (where there is no dn, s, sn and dn are 0, and b)
                const float t = fmaf(b, w[j] * dn[j] - sn * mean, ds[j]), gt = TOKEN ? g[j] * t : t;
                o[j] = ra * (gt * wa[p][j] - on * mo);
                s[j] = t * a.scale;
                if (TOKEN) g[j] = t * on * wa[p][j];
                sb[p][j] = fmaf(dn[j], sn, sb[p][j]);
                sa[p][j] = fmaf(gt, on, sa[p][j]);
            }
            if (left(p) > 0) {
                if (a.d_o.p) store_cols<DT, PAST>(a.d_o, r, col(p), left(p), o);
                if (a.dres.p) store_cols<DT, PAST>(a.dres, r, col(p), left(p), s);
                if (TOKEN && a.dgate.p) store_cols<DT, PAST>(a.dgate, r, col(p), left(p), g);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    // the groups' sums, in order, through LDS
    if (!a.dwa && !a.dwb && !a.dg) return;
    const NormMat out{a.partial + (int64_t)blockIdx.x * 2 * a.H, a.H, true};
    for (int k = 0; k < 2; k++) {
        if (groups > 1) {
            __syncthreads();
#pragma unroll
            for (int p = 0; p < P; p++)
#pragma unroll
                for (int j = 0; j < 8; j++) joined[(group * P * 8 + p * 8 + j) * nt + tid] = k ? sb[p][j] : sa[p][j];
            __syncthreads();
            if (group == 0) {
#pragma unroll
                for (int p = 0; p < P; p++)
#pragma unroll
                    for (int j = 0; j < 8; j++)
                        for (int i = 1; i < groups; i++) {
                            const float v = joined[(i * P * 8 + p * 8 + j) * nt + tid];
                            if (k) sb[p][j] += v;
                            else sa[p][j] += v;
                        }
            }
        }
        if (group == 0) {
#pragma unroll
            for (int p = 0; p < P; p++)
                if (left(p) > 0) store_cols<DT, kCached>(out, k, col(p), left(p), k ? sb[p] : sa[p]);
        }
    }
}

// The slices' sums: 64 columns a block, 16 threads over the slices, 4 loads of
// each together; then dw_a = g sum, dg = w_a sum (a gate by token: dw_a = sum).
template <int DT>
__global__ void __launch_bounds__(1024)
k_norm_sums(NormBackArgs a, int slices, bool token) {
    __shared__ float red[16][64];
    const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6, c = blockIdx.x * 64 + tx, k = blockIdx.y;
    if (k ? !a.dwb : !a.dwa && !a.dg) return;
    const float *p = a.partial + (int64_t)k * a.H + c;
    const int64_t step = 2 * (int64_t)a.H;
    float s = 0.f;
    if (c < a.H)
        for (int i = ty; i < slices; i += 64) {
            float v[4];
#pragma unroll
            for (int j = 0; j < 4; j++) v[j] = i + 16 * j < slices ? p[(i + 16 * j) * step] : 0.f;
#pragma unroll
            for (int j = 0; j < 4; j++) s += v[j];
        }
    red[ty][tx] = s;
    __syncthreads();
    if (ty || c >= a.H) return;
#pragma unroll
    for (int i = 1; i < 16; i++) s += red[i][tx];
    auto put = [&](void *out, int dtype, float v) {
        if (!out) return;
        if (dtype == BITMOE_F32) static_cast<float *>(out)[c] = v;
        else static_cast<uint16_t *>(out)[c] = (uint16_t)elem_pair<DT>(v, 0.f);
    };
    auto at = [&](const void *w) { return w ? elem_f32<DT>(static_cast<const uint16_t *>(w)[c]) : 1.f; };
    if (k) {
        put(a.dwb, a.dw_dtype, s);
    } else {
        put(a.dwa, a.dw_dtype, token ? s : s * at(a.gate.p));
        put(a.dg, a.dg_dtype, s * at(a.wa));
    }
}

inline int64_t norm_bytes(int T, int H, std::initializer_list<const NormMat *> mats) {
    int64_t n = 0;
    for (const NormMat *m : mats)
        if (m->p && m->ld) n += (int64_t)T * H * (m->f32 ? 4 : 2);
    return n;
}

template <int DT>
int launch_norm(const NormArgs &a, hipStream_t st) {
    const int pieces = a.H <= 8192 ? 1 : 2, threads = (a.H + pieces * 512 - 1) / (pieces * 512) * 64;
    constexpr int most = 1 << 21;               // (a launch holds less than 2^32 threads)
    for (int r0 = 0; r0 < a.T; r0 += most) {
        const int rows = std::min(a.T - r0, most);
        if (pieces == 1) k_block_norm<DT, 1><<<rows, threads, 0, st>>>(a, r0);
        else k_block_norm<DT, 2><<<rows, threads, 0, st>>>(a, r0);
        BM_LAUNCH_CHECK();
    }
    return BITMOE_OK;
}

template <int DT>
int launch_norm_backward(const NormBackArgs &a, hipStream_t st) {
    const bm_host::NormShape b = bm_host::norm_shape(a.T, a.H);
    const bool token = a.gate.p && a.gate.ld != 0, wide = a.s.f32 || a.ds.f32;
    const bool past = past_cache(norm_bytes(a.T, a.H, {&a.dn, &a.ds, &a.s, &a.o, &a.gate, &a.d_o, &a.dres, &a.dgate})) != kCached;
    if (b.slices > 0) {
        const size_t lds = b.groups > 1 ? (size_t)b.groups * b.nt * b.pieces * 8 * 4 : 0;
        auto go = [&](auto w, auto t, auto c) {
            constexpr bool W = decltype(w)::value, K = decltype(t)::value;
            constexpr int A = decltype(c)::value ? kLoadsPast : kCached;
            const int n = b.nt * b.groups;
            if (b.pieces == 1) k_block_norm_backward<DT, 1, 256, A, W, K><<<b.slices, n, lds, st>>>(a, b.nt, b.groups);
            else if (b.nt <= 512) k_block_norm_backward<DT, 2, 512, A, W, K><<<b.slices, n, lds, st>>>(a, b.nt, b.groups);
            else k_block_norm_backward<DT, 2, 1024, kCached, W, K><<<b.slices, n, lds, st>>>(a, b.nt, b.groups);
        };
        const std::true_type yes;
        const std::false_type no;
        auto go2 = [&](auto w, auto t) { past ? go(w, t, yes) : go(w, t, no); };
        if (wide) token ? go2(yes, yes) : go2(yes, no);
        else token ? go2(no, yes) : go2(no, no);
        BM_LAUNCH_CHECK();
    }
    if (a.dwa || a.dwb || a.dg) {
        k_norm_sums<DT><<<dim3((a.H + 63) / 64, 2), 1024, 0, st>>>(a, b.slices, token);
        BM_LAUNCH_CHECK();
    }
    return BITMOE_OK;
}

}  // namespace bm
