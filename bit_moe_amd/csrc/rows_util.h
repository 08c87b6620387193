// Device helpers of the row-wise kernels: threads over rows and columns, a
// row's 8-value pieces in and out, past the memory-side cache or through it.
#pragma once

#include <algorithm>
#include <type_traits>

#include "gemm_util.h"

namespace bm {

// A block's 256 threads over the rows' 8-value pieces: 2^cshift of them along
// a row, the rest over further rows.  Of 256, 128 and 64 the widest that leaves
// no more than a sixteenth of the threads without a piece (7168 values are 3.5
// times 256 pieces, 7 times 128: combine of 8192 x 8 x 7168 173 against 179 us;
// x 2560, 64 against 256: 63 and 72).
struct Grid2 {
    dim3 grid;
    int cshift;
};
// (width: values a piece; least: 2^least pieces at least along a row)
inline Grid2 pieces_grid(int rows, int cols, int width = 8, int least = 0) {
    const int per = (cols + width - 1) / width;
    int cs = least;
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
inline int past_cache(int64_t bytes) {
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

// eight values of a row of DT or float32, the first n of them (the rest 0; none
// read for n <= 0), and back
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
// The first n (1 .. 7) of eight elements, the rest 0: all loads at once, those past
// the last one from its address (each behind a test of its own: the norm's backward
// pass of 3001 x 2047, rows on 16 bytes, 67 us against 47).
BM_DEV uint4 load_part(const uint16_t *p, int n) {
    uint32_t e[8], w[4];
#pragma unroll
    for (int j = 0; j < 8; j++) e[j] = p[min(j, n - 1)];
#pragma unroll
    for (int j = 0; j < 4; j++) w[j] = (2 * j < n ? e[2 * j] : 0) | (2 * j + 1 < n ? e[2 * j + 1] << 16 : 0);
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <int DT, int PAST>
BM_DEV void load_values(const void *p, int64_t i, int n, bool f32, float *v) {
    if (f32) {
        const float *q = static_cast<const float *>(p) + i;
        if (n >= 8) {
            const f32x4_any *m = reinterpret_cast<const f32x4_any *>(q);
            const f32x4_any a = PAST == kCached ? m[0] : __builtin_nontemporal_load(m);
            const f32x4_any b = PAST == kCached ? m[1] : __builtin_nontemporal_load(m + 1);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                v[j] = a[j];
                v[4 + j] = b[j];
            }
            return;
        }
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = 0.f;
        if (n <= 0) return;
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = q[min(j, n - 1)];
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = j < n ? v[j] : 0.f;
        return;
    }
    const uint16_t *q = static_cast<const uint16_t *>(p) + i;
    uint4 u = make_uint4(0, 0, 0, 0);
    if (n >= 8) {
        const u32x4_any *m = reinterpret_cast<const u32x4_any *>(q);
        const u32x4_any t = PAST == kCached ? *m : __builtin_nontemporal_load(m);
        u = make_uint4(t[0], t[1], t[2], t[3]);
    } else if (n > 0) {
        u = load_part(q, n);
    }
    values<DT>(u, v);
}
template <int DT, int PAST>
BM_DEV void store_values(void *p, int64_t i, int n, bool f32, const float *v) {
    if (n >= 8 && PAST == kAllPast) {
        if (f32) {
            f32x4_any *q = reinterpret_cast<f32x4_any *>(static_cast<float *>(p) + i);
            __builtin_nontemporal_store(f32x4_any{v[0], v[1], v[2], v[3]}, q);
            __builtin_nontemporal_store(f32x4_any{v[4], v[5], v[6], v[7]}, q + 1);
        } else {
            u32x4_any u;
#pragma unroll
            for (int j = 0; j < 4; j++) u[j] = elem_pair<DT>(v[2 * j], v[2 * j + 1]);
            __builtin_nontemporal_store(u, reinterpret_cast<u32x4_any *>(static_cast<uint16_t *>(p) + i));
        }
    } else {
        store8<DT>(p, i, n, f32, v);
    }
}
// f(past) for the bytes that a call moves
template <class F>
int with_past(int64_t bytes, F f) {
    switch (past_cache(bytes)) {
        case kCached: return f(std::integral_constant<int, kCached>{});
        case kLoadsPast: return f(std::integral_constant<int, kLoadsPast>{});
        default: return f(std::integral_constant<int, kAllPast>{});
    }
}

}  // namespace bm
