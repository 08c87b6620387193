// Checks of the 16-bit expert layer's operands, for its C ABI.
#pragma once

#include <cstdint>

#include "experts.h"

namespace bm_host {

constexpr int kMaxRows = 1 << 24, kMaxCols = 1 << 18, kMaxExperts = 1024;

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool is16(int dtype) { return dtype == BITMOE_BF16 || dtype == BITMOE_F16; }
inline bool out_type(int dtype, int x_dtype) { return dtype == x_dtype || dtype == BITMOE_F32; }
inline size_t esize(int dtype) { return dtype == BITMOE_F32 ? 4 : 2; }

// a matrix operand for R rows of the call; maps only where the call has them
inline int check_rows(const bitmoe_rows *m, int R, int cols, bool maps) {
    if (!m || m->rows < 0 || m->cols != cols || m->ld < m->cols) return BITMOE_EINVAL;
    if (!is16(m->dtype) && m->dtype != BITMOE_F32) return BITMOE_EINVAL;
    if (m->map ? (!maps || m->div < 1 || !aligned(m->map, 4)) : m->rows < R) return BITMOE_EINVAL;
    // (a map may give rows of a matrix that has none: no address is needed)
    if (R > 0 && (m->rows > 0 || !m->map) && (!m->data || !aligned(m->data, esize(m->dtype)))) return BITMOE_EINVAL;
    return BITMOE_OK;
}

inline int check_sizes(int E, int R, int N, int K) {
    if (E < 1 || R < 0 || N < 1 || K < 1) return BITMOE_EINVAL;
    if (E > kMaxExperts || R > kMaxRows || N > kMaxCols || K > kMaxCols) return BITMOE_EUNSUPPORTED;
    return BITMOE_OK;
}

// Division by an invariant: with 2^(s-1) < d <= 2^s, m = floor(2^(31+s) / d) + 1
// gives floor(x / d) = floor(x m / 2^(31+s)) for every x < 2^31 (the excess
// m d - 2^(31+s) is at most d <= 2^s, so x times it stays below 2^(31+s)).
inline GemmRows rows_arg(const bitmoe_rows *m) {
    GemmRows r{m->data, m->map, m->ld, m->rows, 0, 0, span32(m->map ? m->rows : 256, m->ld)};
    if (m->map && m->div > 1) {
        uint32_t s = 0;
        while (((uint64_t)1 << s) < (uint64_t)m->div) s++;
        r.mul = (uint32_t)(((uint64_t)1 << (31 + s)) / (uint64_t)m->div + 1);
        r.shift = s - 1;
    }
    return r;
}

}  // namespace bm_host
