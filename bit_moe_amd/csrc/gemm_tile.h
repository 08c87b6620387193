// The matrix products for rows on 16-byte addresses.
//
// A stage is 64 of the contraction of a BM x BN tile, loaded from memory
// straight into LDS (global_load_lds, 16 bytes a lane, no registers), two
// stages deep.  Each stage is four units, the halves A0, A1 of A's rows and B0,
// B1 of B's, and is multiplied in four phases, a quadrant of the tile each
// (every wave has its part of every quadrant):
//   even stages  A0 B0,  A0 B1,  A1 B1,  A1 B0     (odd: B0 and B1 exchanged)
// A phase reads from LDS what the next one needs and its registers do not
// hold, so a unit is read once, at one known phase, and its place is free for
// the stage after next long before that stage is due:
//   phase            0            1            2            3
//   reads            B second     A1           -            next A0, B first
//   loads (stage+2)  A0           B first      B second     A1
// A load has six phases to arrive.  Of the stage's four phases three begin
// with a barrier.  Loads spread among the products this way because a CU takes
// about 16 cycles for each; rows of 128 bytes because L2 serves 64-byte pieces
// at half the rate (a ring of 32-wide stages ran 8192^3 at 1172 TFLOP/s, 1822
// with its loads left out).
//
// Bound by the matrix cores where K is long: 16384 x 4096 x 7168 in bfloat16
// takes 683 us forward, 685 as rows' gradient and 710 as weights' gradient (1409,
// 1404, 1356 TFLOP/s); 8192^3 744, 753 and 775.  The matrix cores are busy 74% of
// the time at about 1.6 GHz, the clock that their own power leaves.  Where K is short
// the tile's ends show: a round of 256 x 256 tiles costs 9.5 us beside 1.35 us a
// stage, most of it the epilogue's stores (an epilogue without LDS was no faster).  A workgroup stays
// for several tiles and sends the next one's first stages off before the
// epilogue (32 experts' down projection 943 -> 865 us).  Not taken: waits that
// leave the last tile's stores on their way over the next one's first stages
// (weights' gradient 1240 -> 1377 us: registers spilled), a tile's second half
// skipped where its rows end in the first (1308 -> 1279 TFLOP/s in 8192^3 for
// nothing gained over experts), lines of later stages touched into L2 (1308 ->
// 1169).
#pragma once

#include <type_traits>

#include "gemm_i8.h"
#include "gemm_util.h"

namespace bm {

// what a piece outside the operand reads
__device__ const uint4 kZeroPiece = {0, 0, 0, 0};

BM_DEV uint32_t lds_addr(const void *p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char *)p;
}
// a value that is the wave's, told to the compiler
BM_DEV const uint16_t *wave_ptr(const uint16_t *p) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return reinterpret_cast<const uint16_t *>((uint64_t)hi << 32 | lo);
}
// 16 (4) bytes per lane to LDS, lane l's at `lds` (one for the wave) + 16 l
// (4 l).  In asm, because the compiler would wait for it before the next LDS
// read, of whatever stage; phase_barrier() waits instead.  The wait states that
// the compiler would keep are therefore kept here: one between the write of m0
// and the load that reads it (s_nop 0), and five between a vector instruction's
// write of a scalar register (a readlane of a spilled base) and a load at it.  A
// scalar copy of the base needs none on either side, and is the one for m0 too.
BM_DEV void dma16(const void *src, uint32_t lds) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 ::"{m0}"(__builtin_amdgcn_readfirstlane(lds)), "v"(src) : "memory");
}
// the same with a base of the wave's and 32-bit offsets (bytes) of the lanes':
// no arithmetic per load
BM_DEV void dma16_from(const void *base, uint32_t off, uint32_t lds) {
    uint64_t from;
    asm volatile("s_mov_b64 %0, %3\n\tglobal_load_lds_dwordx4 %2, %0"
                 : "=&s"(from) : "{m0}"(__builtin_amdgcn_readfirstlane(lds)), "v"(off), "s"(base) : "memory");
}
BM_DEV void dma4(const void *src, uint32_t lds) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dword %1, off"
                 ::"{m0}"(__builtin_amdgcn_readfirstlane(lds)), "v"(src) : "memory");
}
// all but this wave's last N loads have arrived, its LDS reads are done, and
// so for every wave of the workgroup
template <int N>
BM_DEV void phase_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Dynamic LDS of a workgroup: two stages; the output rows of this tile and the
// next; A's rows; for the weights' gradient a ring of row maps (64 of A's, 64 of
// B's, four stages); in 8 bits the rows' and the
// columns' scales; the epilogue's part, which is its own, so that the next
// tile's first stages can be on their way during it.
template <int LAY, int DT, int BM, int BN, int WM, int WN, bool MAPS>
struct TileLds {
    static constexpr int rows = 2 * (BM + BN) * kBK * 2;
    static constexpr int maps = rows + 3 * BM * 4;
    static constexpr int scales = maps + (MAPS ? 4 * 128 * 4 : 0);
    static constexpr int out = scales + (DT >= kI8 ? 2 * (BM + BN) * 4 : 0);
    static constexpr int bytes = out + WM * WN * epilogue_floats<BN / WN / 16>() * 4;
    static_assert(bytes <= 160 * 1024, "");
};

// The matrix-core operands of a wave by address: `at` is the lane's place for
// product 0 of the first half of a stage; the others follow by constants (an
// exclusive or where the swizzle mixes with them), so that a unit's reads need
// one register, and are made anew each stage for the same reason.
template <bool KC, int X>
BM_DEV uint32_t frag_place(uint32_t unit, int x0, int lane) {
    const int i = lane & 15, q = lane >> 4;
    if (KC) return unit + (x0 + i) * (kBK * 2) + ((q ^ kc_swz(i)) << 4);
    const int k = 8 * q + (i >> 2);
    return unit + k * (X * 2) + (((x0 >> 4) ^ ks_swz<X>(k)) << 5) + ((i & 3) << 3);
}
// product i (rows or columns 16 i.. of the wave's part, which is a multiple of
// a power of two above i), half kk
template <bool KC, int X>
BM_DEV s16x8 frag_at(uint32_t at, int i, int kk) {
#if defined(__HIP_DEVICE_COMPILE__)
    if (KC) {
        typedef const __attribute__((address_space(3))) s16x8 lds_s16x8;
        return *(lds_s16x8 *)((at ^ (uint32_t)(kk * 64)) + i * (16 * kBK * 2));
    }
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const uint32_t p = (at ^ (uint32_t)(i * 32)) + kk * (32 * X * 2);
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * X * 2));
    return s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
#else
    (void)at; (void)i; (void)kk;        // device code only; the host pass sees this body
    return s16x8{};
#endif
}

// MAPS (weights' gradient): the operands' rows are g.arows and g.brows (span32
// is then of the whole operands).  PARTS (gradients): A is in two parts
// (g.a_low); a tile takes all its stages over the low one, then, its sums scaled,
// over the high one, in twice the time (8192 x 2048 x 7168 396 and 384 us).
template <int LAY, int DT, int BM, int BN, int WM, int WN, bool MAPS, bool PARTS>
__global__ void __launch_bounds__(64 * WM * WN)
k_gemm_tile(GemmArgs g, int mtiles, int ntiles) {
    constexpr int NW = WM * WN, UM = BM / 2, UN = BN / 2;                  // a unit's rows
    constexpr int PA = UM * kBK / 8 / (64 * NW), PB = UN * kBK / 8 / (64 * NW);   // a unit's loads per wave
    constexpr int TI = UM / WM / 16, TJ = UN / WN / 16;                    // 16 x 16 products of a wave in a quadrant
    constexpr bool AKC = LAY != kGradWeights, BKC = LAY == kForward;
    static_assert(LAY == kForward || DT < kI8, "");
    static_assert((LAY == kGradWeights || !MAPS) && (LAY == kForward || MAPS ? !PARTS : true), "");
    constexpr int kUA = UM * kBK, kUB = UN * kBK, kStage = 2 * (kUA + kUB);       // elements
    static_assert(PA >= 1 && PB >= 1 && TI >= 1 && TJ >= 1 && BM <= 64 * NW && (DT < kI8 || BN <= 64 * NW), "");
    extern __shared__ __attribute__((aligned(1024))) uint16_t lds[];
    Tile t;
    Tiles<LAY, BM> list;
    list.init(g, mtiles, ntiles * g.splits, blockIdx.x, gridDim.x);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const uint16_t *zero = reinterpret_cast<const uint16_t *>(&kZeroPiece);

    // Piece i of this thread in a unit, in LDS order: tid + 64 NW i.  Its
    // place in the row does not depend on i (the rows of successive pieces
    // differ by a multiple of the swizzles' period), its row does.
    int ar, ac, br, bc;
    piece_at<AKC, UM>(tid, &ar, &ac);
    piece_at<BKC, UN>(tid, &br, &bc);
    constexpr int kRowA = AKC ? 8 * NW : 64 * NW * 8 / UM, kRowB = BKC ? 8 * NW : 64 * NW * 8 / UN;
    static_assert((kRowA % 16 == 0 || PA == 1) && (kRowB % 16 == 0 || PB == 1), "the swizzles' period");
    // What the loads of a tile go by.  By a base of the wave's that moves with
    // the stage and offsets that stay, where the wave's rows are all there, the
    // stage is whole and the operand spans less than 4 GiB; else, for that
    // stage, by addresses made one by one, with the zero piece for what is not
    // there.  Rows past the group, and columns past the matrix, read its last
    // row (first columns): their results are not stored.
    int *srow = reinterpret_cast<int *>(reinterpret_cast<char *>(lds) + TileLds<LAY, DT, BM, BN, WM, WN, MAPS>::rows);
    int *xrow = srow + 2 * BM;
    float *sscale = reinterpret_cast<float *>(reinterpret_cast<char *>(lds) + TileLds<LAY, DT, BM, BN, WM, WN, MAPS>::scales);
    int m0, n0, kbeg, kend, split, stages, whole;  // whole: whole stages
    const uint16_t *A, *B, *abase, *bbase;         // the matrices; what stage 0 goes by
    uint32_t aoff[AKC ? 2 * PA : PA + 2], boff[BKC ? 2 * PB : PB + 2];   // bytes: KC by half and piece;
    bool afast, bfast;                                                   // KS the rows', then the halves' columns
    auto enter = [&](int par) {
        const Span k = span_of<LAY>(g, &t, ntiles);
        m0 = t.m * BM;
        n0 = t.n * BN;
        kbeg = k.beg;
        kend = k.end;
        split = k.split;
        stages = (kend - kbeg + kBK - 1) / kBK;
        whole = (kend - kbeg) / kBK;
        afast = g.a.span32;
        bfast = g.b.span32;
        A = static_cast<const uint16_t *>(g.a.p) + (PARTS ? g.a_low : 0);
        B = static_cast<const uint16_t *>(g.b.p);
        if (LAY != kGradWeights) B += (int64_t)t.e * g.b_stride;
        abase = A;
        bbase = B;
        if (AKC) {
            abase += kbeg;
            if (!g.a.map) abase += (int64_t)(t.r0 + m0) * g.a.ld;
            bool there = true;
#pragma unroll
            for (int h = 0; h < 2; h++)
#pragma unroll
                for (int i = 0; i < PA; i++) {
                    const int r = min(t.r0 + m0 + h * UM + ar + i * kRowA, t.r1 - 1), row = row_of(g.a, r);
                    there = there && row >= 0;
                    aoff[h * PA + i] = (uint32_t)(max(row, 0) - (g.a.map ? 0 : t.r0 + m0)) * (uint32_t)g.a.ld * 2 + 16 * ac;
                }
            afast = afast && __all(there);
            if (tid < BM) xrow[tid] = row_of(g.a, min(t.r0 + m0 + tid, t.r1 - 1));
        } else {
            if (!g.a.map) abase += (int64_t)t.r0 * g.a.ld;
#pragma unroll
            for (int i = 0; i < PA; i++) aoff[i] = (ar + i * kRowA) * (uint32_t)g.a.ld * 2;
#pragma unroll
            for (int h = 0; h < 2; h++)
                aoff[PA + h] = m0 + h * UM + 8 * ac < g.M ? (m0 + h * UM + 8 * ac) * 2 : 0;
        }
        if (BKC) {
            bbase += (int64_t)n0 * g.b.ld + kbeg;
#pragma unroll
            for (int h = 0; h < 2; h++)
#pragma unroll
                for (int i = 0; i < PB; i++)
                    boff[h * PB + i] = (uint32_t)min(h * UN + br + i * kRowB, g.N - 1 - n0) * (uint32_t)g.b.ld * 2 + 16 * bc;
        } else {
            if (LAY == kGradRows) bbase += (int64_t)kbeg * g.b.ld;
            else if (!g.b.map) bbase += (int64_t)t.r0 * g.b.ld;
#pragma unroll
            for (int i = 0; i < PB; i++) boff[i] = (br + i * kRowB) * (uint32_t)g.b.ld * 2;
#pragma unroll
            for (int h = 0; h < 2; h++)
                boff[PB + h] = n0 + h * UN + 8 * bc < g.N ? (n0 + h * UN + 8 * bc) * 2 : 0;
        }
        A = wave_ptr(A);
        B = wave_ptr(B);
        abase = wave_ptr(abase);
        bbase = wave_ptr(bbase);
        set_rows<LAY, BM>(g, t, m0, tid, srow + par * BM);
        if (DT >= kI8 && tid < BM)
            sscale[par * BM + tid] = !g.raw && m0 + tid < t.r1 - t.r0 ? row_scale(g, t.r0 + m0 + tid) : 0.f;
        if (DT >= kI8 && tid < BN) sscale[2 * BM + par * BN + tid] = g.raw ? 0.f : col_scale(g, t.e, n0 + tid);
    };
    // MAPS: the rows that the maps give (g.arows, g.brows), fetched two stages
    // before the loads that go by them; a stage's offsets are made at the
    // operand's first unit and kept for its second.  Every wave fetches them
    // all, to the same place (the same values), and so waits only for its own
    // loads.
    int *maps = reinterpret_cast<int *>(reinterpret_cast<char *>(lds) + TileLds<LAY, DT, BM, BN, WM, WN, MAPS>::maps);
    const uint32_t maps_at = lds_addr(maps);
    auto fetch_map = [&](const int32_t *rows, int s, int b) {
        dma4(rows + t.r0 + min(s * kBK + lane, kend - 1), maps_at + ((s & 3) * 128 + b * 64) * 4);
    };
    // row k of a stage of the weights' gradient, or -1
    auto map_row = [&](int b, int s, int k) {
        if (s * kBK + k >= kend) return -1;
        return MAPS ? maps[(s & 3) * 128 + b * 64 + k] : t.r0 + s * kBK + k;
    };
    bool awhole = false, bwhole = false;           // MAPS: the rows of the stage being loaded are all there
    const uint32_t lds0 = lds_addr(lds) + wave * 1024;
    // load i of A's (B's) half h of stage s (fast: by the base, but for maps)
    auto load_a = [&](auto fast, int s, int buf, int h, int i) {
        const uint32_t to = lds0 + (buf * kStage + h * kUA) * 2 + i * (NW * 1024);
        if (AKC) {
            if (fast) return dma16_from(abase + (int64_t)s * kBK, aoff[h * PA + i], to);
            const int k = kbeg + s * kBK + 8 * ac, row = xrow[h * UM + ar + i * kRowA];
            dma16(k < kend && row >= 0 ? A + (int64_t)row * g.a.ld + k : zero, to);
        } else {
            if (MAPS ? awhole : (bool)fast)
                return dma16_from(MAPS ? A : abase + (int64_t)s * kBK * g.a.ld, aoff[i] + aoff[PA + h], to);
            const int row = map_row(0, s, ar + i * kRowA);
            dma16(row >= 0 ? A + (int64_t)row * g.a.ld + aoff[PA + h] / 2 : zero, to);
        }
    };
    auto load_b = [&](auto fast, int s, int buf, int h, int i) {
        const uint32_t to = lds0 + (buf * kStage + 2 * kUA + h * kUB) * 2 + i * (NW * 1024);
        if (BKC) {
            if (fast) return dma16_from(bbase + (int64_t)s * kBK, boff[h * PB + i], to);
            const int k = kbeg + s * kBK + 8 * bc;
            dma16(k < kend ? B + (int64_t)min(n0 + h * UN + br + i * kRowB, g.N - 1) * g.b.ld + k : zero, to);
        } else {
            if (MAPS ? bwhole : (bool)fast)
                return dma16_from(MAPS ? B : bbase + (int64_t)s * kBK * g.b.ld, boff[i] + boff[PB + h], to);
            const int k = kbeg + s * kBK + br + i * kRowB;
            const int row = LAY == kGradWeights ? map_row(1, s, br + i * kRowB) : k < kend ? k : -1;
            dma16(row >= 0 ? B + (int64_t)row * g.b.ld + boff[PB + h] / 2 : zero, to);
        }
    };
    // what the unit of phase p of stage s needs before its loads
    auto ready = [&](int s, int p) {
        if (!MAPS || p > 1) return;
        bool there = true;
#pragma unroll
        for (int i = 0; i < (p == 0 ? PA : PB); i++) {
            const int row = map_row(p, s, p == 0 ? ar + i * kRowA : br + i * kRowB);
            there = there && row >= 0;
            (p == 0 ? aoff[i] : boff[i]) = (uint32_t)row * (uint32_t)(p == 0 ? g.a.ld : g.b.ld) * 2;
        }
        (p == 0 ? awhole : bwhole) = (p == 0 ? afast : bfast) && __all(there);
        fetch_map(p == 0 ? g.arows : g.brows, s + 2, p);
    };
    // the loads of phase p for stage s, of parity f: its place in LDS, and B's
    // half that comes first
    auto load = [&](auto fast, int s, int f, int p, int i) {
        if (p == 0 || p == 3) {
            if (i < PA) load_a(fast, s, f, p == 3, i);
        } else if (i < PB) {
            load_b(fast, s, f, p == 1 ? f : 1 - f, i);
        }
    };
    constexpr int kLoads = PA > PB ? PA : PB;

    Acc<DT> acc[2 * TI][2 * TJ];
    s16x8 ra0[2][TI], ra1[2][TI], rb0[2][TJ], rb1[2][TJ];       // [half of the stage's contraction]
    static_assert((TI & (TI - 1)) == 0 && (TJ & (TJ - 1)) == 0 && kUA % 512 == 0 && kUB % 512 == 0, "frag_at");
    uint32_t a_at = frag_place<AKC, UM>(lds_addr(lds), wm * (UM / WM), lane);
    uint32_t b_at = frag_place<BKC, UN>(lds_addr(lds) + 4 * kUA, wn * (UN / WN), lane);
    auto read_a = [&](int buf, int h, int kk, s16x8 (&r)[2][TI]) {
#pragma unroll
        for (int i = 0; i < TI; i++) r[kk][i] = frag_at<AKC, UM>(a_at + (buf * kStage + h * kUA) * 2, i, kk);
    };
    auto read_b = [&](int buf, int h, int kk, s16x8 (&r)[2][TJ]) {
#pragma unroll
        for (int j = 0; j < TJ; j++) r[kk][j] = frag_at<BKC, UN>(b_at + (buf * kStage + h * kUB) * 2, j, kk);
    };
    // (B first: a lane then holds four consecutive columns of one row)
    auto multiply = [&](int ih, int jh, int kk, const s16x8 (&a)[2][TI], const s16x8 (&b)[2][TJ]) {
#pragma unroll
        for (int i = 0; i < TI; i++)
#pragma unroll
            for (int j = 0; j < TJ; j++)
                acc[ih * TI + i][jh * TJ + j] = mfma16<DT>(b[kk][j], a[kk][i], acc[ih * TI + i][jh * TJ + j]);
    };
    // loads issued after the ones a phase waits for (the maps' among them)
    constexpr int kWait3 = 2 * PA + 3 * PB + 2 * MAPS, kWait0 = 3 * PA + 2 * PB + 2 * MAPS;
    // stage s of parity f, whose first B half is f: in rbf on entry, with A0 in ra0
    auto stage = [&](auto fast, int s, int f, s16x8 (&rbf)[2][TJ], s16x8 (&rbs)[2][TJ]) {
#pragma unroll
        for (int p = 0; p < 4; p++) {
            if (p == 0 || p == 1) phase_barrier<kWait0>();
            if (p == 3) phase_barrier<kWait3>();
            asm volatile("" : "+v"(a_at), "+v"(b_at));
            ready(s + 2, p);
#pragma unroll
            for (int kk = 0; kk < 2; kk++) {
                if (p == 0) read_b(f, 1 - f, kk, rbs);
                if (p == 1) read_a(f, 1, kk, ra1);
                if (p == 3) {
                    read_a(1 - f, 0, kk, ra0);
                    read_b(1 - f, 1 - f, kk, rbs);
                }
                if (p == 0) multiply(0, f, kk, ra0, rbf);
                if (p == 1) multiply(0, 1 - f, kk, ra0, rbs);
                if (p == 2) multiply(1, 1 - f, kk, ra1, rbs);
                if (p == 3) multiply(1, f, kk, ra1, rbf);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = kk; i < kLoads; i += 2) load(fast, s + 2, f, p, i);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    // the loads of a tile's first two stages
    auto begin = [&]() {
        if (stages == 0) return;
        if (MAPS) {
            for (int s = 0; s < 4; s++) {
                fetch_map(g.arows, s, 0);
                fetch_map(g.brows, s, 1);
            }
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        }
        auto both = [&](auto fast) {
#pragma unroll
            for (int s = 0; s < 2; s++)
#pragma unroll
                for (int p = 0; p < 4; p++) {
                    ready(s, p);
#pragma unroll
                    for (int i = 0; i < kLoads; i++) load(fast, s, s, p, i);
                }
        };
        if (!MAPS && afast && bfast && whole >= 2) both(std::true_type{});
        else both(std::false_type{});
    };
    // a tile that is there
    auto next = [&]() {
        do
            if (!list.next(g, &t)) return false;
        while (LAY == kGradWeights && t.m < 0);
        return true;
    };
    if (!next()) return;
    enter(0);
    __syncthreads();           // xrow
    begin();
    bool low = PARTS;          // A's low part is being multiplied
    for (int par = 0;;) {
        if (low == PARTS) {
#pragma unroll
            for (int i = 0; i < 2 * TI; i++)
#pragma unroll
                for (int j = 0; j < 2 * TJ; j++) acc[i][j] = Acc<DT>{0, 0, 0, 0};
        }
        if (stages > 0) {
            phase_barrier<3 * PA + 3 * PB + 2 * MAPS>();
#pragma unroll
            for (int kk = 0; kk < 2; kk++) {
                read_a(0, 0, kk, ra0);
                read_b(0, 0, kk, rb0);
            }
            int s = 0;
            if (!MAPS && afast && bfast)
                for (; s + 3 < whole; s += 2) {
                    stage(std::true_type{}, s, 0, rb0, rb1);
                    stage(std::true_type{}, s + 1, 1, rb1, rb0);
                }
            for (; s < stages; s += 2) {
                stage(std::false_type{}, s, 0, rb0, rb1);
                if (s + 1 >= stages) break;
                stage(std::false_type{}, s + 1, 1, rb1, rb0);
            }
        }
        // every wave is done with the stages, and the loads past the last
        // stage have arrived: the next tile's, or part's, may begin
        phase_barrier<0>();
        const bool again = PARTS && low;
        const int e = t.e, n = n0, part = split;
        bool more = again;
        if (again) {
            A -= g.a_low;
            abase -= g.a_low;
        } else {
            more = next();
            if (more) enter(par ^ 1);
            __syncthreads();       // xrow; srow, where no stage was
        }
        if (more) begin();
        if constexpr (PARTS) {
            const float scale = again ? 1.f / low_scale<DT>() : 2.f;
#pragma unroll
            for (int i = 0; i < 2 * TI; i++)
#pragma unroll
                for (int j = 0; j < 2 * TJ; j++) acc[i][j] *= scale;
        }
        low = PARTS && !again;
        if (again) continue;
        float *through = reinterpret_cast<float *>(reinterpret_cast<char *>(lds) + TileLds<LAY, DT, BM, BN, WM, WN, MAPS>::out);
        if constexpr (DT >= kI8)
            i8_epilogue<DT, BM, BN, 2>(g, acc, through, srow + par * BM, sscale + par * BM, sscale + 2 * BM + par * BN, part,
                                       n, wm * (UM / WM), wn * (UN / WN), wave, lane);
        else
            tile_epilogue<LAY, DT, BM, BN, 2>(g, acc, through, srow + par * BM, e, part, n, wm * (UM / WM),
                                              wn * (UN / WN), wave, lane);
        if (!more) return;
        par ^= 1;
    }
}

}  // namespace bm
