// Products of e4m3 packages, tiled form for many tokens:
//     y[m, n] = sum_b sx[m, b] sw[n / 128, b] sum_{k in b} cx[m, k] cw[n, k]  (+ bias[n]).
//
// Mathematics.  A block's sum over 128 columns starts at 0 in the matrix instructions and is
// added to y's by one fused multiply-add with f = sx sw, in fp32.  Two ways to that sum:
//  * EXACT: the codes become bf16 (exact) and go through four 16x16x32 instructions, whose
//    sums are fp32's.
//  * otherwise one 16x16x128 e4m3 instruction, of twice the rate.  It lines up each eight
//    products (consecutive bytes of a lane) by the largest and drops what lies 2^-13 below
//    it, so a sum may be off by 7 2^-13 of its largest products.  That is for a caller who
//    asks for it (DMM_SHORT_SUMS) with a bf16 y, whose own rounding is 2^-9 of it.
// Any order of k may be taken that is the same for both operands: lane group g of four takes
// the 16-byte pieces g and 4 + g of a block.
//
// Mapping.  A workgroup owns BM tokens x BN rows of W, its waves equal parts of that.  W is
// the first operand, so a lane ends with four consecutive n of one token, and f is one value
// for each of its tokens.  K is cut into slabs of KD blocks, which take turns in NS LDS
// stages: distinct arrays, so the compiler can tell a load in flight to one from the reads of
// another.  Rows go from global memory straight to LDS in whole lines of 128 bytes, a block
// each, up to NS - 1 slabs ahead; pieces change places within their rows so that a fragment read
// hits all banks (swizzle).  The products f of NS slabs come by way of registers.  What may be under way
// where a slab is waited for stands in waits.h.  (The compiler does not tell the stages of 32 x 64
// apart: it waits there for everything before it reads W's second fragment, so that the slabs ahead
// land within the slab that sent for them.)
//
// Bound.  Sums in fp32, 2048 tokens, 8192 x 8192: 217 to 230 us, 1.2 to 1.27 PFLOP/s, the bf16
// instructions' rate (the vendor's bf16 product of 8192 cubed runs at 1.36 to 1.44: 191 to 202 us).
// Short sums, largest tile, the same product (107 to 126 us by card, 2.2 to 2.6 PFLOP/s): the LDS, whose reads
// and writes of a slab take about as long as its matrix instructions.  Without the reads of x's
// fragments 85 us remain, without the loads 102, without the multiply-adds 102.  What paid:
// overwriting a slab's first half (W, and half of x) at its middle (with the addresses below,
// 162 -> 126 us), adding sums four instructions late (121), the middle's barrier ahead of the
// next read (117).  Eight waves of 64 x 128 need more registers than there are.  Smaller
// tiles: what a compute unit can have under way against the latency of memory.  Experts' tiles
// (2048 tokens top 8 of 64, 2048 x 4096: 319 to 330 us, short sums 224 to 226, where W's bytes take 104 at a
// copy's rate): of the 226, 44 are a tile's beginning and end, 150 remain without loads, and 194 with
// every load a hit in L2.
#include <type_traits>

#include "experts.h"
#include "f8.h"
#include "waits.h"

namespace dmm {

namespace {

constexpr int kRow = kF8Block;                  // bytes of an LDS tile row

__device__ __forceinline__ i32x8 f8_operand(const u32x4* v) {
    return (i32x8){(int)v[0].x, (int)v[0].y, (int)v[0].z, (int)v[0].w,
                   (int)v[1].x, (int)v[1].y, (int)v[1].z, (int)v[1].w};
}

template <int N>
struct Floats {
    typedef float T __attribute__((ext_vector_type(N)));
};

// EXACT: sums in fp32, y as a.y_dtype says; otherwise short sums and a bf16 y.  BM x BN tile of WM x WN waves; KD blocks a slab.  KG groups of
// WM x WN waves take a part of K each, and the first adds up the sums.  NS stages.
template <bool EXACT, int BM, int BN, int WM, int WN, int KD, int KG, int NS, bool GROUPED>
__global__ void __launch_bounds__(64 * WM * WN * KG, 2) f8_gemm_kernel(F8MatmulArgs a) {
    constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;                 // of a group
    constexpr int kXUnit = BM * kRow, kWUnit = BN * kRow;
    constexpr int kXBytes = KD * kXUnit, kWBytes = KD * kWUnit, kStage = kXBytes + kWBytes;
    constexpr int MT = BM / WM / 16, NT = BN / WN / 16;                     // tiles of a wave
    constexpr int kXLoads = kXBytes / 1024 / kWaves, kWLoads = kWBytes / 1024 / kWaves;
    constexpr int NB = BN > 128 ? BN / 128 : 1;                             // scales of W along n
    constexpr int kFSlabs = NS, FU = kFSlabs * KD;  // slabs, blocks of a fetch of scales
    // Two large stages: what the first half of a slab has read is overwritten at its middle
    constexpr bool kEarly = NS == 2 && KD == 1 && KG == 1 && MT >= 4 && !EXACT;
    constexpr StageQueue kQueue = {NS, kXLoads, kWLoads, kEarly};
    static_assert(NT % 4 == 0 || NT < 4, "kLag");
    static_assert(kXLoads * 1024 * kWaves == kXBytes && kWLoads * 1024 * kWaves == kWBytes, "whole loads");
    static_assert(BM * NB <= kThreads, "a thread for each row's scales");
    static_assert(BN / WN <= 128 || NB == 1, "a wave has one scale of W");
    static_assert(NS >= 2 && NS <= 4, "stages");
    // A stage: x's rows by halves (below), then W's.
    __shared__ __attribute__((aligned(1024))) uint8_t stages0[kEarly ? kXBytes / 2 : KG * kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t stages1[kEarly ? kXBytes / 2 : KG * kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t stages2[NS > 2 ? KG * kStage : kEarly ? kXBytes / 2 : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t stages3[NS > 3 ? KG * kStage : kEarly ? kXBytes / 2 : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t rows0[kEarly ? kWBytes : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t rows1[kEarly ? kWBytes : 16];
    // (one index: the compiler sees through a few address computations only, and waits for all loads
    // to LDS before a read that may be of what they write)
    __shared__ float factors[KG * 2 * NB * FU * BM];

    const int kg = KG == 1 ? 0 : readfirstlane((int)threadIdx.x / kThreads);
    const int tid = (int)threadIdx.x - kg * kThreads, lane = tid & 63, wave = readfirstlane(tid >> 6);
    uint8_t* const stage0 = stages0 + (KG > 1 ? kg * kStage : 0);
    uint8_t* const stage1 = stages1 + (KG > 1 ? kg * kStage : 0);
    uint8_t* const stage2 = stages2 + (KG > 1 && NS > 2 ? kg * kStage : 0);
    uint8_t* const stage3 = stages3 + (KG > 1 && NS > 3 ? kg * kStage : 0);
    struct Stage {
        uint8_t *x0, *x1, *w;                   // of unit 0
    };
    const Stage stage[4] = {
        {stage0, kEarly ? stages2 : stage0 + kXUnit / 2, kEarly ? rows0 : stage0 + kXBytes},
        {stage1, kEarly ? stages3 : stage1 + kXUnit / 2, kEarly ? rows1 : stage1 + kXBytes},
        {stage2, stage2 + kXUnit / 2, stage2 + kXBytes},
        {stage3, stage3 + kXUnit / 2, stage3 + kXBytes},
    };
    const int r = lane & 15, g = lane >> 4;
    const int wm = wave / WN, wn = wave % WN;
    const int64_t nb = (a.K + kF8Block - 1) / kF8Block;

    Place p;
    if (GROUPED) {
        if (!place_grouped<BM, BN, 8, kThreads>(a, p)) {
            write_nan_rows(a, p.m0, p.m_end, kThreads);
            return;
        }
    } else {
        p = place_dense<BM, BN>(a);
    }
    const int64_t slots = a.M * a.top_k;

    // Row of tile row i, counted from the tile's first (in a list: the row of x);
    // rows that are not there repeat one that is.
    const int m_rows = (int)(p.m_end - p.m0), n_rows = (int)(a.N - p.n0 < BN ? a.N - p.n0 : BN);
    // (A list's slots come once, to LDS, behind the first rows of W, which the compiler waits for with them.)
    __shared__ int32_t list[GROUPED ? BM : 1];
    int32_t entry = 0;
    if (GROUPED && tid < BM) entry = a.order[p.m0 + (tid < m_rows ? tid : m_rows - 1)];
    auto x_row = [&](int i) -> int64_t {
        const int m = i < m_rows ? i : m_rows - 1;
        if (!GROUPED) return m;
        const int64_t slot = list[m];
        return slot >= 0 && slot < slots ? (int64_t)((uint32_t)slot / (uint32_t)a.top_k) : 0;
    };
    auto w_row = [&](int i) { return i < n_rows ? i : n_rows - 1; };

    // Loads to LDS fill 1024 bytes at a time: eight rows, lane l the piece whose slot is l % 8
    // of row l / 8.  Load j of wave w is row group w + j kWaves of the slab's, unit by unit.
    const int sub = lane >> 3;
    // x's rows lie by halves: first those of the first half of each wave's tiles.
    constexpr int kHalfRows = BM / WM / 2;
    auto x_group = [&](int j) {                 // the row group's first row of the tile, over 8
        const int at = (wave + j * kWaves) % (BM / 8) * 8, half = at / (BM / 2), in = at % (BM / 2);
        return (in / kHalfRows * (BM / WM) + half * kHalfRows + in % kHalfRows) / 8;
    };
    auto x_unit = [&](int j) { return (wave + j * kWaves) / (BM / 8); };
    auto w_group = [&](int j) { return (wave + j * kWaves) % (BN / 8); };
    auto w_unit = [&](int j) { return (wave + j * kWaves) / (BN / 8); };
    auto piece = [&](int group) { return (lane & 7) ^ swizzle(group * 8 + sub); };
    // Offsets from the tile's first row fit 32 bits (kF8MaxK); the rows of a list have 64.
    typedef typename std::conditional<GROUPED, int64_t, uint32_t>::type XOffset;
    const int64_t row_bytes = nb * kRow;
    const uint8_t* const xbase = a.x_codes + (GROUPED ? 0 : p.m0) * row_bytes;
    const uint8_t* const wbase = a.codes + (p.expert * a.N + p.n0) * row_bytes;
    uint32_t wsrc[kWLoads];
#pragma unroll
    for (int j = 0; j < kWLoads; ++j)
        wsrc[j] = lane_offset((uint32_t)w_row(w_group(j) * 8 + sub) * (uint32_t)row_bytes +
                              (uint32_t)(w_unit(j) * kRow + piece(w_group(j)) * 16));
    // Each group has `full` whole slabs one after the other.
    const int64_t full = a.K / kF8Block / KD / KG;
    auto block_of = [&](int64_t t) { return (kg * full + t) * KD; };
    auto start_w = [&](const Stage& st, int64_t t) {            // of slab t, a whole one
        const GlobalBytes wb = scalar_base(wbase + block_of(t) * kRow);
#pragma unroll
        for (int j = 0; j < kWLoads; ++j) load_lds16(wb + lane_offset(wsrc[j]), st.w + (wave + j * kWaves) * 1024);
    };
    asm volatile("" ::: "memory");
    if (full >= NS) {
#pragma unroll
        for (int i = 0; i < NS; ++i) start_w(stage[i], i);
    }
    asm volatile("" ::: "memory");
    if (GROUPED) {
        if (tid < BM) list[tid] = entry;
        lds_barrier();
    }
    XOffset xsrc[kXLoads];
#pragma unroll
    for (int j = 0; j < kXLoads; ++j)
        xsrc[j] = lane_offset((XOffset)x_row(x_group(j) * 8 + sub) * (XOffset)row_bytes +
                              (XOffset)(x_unit(j) * kRow + piece(x_group(j)) * 16));

    // Thread (row, n block) fetches FU scales of both and stages their products.
    typedef typename Floats<FU>::T Scales;
    typedef Scales ScalesAt __attribute__((aligned(4)));
    const int frow = tid % BM, fblk = BM % 64 == 0 ? readfirstlane(tid / BM) : tid / BM;
    const bool stages_f = fblk < NB;
    const int64_t n_blocks = (a.N + 127) / 128, nblk = p.n0 / 128 + fblk;
    const float* const sx = a.x_scales + ((GROUPED ? 0 : p.m0) + (stages_f ? x_row(frow) : 0)) * nb;
    const float* const sw = a.scales + (p.expert * n_blocks + (stages_f && nblk < n_blocks ? nblk : n_blocks - 1)) * nb;
    Scales fx, fw;                              // fw: one for a wave, in scalar registers
    auto fetch_factors = [&](int64_t b, bool whole) {   // of blocks b .. b + FU - 1, as far as there are any
        if (!stages_f) return;
        if (whole || b + FU <= nb) {
            fx = *(const ScalesAt*)(sx + b);
            if (BM % 64 == 0) fw = *(const __attribute__((address_space(4))) ScalesAt*)(sw + b);
            else fw = *(const ScalesAt*)(sw + b);
        } else {
#pragma unroll
            for (int u = 0; u < FU; ++u) {
                fx[u] = b + u < nb ? sx[b + u] : 0.f;
                fw[u] = b + u < nb ? sw[b + u] : 0.f;
            }
        }
    };
    auto store_factors = [&](int buf) {
        if (!stages_f) return;
#pragma unroll
        for (int u = 0; u < FU; ++u) factors[(((kg * 2 + buf) * NB + fblk) * FU + u) * BM + frow] = fx[u] * fw[u];
    };

    f32x4 acc[NT][MT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};

    enum { kAll, kFirst, kSecond };             // of a slab's rows: the first half are W's and x's first half
    auto load_x = [&](const Stage& st, int j, GlobalBytes from) {
        const int at = (wave + j * kWaves) * 1024;
        if (kEarly) load_lds16(from, 2 * j < kXLoads ? st.x0 + at : st.x1 + (at - kXBytes / 2));
        else load_lds16(from, st.x0 + at);
    };
    auto start_x = [&](const Stage& st, int64_t t, int which) {
        const GlobalBytes xb = scalar_base(xbase + block_of(t) * kRow);
#pragma unroll
        for (int j = 0; j < kXLoads; ++j)
            if (which == kAll || (2 * j >= kXLoads) == (which == kSecond)) load_x(st, j, xb + lane_offset(xsrc[j]));
    };
    auto start = [&](const Stage& st, int64_t t, int which) {   // slab t, a whole one
        start_x(st, t, which);
        if (which != kSecond) start_w(st, t);
    };

    // ---- fragments of a unit: the wave's rows of W, held for all of its tokens, and one
    // 16-token tile at a time, read while the one before multiplies.
    typedef typename std::conditional<EXACT, bf16x8, u32x4>::type Part;     // a quarter, or half, of a lane's bytes
    constexpr int kParts = EXACT ? 4 : 2;
    Part wf[NT][kParts];
    u32x4 xf[2][2];
    float f[2];
    int kept = kF8Block;                        // columns of the unit at hand that there are
    const int at0 = r * kRow + ((g ^ swizzle(r)) << 4), at1 = r * kRow + (((4 + g) ^ swizzle(r)) << 4);
    auto read_raw = [&](const uint8_t* row, u32x4* v, bool cut) {
        v[0] = *(const u32x4*)(row + at0);
        v[1] = *(const u32x4*)(row + at1);
        if (cut) {
            v[0] = keep_bytes(v[0], kept - 16 * g);
            v[1] = keep_bytes(v[1], kept - 64 - 16 * g);
        }
    };
    auto as_parts = [&](const u32x4* v, Part* part) {
        if constexpr (EXACT) {
#pragma unroll
            for (int q = 0; q < 4; ++q) part[q] = f8_bf16(v[q >> 1][2 * (q & 1)], v[q >> 1][2 * (q & 1) + 1]);
        } else {
            part[0] = v[0];
            part[1] = v[1];
        }
    };
    auto read_w = [&](const Stage& st, int k, int i, bool cut) {
        u32x4 v[2];
        read_raw(st.w + k * kWUnit + (wn * (BN / WN) + 16 * i) * kRow, v, cut);
        as_parts(v, wf[i]);
    };
    const int fn = NB > 1 ? wn * (BN / WN) / 128 : 0;
    auto read_x = [&](const Stage& st, int buf, int k, int u, int j, bool cut) {
        const int row = wm * kHalfRows + 16 * (j % (MT / 2));
        read_raw((2 * j < MT ? st.x0 : st.x1) + k * kXUnit + row * kRow, xf[j & 1], cut);
        // one address computation (see factors)
        const uint32_t at = lane_offset((uint32_t)((((kg * 2 + buf) * NB + fn) * FU + u) * BM + wm * (BM / WM) + 16 * j + r));
        f[j & 1] = factors[at];
    };
    // A block's sums are added kLag instructions later, when they are long done: a vector
    // instruction that reads one right behind its matrix instruction waits.
    constexpr int kLag = NT < 4 ? NT : 4;
    f32x4 part[kLag];
    float scale = 0.f;
#pragma unroll
    for (int i = 0; i < kLag; ++i) part[i] = (f32x4){0.f, 0.f, 0.f, 0.f};
    auto add = [&](int i, int j, float s) {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(s, part[i % kLag][e], acc[i][j][e]);
        asm volatile("" : "+v"(acc[i][j]));
    };
    auto multiply = [&](int j, auto next) {
        Part x[kParts];
        as_parts(xf[j & 1], x);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            if (i < kLag) add(NT - kLag + i, j == 0 ? MT - 1 : j - 1, scale);
            else add(i - kLag, j, f[j & 1]);
            f32x4 sum = {0.f, 0.f, 0.f, 0.f};
            if constexpr (EXACT) {
#pragma unroll
                for (int q = 0; q < 4; ++q) sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[i][q], x[q], sum, 0, 0, 0);
            } else {
                sum = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(f8_operand(wf[i]), f8_operand(x), sum, 0, 0, 0, 0, 0, 0);
            }
            part[i % kLag] = sum;
            next(i);
        }
        scale = f[j & 1];
        asm volatile("" ::: "memory");
    };
    auto nothing = [](int) {};

    // Slab t in `cur`: its first fragments are in registers.  Before the last tile every wave
    // has read `cur`, and slab t + 1 has landed in `other`: while the last tile
    // multiplies, slab t + NS starts into `cur` and the first fragments of slab t + 1 are read.
    // The products f of slab t are in factors' half (t / kFSlabs) % 2, from block t % kFSlabs KD on.
    // MAIN: all of these slabs, and the next kFSlabs, are there, and the slab's place among kFSlabs is PHASE; without
    // branches the compiler can count the loads behind a fetch of scales and need not wait for them.
    auto slab = [&](const Stage& cur, const Stage& other, int64_t t, auto busy, auto main,
                    auto phase) __attribute__((always_inline)) {
        constexpr bool BUSY = decltype(busy)::value, MAIN = decltype(main)::value;
        const int in = MAIN ? decltype(phase)::value : (int)(t % kFSlabs), next = in + 1 == kFSlabs ? 0 : in + 1;
        const int buf = (int)(t / kFSlabs) & 1, u0 = in * KD, u1 = next * KD, buf1 = next == 0 ? buf ^ 1 : buf;
        if (in == 0) fetch_factors(block_of(t + kFSlabs), MAIN);
#pragma unroll
        for (int k = 0; k < KD; ++k) {
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                if (j + 1 < MT) {
                    // (ahead of the next read, whose return the barrier would wait for)
                    if (kEarly && j == MT / 2 - 1 && (MAIN || t + NS < full)) {
                        lds_barrier();
                        start(cur, t + NS, kFirst);
                    }
                    if constexpr (BUSY) {
                        read_x(cur, buf, k, u0 + k, j + 1, false);
                        multiply(j, nothing);
                    }
                } else if (k + 1 < KD) {
                    if constexpr (BUSY) {
                        read_x(cur, buf, k + 1, u0 + k + 1, 0, false);
                        multiply(j, [&](int i) { read_w(cur, k + 1, i, false); });
                    }
                }
            }
        }
        if (next == 0) store_factors(buf1);
        if (MAIN || t + NS - (kEarly ? 0 : 1) < full) wait_loads<kQueue.slab()>();
        else wait_loads<0>();
        lds_barrier();
        if (MAIN || t + NS < full) start(cur, t + NS, kEarly ? kSecond : kAll);
        if constexpr (BUSY) {
            if (MAIN || t + 1 < full) {
                read_x(other, buf1, 0, u1, 0, false);
                multiply(MT - 1, [&](int i) { read_w(other, 0, i, false); });
            } else {
                multiply(MT - 1, nothing);
            }
        }
    };
    static_assert(MT % 2 == 0, "the last tile's fragments and the next unit's first take turns");
    typedef std::integral_constant<int, 0> P0;
    typedef std::integral_constant<int, 1> P1;
    typedef std::integral_constant<int, 2> P2;
    typedef std::integral_constant<int, 3> P3;
    const std::true_type always;
    const std::false_type maybe;

    if (full >= NS) {                           // every stage is on its way before the first is waited for
        fetch_factors(block_of(0), true);
#pragma unroll
        for (int i = 0; i < NS; ++i) start_x(stage[i], i, kAll);
        store_factors(0);
        wait_loads<kQueue.begin()>();
    } else if (full > 0) {
        fetch_factors(block_of(0), false);
#pragma unroll
        for (int i = 0; i < NS; ++i)
            if (i < full) start(stage[i], i, kAll);
        store_factors(0);
        wait_loads<0>();
    }
    auto slabs = [&](auto busy) __attribute__((always_inline)) {
        lds_barrier();
        if constexpr (decltype(busy)::value) {
            read_x(stage[0], 0, 0, 0, 0, false);
#pragma unroll
            for (int i = 0; i < NT; ++i) read_w(stage[0], 0, i, false);
        }
        int64_t t = 0;
        static_assert(kFSlabs >= NS, "what starts is there");
        for (; t + 2 * kFSlabs <= full; t += kFSlabs) {
            slab(stage[0], stage[1], t, busy, always, P0());
            slab(stage[1], stage[NS > 2 ? 2 : 0], t + 1, busy, always, P1());
            if constexpr (NS > 2) slab(stage[2], stage[NS > 3 ? 3 : 0], t + 2, busy, always, P2());
            if constexpr (NS > 3) slab(stage[3], stage[0], t + 3, busy, always, P3());
        }
        for (; t < full; t += NS) {
            slab(stage[0], stage[1], t, busy, maybe, P0());
            if (t + 1 < full) slab(stage[1], stage[NS > 2 ? 2 : 0], t + 1, busy, maybe, P0());
            if (NS > 2 && t + 2 < full) slab(stage[2], stage[NS > 3 ? 3 : 0], t + 2, busy, maybe, P0());
            if (NS > 3 && t + 3 < full) slab(stage[3], stage[0], t + 3, busy, maybe, P0());
        }
    };
    // A wave whose rows are all behind a list's end brings its loads and no more.
    const bool has_rows = !GROUPED || WM == 1 || wm * (BM / WM) < m_rows;
    if (full > 0) {
        if (has_rows) slabs(std::true_type());
        else if constexpr (GROUPED && WM > 1) slabs(std::false_type());
    }
    // blocks that are left, the last one maybe cut: up to KD for each group
    const int64_t first = (full * KG + kg) * KD;
    if (nb > full * KG * KD) {
        const int rest = nb > first && has_rows ? (int)(nb - first < KD ? nb - first : KD) : 0;
        lds_barrier();
        fetch_factors(first, false);
        store_factors(0);
        // units past the last block repeat it and are not multiplied
        auto unit_of = [&](int u) { return first + u < nb ? first + u : nb - 1; };
#pragma unroll
        for (int j = 0; j < kXLoads; ++j)
            load_x(stage[0], j, (GlobalBytes)xbase + lane_offset(xsrc[j]) + (unit_of(x_unit(j)) - x_unit(j)) * kRow);
#pragma unroll
        for (int j = 0; j < kWLoads; ++j)
            load_lds16((GlobalBytes)wbase + lane_offset(wsrc[j]) + (unit_of(w_unit(j)) - w_unit(j)) * kRow,
                       stage[0].w + (wave + j * kWaves) * 1024);
        wait_loads<0>();
        lds_barrier();
#pragma unroll 1
        for (int k = 0; k < rest; ++k) {
            kept = a.K - (first + k) * kF8Block < kF8Block ? (int)(a.K - (first + k) * kF8Block) : kF8Block;
#pragma unroll
            for (int i = 0; i < NT; ++i) read_w(stage[0], k, i, true);
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                read_x(stage[0], 0, k, k, j, true);
                multiply(j, nothing);
            }
        }
    }

#pragma unroll
    for (int i = NT - kLag; i < NT; ++i) add(i, MT - 1, scale);

    if constexpr (KG > 1) {
        static_assert((KG - 1) * BM * BN * 4 <= KG * kStage, "the sums fit the stages");
        lds_barrier();
        auto sums = [&](int from, int i, int j) -> f32x4& {
            return ((f32x4*)stages0)[((((from - 1) * kWaves + wave) * NT + i) * MT + j) * 64 + lane];
        };
        if (kg > 0) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < MT; ++j) sums(kg, i, j) = acc[i][j];
        }
        lds_barrier();
        if (kg > 0) return;
#pragma unroll
        for (int from = 1; from < KG; ++from)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < MT; ++j) acc[i][j] += sums(from, i, j);
    }

    // lane (r, g) of tile (i, j): token 16 j + r, four n from 16 i + 4 g
    const int64_t n_left = a.N - p.n0;
    auto quad = [&](int i, int j, int col) {
        f32x4 v = acc[i][j];
        if (a.bias) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e < n_left) v[e] += a.bias[p.expert * a.N + p.n0 + col + e];
        }
        return v;
    };
    // Row of y of tile row i (of the workgroup's), -1 for none.
    auto y_row = [&](int i) -> int64_t {
        if (i >= m_rows) return -1;
        if (!GROUPED) return p.m0 + i;
        const int64_t slot = list[i];
        return slot < slots ? slot : -1;
    };
    // Rows of y in 16-byte pieces: the wave's 16 tokens x 16 NT columns of each j change
    // hands in LDS, so that whole lines are written.
    auto write_rows = [&](auto type) {
        typedef decltype(type) T;
        constexpr int kCols = NT * 16, kPitch = kCols * (int)sizeof(T) + 16, kEach = 16 / (int)sizeof(T);
        constexpr int kLanes = kCols / kEach, kAtOnce = 64 / kLanes < 16 ? 64 / kLanes : 16;
        constexpr int kArrays = kEarly ? 4 : 2, kIn = (kWaves + kArrays - 1) / kArrays;         // waves in each
        static_assert(kIn * 16 * kPitch <= (kEarly ? kXBytes / 2 : kStage), "the stages hold the waves' rows");
        uint8_t* const in = wave / kIn == 0 ? stage0 : wave / kIn == 1 ? stage1 : wave / kIn == 2 ? stages2 : stages3;
        uint8_t* const mine = in + wave % kIn * (16 * kPitch);
        const int c = lane % kLanes, col = wn * (BN / WN) + c * kEach;
#pragma unroll
        for (int j = 0; j < MT; ++j) {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const int at = 16 * i + 4 * g;
                const f32x4 v = quad(i, j, wn * (BN / WN) + at);
                if constexpr (sizeof(T) == 4) *(f32x4*)(mine + r * kPitch + at * 4) = v;
                else *(u32x2*)(mine + r * kPitch + at * 2) = (u32x2){bf16_pair(v.x, v.y), bf16_pair(v.z, v.w)};
            }
            asm volatile("" ::: "memory");      // a wave's LDS accesses happen in order
#pragma unroll
            for (int k = 0; k < 16; k += kAtOnce) {
                const int row = k + lane / kLanes;
                if (row >= 16) continue;
                const u32x4 d = *(const u32x4*)(mine + row * kPitch + c * 16);
                const int64_t out = y_row(wm * (BM / WM) + 16 * j + row);
                if (out >= 0 && col < n_left) *(u32x4*)((T*)a.y + out * a.N + p.n0 + col) = d;
            }
            asm volatile("" ::: "memory");
        }
    };
    const bool f32 = EXACT && a.y_dtype == TQ_F32;
    if (a.N % (f32 ? 4 : 8) == 0 && ((uintptr_t)a.y & 15) == 0) {
        lds_barrier();                          // every wave is done with the stages
        if constexpr (EXACT) {
            if (f32) {
                write_rows(float());
                return;
            }
        }
        write_rows(uint16_t());
        return;
    }
#pragma unroll
    for (int j = 0; j < MT; ++j) {
        const int64_t out = y_row(wm * (BM / WM) + 16 * j + r);
        if (out < 0) continue;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int col = wn * (BN / WN) + 16 * i + 4 * g;
            const f32x4 v = quad(i, j, col);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (col + e >= n_left) continue;
                const int64_t at = out * a.N + p.n0 + col + e;
                if (f32) ((float*)a.y)[at] = v[e];
                else ((uint16_t*)a.y)[at] = f32_to_bf16_rne(v[e]);
            }
        }
    }
}

template <bool EXACT, int BM, int BN, int WM, int WN, int KD, int KG, int NS, bool GROUPED>
hipError_t launch(const F8MatmulArgs& a, hipStream_t s) {
    constexpr int kThreads = 64 * WM * WN * KG;
    const int64_t nt = (a.N + BN - 1) / BN;
    int64_t blocks = (a.M + BM - 1) / BM * nt;
    if (GROUPED) blocks = grouped_blocks<BM>(a, nt);
    if (!grid_fits(blocks, kThreads)) return hipErrorInvalidConfiguration;
    f8_gemm_kernel<EXACT, BM, BN, WM, WN, KD, KG, NS, GROUPED><<<(unsigned)blocks, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

namespace {

template <bool EXACT>
hipError_t by_size(const F8MatmulArgs& a, hipStream_t s) {
    if (a.n_experts > 0)
        return a.M * a.top_k < 64 * (int64_t)a.n_experts ? launch<EXACT, 64, 128, 1, 4, 1, 1, 3, true>(a, s)
                                                         : launch<EXACT, 128, 128, 2, 2, 1, 1, 2, true>(a, s);
    const int64_t cus = compute_unit_count();
    auto tiles = [&](int64_t side) { return ((a.M + side - 1) / side) * ((a.N + side - 1) / side); };
    if (tiles(32) <= cus) return launch<EXACT, 32, 32, 1, 1, 1, 4, 4, false>(a, s);
    if (tiles(32) <= 2 * cus) return launch<EXACT, 32, 64, 1, 2, 1, 4, 3, false>(a, s);
    if constexpr (!EXACT)
        if (4 * tiles(256) >= 3 * cus) return launch<EXACT, 256, 256, 2, 4, 1, 1, 2, false>(a, s);
    if (4 * tiles(128) >= 3 * cus) return launch<EXACT, 128, 128, 2, 2, 1, 1, 2, false>(a, s);
    return tiles(64) <= cus ? launch<EXACT, 64, 64, 2, 2, 2, 1, 4, false>(a, s) : launch<EXACT, 64, 64, 2, 2, 2, 1, 2, false>(a, s);
}

}  // namespace

// The largest tile that still gives nearly every compute unit one (its rate is the highest, 2.3
// PFLOP/s, but a wave of tiles costs its time whether it fills the chip or not); tiles of 128 x
// 128 share a unit's LDS by twos.  us, bf16 y, graph replays over 600 MB of weights, short sums:
//                          256 x 256   128 x 128   64 x 64, 2 stages / 4   32 x 64, 3   32 x 32, 4
//   M = 2048  8192 x 8192     126         151         256 / 413
//   M = 1024  14336 x 4096     62          76         108 / 187
//   M =  512  8192 x 8192      94          45          58 /  92
//   M =  256  8192 x 8192      98          48          43 /  56           91           112
//   M =  128  8192 x 8192      94          48          34 /  27           49            59
//   M =   64  8192 x 8192      93          44          34 /  31           26            33
//   M =   64  4096 x 4096      50          24          18 /  17           16            10
//   M =   32  8192 x 8192      93          43          32 /  29           27            20
// Sums in fp32 (256 x 256 would need more registers than there are):
//                          128 x 128   64 x 64, 2 stages / 4   32 x 64, 3   32 x 32, 4
//   M = 2048  8192 x 8192     224         329 / 464
//   M = 1024  14336 x 4096    112         146 / 224
//   M =  512  8192 x 8192      65          86 / 115
//   M =  256  8192 x 8192      66          48 /  61           93           105
//   M =  128  8192 x 8192      66          34 /  33           49            56
//   M =   64  8192 x 8192      65          34 /  32           27            32
//   M =   64  4096 x 4096      35          19 /  19           15            11
//   M =   32  8192 x 8192      64          33 /  32           28            20
// Where few tiles leave units idle, four groups of a workgroup's waves take a part of K each; the
// four stages of 32 x 32 and of the 64 x 64 tiles that fill the chip once hide latency.
// Experts, by the slots an expert has on average (64 experts of 2048 x 4096), 64 x 128 with 3
// stages / 128 x 128 with 2, short sums:
//   16   115 / 121     32   125 / 138     48   128 / 134     64   138 / 137     128   179 / 161
//   256   274 / 226
// and sums in fp32:
//   8   112 / 123      16   116 / 127     32   128 / 150     48   141 / 151     64   158 / 152
//   128   230 / 209    256   368 / 321
// (Before a list's slots came by LDS, its idle waves rested and its tiles shared W, 128 x 128 took 190
// at 128 slots and 255 at 256; 128 x 256 then 202 and 275, 256 x 256 204 and 262, 64 x 256 with 2
// stages 236 and 357.)
hipError_t launch_f8_gemm(const F8MatmulArgs& a, hipStream_t s) {
    return a.short_sums ? by_size<false>(a, s) : by_size<true>(a, s);
}

}  // namespace dmm
