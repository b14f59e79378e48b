// Products of e4m3 packages, tiled form for many tokens:
//     y[m, n] = sum_b sx[m, b] sw[n / 128, b] sum_{k in b} cx[m, k] cw[n, k]  (+ bias[n]).
//
// Mathematics.  A block's sum over 128 columns starts at 0 in the matrix instructions and is
// added to y's by one fused multiply-add with f = sx sw, in fp32.  Two ways to that sum:
//  * EXACT: the codes become bf16 (exact) and go through four 16x16x32 instructions, whose
//    sums are fp32's.
//  * otherwise one 16x16x128 e4m3 instruction, of twice the rate.  It lines up each eight
//    products (consecutive bytes of a lane) by the largest and drops what lies 2^-13 below
//    it, so a sum may be off by 7 2^-13 of its largest products.  That is for a bf16 y,
//    whose own rounding is 2^-9 of it.
// Any order of k may be taken that is the same for both operands: lane group g of four takes
// the 16-byte pieces g and 4 + g of a block.
//
// Mapping.  A workgroup owns BM tokens x BN rows of W, its waves equal parts of that.  W is
// the first operand, so a lane ends with four consecutive n of one token, and f is one value
// for each of its tokens.  K is cut into slabs of KD blocks, which take turns in two LDS
// arrays: distinct ones, so the compiler can tell a load in flight to one from the reads of
// the other.  Rows go from global memory straight to LDS in whole lines of 128 bytes, a block
// each, a slab ahead; pieces change places within their rows so that a fragment read
// hits all banks (swizzle).  The products f of FU blocks come by way of registers.
#include <type_traits>

#include "experts.h"
#include "f8.h"

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

// BM x BN tile of WM x WN waves; KD blocks a slab.  KG groups of WM x WN waves take every
// KG-th slab each, and the first adds up the sums.
template <bool EXACT, int BM, int BN, int WM, int WN, int KD, int KG, bool GROUPED>
__global__ void __launch_bounds__(64 * WM * WN * KG, 2) f8_gemm_kernel(F8MatmulArgs a) {
    constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;                 // of a group
    constexpr int kXUnit = BM * kRow, kWUnit = BN * kRow;
    constexpr int kXBytes = KD * kXUnit, kWBytes = KD * kWUnit, kStage = kXBytes + kWBytes;
    constexpr int MT = BM / WM / 16, NT = BN / WN / 16;                     // tiles of a wave
    constexpr int kXLoads = kXBytes / 1024 / kWaves, kWLoads = kWBytes / 1024 / kWaves;
    constexpr int NB = BN > 128 ? BN / 128 : 1;                             // scales of W along n
    constexpr int FU = KG > 1 || KD > 4 ? KD : 4, kFSlabs = FU / KD;        // blocks, slabs of a fetch of scales
    static_assert(kXLoads * 1024 * kWaves == kXBytes && kWLoads * 1024 * kWaves == kWBytes, "whole loads");
    static_assert(BM * NB <= kThreads, "a thread for each row's scales");
    static_assert(BN / WN <= 128 || NB == 1, "a wave has one scale of W");
    static_assert(FU % KD == 0 && (kFSlabs == 1 || kFSlabs >= 2), "whole slabs");
    __shared__ __attribute__((aligned(1024))) uint8_t stages0[KG * kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t stages1[KG * kStage];
    __shared__ float factors[KG][2][NB][FU][BM];

    const int kg = KG == 1 ? 0 : readfirstlane((int)threadIdx.x / kThreads);
    const int tid = (int)threadIdx.x - kg * kThreads, lane = tid & 63, wave = readfirstlane(tid >> 6);
    uint8_t* const stage0 = stages0 + kg * kStage;
    uint8_t* const stage1 = stages1 + kg * kStage;
    const int r = lane & 15, g = lane >> 4;
    const int wm = wave / WN, wn = wave % WN;
    const int64_t nb = (a.K + kF8Block - 1) / kF8Block;

    Place p;
    if (GROUPED) {
        if (!place_grouped<BM, BN, kThreads>(a, p)) {
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
    auto x_row = [&](int i) -> int64_t {
        const int m = i < m_rows ? i : m_rows - 1;
        if (!GROUPED) return m;
        const int64_t slot = a.order[p.m0 + m];
        return slot >= 0 && slot < slots ? (int64_t)((uint32_t)slot / (uint32_t)a.top_k) : 0;
    };
    auto w_row = [&](int i) { return i < n_rows ? i : n_rows - 1; };

    // Loads to LDS fill 1024 bytes at a time: eight rows, lane l the piece whose slot is l % 8
    // of row l / 8.  Load j of wave w is row group w + j kWaves of the slab's, unit by unit.
    const int sub = lane >> 3;
    auto x_group = [&](int j) { return (wave + j * kWaves) % (BM / 8); };
    auto x_unit = [&](int j) { return (wave + j * kWaves) / (BM / 8); };
    auto w_group = [&](int j) { return (wave + j * kWaves) % (BN / 8); };
    auto w_unit = [&](int j) { return (wave + j * kWaves) / (BN / 8); };
    auto piece = [&](int group) { return (lane & 7) ^ swizzle(group * 8 + sub); };
    // Offsets from the tile's first row fit 32 bits (kF8MaxK); the rows of a list have 64.
    typedef typename std::conditional<GROUPED, int64_t, uint32_t>::type XOffset;
    const int64_t row_bytes = nb * kRow;
    const uint8_t* const xbase = a.x_codes + (GROUPED ? 0 : p.m0) * row_bytes;
    const uint8_t* const wbase = a.codes + (p.expert * a.N + p.n0) * row_bytes;
    XOffset xsrc[kXLoads];
    uint32_t wsrc[kWLoads];
#pragma unroll
    for (int j = 0; j < kXLoads; ++j)
        xsrc[j] = lane_offset((XOffset)x_row(x_group(j) * 8 + sub) * (XOffset)row_bytes +
                              (XOffset)(x_unit(j) * kRow + piece(x_group(j)) * 16));
#pragma unroll
    for (int j = 0; j < kWLoads; ++j)
        wsrc[j] = lane_offset((uint32_t)w_row(w_group(j) * 8 + sub) * (uint32_t)row_bytes +
                              (uint32_t)(w_unit(j) * kRow + piece(w_group(j)) * 16));

    // Thread (row, n block) fetches FU scales of both and stages their products.
    typedef typename Floats<FU>::T Scales;
    typedef Scales ScalesAt __attribute__((aligned(4)));
    const int frow = tid % BM, fblk = tid / BM;
    const bool stages_f = fblk < NB;
    const int64_t n_blocks = (a.N + 127) / 128, nblk = p.n0 / 128 + fblk;
    const float* const sx = a.x_scales + ((GROUPED ? 0 : p.m0) + (stages_f ? x_row(frow) : 0)) * nb;
    const float* const sw = a.scales + (p.expert * n_blocks + (stages_f && nblk < n_blocks ? nblk : n_blocks - 1)) * nb;
    Scales fx, fw;
    auto fetch_factors = [&](int64_t b) {       // of blocks b .. b + FU - 1, as far as there are any
        if (!stages_f) return;
        if (b + FU <= nb) {
            fx = *(const ScalesAt*)(sx + b);
            fw = *(const ScalesAt*)(sw + b);
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
        for (int u = 0; u < FU; ++u) factors[kg][buf][fblk][u][frow] = fx[u] * fw[u];
    };

    f32x4 acc[NT][MT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};

    auto start = [&](uint8_t* st, int64_t t) {  // slab t, a whole one
        const GlobalBytes xb = scalar_base(xbase + (t * KG + kg) * (KD * kRow));
        const GlobalBytes wb = scalar_base(wbase + (t * KG + kg) * (KD * kRow));
#pragma unroll
        for (int j = 0; j < kXLoads; ++j) {
            if (BM == 32 && x_group(j) * 8 >= m_rows) continue;     // rows no token reads
            load_lds16(xb + lane_offset(xsrc[j]), st + (wave + j * kWaves) * 1024);
        }
#pragma unroll
        for (int j = 0; j < kWLoads; ++j)
            load_lds16(wb + lane_offset(wsrc[j]), st + kXBytes + (wave + j * kWaves) * 1024);
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
    auto read_w = [&](const uint8_t* st, int k, int i, bool cut) {
        u32x4 v[2];
        read_raw(st + kXBytes + k * kWUnit + (wn * (BN / WN) + 16 * i) * kRow, v, cut);
        as_parts(v, wf[i]);
    };
    const int fn = NB > 1 ? wn * (BN / WN) / 128 : 0;
    auto read_x = [&](const uint8_t* st, int buf, int k, int u, int j, bool cut) {
        read_raw(st + k * kXUnit + (wm * (BM / WM) + 16 * j) * kRow, xf[j & 1], cut);
        f[j & 1] = factors[kg][buf][fn][u][wm * (BM / WM) + 16 * j + r];
    };
    auto multiply = [&](int j, auto next) {
        Part x[kParts];
        as_parts(xf[j & 1], x);
        const float s = f[j & 1];
        f32x4 part[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            part[i] = (f32x4){0.f, 0.f, 0.f, 0.f};
            if constexpr (EXACT) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    part[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[i][q], x[q], part[i], 0, 0, 0);
            } else {
                part[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(f8_operand(wf[i]), f8_operand(x), part[i],
                                                                           0, 0, 0, 0, 0, 0);
            }
            next(i);
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(s, part[i][e], acc[i][j][e]);
            asm volatile("" : "+v"(acc[i][j]));
        }
        asm volatile("" ::: "memory");
    };
    auto nothing = [](int) {};

    // Slab t in `cur`: its first fragments are in registers.  Before the last tile every wave
    // has read `cur`, and slab t + 1 has landed in `other`: while the last tile
    // multiplies, slab t + 2 starts into `cur` and the first fragments of slab t + 1 are read.
    // The products f of slab t are in factors' half (t / kFSlabs) % 2, from block t % kFSlabs KD on.
    const int64_t full = a.K / kF8Block / KD / KG;
    auto block_of = [&](int64_t t) { return (t * KG + kg) * KD; };
    auto slab = [&](uint8_t* cur, uint8_t* other, int64_t t) {
        const int buf = (int)(t / kFSlabs) & 1, u0 = (int)(t % kFSlabs) * KD;
        const int buf1 = (int)((t + 1) / kFSlabs) & 1, u1 = (int)((t + 1) % kFSlabs) * KD;
        if (u0 == 0) fetch_factors(block_of(t + kFSlabs));
#pragma unroll
        for (int k = 0; k < KD; ++k) {
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                if (j + 1 < MT) {
                    read_x(cur, buf, k, u0 + k, j + 1, false);
                    multiply(j, nothing);
                } else if (k + 1 < KD) {
                    read_x(cur, buf, k + 1, u0 + k + 1, 0, false);
                    multiply(j, [&](int i) { read_w(cur, k + 1, i, false); });
                }
            }
        }
        if ((t + 1) % kFSlabs == 0) store_factors(buf1);
        wait_loads<0>();
        lds_barrier();
        if (t + 2 < full) start(cur, t + 2);
        if (t + 1 < full) {
            read_x(other, buf1, 0, u1, 0, false);
            multiply(MT - 1, [&](int i) { read_w(other, 0, i, false); });
        } else {
            multiply(MT - 1, nothing);
        }
    };
    static_assert(MT % 2 == 0, "the last tile's fragments and the next unit's first take turns");

    fetch_factors(block_of(0));
    if (full > 0) start(stage0, 0);
    store_factors(0);
    if (full > 0) {
        wait_loads<0>();
        lds_barrier();
        if (full > 1) start(stage1, 1);
        read_x(stage0, 0, 0, 0, 0, false);
#pragma unroll
        for (int i = 0; i < NT; ++i) read_w(stage0, 0, i, false);
        for (int64_t t = 0; t < full; t += 2) {
            slab(stage0, stage1, t);
            if (t + 1 < full) slab(stage1, stage0, t + 1);
        }
    }
    // blocks that are left, the last one maybe cut: up to KD for each group
    const int64_t first = block_of(full);
    if (nb > full * KG * KD) {
        const int rest = nb > first ? (int)(nb - first < KD ? nb - first : KD) : 0;
        lds_barrier();
        // units past the last block repeat it and are not multiplied
        auto unit_of = [&](int u) { return first + u < nb ? first + u : nb - 1; };
#pragma unroll
        for (int j = 0; j < kXLoads; ++j)
            load_lds16((GlobalBytes)xbase + lane_offset(xsrc[j]) + (unit_of(x_unit(j)) - x_unit(j)) * kRow,
                       stage0 + (wave + j * kWaves) * 1024);
#pragma unroll
        for (int j = 0; j < kWLoads; ++j)
            load_lds16((GlobalBytes)wbase + lane_offset(wsrc[j]) + (unit_of(w_unit(j)) - w_unit(j)) * kRow,
                       stage0 + kXBytes + (wave + j * kWaves) * 1024);
        wait_loads<0>();
        lds_barrier();
        const int buf = (int)(full / kFSlabs) & 1, u0 = (int)(full % kFSlabs) * KD;
#pragma unroll 1
        for (int k = 0; k < rest; ++k) {
            kept = a.K - (first + k) * kF8Block < kF8Block ? (int)(a.K - (first + k) * kF8Block) : kF8Block;
#pragma unroll
            for (int i = 0; i < NT; ++i) read_w(stage0, k, i, true);
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                read_x(stage0, buf, k, u0 + k, j, true);
                multiply(j, nothing);
            }
        }
    }

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
        const int64_t slot = a.order[p.m0 + i];
        return slot < slots ? slot : -1;
    };
    // Rows of y in 16-byte pieces: the wave's 16 tokens x 16 NT columns of each j change
    // hands in LDS, so that whole lines are written.
    auto write_rows = [&](auto type) {
        typedef decltype(type) T;
        constexpr int kCols = NT * 16, kPitch = kCols * (int)sizeof(T) + 16, kEach = 16 / (int)sizeof(T);
        constexpr int kLanes = kCols / kEach, kAtOnce = 64 / kLanes < 16 ? 64 / kLanes : 16;
        constexpr int kHalf = (kWaves + 1) / 2; // waves a stage
        static_assert(kHalf * 16 * kPitch <= kStage, "the stages hold the waves' rows");
        uint8_t* const mine = (wave < kHalf ? stage0 : stage1) + wave % kHalf * (16 * kPitch);
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
    const bool f32 = a.y_dtype == TQ_F32;
    if (a.N % (f32 ? 4 : 8) == 0 && ((uintptr_t)a.y & 15) == 0) {
        lds_barrier();                          // every wave is done with the stages
        if (f32) write_rows(float());
        else write_rows((uint16_t)0);
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

template <bool EXACT, int BM, int BN, int WM, int WN, int KD, int KG, bool GROUPED>
hipError_t launch(const F8MatmulArgs& a, hipStream_t s) {
    constexpr int kThreads = 64 * WM * WN * KG;
    const int64_t nt = (a.N + BN - 1) / BN;
    int64_t blocks = (a.M + BM - 1) / BM * nt;
    if (GROUPED) blocks = grouped_blocks<BM>(a, nt);
    if (!grid_fits(blocks, kThreads)) return hipErrorInvalidConfiguration;
    f8_gemm_kernel<EXACT, BM, BN, WM, WN, KD, KG, GROUPED><<<(unsigned)blocks, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_f8_gemm(const F8MatmulArgs& a, hipStream_t s) {
    const bool exact = a.y_dtype == TQ_F32;
    if (a.n_experts > 0) {
        if (a.M * a.top_k < 40 * (int64_t)a.n_experts)
            return exact ? launch<true, 32, 128, 1, 4, 2, 1, true>(a, s) : launch<false, 32, 128, 1, 4, 2, 1, true>(a, s);
        return exact ? launch<true, 128, 128, 2, 2, 1, 1, true>(a, s) : launch<false, 128, 256, 2, 4, 1, 1, true>(a, s);
    }
    const int64_t cus = compute_unit_count();
    auto tiles = [&](int64_t side) { return ((a.M + side - 1) / side) * ((a.N + side - 1) / side); };
    if (tiles(32) <= 2 * cus)
        return exact ? launch<true, 32, 32, 1, 1, 2, 4, false>(a, s) : launch<false, 32, 32, 1, 1, 2, 4, false>(a, s);
    if (!exact && 4 * tiles(256) >= 3 * cus) return launch<false, 256, 256, 2, 4, 1, 1, false>(a, s);
    if (4 * tiles(128) >= 3 * cus)
        return exact ? launch<true, 128, 128, 2, 2, 1, 1, false>(a, s) : launch<false, 128, 128, 2, 2, 1, 1, false>(a, s);
    return exact ? launch<true, 64, 64, 2, 2, 2, 1, false>(a, s) : launch<false, 64, 64, 2, 2, 2, 1, false>(a, s);
}

}  // namespace dmm
