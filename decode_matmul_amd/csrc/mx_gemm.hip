// MXFP4 products, tiled form for many tokens: y[m, n] = sum_k x[m, k] w_hat[n, k] (+ bias[n]).
//
// Mathematics.  As in mx_gemv.hip, a lane's 16 code bytes are the operand of
// the 16x16x128 scaled matrix instruction (MXFP4 activations), and four
// scaled conversions turn eight codes into eight exact bf16 values, here for the
// 32x32x16 bf16 instruction (bf16 activations).  Any order of k may be taken
// that is the same for both operands: with bf16 activations lane half g takes
// block g of each 64-wide unit, octet s in step s, so its codes are 16
// consecutive bytes and one scale.
//
// Mapping.  A workgroup owns BM tokens x BN rows of W, its waves equal parts of
// that (the largest tile: 256 x 256, 8 waves of 128 x 64, 128 accumulators a
// lane).  W is the first operand, so a lane ends with four consecutive n of one
// token.  K is cut into slabs, which take turns in two LDS arrays: distinct
// ones, so the compiler can tell a load in flight to one from the reads of the
// other.  Rows go from global memory straight to LDS in whole lines of 128 bytes
// (64 bf16 or 256 codes; slabs of 128 columns have 64 bytes of codes), a slab
// ahead; fragments go to registers a step ahead.  Chunks (16 bytes) change places
// within their rows so that a fragment read hits all banks (swizzle, w_slot).
//
// Bound.  The largest tile: the matrix instructions and the power they draw
// (bf16 2048 x 8192 x 8192: 1.3 PFLOP/s at 2.1 GHz; MXFP4 activations: with the
// loads left out 62 of 75 us remain, and the same instructions from registers
// alone reach 7.3 PFLOP/s).  Smaller tiles: what a compute unit can have under
// way, about 40 KB, against the latency of memory, and the requests for it (one for
// 8 bytes costs as much as one for a line).
#include <type_traits>

#include "experts.h"

namespace dmm {

namespace {

constexpr int kRow = 128;                       // bytes of an LDS tile row (activations; codes with MXFP4 ones)
constexpr int64_t kMaxTiledBytes = (int64_t)1 << 24;   // of a row in the tiled form: 256 rows fit 32-bit offsets

typedef float f32x16 __attribute__((ext_vector_type(16)));

// Which slot of W's rows of LANES chunks chunk 0 takes (rows of 128 bytes as the
// activations'; of rows of 64, four of which fill the banks, likewise).
template <int LANES>
__device__ __forceinline__ int w_slot(int row) {
    return LANES == 8 ? swizzle(row) : ((row >> 2) ^ (row >> 3)) & 3;
}

// MXX: activations in MXFP4.  DIRECT: whole slabs of bf16 activations (MXX: of
// scales) go straight to LDS, their rows aligned; otherwise through registers.  BM x BN
// tile of WM x WN waves; KD units (64 columns, or 256 with MXX) a slab.  KG
// groups of WM x WN waves take every KG-th slab each, and the first adds up the sums.
template <bool MXX, bool DIRECT, int BM, int BN, int WM, int WN, int KD, int KG, bool GROUPED>
__global__ void __launch_bounds__(64 * WM * WN * KG, 2) mx_gemm_kernel(MxMatmulArgs a) {
    constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;                 // of a group
    constexpr int kUnit = MXX ? 256 : 64, kSlab = KD * kUnit;
    constexpr int kWRow = MXX ? kRow : KD * 32;         // bytes of W's rows in LDS: a unit, or with bf16 activations a slab
    constexpr int kXUnit = BM * kRow, kWUnit = BN * kRow;
    constexpr int kXBytes = KD * kXUnit, kWBytes = BN * (kSlab / 2);
    constexpr int kSRow = 8 * KD, kSBytes = MXX ? (BM + BN) * kSRow : 0;
    constexpr int kStage = kXBytes + kWBytes + kSBytes;
    constexpr int TR = MXX ? 16 : 32;           // rows of a matrix instruction's tile
    constexpr int MT = BM / WM / TR, NT = BN / WN / TR; // tiles of a wave
    constexpr int HT = MXX ? MT / 2 : MT;       // tiles along M of a step
    constexpr int kXLoads = kXBytes / 1024 / kWaves, kWLoads = kWBytes / 1024 / kWaves;
    constexpr bool kOneWave = kWaves * KG <= 4 && 2 * (2 * KG * kStage + (GROUPED ? 256 : 0)) > 160 * 1024;   // a SIMD
    static_assert(kXLoads * 1024 * kWaves == kXBytes && kWLoads * 1024 * kWaves == kWBytes, "whole loads");
    static_assert(kXUnit % 1024 == 0 && kXLoads % KD == 0, "a load stays in a unit");
    static_assert(MXX || KD == 2 || KD == 4, "w_slot");
    static_assert(!MXX || BM + BN <= kThreads, "a thread for each row's scales");
    static_assert(KG == 1 || (!GROUPED && (MXX || KG * KD >= 8)), "a group fetches the scales of each of its slabs");
    __shared__ __attribute__((aligned(1024))) uint8_t stages0[KG * kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t stages1[KG * kStage];

    const int kg = KG == 1 ? 0 : readfirstlane((int)threadIdx.x / kThreads);
    const int tid = (int)threadIdx.x - kg * kThreads, lane = tid & 63, wave = readfirstlane(tid >> 6);
    uint8_t* const stage0 = stages0 + kg * kStage;
    uint8_t* const stage1 = stages1 + kg * kStage;
    const int r = lane % TR, g = lane / TR;
    const int wm = wave / WN, wn = wave % WN;
    const int64_t nb = (a.K + 31) / 32;

    Place p;
    if (GROUPED) {
        if (!place_grouped<BM, BN, 1, kThreads>(a, p)) {
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

    // Loads to LDS fill 1024 bytes at a time: eight rows of 128 bytes, lane l the
    // chunk whose slot is l % 8 of row l / 8 (W's rows of 64 bytes likewise, four lanes
    // each).  Load j of wave w is row group w + (j % (kXLoads / KD)) kWaves of a unit;
    // a wave's row groups repeat from unit to unit.
    const int x_sub = lane >> 3;
    auto x_group = [&](int j) { return wave + (j % (kXLoads / KD)) * kWaves; };
    auto x_unit = [&](int j) { return j / (kXLoads / KD); };
    auto x_chunk = [&](int j) { return (lane & 7) ^ swizzle(x_group(j) * 8 + x_sub); };
    // W's loads are dealt over the whole slab (a unit may have fewer than there are
    // waves).  Whole lines of the rows' codes, as far as a slab has them: with bf16
    // activations a unit is only 32 bytes of a row, and loads of such pieces cost as
    // much as loads of lines.
    constexpr int kWLanes = kWRow / 16, kWRows = 64 / kWLanes, kWGroups = BN / kWRows;  // lanes a row, rows a load
    auto w_all = [&](int j) { return wave + j * kWaves; };
    auto w_tile_row = [&](int j) { return w_all(j) % kWGroups * kWRows + lane / kWLanes; };
    auto w_unit = [&](int j) { return MXX ? w_all(j) / kWGroups : 0; };
    auto w_chunk = [&](int j) { return (lane & (kWLanes - 1)) ^ w_slot<kWLanes>(w_tile_row(j)); };
    // Offsets from the tile's first row fit 32 bits (mx_gemm_takes); the rows of a list have 64.
    typedef typename std::conditional<GROUPED, int64_t, uint32_t>::type XOffset;
    const uint8_t* const xbase = MXX ? a.x_codes + p.m0 * nb * 16 : (const uint8_t*)(a.x + (GROUPED ? 0 : p.m0) * a.ldx);
    const int64_t xrow_bytes = MXX ? nb * 16 : a.ldx * 2;
    XOffset xsrc[kXLoads / KD];
#pragma unroll
    for (int j = 0; j < kXLoads / KD; ++j)
        xsrc[j] = lane_offset((XOffset)x_row(x_group(j) * 8 + x_sub) * (XOffset)xrow_bytes + (XOffset)(x_chunk(j) * 16));
    const uint8_t* const wbase = a.codes + (p.expert * a.N + p.n0) * nb * 16;
    uint32_t wsrc[kWLoads];
#pragma unroll
    for (int j = 0; j < kWLoads; ++j) {
        wsrc[j] = lane_offset((uint32_t)w_row(w_tile_row(j)) * ((uint32_t)nb * 16u) + (uint32_t)(w_chunk(j) * 16 + w_unit(j) * (kUnit / 2)));
    }
    // Scales.  MXX: thread tid stages a slab's bytes of one row of W (the first BN
    // threads) or x, or (DIRECT) 16 bytes a row go straight to LDS.  Otherwise lane
    // (r, g) keeps 16 bytes, the scales of eight units, of each of its rows of W.
    const uint8_t* const wscales = a.scales + (p.expert * a.N + p.n0) * nb;
    const uint8_t* const xscales = MXX ? a.x_scales + p.m0 * nb : nullptr;
    static_assert(!MXX || !DIRECT || kSRow == 16, "a lane brings a row's scales");
    uint32_t ssrc[NT];
    const bool stages_w = BN % 64 == 0 ? wave < BN / 64 : tid < BN;
    if (MXX) {
        ssrc[0] = lane_offset((uint32_t)(stages_w ? w_row(tid) : (int)x_row((tid - BN) & (BM - 1))) * (uint32_t)nb);
    } else {
#pragma unroll
        for (int i = 0; i < NT; ++i) ssrc[i] = lane_offset((uint32_t)w_row(wn * (BN / WN) + TR * i + r) * (uint32_t)nb);
    }

    typedef typename std::conditional<MXX, f32x4, f32x16>::type Acc;
    Acc acc[NT][MT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[i][j] = (Acc)(0.f);

    // ---- a slab on its way to LDS
    u32x4 xr[kXLoads];                          // activations on the way through registers (!DIRECT)
    auto x_lds = [&](int j) { return x_unit(j) * kXUnit + x_group(j) * 1024; };
    auto w_lds = [&](int j) { return kXBytes + w_all(j) * 1024; };
    auto store_x = [&](uint8_t* st) {
#pragma unroll
        for (int j = 0; j < kXLoads; ++j) *(u32x4*)(st + x_lds(j) + lane * 16) = xr[j];
    };
    typedef uint32_t Scales __attribute__((ext_vector_type(2 * KD)));
    typedef Scales ScalesAt __attribute__((aligned(1)));
    Scales sreg;                                // MXX: scales on their way
    auto start = [&](uint8_t* st, int64_t t) {  // slab t, a whole one
        if (MXX) {
            const uint8_t* const rows = (stages_w ? wscales : xscales) + (t * KG + kg) * kSRow;
            const GlobalBytes from = (BN % 64 == 0 ? scalar_base(rows) : (GlobalBytes)rows) + lane_offset(ssrc[0]);
            if (!DIRECT) sreg = *(const __attribute__((address_space(1))) ScalesAt*)from;
            else if (wave < (BM + BN) / 64) load_lds16(from, st + kXBytes + kWBytes + wave * 1024);
        }
        const GlobalBytes xb = scalar_base(xbase + (t * KG + kg) * (KD * kRow));
        const GlobalBytes wb = scalar_base(wbase + (t * KG + kg) * (kSlab / 2));
#pragma unroll
        for (int j = 0; j < kXLoads; ++j) {
            if (BM == 32 && x_group(j) * 8 >= m_rows) continue;     // rows no token reads: few tokens fetch less
            const GlobalBytes from = xb + lane_offset(xsrc[j % (kXLoads / KD)]) + x_unit(j) * kRow;
            if (MXX || DIRECT) load_lds16(from, st + x_lds(j));
            else xr[j] = *(const __attribute__((address_space(1))) u32x4h*)from;
        }
#pragma unroll
        for (int j = 0; j < kWLoads; ++j) load_lds16(wb + lane_offset(wsrc[j]), st + w_lds(j));
    };
    auto finish = [&](uint8_t* st) {            // what came to registers
        if (MXX && !DIRECT && tid < BM + BN) *(Scales*)(st + kXBytes + kWBytes + tid * kSRow) = sreg;
        if (!MXX && !DIRECT) store_x(st);
    };
    // bf16 activations: scales of the units at hand and of the next, 16 bytes (eight
    // units) of a row at a time; 8 at a time were a third of a slab's requests.
    typedef uint64_t Sixteen __attribute__((ext_vector_type(2)));
    typedef Sixteen SixteenAt __attribute__((aligned(1)));
    const int64_t last = nb > 16 ? nb - 16 : 0;
    Sixteen sc[NT], sc_next[NT];
    auto fetch_scales = [&](int64_t q) {        // of units q .. q + 7, as far as there are any: the last 16
        const int64_t b = 2 * q < last ? 2 * q : last;
        const GlobalBytes sb = scalar_base(wscales + b);
#pragma unroll
        for (int i = 0; i < NT; ++i)
            sc_next[i] = *(const __attribute__((address_space(1))) SixteenAt*)(sb + lane_offset(ssrc[i]));
    };
    auto take_scales = [&](int64_t q) {         // q a multiple of 8 (of KD, where there are groups)
        const int64_t b = 2 * q < last ? 2 * q : last;
        const int skip = 8 * (int)(2 * q - b);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            sc[i] = sc_next[i];
            if (skip >= 64) sc[i] = (Sixteen){sc[i].y >> (skip - 64), 0};
            else if (skip > 0) sc[i] = (Sixteen){sc[i].x >> skip | sc[i].y << (64 - skip), sc[i].y >> skip};
        }
        constexpr int kNext = KG == 1 ? 8 : KG * KD;        // units to the next take
        if (2 * (q + kNext) < nb) fetch_scales(q + kNext);
    };

    // ---- fragments: step s (of four) of a unit from LDS to registers, then
    // multiplied.  bf16 activations: 16 columns a step.  MXX: 128 columns, of
    // half of the wave's tokens (fewer fragments at a time: 256 registers hold
    // them beside 128 accumulators).
    u32x4 wf[2][NT], xf[2][HT];                 // bf16 activations: wf[0] is a unit's codes
    u32x4 wc[NT];                               // bf16 activations: the codes at hand
    u32x2 sw_raw[NT], sx_raw[MT];
    int sw[NT], sx[MT];
    auto read = [&](const uint8_t* st, int k, int s) {
        const uint8_t* const xt = st + k * kXUnit + wm * (BM / WM) * kRow;
        const uint8_t* const wt = st + kXBytes + (MXX ? k * kWUnit : 0) + wn * (BN / WN) * kWRow;
        const int at = r * kRow + (((MXX ? 4 * (s >> 1) + g : 4 * g + s) ^ swizzle(r)) << 4);
        if (MXX && s == 0) {
            const uint8_t* const ws = st + kXBytes + kWBytes + wn * (BN / WN) * kSRow + 8 * k;
            const uint8_t* const xs = st + kXBytes + kWBytes + (BN + wm * (BM / WM)) * kSRow + 8 * k;
#pragma unroll
            for (int i = 0; i < NT; ++i) sw_raw[i] = *(const u32x2*)(ws + (TR * i + r) * kSRow);
#pragma unroll
            for (int j = 0; j < MT; ++j) sx_raw[j] = *(const u32x2*)(xs + (TR * j + r) * kSRow);
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            if (MXX && s % 2 == 0) wf[s >> 1][i] = *(const u32x4*)(wt + TR * i * kRow + at);
            if (!MXX && s == 0) wf[0][i] = *(const u32x4*)(wt + (TR * i + r) * kWRow + (((2 * k + g) ^ w_slot<kWLanes>(r)) << 4));
        }
#pragma unroll
        for (int j = 0; j < HT; ++j)
            xf[s & 1][j] = *(const u32x4*)(xt + TR * ((MXX ? (s & 1) * HT : 0) + j) * kRow + at);
    };
    auto multiply = [&](auto step) {
        constexpr int s = decltype(step)::value;
        if constexpr (MXX) {
            if (s == 0) {
                // bytes g and 4 + g of a row's eight scales: this lane's blocks of the two halves of a unit
                const uint32_t sel = 0x0c0c0400u + 0x0101u * (uint32_t)g;
#pragma unroll
                for (int i = 0; i < NT; ++i) sw[i] = (int)perm_b32(sw_raw[i].y, sw_raw[i].x, sel);
#pragma unroll
                for (int j = 0; j < MT; ++j) sx[j] = (int)perm_b32(sx_raw[j].y, sx_raw[j].x, sel);
            }
            constexpr int h = s >> 1, j0 = (s & 1) * HT;
#pragma unroll
            for (int j = 0; j < HT; ++j)
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    acc[i][j0 + j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        mx_operand(wf[h][i]), mx_operand(xf[s & 1][j]), acc[i][j0 + j], 4, 4, h, sw[i], h, sx[j0 + j]);
        } else {
            bf16x8 w[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                if (s == 0) wc[i] = wf[0][i];
                const uint32_t b = (uint32_t)(sc[i].x >> (8 * g)) & 0xffu;
                w[i] = mx_decode8(wc[i][s], e8m0_bits(b));
                if (s == 3) sc[i] = (Sixteen){sc[i].x >> 16 | sc[i].y << 48, sc[i].y >> 16};
            }
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[i], __builtin_bit_cast(bf16x8, xf[s & 1][j]),
                                                                        acc[i][j], 0, 0, 0);
        }
        // Keep the step where it is: without this its matrix instructions, which
        // touch no memory, may be put behind the reads of later steps, whose
        // fragments then are all held at once.
#pragma unroll
        for (int j = 0; j < HT; ++j)
#pragma unroll
            for (int i = 0; i < NT; ++i) hold_acc<kOneWave>(acc[i][(MXX ? (s & 1) * HT : 0) + j]);
        asm volatile("" ::: "memory");
    };
    typedef std::integral_constant<int, 0> S0;
    typedef std::integral_constant<int, 1> S1;
    typedef std::integral_constant<int, 2> S2;
    typedef std::integral_constant<int, 3> S3;

    // Slab t in `cur`: its first step is in registers.  A step is read while the
    // one before multiplies.  Before the last step every wave has read `cur`, and
    // slab t + 1 has landed in `other` (what of it came to registers is stored
    // there): while the last step multiplies, slab t + 2 starts into `cur` and the
    // first step of slab t + 1 is read.
    // (a group's slab t is slab t KG + kg of the rows)
    const int64_t full = a.K / kSlab / KG;
    auto slab = [&](uint8_t* cur, uint8_t* other, int64_t t) {
#pragma unroll
        for (int k = 0; k < KD; ++k) {
            if (!MXX && (KG > 1 ? k == 0 : (t * KD + k) % 8 == 0)) take_scales((t * KG + kg) * KD + k);
            read(cur, k, 1);
            multiply(S0());
            read(cur, k, 2);
            multiply(S1());
            read(cur, k, 3);
            multiply(S2());
            if (k + 1 < KD) {
                read(cur, k + 1, 0);
                multiply(S3());
            }
        }
        if (t + 1 < full) finish(other);
        wait_loads<0>();
        lds_barrier();
        if (t + 2 < full) start(cur, t + 2);
        if (t + 1 < full) read(other, 0, 0);
        multiply(S3());
    };

    if (!MXX) {
        if (nb >= 16) {
            fetch_scales(kg * KD);
        } else {                                // fewer than 16 bytes a row: all that there will be
#pragma unroll
            for (int i = 0; i < NT; ++i)
                sc_next[i] = (Sixteen){scales8(wscales + ssrc[i], 0, nb), scales8(wscales + ssrc[i], 8, nb)};
        }
    }
    if (full > 0) {
        start(stage0, 0);
        finish(stage0);
        wait_loads<0>();
        lds_barrier();
        if (full > 1) start(stage1, 1);
        read(stage0, 0, 0);
        for (int64_t t = 0; t < full; t += 2) {
            slab(stage0, stage1, t);
            if (t + 1 < full) slab(stage1, stage0, t + 1);
        }
    }
    // units that are left, the last one maybe cut: up to KD for each group
    const int64_t first = (full * KG + kg) * KD, units = (nb * 32 + kUnit - 1) / kUnit;
    if (units > full * KG * KD) {
        const int rest = units > first ? (int)(units - first < KD ? units - first : KD) : 0;
        // The slab that ends past K: activations through registers, zeros past K;
        // W's chunks past its last block repeat it (their products are 0).
        lds_barrier();
#pragma unroll
        for (int j = 0; j < kXLoads; ++j) {
            const int64_t u = first + x_unit(j);
            const uint8_t* const row = xbase + lane_offset(xsrc[j % (kXLoads / KD)]) - x_chunk(j) * 16;
            if (MXX) {
                xr[j] = (u32x4){0u, 0u, 0u, 0u};
                if (u * 8 + x_chunk(j) < nb) xr[j] = *(const u32x4*)(row + (u * 8 + x_chunk(j)) * 16);
            } else {
                xr[j] = load_x8((const uint16_t*)row, u * 64 + x_chunk(j) * 8, a.K);
            }
        }
        store_x(stage0);
#pragma unroll
        for (int j = 0; j < kWLoads; ++j) {
            const int64_t c = w_unit(j) * (kUnit / 32) + w_chunk(j), b = first * (kUnit / 32) + c;
            load_lds16((GlobalBytes)(wbase + lane_offset(wsrc[j]) + ((b < nb ? b : nb - 1) - c) * 16), stage0 + w_lds(j));
        }
        if (MXX && tid < BM + BN) {
#pragma unroll
            for (int k = 0; k < KD; ++k)
                *(uint64_t*)(stage0 + kXBytes + kWBytes + tid * kSRow + 8 * k) =
                    scales8((stages_w ? wscales : xscales) + ssrc[0], (first + k) * 8, nb);
        }
        wait_loads<0>();
        lds_barrier();
#pragma unroll 1
        for (int k = 0; k < rest; ++k) {
            if (!MXX && (KG > 1 ? k == 0 : (first + k) % 8 == 0)) take_scales(first + k);
            read(stage0, k, 0);
            read(stage0, k, 1);
            if (!MXX && a.K % 32 != 0 && k + 1 == units - first && 2 * (int)(first + k) + g == (int)nb - 1) {
#pragma unroll
                for (int i = 0; i < NT; ++i) wf[0][i] = cut_codes(wf[0][i], (int)(a.K % 32));
            }
            multiply(S0());
            read(stage0, k, 2);
            multiply(S1());
            read(stage0, k, 3);
            multiply(S2());
            multiply(S3());
        }
    }

    if constexpr (KG > 1) {
        constexpr int Q = TR * TR / 256;        // quads of a lane's sums
        static_assert((KG - 1) * BM * BN * 4 <= KG * kStage, "the sums fit the stages");
        lds_barrier();
        auto sums = [&](int from, int i, int j, int q) -> f32x4& {
            return ((f32x4*)stages0)[((((from - 1) * kWaves + wave) * NT + i) * MT + j) * (Q * 64) + q * 64 + lane];
        };
        if (kg > 0) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < MT; ++j)
#pragma unroll
                    for (int q = 0; q < Q; ++q)
                        sums(kg, i, j, q) = (f32x4){acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        }
        lds_barrier();
        if (kg > 0) return;
#pragma unroll
        for (int from = 1; from < KG; ++from)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < MT; ++j)
#pragma unroll
                    for (int q = 0; q < Q; ++q) {
                        const f32x4 v = sums(from, i, j, q);
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[i][j][4 * q + e] += v[e];
                    }
    }

    // lane (r, g) of tile (i, j): token TR j + r, four n from TR i + 8 q + 4 g for
    // each q (16 x 16 tiles: from 4 g)
    const int64_t n_left = a.N - p.n0;
    auto quad = [&](int i, int j, int q, int col) {
        f32x4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
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
    // Rows of y in 16-byte pieces: the wave's TR tokens x NT TR columns of each j
    // change hands in LDS, so that whole lines are written.
    auto write_rows = [&](auto type) {
        typedef decltype(type) T;
        constexpr int kCols = NT * TR, kPitch = kCols * (int)sizeof(T) + 16, kEach = 16 / (int)sizeof(T);
        constexpr int kLanes = kCols / kEach, kAtOnce = 64 / kLanes;
        constexpr int kHalf = (kWaves + 1) / 2; // waves a stage
        static_assert(kHalf * TR * kPitch <= kStage && TR % kAtOnce == 0, "the stages hold the waves' rows");
        uint8_t* const mine = (wave < kHalf ? stage0 : stage1) + wave % kHalf * (TR * kPitch);
        const int c = lane % kLanes, col = wn * (BN / WN) + c * kEach;
#pragma unroll
        for (int j = 0; j < MT; ++j) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int q = 0; q < TR * TR / 256; ++q) {
                    const int at = TR * i + 8 * q + 4 * g;
                    const f32x4 v = quad(i, j, q, wn * (BN / WN) + at);
                    if constexpr (sizeof(T) == 4) *(f32x4*)(mine + r * kPitch + at * 4) = v;
                    else *(u32x2*)(mine + r * kPitch + at * 2) = (u32x2){bf16_pair(v.x, v.y), bf16_pair(v.z, v.w)};
                }
            asm volatile("" ::: "memory");      // a wave's LDS accesses happen in order
#pragma unroll
            for (int k = 0; k < TR; k += kAtOnce) {
                const int row = k + lane / kLanes;
                const u32x4 d = *(const u32x4*)(mine + row * kPitch + c * 16);
                const int64_t out = y_row(wm * (BM / WM) + TR * j + row);
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
        const int64_t out = y_row(wm * (BM / WM) + TR * j + r);
        if (out < 0) continue;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int q = 0; q < TR * TR / 256; ++q) {
                const int col = wn * (BN / WN) + TR * i + 8 * q + 4 * g;
                const f32x4 v = quad(i, j, q, col);
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

template <bool MXX, bool DIRECT, int BM, int BN, int WM, int WN, int KD, int KG, bool GROUPED>
hipError_t launch(const MxMatmulArgs& a, hipStream_t s) {
    constexpr int kThreads = 64 * WM * WN * KG;
    const int64_t nt = (a.N + BN - 1) / BN;
    int64_t blocks = (a.M + BM - 1) / BM * nt;
    if (GROUPED) blocks = grouped_blocks<BM>(a, nt);
    if (!grid_fits(blocks, kThreads)) return hipErrorInvalidConfiguration;
    mx_gemm_kernel<MXX, DIRECT, BM, BN, WM, WN, KD, KG, GROUPED><<<(unsigned)blocks, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

template <int BM, int BN, int WM, int WN, int KD, int KG, bool GROUPED>
hipError_t launch_bf16(const MxMatmulArgs& a, hipStream_t s) {
    const bool direct = ((uintptr_t)a.x & 15) == 0 && (a.ldx % 8 == 0 || a.M == 1);
    return direct ? launch<false, true, BM, BN, WM, WN, KD, KG, GROUPED>(a, s)
                  : launch<false, false, BM, BN, WM, WN, KD, KG, GROUPED>(a, s);
}

}  // namespace

bool mx_gemm_takes(const MxMatmulArgs& a) {
    return a.K * 2 < kMaxTiledBytes &&
           (a.x_codes || a.n_experts > 0 || a.M == 1 || a.ldx * 2 < kMaxTiledBytes);
}

// The largest tile that still gives every compute unit one (its rate is the
// highest, 1.3 PFLOP/s with bf16 and 3.6 with MXFP4 activations, but a wave of
// tiles costs its time whether it fills the chip or not).  us by tile, in one run (graph
// replays, as at launch_mx_matmul):
//   bf16    256 x 256 / 128 x 128 / 64 x 64
//     M = 2048, 8192 x 8192   205 /  239 /  334
//     M = 1024, 4096 x 4096    82 /   41 /   47
//     M =  512, 4096 x 4096    81 /   36 /   25
//     M =   64, 8192 x 8192   153 /   67 /   34
//   MXFP4
//     M = 2048, 8192 x 8192    73 /   97 /  154
//     M = 1024, 4096 x 4096    32 /   18 /   23
//     M =  512, 4096 x 4096    31 /   16 /   13
// Few tiles leave compute units idle and each other one with more to fetch than it
// can have under way: up to two tiles of 32 x 32 a unit take those, dealt over K to
// four groups of one wave (a slab of 256 columns each where a unit has one tile, of
// 128 where two share its LDS).  us, bf16, 32 x 32 / 64 x 64:
//     M = 32, 8192 x 8192   17 / 33     M =  64, 4096 x 4096    8.9 / 15.7
//     M = 64, 8192 x 8192   27 / 33     M = 128, 4096 x 4096   11.7 / 15.8
//     M = 64, 4096 x 14336  24 / 55     M = 256, 4096 x 4096   21.1 / 16.3
// MXFP4 (slabs of 256 columns), 32 x 32 / 64 x 64:
//     M = 32, 8192 x 8192   12.5 / 18.4   M =  64, 4096 x 4096  6.3 / 8.4
//     M = 64, 8192 x 8192   15.9 / 19.6   M = 256, 4096 x 4096  12.8 / 8.6
// (two groups of 64 x 64 gain nothing, 37.6 at M = 64, 8192 x 8192: the bytes a unit
// fetches stay the same.)
// Experts: by the slots an expert has on average, 32 x 128 / 64 x 256
//     (64 experts of 2048 x 4096)
//     32   96 / 102     48   116 / 105     256   390 / 289
// (four waves of 64 x 64 a tile of 64 x 256; eight of 32 x 64 took 348 where they
// took 326, tiles of 128 x 256 took 333 there and 181 against 134 at 64 slots).
hipError_t launch_mx_gemm(const MxMatmulArgs& a, hipStream_t s) {
    if (a.n_experts > 0)
        return a.M * a.top_k < 40 * (int64_t)a.n_experts ? launch_bf16<32, 128, 1, 4, 4, 1, true>(a, s)
                                                         : launch_bf16<64, 256, 1, 4, 2, 1, true>(a, s);
    const int64_t cus = compute_unit_count();
    auto tiles = [&](int64_t side) { return ((a.M + side - 1) / side) * ((a.N + side - 1) / side); };
    if (tiles(32) <= 2 * cus) {
        if (a.x_codes) return launch<true, false, 32, 32, 1, 1, 1, 4, false>(a, s);
        return tiles(32) <= cus ? launch_bf16<32, 32, 1, 1, 4, 4, false>(a, s) : launch_bf16<32, 32, 1, 1, 2, 4, false>(a, s);
    }
    if (4 * tiles(256) >= 3 * cus)
        return a.x_codes ? launch<true, false, 256, 256, 2, 4, 1, 1, false>(a, s) : launch_bf16<256, 256, 2, 4, 2, 1, false>(a, s);
    if (4 * tiles(128) >= 3 * cus)
        return a.x_codes ? launch<true, false, 128, 128, 2, 2, 1, 1, false>(a, s) : launch_bf16<128, 128, 2, 2, 2, 1, false>(a, s);
    if (!a.x_codes) return launch_bf16<64, 64, 2, 2, 4, 1, false>(a, s);
    // Aligned scales straight to LDS: 11.3 us against 12.1 at M = 512, 4096 x 4096.
    // The larger tiles' slabs have 8 bytes a row, two lanes of 4, which gained nothing.
    const bool aligned = a.K % 512 == 0 && (((uintptr_t)a.scales | (uintptr_t)a.x_scales) & 15) == 0;
    return aligned ? launch<true, true, 64, 64, 2, 2, 2, 1, false>(a, s) : launch<true, false, 64, 64, 2, 2, 2, 1, false>(a, s);
}

}  // namespace dmm
