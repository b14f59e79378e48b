// Products of e4m3 packages, weight-streaming form for few tokens:
//     y[m, n] = sum_b sx[m, b] sw[n / 128, b] sum_{k in b} cx[m, k] cw[n, k]  (+ bias[n]).
//
// Mathematics.  A block's 128 columns are four 16x16x32 bf16 matrix instructions (e4m3 values
// are exact in bf16; the e4m3 instructions lose bits of their sums), whose sum starts at 0
// and is added to y's by one fused multiply-add with f = sx sw, in fp32.  Any order of k may
// be taken that is the same for both operands: lane group g of four takes the 16-byte pieces
// g and 4 + g of a block.
//
// Bound: the package's bytes.  A workgroup owns 16 NT rows and its W waves take the blocks in
// turn, each with up to NBUF blocks' loads in flight (for passes of 8 tokens the compiler waits for all of
// them once a round, before it reads the first buffer's fragments of W); the waves' sums meet in
// LDS, in wave order.
// Codes go straight to LDS, whole lines of 8 rows a load; pieces change places within their
// rows so that the 16 rows of a fragment read hit all banks.  The products f of up to
// kSegBlocks blocks are staged once by the workgroup.  (14336 x 4096, 8 tokens, (1, 8) 2, caches
// not passed: 16.3 us, 14.3 without the products, 13.6 without the activations' loads as well,
// whether a load takes 128 bytes of eight rows or 1024 of one.)
#include "f8.h"
#include "waits.h"

namespace dmm {

namespace {

// An entry of the order list, wave-uniform.
__device__ __forceinline__ int order_at(const int32_t* order, int64_t i) {
    return ((const __attribute__((address_space(4))) int32_t*)order)[i];
}

// TB: tokens of a pass (8 or 16).  NT: 16-row tiles.  W: waves.  NBUF: blocks of a wave under way.
template <int TB, int NT, int W, int NBUF, bool GROUPED>
__global__ void __launch_bounds__(64 * W, 2) f8_gemv_kernel(F8MatmulArgs a) {
    constexpr int rows = 16 * NT, kThreads = 64 * W;
    constexpr int kWBytes = NT * 2048, kXBytes = TB * kF8Block, kBuf = kWBytes + kXBytes;
    constexpr int kXLoads = TB / 8, kLoads = 2 * NT + kXLoads;      // loads of a block
    static_assert(128 % rows == 0, "a tile has one scale of W a block");
    constexpr int kSegBlocks = W * NBUF * ((64 + W * NBUF - 1) / (W * NBUF));   // whose factors are staged together
    constexpr int kEach = (TB * kSegBlocks + kThreads - 1) / kThreads;          // factors a thread
    // distinct arrays: the compiler can tell a load in flight to one from the reads of another
    __shared__ __attribute__((aligned(1024))) uint8_t buf0[W][kBuf];
    __shared__ __attribute__((aligned(1024))) uint8_t buf1[W][kBuf];
    __shared__ __attribute__((aligned(1024))) uint8_t buf2[NBUF > 2 ? W : 1][NBUF > 2 ? kBuf : 16];
    __shared__ float factors[kSegBlocks][TB];
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = readfirstlane(tid >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int nb = (int)((a.K + kF8Block - 1) / kF8Block);
    const uint32_t ntiles = (uint32_t)((a.N + rows - 1) / rows), by = GROUPED ? blockIdx.x / ntiles : 0u;
    const int64_t n0 = (int64_t)(blockIdx.x - by * ntiles) * rows;
    const int nrows = (int)(a.N - n0 < rows ? a.N - n0 : rows);
    const int64_t expert = by;

    int64_t begin = 0, end = a.M;                               // tokens, or positions in the order list
    const int64_t slots = a.M * a.top_k;
    if (GROUPED) {
        begin = order_at(a.offsets, expert);
        end = expert < a.n_experts ? (int64_t)order_at(a.offsets, expert + 1) : slots;
        begin = begin < 0 ? 0 : begin;
        end = end > slots ? slots : end;
        if (expert == a.n_experts) {                            // slots of no expert
            for (int64_t i = begin; i < end; ++i) {
                const int64_t slot = a.order[i];
                if (slot < 0 || slot >= slots || tid >= nrows) continue;
                if (a.y_dtype == TQ_F32) ((float*)a.y)[slot * a.N + n0 + tid] = __builtin_nanf("");
                else ((uint16_t*)a.y)[slot * a.N + n0 + tid] = 0x7fc0u;
            }
            return;
        }
    }
    // offsets from the tile's first row (32 bits hold them: kF8MaxK); rows past the tile repeat its last
    const uint8_t* const wbase = a.codes + (expert * a.N + n0) * nb * kF8Block;
    const float* const sw = a.scales + (expert * ((a.N + 127) / 128) + n0 / 128) * nb;
    // of row l / 8 of the i-th eight rows: the piece that lane l brings
    auto piece = [&](int l, int i) { return (l & 7) ^ swizzle((i & 1) * 8 + (l >> 3)); };
    uint32_t woff[2 * NT];
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i) {
        const int row = 8 * i + (lane >> 3);
        woff[i] = (uint32_t)(row < nrows ? row : nrows - 1) * (uint32_t)nb * kF8Block + (uint32_t)(piece(lane, i) << 4);
    }

    const bool once = !GROUPED || end - begin <= TB;            // W is read once
    for (int64_t t0 = begin; t0 < end; t0 += TB) {
        const int count = (int)(end - t0 < TB ? end - t0 : TB);
        // x's row of token i of the pass; tokens past it repeat its last
        auto x_row = [&](int i) -> int64_t {
            const int64_t at = t0 + (i < count ? i : count - 1);
            if (!GROUPED) return at;
            const uint32_t s = (uint32_t)a.order[at];
            return (int64_t)((s < (uint32_t)slots ? s : 0u) / (uint32_t)a.top_k);
        };
        int64_t xoff[kXLoads];
#pragma unroll
        for (int j = 0; j < kXLoads; ++j) xoff[j] = x_row(8 * j + (lane >> 3)) * nb * kF8Block + (piece(lane, j) << 4);
        const int xr = (r & (TB - 1)) * kF8Block, wr = r * kF8Block;
        const int at0 = (g ^ swizzle(r & (TB - 1))) << 4, at1 = ((4 + g) ^ swizzle(r & (TB - 1))) << 4;
        const int wt0 = (g ^ swizzle(r)) << 4, wt1 = ((4 + g) ^ swizzle(r)) << 4;
        auto load = [&](uint8_t* b, int c) {
            const GlobalBytes wb = scalar_base(wbase + (int64_t)c * kF8Block);
#pragma unroll
            for (int i = 0; i < 2 * NT; ++i) {
                if (once) load_lds16<true>(wb + lane_offset(woff[i]), b + i * 1024);
                else load_lds16(wb + lane_offset(woff[i]), b + i * 1024);
            }
            const GlobalBytes xb = scalar_base(a.x_codes + (int64_t)c * kF8Block);
#pragma unroll
            for (int j = 0; j < kXLoads; ++j) load_lds16(xb + lane_offset(xoff[j]), b + kWBytes + j * 1024);
        };
        f32x4 acc[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[i] = (f32x4){0.f, 0.f, 0.f, 0.f};
        auto multiply = [&](const uint8_t* b, int c, int kept) {
            const float f = factors[c % kSegBlocks][r & (TB - 1)];
            bf16x8 x[4];
            auto fragment = [&](const uint8_t* row, int p0, int p1, bf16x8* v) {
                u32x4 d[2] = {*(const u32x4*)(row + p0), *(const u32x4*)(row + p1)};
                if (kept < kF8Block) {
                    d[0] = keep_bytes(d[0], kept - 16 * g);
                    d[1] = keep_bytes(d[1], kept - 64 - 16 * g);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] = f8_bf16(d[q >> 1][2 * (q & 1)], d[q >> 1][2 * (q & 1) + 1]);
            };
            // tokens past the pass read another's: their columns are not stored
            fragment(b + kWBytes + xr, at0, at1, x);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                bf16x8 w[4];
                fragment(b + i * 2048 + wr, wt0, wt1, w);
                f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int q = 0; q < 4; ++q) part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[q], x[q], part, 0, 0, 0);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][e] = __builtin_fmaf(f, part[e], acc[i][e]);
                asm volatile("" : "+v"(acc[i]));
            }
            asm volatile("" ::: "memory");
        };
        auto kept_of = [&](int c) {
            const int64_t left = a.K - (int64_t)c * kF8Block;
            return left < kF8Block ? (int)left : kF8Block;
        };
        // factors of blocks s0 .. s0 + kSegBlocks - 1: thread q's are numbers q, q + kThreads, ..
        float fx[kEach], fw[kEach];
        auto fetch_factors = [&](int s0) {
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int q = tid + i * kThreads, m = q / kSegBlocks, b = s0 + q % kSegBlocks;
                const bool there = m < count && b < nb;
                fx[i] = a.x_scales[there ? x_row(m) * nb + b : 0];
                fw[i] = there ? sw[b] : 0.f;
                if (!there) fx[i] = 0.f;
            }
        };
        auto store_factors = [&]() {
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int q = tid + i * kThreads;
                if (q < TB * kSegBlocks) factors[q % kSegBlocks][q / kSegBlocks] = fx[i] * fw[i];
            }
        };

        // This wave's blocks are wave, wave + W, ..: NBUF under way, waited for by count.
        static_assert(NBUF == 2 || NBUF == 3, "as many buffers");
        uint8_t* const bufs[3] = {buf0[wave], buf1[wave], NBUF > 2 ? buf2[wave] : nullptr};
        if (nb > 0) {
            fetch_factors(0);
            asm volatile("" ::: "memory");
#pragma unroll
            for (int i = 0; i < NBUF; ++i) {
                load(bufs[i], wave + i * W < nb ? wave + i * W : nb - 1);       // one that is not there: the last, again
                asm volatile("" ::: "memory");
            }
        }
        for (int s0 = 0; s0 < nb; s0 += kSegBlocks) {
            if (s0 > 0) {
                lds_barrier();                  // every wave has read the segment before
                fetch_factors(s0);
            }
            store_factors();
            lds_barrier();
            const int c_end = s0 + kSegBlocks < nb ? s0 + kSegBlocks : nb;
            for (int c0 = s0 + wave; c0 < c_end; c0 += NBUF * W) {
#pragma unroll
                for (int i = 0; i < NBUF; ++i) {
                    const int c = c0 + i * W;
                    if (c >= c_end) break;
                    const int behind = blocks_behind(c, W, NBUF, nb);
                    if (behind == NBUF - 1) wait_loads<(NBUF - 1) * kLoads>();
                    else if (behind == 1) wait_loads<kLoads>();
                    else wait_loads<0>();
                    multiply(bufs[i], c, kept_of(c));
                    if (c + NBUF * W < nb) load(bufs[i], c + NBUF * W);
                }
            }
        }
        wait_loads<0>();
        lds_barrier();
        f32x4* const red = (f32x4*)&buf0[0][0];                     // [W][NT][64]: the buffers are free now
#pragma unroll
        for (int i = 0; i < NT; ++i) red[(wave * NT + i) * 64 + lane] = acc[i];
        lds_barrier();
        // lane (m, q) of tile i holds y[m, n0 + 16 i + 4 q ..]
        const int l = (int)lane_offset((uint32_t)lane), m = l & 15;
        if (wave < NT && m < count) {
            const int i = wave;
            f32x4 v = red[i * 64 + l];
#pragma unroll
            for (int w = 1; w < W; ++w) v += red[(w * NT + i) * 64 + l];
            int64_t out = t0 + m;
            if (GROUPED) out = a.order[out];
            if (out >= 0 && out < slots) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int row = 16 * i + 4 * (l >> 4) + q;
                    if (row >= nrows) continue;
                    const int64_t col = n0 + row;
                    const float y = a.bias ? v[q] + a.bias[expert * a.N + col] : v[q];
                    if (a.y_dtype == TQ_F32) ((float*)a.y)[out * a.N + col] = y;
                    else ((uint16_t*)a.y)[out * a.N + col] = f32_to_bf16_rne(y);
                }
            }
        }
        lds_barrier();
    }
}

template <int TB, int NT, int W, int NBUF, bool GROUPED>
hipError_t launch(const F8MatmulArgs& a, hipStream_t s) {
    static_assert(NT <= W, "a wave for each tile at the end");
    constexpr int rows = 16 * NT;
    const int64_t blocks = (a.N + rows - 1) / rows * (GROUPED ? (int64_t)a.n_experts + 1 : 1);
    if (!grid_fits(blocks, 64 * W)) return hipErrorInvalidConfiguration;
    f8_gemv_kernel<TB, NT, W, NBUF, GROUPED><<<(unsigned)blocks, 64 * W, 0, s>>>(a);
    return hipGetLastError();
}

// One token: a wave takes kTokenRows rows as they lie in memory, 1 KB (eight blocks) of a row a load,
// S of each row under way at once and all of a short row's (4096 columns: the whole matrix is on its
// way, in registers).  The products are fp32 ones of the vector units, a block's sum within its
// eight lanes times f; the lanes' sums meet at the end.
constexpr int kTokenRows = 2;

template <int S>
__global__ void __launch_bounds__(256) f8_token_kernel(F8MatmulArgs a) {
    const int lane = (int)threadIdx.x & 63, wave = readfirstlane((int)threadIdx.x >> 6);
    const int64_t n0 = ((int64_t)blockIdx.x * 4 + wave) * kTokenRows;
    if (n0 >= a.N) return;
    const int nb = (int)((a.K + kF8Block - 1) / kF8Block), segs = (nb + 7) / 8;
    const float* const sw = a.scales + n0 / 128 * nb;           // kTokenRows divides 128
    const uint8_t* wrow[kTokenRows];
#pragma unroll
    for (int i = 0; i < kTokenRows; ++i) wrow[i] = a.codes + (n0 + i < a.N ? n0 + i : n0) * nb * kF8Block;
    float acc[kTokenRows];
#pragma unroll
    for (int i = 0; i < kTokenRows; ++i) acc[i] = 0.f;
    for (int s0 = 0; s0 < segs; s0 += S) {
        u32x4 w[S][kTokenRows], x[S];
        float fx[S], fw[S];
#pragma unroll
        for (int s = 0; s < S; ++s) {
            // a block that is not there: the row's first, times 0
            const int blk = (s0 + s) * 8 + lane / 8, at = blk < nb ? (s0 + s) * 1024 + lane * 16 : 0;
#pragma unroll
            for (int i = 0; i < kTokenRows; ++i) w[s][i] = __builtin_nontemporal_load((const u32x4*)(wrow[i] + at));
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int blk = (s0 + s) * 8 + lane / 8, at = blk < nb ? (s0 + s) * 1024 + lane * 16 : 0;
            x[s] = *(const u32x4*)(a.x_codes + at);
            fx[s] = a.x_scales[blk < nb ? blk : 0];
            fw[s] = sw[blk < nb ? blk : 0];
        }
        auto decode = [](uint32_t c, float* v) {
            const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false);
            const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
            v[0] = lo.x;
            v[1] = lo.y;
            v[2] = hi.x;
            v[3] = hi.y;
        };
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int64_t left = a.K - ((int64_t)(s0 + s) * 1024 + lane * 16);
            const int kept = left < 0 ? 0 : left < 16 ? (int)left : 16;
            const float f = left > 0 ? fx[s] * fw[s] : 0.f;
            float xv[16];
            x[s] = keep_bytes(x[s], kept);
#pragma unroll
            for (int q = 0; q < 4; ++q) decode(x[s][q], xv + 4 * q);
#pragma unroll
            for (int i = 0; i < kTokenRows; ++i) {
                const u32x4 c = keep_bytes(w[s][i], kept);
                float part = 0.f;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float v[4];
                    decode(c[q], v);
#pragma unroll
                    for (int e = 0; e < 4; ++e) part = __builtin_fmaf(v[e], xv[4 * q + e], part);
                }
                acc[i] = __builtin_fmaf(f, part, acc[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kTokenRows; ++i) acc[i] = group_sum<64>(acc[i]);
    if (lane < kTokenRows && n0 + lane < a.N) {
        float v = acc[0];
#pragma unroll
        for (int i = 1; i < kTokenRows; ++i) v = lane == i ? acc[i] : v;
        const int64_t n = n0 + lane;
        if (a.bias) v += a.bias[n];
        if (a.y_dtype == TQ_F32) ((float*)a.y)[n] = v;
        else ((uint16_t*)a.y)[n] = f32_to_bf16_rne(v);
    }
}

template <int S>
hipError_t launch_token(const F8MatmulArgs& a, hipStream_t s) {
    const int64_t blocks = (a.N + 4 * kTokenRows - 1) / (4 * kTokenRows);
    if (!grid_fits(blocks, 256)) return hipErrorInvalidConfiguration;
    f8_token_kernel<S><<<(unsigned)blocks, 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

// us a call in a replayed graph, each call with other weights (600 MB of them in turn):
//                 14336 x 4096  28672 x 8192  4096 x 14336  4096 x 4096  8192 x 8192  20480 x 5120
//   M = 1   by a token's kernel, four segments under way / two, against (1, 8) of three blocks
//                 11.7 / 12.5 / 16.1   38.5 / 40.5 / 40.7   14.3 / 13.2 / 14.4   5.6 / 5.7 / 6.9   14.1 / 15.4 / 14.2
//                                                                                   23.3 / 20.3 / 22.0
//   by (tiles of 16 rows, waves) of a workgroup and blocks of a wave under way:
//   M = 8   (1, 8) 2   15.5          40.8          15.4          7.7          16.1         21.1
//           (1, 8) 3   16.6          42.3          15.1          7.0          14.7         24.4
//           (2, 4) 3   14.5          50.2          21.9          9.4          19.2         24.0
//   M = 16  (1, 8) 2   17.8          47.3          16.2          8.0          16.6         27.3
//           (1, 8) 3   23.9          59.3          16.6          7.9          19.5         35.5
//           (2, 4) 3   14.8          50.5          20.5          9.6          19.0         24.9
// Weights past the caches gain 6 to 8 % of these.
// Experts, by the slots an expert has on average (64 of 2048 x 4096), streamed by (2, 4) 2 / tiles:
//   3   68 / -     4   82 / 99     6   108 / 106     8   126 / 108     12   170 / 111
// (2 on average: 54.7, 5.2 TB/s of the touched experts' packages.)
hipError_t launch_f8_matmul(const F8MatmulArgs& a, hipStream_t s) {
    const int64_t tiles = (a.N + 15) / 16, cus = compute_unit_count();
    if (a.n_experts > 0)
        return a.M * a.top_k >= 8 * (int64_t)a.n_experts ? launch_f8_gemm(a, s) : launch<8, 2, 4, 2, true>(a, s);
    if (a.M > 16) return launch_f8_gemm(a, s);
    if (a.M == 1) {
        const int64_t segs = (a.K + 1023) / 1024;               // four at a time, unless half of the last would be idle
        return segs % 4 == 0 || segs % 4 == 3 ? launch_token<4>(a, s) : launch_token<2>(a, s);
    }
    if (a.M <= 8) return tiles <= 2 * cus ? launch<8, 1, 8, 3, false>(a, s) : launch<8, 1, 8, 2, false>(a, s);
    // many tiles of short rows share their activations
    return tiles > 2 * cus && a.K <= 6144 ? launch<16, 2, 4, 3, false>(a, s) : launch<16, 1, 8, 2, false>(a, s);
}

}  // namespace dmm
