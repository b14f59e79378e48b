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
// turn, each with two blocks' loads in flight; the waves' sums meet in LDS, in wave order.
// Codes go straight to LDS, whole lines of 8 rows a load; pieces change places within their
// rows so that the 16 rows of a fragment read hit all banks.  The products f of up to
// kSegBlocks blocks are staged once by the workgroup.
#include "f8.h"

namespace dmm {

namespace {

constexpr int kSegBlocks = 64;

// An entry of the order list, wave-uniform.
__device__ __forceinline__ int order_at(const int32_t* order, int64_t i) {
    return ((const __attribute__((address_space(4))) int32_t*)order)[i];
}

// TB: tokens of a pass (8 or 16).  NT: 16-row tiles.  W: waves.
template <int TB, int NT, int W, bool GROUPED>
__global__ void __launch_bounds__(64 * W, 2) f8_gemv_kernel(F8MatmulArgs a) {
    constexpr int rows = 16 * NT, kThreads = 64 * W;
    constexpr int kWBytes = NT * 2048, kXBytes = TB * kF8Block, kBuf = kWBytes + kXBytes;
    constexpr int kXLoads = TB / 8, kLoads = 2 * NT + kXLoads;      // loads of a block
    static_assert(128 % rows == 0, "a tile has one scale of W a block");
    __shared__ __attribute__((aligned(1024))) uint8_t buf0[W][kBuf];
    __shared__ __attribute__((aligned(1024))) uint8_t buf1[W][kBuf];
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
            for (int i = 0; i < 2 * NT; ++i) load_lds16(wb + lane_offset(woff[i]), b + i * 1024);
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
        auto stage_factors = [&](int s0) {      // of blocks s0 .. s0 + kSegBlocks - 1
            const int n = nb - s0 < kSegBlocks ? nb - s0 : kSegBlocks;
            for (int q = tid; q < TB * kSegBlocks; q += kThreads) {
                const int m = q / kSegBlocks, b = q % kSegBlocks;
                if (b < n) factors[b][m] = m < count ? a.x_scales[x_row(m) * nb + s0 + b] * sw[s0 + b] : 0.f;
            }
        };

        // This wave's blocks are wave, wave + W, ..: two in flight, waited for by count.
        uint8_t* const b0 = buf0[wave];
        uint8_t* const b1 = buf1[wave];
        if (wave < nb) load(b0, wave);
        asm volatile("" ::: "memory");
        if (wave + W < nb) load(b1, wave + W);
        asm volatile("" ::: "memory");
        for (int s0 = 0; s0 < nb; s0 += kSegBlocks) {
            if (s0 > 0) lds_barrier();          // every wave has read the segment before
            stage_factors(s0);
            lds_barrier();
            const int c_end = s0 + kSegBlocks < nb ? s0 + kSegBlocks : nb;
            static_assert(kSegBlocks % (2 * W) == 0, "a wave's blocks of a segment go on where the last ended");
            for (int c = s0 + wave; c < c_end; c += 2 * W) {
                if (c + W < nb) wait_loads<kLoads>();
                else wait_loads<0>();
                multiply(b0, c, kept_of(c));
                if (c + 2 * W < nb) load(b0, c + 2 * W);
                if (c + W >= c_end) break;
                if (c + 2 * W < nb) wait_loads<kLoads>();
                else wait_loads<0>();
                multiply(b1, c + W, kept_of(c + W));
                if (c + 3 * W < nb) load(b1, c + 3 * W);
            }
        }
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

template <int TB, int NT, int W, bool GROUPED>
hipError_t launch(const F8MatmulArgs& a, hipStream_t s) {
    static_assert(NT <= W, "a wave for each tile at the end");
    constexpr int rows = 16 * NT;
    const int64_t blocks = (a.N + rows - 1) / rows * (GROUPED ? (int64_t)a.n_experts + 1 : 1);
    if (!grid_fits(blocks, 64 * W)) return hipErrorInvalidConfiguration;
    f8_gemv_kernel<TB, NT, W, GROUPED><<<(unsigned)blocks, 64 * W, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_f8_matmul(const F8MatmulArgs& a, hipStream_t s) {
    const int64_t tiles = (a.N + 15) / 16, cus = compute_unit_count();
    if (a.n_experts > 0)
        return a.M * a.top_k >= 8 * (int64_t)a.n_experts ? launch_f8_gemm(a, s) : launch<8, 2, 4, true>(a, s);
    if (a.M > 16) return launch_f8_gemm(a, s);
    if (a.M <= 8) return tiles <= 2 * cus ? launch<8, 1, 8, false>(a, s) : launch<8, 2, 4, false>(a, s);
    return tiles <= 2 * cus ? launch<16, 1, 8, false>(a, s) : launch<16, 2, 4, false>(a, s);
}

}  // namespace dmm
