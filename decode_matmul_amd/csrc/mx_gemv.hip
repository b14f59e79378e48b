// MXFP4 products, weight-streaming form for few tokens: y[m, n] = sum_k x[m, k] w_hat[n, k] (+ bias[n]).
//
// Mathematics.  Lane (r, g) = (lane % 16, lane / 16) takes block 4 u + g of 128
// columns of row r: with the block's 16 code bytes and one scale byte that is
// the operand layout of the 16x16x128 scaled matrix instruction, which takes
// MXFP4 activations loaded the same way (mx_matmul_mx).  For bf16 activations
// the hardware turns eight codes and their scale into eight exact bf16 values
// (four conversions), and the four octets of the lane's block go through four
// 16x16x32 bf16 matrix instructions; the sum over k may be taken in any order,
// so octet j pairs w[n, 32 b + 8 j ..] with x[m, 32 b + 8 j ..].
//
// Bound: the package's bytes.  Few tokens leave no other work to spread over
// the chip, so a workgroup owns 16 NT rows and its W waves take the 256-wide
// chunks of K in turn, each with two chunks' loads in flight; the waves' sums
// meet in LDS, in wave order.  Everything read once goes through LDS:
//  * Codes by loads straight to LDS, whole 128-byte lines of 8 rows an
//    instruction.  Read in the matrix instruction's layout instead (16 rows x
//    64 bytes), 31 MB took 7.4 us against 6.2 in a bare read.
//  * Scales, 256 bytes a row for 8192 columns, loaded once by the workgroup:
//    read by each wave, 8 bytes of 16 rows at a time, they cost 1.4 us of 8.8.
//  * bf16 activations of a chunk, straight to a buffer of the wave's own.
// 16-byte pieces are permuted within their rows so that the 16 rows of a
// fragment read hit all banks.
#include <type_traits>

#include "mx.h"

namespace dmm {

namespace {

constexpr int kChunk = 256;                     // columns: 8 blocks, 128 bytes of codes
constexpr int kSegChunks = 32;                  // chunks whose scales are staged together: 256 bytes a row

// An entry of the order list, wave-uniform.
__device__ __forceinline__ int order_at(const int32_t* order, int64_t i) {
    return ((const __attribute__((address_space(4))) int32_t*)order)[i];
}

// MXX: activations in MXFP4.  TB: tokens of a pass.  NT: 16-row tiles.  W:
// waves.  DIRECT: bf16 activations 16-byte aligned.
template <bool MXX, int TB, int NT, int W, bool DIRECT, bool GROUPED>
__global__ void __launch_bounds__(64 * W, 2) mx_gemv_kernel(MxMatmulArgs a, int scale_lines) {
    constexpr int rows = 16 * NT;
    constexpr int kThreads = 64 * W;
    constexpr int kWBytes = NT * 2048, kXBytes = MXX ? 0 : TB * 512, kBuf = kWBytes + kXBytes;
    constexpr int kXLoads = MXX ? 3 : DIRECT ? TB / 2 : 0, kLoads = 2 * NT + kXLoads;     // loads of a chunk
    constexpr bool kOneWave = W <= 4 && 2 * (2 * W * kBuf + NT * 4096) > 160 * 1024;   // a SIMD
    __shared__ __attribute__((aligned(1024))) uint8_t buf0[W][kBuf];
    __shared__ __attribute__((aligned(1024))) uint8_t buf1[W][kBuf];
    __shared__ __attribute__((aligned(1024))) uint8_t sbuf[NT * 4096];
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = readfirstlane(tid >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int nb = (int)((a.K + 31) / 32);
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
    // offsets from the tile's first row (32 bits hold them: kMxMaxK); rows past the tile repeat its last
    const uint8_t* const wbase = a.codes + (expert * a.N + n0) * nb * 16;
    const uint8_t* const sbase = a.scales + (expert * a.N + n0) * nb;
    // of row l / 8 of the i-th eight rows: the piece that lane l brings
    auto piece = [&](int l, int i) { return (l & 7) ^ swizzle((i & 1) * 8 + (l >> 3)); };
    uint32_t woff[2 * NT];
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i) {
        const int row = 8 * i + (lane >> 3);
        woff[i] = (uint32_t)(row < nrows ? row : nrows - 1) * (uint32_t)nb * 16u;
    }
    const int full = (int)(a.K / kChunk), chunks = (int)((a.K + kChunk - 1) / kChunk);
    const int segs = (chunks + kSegChunks - 1) / kSegChunks;
    // Where piece 0 (16 bytes) of token i's 512 bytes sits: the tokens that are read
    // together, 0-3 and 12-15 a lane group ahead of 4-11, hit different banks (see swizzle).
    auto token_slot = [](int i) { return (i & 3) | ((i >> 3) & 1) << 2 | (((i >> 3) ^ (i >> 2)) & 1) << 3; };

    for (int64_t t0 = begin; t0 < end; t0 += TB) {
        const int count = (int)(end - t0 < TB ? end - t0 : TB);
        // Two tokens a load: lanes 0..31 and 32..63 bring 512 bytes each.
        int64_t xoff[TB / 2];
        auto find_x = [&]() {
            // by scalar loads: a vector load would be waited for behind those to LDS
            int slot[TB];
#pragma unroll
            for (int i = 0; i < TB; ++i) slot[i] = GROUPED ? order_at(a.order, t0 + (i < count ? i : count - 1)) : 0;
#pragma unroll
            for (int j = 0; j < TB / 2; ++j) {
                const int i = 2 * j + (lane >> 5);
                int64_t row = t0 + (i < count ? i : count - 1);     // tokens past the pass repeat its last
                if (GROUPED) {
                    const uint32_t s = (uint32_t)(lane < 32 ? slot[2 * j] : slot[2 * j + 1]);
                    row = (int64_t)((s < (uint32_t)slots ? s : 0u) / (uint32_t)a.top_k);
                }
                xoff[j] = (row * a.ldx + (((lane & 31) ^ token_slot(i)) << 3)) * 2;
            }
        };
        const uint8_t* const xcbase = MXX ? a.x_codes + t0 * nb * 16 : nullptr;
        const uint8_t* const xsbase = MXX ? a.x_scales + t0 * nb : nullptr;
        const uint32_t xr = (uint32_t)(r < count ? r : count - 1) * (uint32_t)nb;
        // where the lane's four octets of a token's 128 columns, and its two blocks of a row, sit
        uint32_t xat[4], wat[2];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            xat[j] = (uint32_t)((r & (TB - 1)) * 512 + (((4 * g + j) ^ token_slot(r & (TB - 1))) << 4));
#pragma unroll
        for (int u = 0; u < 2; ++u) wat[u] = (uint32_t)(r * 128 + (((4 * u + g) ^ swizzle(r)) << 4));

        // MXX: activations of the chunks in flight
        u32x4 xc0[2], xc1[2];
        uint64_t xs0 = 0, xs1 = 0;
        auto load_w = [&](uint8_t* b, int c) {
            const GlobalBytes cb = scalar_base(wbase + (int64_t)c * 128);
#pragma unroll
            for (int i = 0; i < 2 * NT; ++i)
                load_lds16(cb + lane_offset(woff[i] + (uint32_t)((piece(lane, i)) << 4)), b + i * 1024);
        };
        auto load_x = [&](uint8_t* b, u32x4* xc, uint64_t& xs, int c) {
            if (MXX) {
                const GlobalBytes xb = scalar_base(xcbase + (int64_t)c * 128), sb = scalar_base(xsbase + (int64_t)c * 8);
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    xc[u] = *(const __attribute__((address_space(1))) u32x4*)(xb + lane_offset((xr + (uint32_t)g) * 16u) + u * 64);
                xs = *(const __attribute__((address_space(1))) u64u*)(sb + lane_offset(xr));
            } else {
                const GlobalBytes xb = scalar_base((const uint8_t*)a.x + (int64_t)c * (2 * kChunk));
#pragma unroll
                for (int j = 0; j < TB / 2; ++j) {
                    if (DIRECT) load_lds16(xb + lane_offset(xoff[j]), b + kWBytes + j * 1024);
                    else
                        *(u32x4*)(b + kWBytes + j * 1024 + lane * 16) =
                            *(const __attribute__((address_space(1))) u32x4h*)(xb + lane_offset(xoff[j]));
                }
            }
        };
        auto load = [&](uint8_t* b, u32x4* xc, uint64_t& xs, int c) {
            load_w(b, c);
            load_x(b, xc, xs, c);
        };
        // the chunk that ends past K: zeros for the activations that are not
        // there; W's blocks past the last repeat it
        auto load_tail = [&](uint8_t* b, u32x4* xc, uint64_t& xs, int c) {
            const int l = (int)lane_offset((uint32_t)lane), lg = l >> 4;
            if (MXX) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    xc[u] = (u32x4){0u, 0u, 0u, 0u};
                    if (8 * c + 4 * u + lg < nb)
                        xc[u] = *(const u32x4*)(xcbase + lane_offset((xr + (uint32_t)lg) * 16u) + (int64_t)c * 128 + u * 64);
                }
                xs = scales8(xsbase + lane_offset(xr), 8 * (int64_t)c, nb);
            } else {
#pragma unroll
                for (int j = 0; j < TB / 2; ++j) {
                    const int q = ((l & 31) ^ token_slot(2 * j + (l >> 5))) << 3;
                    *(u32x4*)(b + kWBytes + j * 1024 + l * 16) =
                        load_x8(a.x + (lane_offset(xoff[j]) >> 1) - q, (int64_t)c * kChunk + q, a.K);
                }
            }
#pragma unroll
            for (int i = 0; i < 2 * NT; ++i) {
                int q = 8 * c + piece(l, i);
                q = q < nb ? q : nb - 1;
                load_lds16((GlobalBytes)wbase + lane_offset(woff[i] + (uint32_t)q * 16u), b + i * 1024);
            }
        };
        f32x4 acc[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[i] = (f32x4){0.f, 0.f, 0.f, 0.f};
        auto multiply = [&](const uint8_t* b, const u32x4* xc, uint64_t xs, int c, auto tail) {
            uint64_t sc[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i)
                sc[i] = *(const uint64_t*)(sbuf + (16 * i + r) * 256 + ((((c & 31) >> 1) ^ r) << 4) + (c & 1) * 8);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                u32x4 w[NT];
#pragma unroll
                for (int i = 0; i < NT; ++i) w[i] = *(const u32x4*)(b + i * 2048 + wat[u]);
                if constexpr (!MXX && decltype(tail)::value) {
                    const int left = (int)lane_offset((uint32_t)a.K) - 32 * (8 * c + 4 * u + g);
#pragma unroll
                    for (int i = 0; i < NT; ++i) w[i] = cut_codes(w[i], left < 0 ? 0 : left < 32 ? left : 32);
                }
                if (MXX) {
                    const int s = (int)((uint32_t)(xs >> (32 * u)) >> (8 * g));
#pragma unroll
                    for (int i = 0; i < NT; ++i)
                        acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            mx_operand(w[i]), mx_operand(xc[u]), acc[i], 4, 4, 0,
                            (int)((uint32_t)(sc[i] >> (32 * u)) >> (8 * g)), 0, s);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        // tokens past the pass read another's: their columns are not stored
                        const bf16x8 x = *(const bf16x8*)(b + kWBytes + xat[j] + u * 256);
#pragma unroll
                        for (int i = 0; i < NT; ++i) {
                            const uint32_t s = ((uint32_t)(sc[i] >> (32 * u)) >> (8 * g)) & 0xffu;
                            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(mx_decode8(w[i][j], e8m0_bits(s)), x, acc[i],
                                                                             0, 0, 0);
                        }
                    }
                }
                // keeps each half's operands to that half
#pragma unroll
                for (int i = 0; i < NT; ++i) hold_acc<kOneWave>(acc[i]);
                asm volatile("" ::: "memory");
            }
        };
        // Scales of segment s, 16 pieces of 16 bytes a row: piece q of row i sits at
        // q ^ (i % 16).  With scale_lines (rows of whole, aligned pieces) wave w
        // brings them straight to LDS, four rows a load; what lies past the row
        // repeats its last piece.  Otherwise a thread brings a row's piece through
        // registers.  Bytes behind a row multiply zeros.
        constexpr int kScaleLoads = 4 * NT;
        auto start_scales = [&](int s) {
#pragma unroll
            for (int j = 0; j < (kScaleLoads + W - 1) / W; ++j) {
                const int i = wave + j * W;
                if (i >= kScaleLoads) break;
                const int l = (int)lane_offset((uint32_t)lane), row = 4 * i + (l >> 4);
                const int b = s * (8 * kSegChunks) + (((l ^ row) & 15) << 4);
                load_lds16((GlobalBytes)sbase + ((int64_t)(row < nrows ? row : nrows - 1) * nb + (b < nb ? b : nb - 16)),
                           sbuf + i * 1024);
            }
        };
        auto copy_scales = [&](int s) {
#pragma unroll 1
            for (int q = tid; q < 256 * NT; q += kThreads) {
                const int row = q >> 4, b = s * (8 * kSegChunks) + (q & 15) * 16;
                if (b >= nb) continue;
                const uint8_t* const p = sbase + (int64_t)(row < nrows ? row : nrows - 1) * nb;
                const uint64_t lo = scales8(p, b, nb), hi = scales8(p, b + 8, nb);
                *(u32x4*)(sbuf + row * 256 + (((q ^ row) & 15) << 4)) =
                    (u32x4){(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
            }
        };

        // This wave's chunks are wave, wave + W, ..: two in flight, waited for by
        // count (at most the loads issued after them outstanding; the first two
        // send for their codes before their activations, whose addresses come later).
        uint8_t* const b0 = buf0[wave];
        uint8_t* const b1 = buf1[wave];
        if (segs > 0) {                                             // K = 0: nothing to read
            if (scale_lines) start_scales(0);
            else copy_scales(0);
        }
        asm volatile("" ::: "memory");
        if (wave < full) load_w(b0, wave);
        if (wave + W < full) load_w(b1, wave + W);
        asm volatile("" ::: "memory");
        if (!MXX) find_x();
        if (wave < full) load_x(b0, xc0, xs0, wave);
        asm volatile("" ::: "memory");
        if (wave + W < full) load_x(b1, xc1, xs1, wave + W);
        if (wave + W < full) wait_loads<2 * kLoads>();
        else if (wave < full) wait_loads<kLoads>();
        else wait_loads<0>();
        for (int s = 0; s < segs; ++s) {
            if (s > 0) {
                lds_barrier();                                      // every wave has read the segment before
                if (scale_lines) start_scales(s);
                else copy_scales(s);
                wait_loads<0>();
            }
            lds_barrier();
            const int c_end = (s + 1) * kSegChunks < full ? (s + 1) * kSegChunks : full;
            for (int c = s * kSegChunks + wave; c < c_end; c += 2 * W) {
                if (c == wave && c + W < full) wait_loads<kXLoads>();
                else if (c + W < full) wait_loads<kLoads>();
                else wait_loads<0>();
                multiply(b0, xc0, xs0, c, std::false_type());
                if (c + 2 * W < full) load(b0, xc0, xs0, c + 2 * W);
                if (c + W >= c_end) break;
                if (c + 2 * W < full) wait_loads<kLoads>();
                else wait_loads<0>();
                multiply(b1, xc1, xs1, c + W, std::false_type());
                if (c + 3 * W < full) load(b1, xc1, xs1, c + 3 * W);
            }
        }
        if (full < chunks && full % W == wave) {
            load_tail(b0, xc0, xs0, full);
            wait_loads<0>();
            multiply(b0, xc0, xs0, full, std::true_type());
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

template <bool MXX, int TB, int NT, int W, bool DIRECT, bool GROUPED>
hipError_t launch(const MxMatmulArgs& a, hipStream_t s) {
    constexpr int rows = 16 * NT;
    const int64_t blocks = (a.N + rows - 1) / rows * (GROUPED ? (int64_t)a.n_experts + 1 : 1);
    if (!grid_fits(blocks, 64 * W)) return hipErrorInvalidConfiguration;
    const int scale_lines = a.K % 512 == 0 && ((uintptr_t)a.scales & 15) == 0;
    mx_gemv_kernel<MXX, TB, NT, W, DIRECT, GROUPED><<<(unsigned)blocks, 64 * W, 0, s>>>(a, scale_lines);
    return hipGetLastError();
}

template <int TB, int NT, int W, bool GROUPED>
hipError_t launch_bf16(const MxMatmulArgs& a, hipStream_t s) {
    const bool direct = ((uintptr_t)a.x & 15) == 0 && (a.ldx % 8 == 0 || a.M == 1);
    return direct ? launch<false, TB, NT, W, true, GROUPED>(a, s) : launch<false, TB, NT, W, false, GROUPED>(a, s);
}

}  // namespace

hipError_t launch_mx_matmul(const MxMatmulArgs& a, hipStream_t s) {
    const int64_t tiles = (a.N + 15) / 16, cus = compute_unit_count();
    // Times here and in mx_gemm.hip are us a call in a replayed graph, each call with
    // other weights (600 MB of them, or 24 sets, in turn).
    // One pass of 16 tokens against the tiled form (tiled from the second figure on):
    //   bf16   M = 16   8192 x 8192  14.6 / 14.6   4096 x 4096  6.6 / 7.9   14336 x 4096  12.3 / 13.9
    //          M = 32   8192 x 8192  22.1 / 16.8   4096 x 4096  10.1 / 8.6  14336 x 4096  19.1 / 16.6
    // MXFP4 activations, whose tiles fetch little, pass earlier where the 32 x 32 tiles
    // of one row of them fill the chip (past two a unit, 64 x 64 tiles are no faster for
    // one token):
    //   M = 1      8192 x 8192  11.3 / 11.6   14336 x 4096  9.4 / 8.7    28672 x 8192  26.5 / 26.8
    //   M = 16     8192 x 8192  14.0 / 12.1   14336 x 4096  10.4 / 9.5   28672 x 8192  30.0 / 28.0
    //              4096 x 4096  6.1 / 5.9      4096 x 14336 11.7 / 17.4
    // and for experts from six slots each on (64 experts of 2048 x 4096: 61 / 57 us at 4
    // slots, just past where they cross, 82 / 62 at 6, 95 / 64 at 8).  That is by the
    // average, for fairly even lists: how long each is only the GPU knows.  300 slots
    // that all go to one expert take 153 us here, 384 in tiles 20; and the 320 slots of
    // no expert beside 56 that have one take 50 of 87, as the last workgroups write their
    // rows one after another.
    const int64_t halves = (a.N + 31) / 32;
    const int64_t few = !a.x_codes || 2 * halves <= cus || halves > 2 * cus ? 16 : halves <= cus ? 8 : 0;
    const bool many = a.n_experts > 0 ? a.M * a.top_k >= 6 * (int64_t)a.n_experts : a.M > few;
    if (many && mx_gemm_takes(a)) return launch_mx_gemm(a, s);
    if (a.n_experts > 0)
        return launch_bf16<8, 2, 4, true>(a, s);
    // Tiles of 16 rows a compute unit decide the shape: few tiles take 8 waves each
    // (K is what there is to spread), more share a workgroup, so that its
    // activations are read once for them.  us at 14336 x 4096 (3.5 tiles a unit) /
    // 8192 x 8192 (2) / 4096 x 4096 (1), by (tiles, waves) of a workgroup:
    //   M = 1:  (1, 8) 10.4 / 11.1 / 5.2   (2, 4)  9.3 / 12.7 / 6.3   (4, 4) 11.2 / 14.9 / 8.0
    //   M = 8:  (1, 8) 17.6 / 15.2 / 5.6   (2, 8) 13.6 / 12.6 / 6.2   (2, 4) 10.9 / 13.2 / 6.8
    //   M = 16: (1, 4) 21.7 / 19.5 / 6.6   (2, 4) 15.8 / 14.6 / 7.3   (4, 4) 12.3 / 17.6 / 8.9
    if (a.x_codes)
        return tiles <= 2 * cus ? launch<true, 16, 1, 8, true, false>(a, s) : launch<true, 16, 2, 4, true, false>(a, s);
    if (a.M <= 2) return tiles <= 2 * cus ? launch_bf16<2, 1, 8, false>(a, s) : launch_bf16<2, 2, 4, false>(a, s);
    if (a.M <= 4) return tiles <= 2 * cus ? launch_bf16<4, 1, 8, false>(a, s) : launch_bf16<4, 2, 4, false>(a, s);
    if (a.M <= 8)
        return tiles <= cus ? launch_bf16<8, 1, 8, false>(a, s)
               : tiles <= 2 * cus ? launch_bf16<8, 2, 8, false>(a, s)
                                  : launch_bf16<8, 2, 4, false>(a, s);
    return tiles <= cus ? launch_bf16<16, 1, 4, false>(a, s)
           : tiles <= 2 * cus ? launch_bf16<16, 2, 4, false>(a, s)
                              : launch_bf16<16, 4, 4, false>(a, s);
}

}  // namespace dmm
