// f8_pack, f8_unpack and f8_norm_pack: e4m3 values in blocks of 128 columns, with a scale
// for one row (activations) or for 128 (weights).
//
// Mathematics.  A block with a = max |w| has the least power of two s with a / s <= 448,
// the largest e4m3 value.  e4m3 keeps its four bits down to 2^-6, so a power of two loses
// nothing that a / 448 would keep but half a binade of subnormals, and w / s is exact: the
// hardware's nearest-even conversion is the only rounding.
//
// All of them move each byte once and compute a few operations a value: they are bound by
// memory, or for few rows by the launch.  A lane has eight consecutive values, sixteen
// lanes a block's 128; its largest magnitude takes four data-parallel moves.
#include "f8.h"

namespace dmm {

namespace {

constexpr int kThreads = 256;

// Packing by rows: a lane for eight values of the padded rows, `pieces` of them.
template <bool BF16, bool FLAT>
__global__ void __launch_bounds__(kThreads) f8_pack_kernel(const void* W, int64_t K, int64_t ldw, int64_t nb,
                                                           int64_t pieces, uint8_t* codes, float* scales,
                                                           int32_t* status) {
    const int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const bool live = t < pieces;
    float v[8];
    if (FLAT) {                                 // whole blocks without gaps: one long row
        load_row8<BF16>(W, t * 8, live ? 8 : 0, v, 0.f);
    } else {
        const int64_t blk = live ? t >> 4 : 0, row = blk / nb;
        const int64_t k = (blk - row * nb) * kF8Block + (t & 15) * 8, left = K - k;
        load_row8<BF16>(W, row * ldw + k, !live || left < 0 ? 0 : (int)(left < 8 ? left : 8), v, 0.f);
    }
    const uint32_t s = f8_scale_bits(over_group<16>(largest8(v), larger));
    if (!live) return;
    *(u32x2*)(codes + t * 8) = f8_encode8(v, s);
    if ((t & 15) == 0) {
        scales[t >> 4] = __builtin_bit_cast(float, s);
        if (s == kF8NaN) atomic_or_status(status, TQ_DATA_RANGE);
    }
}

// Packing 128 x 128: a workgroup a block, a thread eight values of every 16th row.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) f8_pack_square_kernel(const void* W, int64_t rows, int64_t K, int64_t ldw,
                                                                  int64_t nb, uint8_t* codes, float* scales,
                                                                  int32_t* status) {
    __shared__ uint32_t most[kThreads / 64];
    const int tid = (int)threadIdx.x;
    const int64_t br = blockIdx.x / nb, b = blockIdx.x - br * nb;
    const int64_t r0 = br * 128 + (tid >> 4), k = b * kF8Block + (tid & 15) * 8, left = K - k;
    const int have = left < 0 ? 0 : (int)(left < 8 ? left : 8);
    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + 16 * i;
        load_row8<BF16>(W, r < rows ? r * ldw + k : 0, r < rows ? have : 0, v[i], 0.f);
    }
    uint32_t a = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = larger(a, largest8(v[i]));
    a = over_group<64>(a, larger);
    if ((tid & 63) == 0) most[tid >> 6] = a;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) a = larger(a, most[w]);
    const uint32_t s = f8_scale_bits(a);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + 16 * i;
        if (r < rows) *(u32x2*)(codes + (r * nb + b) * kF8Block + (tid & 15) * 8) = f8_encode8(v[i], s);
    }
    if (tid == 0) {
        scales[blockIdx.x] = __builtin_bit_cast(float, s);
        if (s == kF8NaN) atomic_or_status(status, TQ_DATA_RANGE);
    }
}

// Decoding: a lane for eight codes of the padded rows.  A value is the fp32 product of code and
// scale (exact for a power of two), then rounded to bf16.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) f8_unpack_kernel(const uint8_t* codes, const float* scales, int64_t K,
                                                             int64_t nb, int64_t pieces, int shift, void* out,
                                                             int32_t* status) {
    const int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (t >= pieces) return;
    const int64_t blk = t >> 4, row = blk / nb, b = blk - row * nb;
    const int64_t k = b * kF8Block + (t & 15) * 8, left = K - k;
    const int have = left < 0 ? 0 : (int)(left < 8 ? left : 8);
    const u32x2 c = *(const u32x2*)(codes + t * 8);
    const float s = scales[(row >> shift) * nb + b];
    float v[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[h], false);
        const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[h], true);
        v[4 * h] = lo.x * s;
        v[4 * h + 1] = lo.y * s;
        v[4 * h + 2] = hi.x * s;
        v[4 * h + 3] = hi.y * s;
    }
    if (status) {
        bool nan = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) nan |= i < have && !(__builtin_fabsf(v[i]) < __builtin_inff());
        if (nan || !(__builtin_fabsf(s) < __builtin_inff())) atomic_or_status(status, TQ_DATA_RANGE);
        bool rest = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) rest |= i >= have && ((c[i >> 2] >> (8 * (i & 3))) & 0xffu) != 0u;
        if (rest) atomic_or_status(status, TQ_DATA_PADDING);
    }
    if (have > 0) store_row8<BF16>(out, row * K + k, have, v);
}

// ------------------------------------------------------------------- norm
//
// h = x + residual, rounded to the type of x, as it is stored; f = (mean h^2 + eps)^-1/2
// from a sum in float64 (squares of fp32 are exact there, and float64 runs at the rate of
// fp32), rounded to fp32; y = h f weight, each product rounded to fp32; y's package.
// The factor does not depend on how the sum is split, up to float64's own rounding, so that the package hardly ever does.
//
// WAVES waves a row, 4 / WAVES rows a workgroup of four.  HELD: the row's values stay in
// registers, CHUNKS times eight a lane; longer rows are read twice.
template <bool BF16, int WAVES, int CHUNKS, bool HELD>
__global__ void __launch_bounds__(WAVES > 4 ? 64 * WAVES : kThreads) f8_norm_pack_kernel(F8NormArgs a) {
    constexpr int kLanes = 64 * WAVES, kRows = WAVES > 4 ? 1 : 4 / WAVES;
    __shared__ double part[kRows * WAVES];
    const int lane = (int)threadIdx.x % kLanes, in = (int)threadIdx.x / kLanes;
    const int64_t row = (int64_t)blockIdx.x * kRows + in;
    const bool live = row < a.M;
    const int64_t nb = (a.K + kF8Block - 1) / kF8Block, pieces = live ? nb * 16 : 0;
    auto have_of = [&](int64_t p) {             // values of piece p (eight columns) that there are
        const int64_t left = a.K - p * 8;
        return left < 0 || p >= pieces ? 0 : (int)(left < 8 ? left : 8);
    };
    auto load_h = [&](int64_t p, float* h) {
        const int have = have_of(p);
        load_row8<BF16>(a.x, row * a.ldx + p * 8, have, h, 0.f);
        if (a.residual) {
            float r[8];
            load_row8<BF16>(a.residual, row * a.ldr + p * 8, have, r, 0.f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[i] += r[i];
                if (BF16) h[i] = bf16_bits_to_f32(f32_to_bf16_rne(h[i]));
            }
        }
    };
    float h[HELD ? CHUNKS : 1][8];
    double sum = 0.0;
    auto square = [&](const float* v) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = __builtin_fma((double)v[i], (double)v[i], sum);
    };
    if (HELD) {
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) load_h(lane + c * kLanes, h[c]);
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) square(h[c]);
    } else {
        for (int64_t p = lane; p < pieces; p += kLanes) {
            load_h(p, h[0]);
            square(h[0]);
        }
    }
    sum = wave_sum(sum);
    if (WAVES > 1) {
        if (lane % 64 == 0) part[in * WAVES + lane / 64] = sum;
        __syncthreads();
        sum = 0.0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) sum += part[in * WAVES + w];
    }
    const float f = (float)(1.0 / __builtin_sqrt(sum / (double)a.K + a.eps));
    auto finish = [&](int64_t p, const float* v) {
        const int have = have_of(p);
        if (p >= pieces) return;                // all sixteen lanes of a block alike
        float w[8], y[8];
        if (a.w_dtype == TQ_BF16) load_row8<true>(a.weight, p * 8, have, w, 0.f);
        else load_row8<false>(a.weight, p * 8, have, w, 0.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = v[i] * f * w[i];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = i < have ? y[i] : 0.f;   // a factor that is not finite
        if (a.h) store_row8<BF16>(a.h, row * a.ldh + p * 8, have, v);
        if (a.y) store_row8<BF16>(a.y, row * a.ldy + p * 8, have, y);
        const uint32_t s = f8_scale_bits(over_group<16>(largest8(y), larger));
        *(u32x2*)(a.codes + (row * nb * 16 + p) * 8) = f8_encode8(y, s);
        if (p % 16 == 0) {
            a.scales[row * nb + p / 16] = __builtin_bit_cast(float, s);
            if (s == kF8NaN) atomic_or_status(a.status, TQ_DATA_RANGE);
        }
    };
    if (HELD) {
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) finish(lane + c * kLanes, h[c]);
    } else {
        for (int64_t p = lane; p < pieces; p += kLanes) {
            load_h(p, h[0]);
            finish(p, h[0]);
        }
    }
}

template <bool BF16, int WAVES, int CHUNKS, bool HELD>
hipError_t norm(const F8NormArgs& a, hipStream_t s) {
    constexpr int kRows = WAVES > 4 ? 1 : 4 / WAVES, kAll = WAVES > 4 ? 64 * WAVES : kThreads;
    const int64_t blocks = (a.M + kRows - 1) / kRows;
    if (!grid_fits(blocks, kAll)) return hipErrorInvalidConfiguration;
    f8_norm_pack_kernel<BF16, WAVES, CHUNKS, HELD><<<(unsigned)blocks, kAll, 0, s>>>(a);
    return hipGetLastError();
}

template <bool BF16>
hipError_t norm_by_size(const F8NormArgs& a, hipStream_t s) {
    const int64_t pieces = (a.K + kF8Block - 1) / kF8Block * 16;
    if (pieces <= 256) return norm<BF16, 1, 4, true>(a, s);
    if (pieces <= 1024) return norm<BF16, 4, 4, true>(a, s);
    return norm<BF16, 8, 1, false>(a, s);
}

}  // namespace

hipError_t launch_f8_pack(const void* W, int w_dtype, int64_t rows, int64_t K, int64_t ldw, int block_rows,
                          uint8_t* codes, float* scales, int32_t* status, hipStream_t s) {
    const int64_t nb = (K + kF8Block - 1) / kF8Block;
    if (rows == 0 || nb == 0) return hipSuccess;
    if (block_rows == 128) {
        const int64_t blocks = (rows + 127) / 128 * nb;
        if (!grid_fits(blocks, kThreads)) return hipErrorInvalidConfiguration;
        if (w_dtype == TQ_BF16)
            f8_pack_square_kernel<true><<<(unsigned)blocks, kThreads, 0, s>>>(W, rows, K, ldw, nb, codes, scales, status);
        else
            f8_pack_square_kernel<false><<<(unsigned)blocks, kThreads, 0, s>>>(W, rows, K, ldw, nb, codes, scales, status);
        return hipGetLastError();
    }
    const int64_t pieces = rows * nb * 16, blocks = (pieces + kThreads - 1) / kThreads;
    if (!grid_fits(blocks, kThreads)) return hipErrorInvalidConfiguration;
    const bool flat = K % kF8Block == 0 && (rows == 1 || ldw == K);
    auto go = [&](auto kernel) {
        kernel<<<(unsigned)blocks, kThreads, 0, s>>>(W, K, ldw, nb, pieces, codes, scales, status);
        return hipGetLastError();
    };
    if (w_dtype == TQ_BF16) return flat ? go(f8_pack_kernel<true, true>) : go(f8_pack_kernel<true, false>);
    return flat ? go(f8_pack_kernel<false, true>) : go(f8_pack_kernel<false, false>);
}

hipError_t launch_f8_unpack(const uint8_t* codes, const float* scales, int64_t rows, int64_t K, int block_rows,
                            void* out, int out_dtype, int32_t* status, hipStream_t s) {
    const int64_t nb = (K + kF8Block - 1) / kF8Block, pieces = rows * nb * 16;
    if (pieces == 0) return hipSuccess;
    const int64_t blocks = (pieces + kThreads - 1) / kThreads;
    if (!grid_fits(blocks, kThreads)) return hipErrorInvalidConfiguration;
    const int shift = block_rows == 128 ? 7 : 0;
    if (out_dtype == TQ_BF16)
        f8_unpack_kernel<true><<<(unsigned)blocks, kThreads, 0, s>>>(codes, scales, K, nb, pieces, shift, out, status);
    else
        f8_unpack_kernel<false><<<(unsigned)blocks, kThreads, 0, s>>>(codes, scales, K, nb, pieces, shift, out, status);
    return hipGetLastError();
}

hipError_t launch_f8_norm_pack(const F8NormArgs& a, hipStream_t s) {
    if (a.M == 0 || a.K == 0) return hipSuccess;
    return a.x_dtype == TQ_BF16 ? norm_by_size<true>(a, s) : norm_by_size<false>(a, s);
}

}  // namespace dmm
