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
// lanes a block's 128; its largest magnitude takes four data-parallel moves.  us in a
// replayed graph, bf16: pack 2048 x 8192 9.4 (5.4 TB/s), 14336 x 4096 by 128 x 128 33.8 (5.2),
// unpack of it 26.3 (6.7); norm with residual, sum and rows 2048 x 8192 30.8 (4.9), 4096 x 4096
// 28.4 (5.3), 1 x 4096 2.8.
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
    if (have > 0) store_row8<BF16, true>(out, row * K + k, have, v);
}

// ------------------------------------------------------------------- norm
//
// h = x + residual, rounded to the type of x, as it is stored; f = (mean h^2 + eps)^-1/2
// from a sum in float64 (squares of fp32 are exact there, and float64 runs at the rate of
// fp32), rounded to fp32; y = h f weight, each product rounded to fp32; y's package.
// The factor does not depend on how the sum is split, up to float64's own rounding, so that the package hardly ever does.
//
// WAVES waves a row, 4 / WAVES rows a workgroup of four.  HELD: the row's values and its weights
// stay in registers, CHUNKS times eight a lane, all of them on their way at once; longer
// rows are read twice.
__device__ __forceinline__ double moved_sum(double v) {         // over the wave, in all lanes
    auto add = [&](double o) { v += o; };
    auto both = [&](auto f) {
        const uint64_t u = __builtin_bit_cast(uint64_t, v);
        return __builtin_bit_cast(double, (uint64_t)f((uint32_t)(u >> 32)) << 32 | f((uint32_t)u));
    };
    add(both([](uint32_t x) { return moved<0xb1>(x); }));
    add(both([](uint32_t x) { return moved<0x4e>(x); }));
    add(both([](uint32_t x) { return moved<0x141>(x); }));
    add(both([](uint32_t x) { return moved<0x140>(x); }));
    add(both([](uint32_t x) { return (uint32_t)__builtin_amdgcn_ds_swizzle((int)x, 0x401f); }));     // lane ^ 16
    add(both([](uint32_t x) { return (uint32_t)__shfl_xor((int)x, 32); }));
    return v;
}

// a^-1/2 in float64: the hardware's estimate and one step of third order.
__device__ __forceinline__ double inverse_root(double a) {
    if (!(a > 0.0 && a < __builtin_inf())) return 1.0 / __builtin_sqrt(a);
    const double y = __builtin_amdgcn_rsq(a);
    const double e = __builtin_fma(-a * y, y, 1.0);
    return __builtin_fma(y * e, __builtin_fma(e, 0.375, 0.5), y);
}

// Eight values as they lie in memory.
template <bool BF16>
struct Eight {
    uint32_t d[BF16 ? 4 : 8];
    __device__ __forceinline__ void load(const void* base, int64_t at, int have) {
        if (have >= 8) {
            const u32x4 v = *(const u32x4h*)((const uint8_t*)base + at * (BF16 ? 2 : 4));
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] = v[i];
            if (!BF16) {
                const u32x4 w = *(const u32x4h*)((const uint8_t*)base + at * 4 + 16);
#pragma unroll
                for (int i = 0; i < 4; ++i) d[(BF16 ? 0 : 4) + i] = w[i];
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < (BF16 ? 4 : 8); ++i) d[i] = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i >= have) continue;
            if (BF16) d[i / 2] |= (uint32_t)((const uint16_t*)base)[at + i] << (16 * (i & 1));
            else d[BF16 ? 0 : i] = ((const uint32_t*)base)[at + i];
        }
    }
    __device__ __forceinline__ float operator[](int i) const {
        if (!BF16) return __builtin_bit_cast(float, d[BF16 ? 0 : i]);
        return __builtin_bit_cast(float, (i & 1) ? d[i / 2] & 0xffff0000u : d[i / 2] << 16);
    }
};

template <bool BF16, bool WBF16, int WAVES, int CHUNKS, bool HELD>
__global__ void __launch_bounds__(WAVES > 4 ? 64 * WAVES : kThreads) f8_norm_pack_kernel(F8NormArgs a) {
    constexpr int kLanes = 64 * WAVES, kRows = WAVES > 4 ? 1 : 4 / WAVES, kHeld = HELD ? CHUNKS : 1;
    __shared__ double part[kRows * WAVES];
    const int lane = (int)threadIdx.x % kLanes, in = (int)threadIdx.x / kLanes;
    const int64_t row = (int64_t)blockIdx.x * kRows + in;
    const bool live = row < a.M;
    const int64_t nb = (a.K + kF8Block - 1) / kF8Block, pieces = live ? nb * 16 : 0;
    auto have_of = [&](int64_t p) {             // values of piece p (eight columns) that there are
        const int64_t left = a.K - p * 8;
        return left < 0 || p >= pieces ? 0 : (int)(left < 8 ? left : 8);
    };
    Eight<BF16> h[kHeld], res[kHeld];
    Eight<WBF16> weight[kHeld];
    auto load = [&](int c, int64_t p) {
        const int have = have_of(p);
        h[c].load(a.x, row * a.ldx + p * 8, have);
        if (a.residual) res[c].load(a.residual, row * a.ldr + p * 8, have);
    };
    auto add = [&](int c) {
        if (!a.residual) return;
        if (BF16) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                h[c].d[i] = bf16_pair(h[c][2 * i] + res[c][2 * i], h[c][2 * i + 1] + res[c][2 * i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) h[c].d[BF16 ? 0 : i] = __builtin_bit_cast(uint32_t, h[c][i] + res[c][i]);
        }
    };
    double sum = 0.0;
    auto square = [&](int c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = __builtin_fma((double)h[c][i], (double)h[c][i], sum);
    };
    if (HELD) {
#pragma unroll
        for (int c = 0; c < kHeld; ++c) load(c, lane + c * kLanes);
#pragma unroll
        for (int c = 0; c < kHeld; ++c)
            weight[c].load(a.weight, (int64_t)(lane + c * kLanes) * 8, have_of(lane + c * kLanes));
#pragma unroll
        for (int c = 0; c < kHeld; ++c) {
            add(c);
            square(c);
        }
    } else {
        for (int64_t p = lane; p < pieces; p += kLanes) {
            load(0, p);
            add(0);
            square(0);
        }
    }
    sum = moved_sum(sum);
    if (WAVES > 1) {
        if (lane % 64 == 0) part[in * WAVES + lane / 64] = sum;
        __syncthreads();
        sum = 0.0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) sum += part[in * WAVES + w];
    }
    const float f = (float)inverse_root(sum / (double)a.K + a.eps);
    auto finish = [&](int c, int64_t p) {
        if (p >= pieces) return;                // all sixteen lanes of a block alike
        const int have = have_of(p);
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = i < have ? h[c][i] * f * weight[c][i] : 0.f;
        if (a.h) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = h[c][i];
            store_row8<BF16, true>(a.h, row * a.ldh + p * 8, have, v);
        }
        if (a.y) store_row8<BF16, true>(a.y, row * a.ldy + p * 8, have, y);
        const uint32_t s = f8_scale_bits(over_group<16>(largest8(y), larger));
        *(u32x2*)(a.codes + (row * nb * 16 + p) * 8) = f8_encode8(y, s);
        if (p % 16 == 0) {
            a.scales[row * nb + p / 16] = __builtin_bit_cast(float, s);
            if (s == kF8NaN) atomic_or_status(a.status, TQ_DATA_RANGE);
        }
    };
    if (HELD) {
#pragma unroll
        for (int c = 0; c < kHeld; ++c) finish(c, lane + c * kLanes);
    } else {
        for (int64_t p = lane; p < pieces; p += kLanes) {
            load(0, p);
            weight[0].load(a.weight, p * 8, have_of(p));
            add(0);
            finish(0, p);
        }
    }
}

template <bool BF16, bool WBF16, int WAVES, int CHUNKS, bool HELD>
hipError_t norm(const F8NormArgs& a, hipStream_t s) {
    constexpr int kRows = WAVES > 4 ? 1 : 4 / WAVES, kAll = WAVES > 4 ? 64 * WAVES : kThreads;
    const int64_t blocks = (a.M + kRows - 1) / kRows;
    if (!grid_fits(blocks, kAll)) return hipErrorInvalidConfiguration;
    f8_norm_pack_kernel<BF16, WBF16, WAVES, CHUNKS, HELD><<<(unsigned)blocks, kAll, 0, s>>>(a);
    return hipGetLastError();
}

template <bool BF16, bool WBF16>
hipError_t norm_by_size(const F8NormArgs& a, hipStream_t s) {
    const int64_t pieces = (a.K + kF8Block - 1) / kF8Block * 16;
    // A lane for each piece as far as a workgroup goes (us, bf16 with residual and both outputs, by
    // pieces a lane: 8192 x 2048 four 36.4, one 29.9; 4096 x 4096 four 34.3, two 33.4, one 30.5;
    // 2048 x 8192 four 36.6, two 33.5, one 33.0; 1 x 8192 four 4.6, one 3.6; all with
    // stores that stay in the caches, which cost 2 us of 30 at 4096 x 4096).
    if (pieces <= 64) return norm<BF16, WBF16, 1, 1, true>(a, s);
    if (pieces <= 128) return norm<BF16, WBF16, 2, 1, true>(a, s);
    if (pieces <= 256) return norm<BF16, WBF16, 4, 1, true>(a, s);
    if (pieces <= 512) return norm<BF16, WBF16, 8, 1, true>(a, s);
    if (pieces <= 1024) return norm<BF16, WBF16, 16, 1, true>(a, s);
    if (pieces <= 2048) return norm<BF16, WBF16, 16, 2, true>(a, s);
    return norm<BF16, WBF16, 16, 1, false>(a, s);
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
    if (a.x_dtype == TQ_BF16) return a.w_dtype == TQ_BF16 ? norm_by_size<true, true>(a, s) : norm_by_size<true, false>(a, s);
    return a.w_dtype == TQ_BF16 ? norm_by_size<false, true>(a, s) : norm_by_size<false, false>(a, s);
}

}  // namespace dmm
