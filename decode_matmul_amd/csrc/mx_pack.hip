// mx_pack and mx_unpack: MXFP4 quantization and decoding.
//
// Mathematics.  A block of 32 values with a = max |w| has the scale 2^e,
// e = floor(log2 a) - 2, so that a 2^-e lies in [4, 8) and the largest
// magnitude, 6, is in reach; floor(log2 a) is the exponent field of a.  w 2^-e
// is exact in fp32 for every w that does not round to 0, so the hardware's
// nearest-even conversion to e2m1 (which saturates at 6) is the only rounding.
//
// Both kernels move each byte once and compute about four operations a value:
// they are bound by memory.  Four lanes share a block, eight values each, so a
// wave reads 1 KiB (bf16) or 2 KiB (fp32) of consecutive values with 16-byte
// loads and writes 256 consecutive code bytes; the block maximum takes two
// exchanges within the four lanes.  A matrix without gaps and with whole blocks
// is one long row.  Decoding stores past the caches (bf16 14336 x 4096: 32.0 us
// without), whole lines at a time: fp32 values go four a lane.
#include "mx.h"

namespace dmm {

namespace {

constexpr int kThreads = 256;

// Eight values at p (aligned to their type), the first `have` of them real.
template <bool BF16>
__device__ __forceinline__ void load8(const void* base, int64_t at, int have, float* v) {
    if (have >= 8) {
        if (BF16) {
            const u32x4 d = *(const u32x4h*)((const uint16_t*)base + at);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __builtin_bit_cast(float, d[i] << 16);
                v[2 * i + 1] = __builtin_bit_cast(float, d[i] & 0xffff0000u);
            }
        } else {
            const f32x4 a = *(const f32x4a*)((const float*)base + at);
            const f32x4 b = *(const f32x4a*)((const float*)base + at + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = a[i];
                v[4 + i] = b[i];
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = 0.f;
        if (i < have)
            v[i] = BF16 ? bf16_bits_to_f32(((const uint16_t*)base)[at + i]) : ((const float*)base)[at + i];
    }
}

// Eight values to their codes; the block's scale byte goes to s.
__device__ __forceinline__ uint32_t encode8(float* v, int& s) {
    // the largest magnitude: bit patterns of nonnegative floats order as integers
    uint32_t a = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t u = __builtin_bit_cast(uint32_t, v[i]) & 0x7fffffffu;
        a = a > u ? a : u;
    }
    uint32_t o = (uint32_t)__shfl_xor((int)a, 1);
    a = a > o ? a : o;
    o = (uint32_t)__shfl_xor((int)a, 2);
    a = a > o ? a : o;
    const int field = (int)(a >> 23);
    s = field == 255 ? 255 : (field > 2 ? field - 2 : 0);
    if (field == 255) return 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __builtin_amdgcn_ldexpf(v[i], 127 - s);
    uint32_t c = 0u;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], 1.f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], 1.f, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], 1.f, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], 1.f, 3);
    return c;
}

// Rows with gaps or cut blocks: one lane per eight values of the padded rows.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) mx_pack_rows_kernel(const void* W, int64_t K, int64_t ldw, int64_t nb,
                                                                int64_t blocks, uint8_t* codes, uint8_t* scales,
                                                                int32_t* status) {
    const int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t blk = t >> 2;
    const int part = (int)t & 3;
    const bool live = blk < blocks;
    const int64_t row = live ? blk / nb : 0;
    const int64_t k = (live ? blk - row * nb : 0) * 32 + part * 8;
    float v[8];
    load8<BF16>(W, row * ldw + k, live ? (int)(K - k < 8 ? K - k : 8) : 0, v);
    int s;
    const uint32_t c = encode8(v, s);
    if (!live) return;
    ((uint32_t*)codes)[t] = c;
    if (part == 0) {
        scales[blk] = (uint8_t)s;
        if (s == 255) atomic_or_status(status, TQ_DATA_RANGE);
    }
}

// One row of n8 eighths of a block (n8 a multiple of 4).
template <bool BF16>
__global__ void __launch_bounds__(kThreads) mx_pack_flat_kernel(const void* W, int64_t n8, uint8_t* codes,
                                                                uint8_t* scales, int32_t* status) {
    const int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    float v[8];
    load8<BF16>(W, t * 8, t < n8 ? 8 : 0, v);
    int s;
    const uint32_t c = encode8(v, s);
    if (t >= n8) return;
    ((uint32_t*)codes)[t] = c;
    if ((t & 3) == 0) {
        scales[t >> 2] = (uint8_t)s;
        if (s == 255) atomic_or_status(status, TQ_DATA_RANGE);
    }
}

// Eight codes and their scale to `have` values of row `out`, from column k.
template <bool BF16>
__device__ __forceinline__ void decode8(uint32_t c, uint32_t s, void* out, int64_t at, int have) {
    const float scale = e8m0_bits(s);
    if (BF16) {
        union {
            bf16x8 v;
            u32x4 d;
            uint16_t h[8];
        } u;
        u.v = mx_decode8(c, scale);
        uint16_t* p = (uint16_t*)out + at;
        if (have >= 8) {
            __builtin_nontemporal_store(u.d, (u32x4h*)p);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < have) p[i] = u.h[i];
        }
    } else {
        union {
            f32x2 h[4];
            float f[8];
            u32x4 d[2];
        } u;
        u.h[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 0);
        u.h[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 1);
        u.h[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 2);
        u.h[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 3);
        float* p = (float*)out + at;
        if (have >= 8) {
            *(u32x4a*)p = u.d[0];
            *(u32x4a*)(p + 4) = u.d[1];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < have) p[i] = u.f[i];
        }
    }
}

// Rows with cut blocks: one lane per eight values of the padded rows.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) mx_unpack_rows_kernel(const uint8_t* codes, const uint8_t* scales,
                                                                  int64_t K, int64_t nb, int64_t blocks, void* out,
                                                                  int32_t* status) {
    const int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t blk = t >> 2;
    if (blk >= blocks) return;
    const int64_t row = blk / nb;
    const int64_t k = (blk - row * nb) * 32 + ((int)t & 3) * 8;
    const uint32_t c = ((const uint32_t*)codes)[t];
    const uint32_t s = scales[blk];
    const int have = (int)(K - k < 8 ? K - k : 8);
    if (status) {
        if (s == 255u) atomic_or_status(status, TQ_DATA_RANGE);
        if (have < 8 && (have <= 0 ? c : c >> (4 * have)) != 0u) atomic_or_status(status, TQ_DATA_PADDING);
    }
    if (have > 0) decode8<BF16>(c, s, out, row * K + k, have);
}

// Whole blocks: one row of n lanes' values, eight (bf16) or four (fp32) each.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) mx_unpack_flat_kernel(const uint8_t* codes, const uint8_t* scales,
                                                                  int64_t n, void* out, int32_t* status) {
    const int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (t >= n) return;
    const uint32_t s = scales[t >> (BF16 ? 2 : 3)];
    if (BF16) {
        decode8<true>(((const uint32_t*)codes)[t], s, out, t * 8, 8);
    } else {
        const uint32_t c = ((const uint16_t*)codes)[t];
        union {
            f32x2 h[2];
            u32x4 d;
        } u;
        u.h[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, e8m0_bits(s), 0);
        u.h[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, e8m0_bits(s), 1);
        __builtin_nontemporal_store(u.d, (u32x4a*)((float*)out + t * 4));
    }
    if (status && s == 255u) atomic_or_status(status, TQ_DATA_RANGE);
}

template <bool BF16>
hipError_t pack(const void* W, int64_t rows, int64_t K, int64_t ldw, uint8_t* codes, uint8_t* scales, int32_t* status,
                hipStream_t s) {
    const int64_t nb = (K + 31) / 32, blocks = rows * nb, n8 = blocks * 4;
    const unsigned grid = (unsigned)((n8 + kThreads - 1) / kThreads);
    if (K % 32 == 0 && (rows == 1 || ldw == K))
        mx_pack_flat_kernel<BF16><<<grid, kThreads, 0, s>>>(W, n8, codes, scales, status);
    else
        mx_pack_rows_kernel<BF16><<<grid, kThreads, 0, s>>>(W, K, ldw, nb, blocks, codes, scales, status);
    return hipGetLastError();
}

template <bool BF16>
hipError_t unpack(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, void* out, int32_t* status,
                  hipStream_t s) {
    const int64_t nb = (K + 31) / 32, blocks = rows * nb, n = blocks * (BF16 || K % 32 != 0 ? 4 : 8);
    const unsigned grid = (unsigned)((n + kThreads - 1) / kThreads);
    if (K % 32 == 0)
        mx_unpack_flat_kernel<BF16><<<grid, kThreads, 0, s>>>(codes, scales, n, out, status);
    else
        mx_unpack_rows_kernel<BF16><<<grid, kThreads, 0, s>>>(codes, scales, K, nb, blocks, out, status);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_pack(const void* W, int w_dtype, int64_t rows, int64_t K, int64_t ldw, uint8_t* codes,
                          uint8_t* scales, int32_t* status, hipStream_t s) {
    const int64_t blocks = rows * ((K + 31) / 32);
    if (blocks == 0) return hipSuccess;
    if (!grid_fits((blocks * 4 + kThreads - 1) / kThreads, kThreads)) return hipErrorInvalidConfiguration;
    return w_dtype == TQ_BF16 ? pack<true>(W, rows, K, ldw, codes, scales, status, s)
                              : pack<false>(W, rows, K, ldw, codes, scales, status, s);
}

hipError_t launch_mx_unpack(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, void* out,
                            int out_dtype, int32_t* status, hipStream_t s) {
    const int64_t blocks = rows * ((K + 31) / 32);
    if (blocks == 0) return hipSuccess;
    if (!grid_fits((blocks * 8 + kThreads - 1) / kThreads, kThreads)) return hipErrorInvalidConfiguration;
    return out_dtype == TQ_BF16 ? unpack<true>(codes, scales, rows, K, out, status, s)
                                : unpack<false>(codes, scales, rows, K, out, status, s);
}

}  // namespace dmm
