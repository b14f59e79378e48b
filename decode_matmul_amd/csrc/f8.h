// Helpers shared by the f8_* kernels: e4m3 values in blocks of 128 columns with an
// fp32 scale each (gfx950 converts and multiplies e4m3 in hardware).
#pragma once

#include "lanes.h"

namespace dmm {

constexpr int kF8Block = 128;                   // columns of a scale, bytes of a block's codes
constexpr uint32_t kF8NaN = 0x7fc00000u;        // the scale of a block that is not finite

// The scale of a block whose largest magnitude has the bits a: the least power of two
// with a / scale <= 448 = 1.75 2^8, at least 2^-126 (a mantissa above 1.75 carries into the
// exponent).  A power of two scales exactly, so that a value is rounded once.
__device__ __forceinline__ uint32_t f8_scale_bits(uint32_t a) {
    if (a >= 0x7f800000u) return kF8NaN;
    const uint32_t e = (a + 0x1fffffu) >> 23;
    return (e > 8u ? e - 8u : 1u) << 23;
}

// Eight values over a scale as e4m3, nearest, ties to even (0 under a scale that is NaN).
__device__ __forceinline__ u32x2 f8_encode8(const float* v, uint32_t scale) {
    if (scale == kF8NaN) return (u32x2){0u, 0u};
    const float r = __builtin_bit_cast(float, (254u << 23) - scale);    // 1 / scale
    u32x2 c;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h] * r, v[4 * h + 1] * r, 0, false);
        c[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2] * r, v[4 * h + 3] * r, w, true);
    }
    return c;
}

// Eight e4m3 codes as bf16 (exact: four significant bits).
__device__ __forceinline__ bf16x8 f8_bf16(uint32_t lo, uint32_t hi) {
    union {
        bf16x2 h[4];
        bf16x8 v;
    } u;
    u.h[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 1.f, false);
    u.h[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 1.f, true);
    u.h[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 1.f, false);
    u.h[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 1.f, true);
    return u.v;
}

// The first `kept` (any number) of 16 bytes; zeros behind.
__device__ __forceinline__ u32x4 keep_bytes(u32x4 v, int kept) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = kept - 4 * i;
        v[i] &= n >= 4 ? 0xffffffffu : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
    }
    return v;
}

// Bits of the largest magnitude of eight values (those of nonnegative floats order as integers).
__device__ __forceinline__ uint32_t largest8(const float* v) {
    uint32_t a = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t u = __builtin_bit_cast(uint32_t, v[i]) & 0x7fffffffu;
        a = a > u ? a : u;
    }
    return a;
}

__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }

}  // namespace dmm
