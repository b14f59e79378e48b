// MXFP4 helpers shared by the mx_* kernels (gfx950 converts and multiplies
// e2m1 values with E8M0 block scales in hardware).
#pragma once

#include "common.h"

namespace dmm {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4a __attribute__((ext_vector_type(4), aligned(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// An E8M0 byte as the fp32 whose exponent field it is: what the scaled
// conversions take (0 stands for 2^-127 and 255 for NaN there).
__device__ __forceinline__ float e8m0_bits(uint32_t s) {
    return __builtin_bit_cast(float, s << 23);
}

// The eight codes of a dword times their block's scale, as eight bf16 values
// (exact: an e2m1 value has two significant bits).
__device__ __forceinline__ bf16x8 mx_decode8(uint32_t c, float scale) {
    union {
        bf16x2 h[4];
        bf16x8 v;
    } u;
    u.h[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0);
    u.h[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1);
    u.h[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2);
    u.h[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3);
    return u.v;
}

// The scaled matrix instruction's operand of 32 codes (16 bytes; the upper
// half of the register group is not read for 4-bit types).
__device__ __forceinline__ i32x8 mx_operand(u32x4 c) {
    return (i32x8){(int)c.x, (int)c.y, (int)c.z, (int)c.w, 0, 0, 0, 0};
}

}  // namespace dmm
