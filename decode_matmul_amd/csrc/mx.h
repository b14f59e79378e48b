// MXFP4 helpers shared by the mx_* kernels (gfx950 converts and multiplies
// e2m1 values with E8M0 block scales in hardware).
#pragma once

#include "common.h"

namespace dmm {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4a __attribute__((ext_vector_type(4), aligned(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint64_t u64u __attribute__((aligned(1)));

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

// Two fp32 values as bf16, nearest-even, in one dword.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

// The scaled matrix instruction's operand of 32 codes (16 bytes; the upper
// half of the register group is not read for 4-bit types).
__device__ __forceinline__ i32x8 mx_operand(u32x4 c) {
    return (i32x8){(int)c.x, (int)c.y, (int)c.z, (int)c.w, 0, 0, 0, 0};
}

// Scale bytes b .. b + 7 of a row of nb (those past the row are 127).
__device__ __forceinline__ uint64_t scales8(const uint8_t* row, int64_t b, int64_t nb) {
    if (b + 8 <= nb) return *(const u64u*)(row + b);
    uint64_t v = 0x7f7f7f7f7f7f7f7full;
#pragma unroll 1
    for (int i = 0; b + i < nb; ++i) v ^= (uint64_t)(row[b + i] ^ 0x7fu) << (8 * i);
    return v;
}

// Eight activations at column k of a row (past K they are 0).
__device__ __forceinline__ u32x4 load_x8(const uint16_t* row, int64_t k, int64_t K) {
    if (k + 8 <= K) return *(const u32x4h*)(row + k);
    uint64_t lo = 0, hi = 0;
#pragma unroll 1
    for (int i = 0; i < 7 && k + i < K; ++i) {
        if (i < 4) lo |= (uint64_t)row[k + i] << (16 * i);
        else hi |= (uint64_t)row[k + i] << (16 * (i - 4));
    }
    const u32x4 v = {(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
    return v;
}

// The codes of a cut block, of which the first `kept` (0 .. 32) count.  The others meet
// activations that are 0, but with the largest scales they stand for infinities.
__device__ __forceinline__ u32x4 cut_codes(u32x4 c, int kept) {
    const uint64_t lo = kept < 16 ? (1ull << (4 * kept)) - 1ull : ~0ull;
    const uint64_t hi = kept > 16 ? ~0ull >> (128 - 4 * kept) : 0ull;
    return c & (u32x4){(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// A uniform pointer the compiler keeps in scalar registers as it is, so that a
// lane's address stays base + 32-bit offset (folded into per-lane pointers,
// the slabs' addresses take more registers than there are).
typedef const __attribute__((address_space(1))) uint8_t* GlobalBytes;
__device__ __forceinline__ GlobalBytes scalar_base(const uint8_t* p) {
    GlobalBytes q = (GlobalBytes)p;
    asm("" : "+s"(q));
    return q;
}

// A lane's value, likewise kept as it is where it stands: what is computed from
// it is computed there (widened or added ahead of a loop, offsets take
// registers all through it).
__device__ __forceinline__ uint32_t lane_offset(uint32_t o) {
    asm volatile("" : "+v"(o));
    return o;
}
__device__ __forceinline__ int64_t lane_offset(int64_t o) {
    asm volatile("" : "+v"(o));
    return o;
}

// 16 bytes a lane from global memory to LDS: lane l's land at lds + 16 l.  STREAM: what is read
// once, past the caches.
template <bool STREAM = false>
__device__ __forceinline__ void load_lds16(GlobalBytes g, void* lds) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)g,
                                     (__attribute__((address_space(3))) void*)lds, 16, 0, STREAM ? 2 : 0);
}

// Which of a 128-byte row's eight slots chunk 0 takes.  A 16-byte LDS read serves
// lanes 0-3, 12-15, 20-23 and 24-27 together, then 4-11, 16-19 and 28-31, and the
// upper half alike.  Two rows fill the 64 banks, so in either set the eight even
// (and odd) rows have to differ, also where half of them read the neighbouring
// chunk (16 x 16 tiles): the Gray code of row / 2 does that.  (With row % 8 ^ row /
// 8 % 2, 40 % of the LDS cycles of the MXFP4 tiles were conflicts.)
__device__ __forceinline__ int swizzle(int row) { return ((row >> 1) & 7) ^ ((row >> 2) & 3); }

// Keeps an accumulator's matrix instructions ahead of what follows.  A kernel
// with one wave a SIMD has its accumulators in the accumulation registers;
// asking for them elsewhere would copy them there and back.
template <bool ONE_WAVE, class T>
__device__ __forceinline__ void hold_acc(T& acc) {
    if constexpr (ONE_WAVE) asm volatile("" : "+a"(acc));
    else asm volatile("" : "+v"(acc));
}

// At most VM vector loads of this wave outstanding.
template <int VM>
__device__ __forceinline__ void wait_loads() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((VM & 15) | ((VM >> 4) << 14) | 0xf70);
    asm volatile("" ::: "memory");
}

// The workgroup's barrier for LDS accesses: this wave's are done, its loads
// may be on their way.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xc07f);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

}  // namespace dmm
